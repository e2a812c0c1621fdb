// tile_common.cuh -- what the tcgen05 kernels of linear attention share: waits
// taken by whole warps, loads and stores of tensor memory in 16 columns, paired
// fp32 arithmetic.
#pragma once
#include "attn_common.cuh"

namespace ikbo {

// A wait taken by a whole warp: the lanes agree on its outcome, so that a limit
// that expires while the barrier completes never splits the warp before its next
// warp-wide instruction.  X has the CTA's abort word, P the limit.
template <typename X, typename P>
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, X& x, const P& p) {
  const bool ok = mbar_wait(bar, parity, &x.abort, p.timeout_ns, 1);
  return __all_sync(0xffffffffu, ok);
}

__device__ __forceinline__ void warp_arrive(uint64_t* bar) {
  __syncwarp();
  if (lane_id() == 0) mbar_arrive(bar);
}

// Ends when `bar` completes its phase, or a second is over.
__device__ __forceinline__ void wait_a_second(uint64_t* bar, uint32_t parity) {
  const uint64_t t0 = globaltimer_ns();
  while (!mbar_try_wait(bar, parity) && globaltimer_ns() - t0 < 1000000000ull) {}
}

// An issuer leaves when its products in flight have ended, or a second is over.
__device__ __forceinline__ void drain(uint64_t* bar) {
  __syncwarp();
  if (elect_one()) mma_commit(bar);
  __syncwarp();
  wait_a_second(bar, 0);
  __syncwarp();
}

// 32 lanes x 16 columns from, or 8 columns to, tensor memory.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]),
        "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
// Waits for loads, and keeps uses of r behind that.
__device__ __forceinline__ void tmem_ld16_wait(uint32_t (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]),
                 "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
               :
               : "memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]),
               "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
// (r0, r1) = (a0, a1) * (b0, b1)
__device__ __forceinline__ void mul2(float& r0, float& r1, float a0, float a1, float b0, float b1) {
  asm("{.reg .b64 x, y, w;\n\t"
      "mov.b64 x, {%2, %3};\n\t"
      "mov.b64 y, {%4, %5};\n\t"
      "mul.rn.f32x2 w, x, y;\n\t"
      "mov.b64 {%0, %1}, w;}"
      : "=f"(r0), "=f"(r1)
      : "f"(a0), "f"(a1), "f"(b0), "f"(b1));
}

// (r0, r1) = (a0, a1) * b + (c0, c1)
__device__ __forceinline__ void fma2v(float& r0, float& r1, float a0, float a1, float b, float c0, float c1) {
  asm("{.reg .b64 x, y, z, w;\n\t"
      "mov.b64 x, {%2, %3};\n\t"
      "mov.b64 y, {%4, %4};\n\t"
      "mov.b64 z, {%5, %6};\n\t"
      "fma.rn.f32x2 w, x, y, z;\n\t"
      "mov.b64 {%0, %1}, w;}"
      : "=f"(r0), "=f"(r1)
      : "f"(a0), "f"(a1), "f"(b), "f"(c0), "f"(c1));
}
}  // namespace ikbo
