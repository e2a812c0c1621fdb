// mma_common.cuh -- warp-level pieces that the kernels on the 16x8x16 matrix
// instruction share: the product, 8x8 loads from shared memory, asynchronous
// 16-byte copies, and splitting an fp32 pair into two bf16 pairs.
#pragma once
#include <cstdint>

#include "ptx.cuh"

namespace ikbo {

__device__ __forceinline__ void mma_16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Four 8x8 matrices of 16-bit elements from shared memory; lane 8i + r gives
// row r of matrix i.
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

// An 8x8 matrix of 16-bit elements, two a lane, turned.
__device__ __forceinline__ uint32_t turn8x8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// 16 bytes of global memory to shared memory, or 16 zeros.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kPending>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kPending) : "memory");
}

// a, b = hi + lo to 16 bits of mantissa (2^-17 relative).
__device__ __forceinline__ void split_bf16x2(float a, float b, uint32_t& hi, uint32_t& lo) {
  hi = pack_bf16x2(a, b);
  lo = pack_bf16x2(a - __uint_as_float(hi << 16), b - __uint_as_float(hi & 0xffff0000u));
}
// Bits 15 and 31: whether the halves of x, a bf16 pair, are infinite or NaN (the exponent's carry).
__device__ __forceinline__ uint32_t not_finite(uint32_t x) { return (x & 0x7f807f80u) + 0x00800080u; }
__device__ __forceinline__ uint32_t not_finite(const uint4& x) {
  return not_finite(x.x) | not_finite(x.y) | not_finite(x.z) | not_finite(x.w);
}
// x without its halves that are infinite or NaN, and ones where they are.
__device__ __forceinline__ uint32_t finite_part(uint32_t x) { return x & ~(((not_finite(x) & 0x80008000u) >> 15) * 0xffffu); }
__device__ __forceinline__ uint32_t odd_ones(uint32_t x) { return ((not_finite(x) & 0x80008000u) >> 15) * 0x3f80u; }
// 0 times the halves of bf16 pairs: 0, of either sign, where none is infinite or NaN, else NaN; `or`ed.
__device__ __forceinline__ uint32_t times_zero(uint32_t x) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(0u));
  return r;
}
__device__ __forceinline__ uint32_t times_zero(const uint4& x) {
  return times_zero(x.x) | times_zero(x.y) | times_zero(x.z) | times_zero(x.w);
}
__device__ __forceinline__ uint32_t times_zero(const uint32_t (&x)[4]) {
  return times_zero(x[0]) | times_zero(x[1]) | times_zero(x[2]) | times_zero(x[3]);
}
__device__ __forceinline__ bool is_finite(float x) { return fabsf(x) < INFINITY; }
__device__ __forceinline__ float bf16_lo(uint32_t x) { return __uint_as_float(x << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t x) { return __uint_as_float(x & 0xffff0000u); }

}  // namespace ikbo
