// linread.cu -- candidates' queries of their user's state of linear attention,
// read through the map, and the gradient.
//
//   O[i,h] = scale Q[i,h] S[map[i],h]
//   dQ[i,h] = scale dO[i,h] S[map[i],h]^T,   dS[u,h] = scale sum_{map[i]=u} Q[i,h]^T dO[i,h]
//
// The broadcast's linear form: a user's 64 KB state serves all of its
// candidates, grouped by the plan's work list as the attention's are, and the
// gradient of the state is the sum over them.
#include <cuda_bf16.h>

#include "linattn_internal.h"
#include "mma_common.cuh"

namespace ikbo {
namespace {

constexpr int RD_THREADS = 256;
constexpr int RD_ROWS = 128;  // of a unit, at most (16 a warp)
constexpr int RD_TILE = RD_ROWS * LIN_D * 2;

// Whether unit i exists and is sound (n is the list's length).
__device__ __forceinline__ bool read_unit(const LinReadParams& p, int i, int4& w) {
  w = __ldg(reinterpret_cast<const int4*>(p.work) + i);
  if (w.x >= 0 && w.x < p.n_users && w.y >= 0 && w.y < p.H && w.z >= 0 && w.w > 0 && w.z + w.w <= p.n_cand && w.w * p.Lq <= RD_ROWS) return true;
  if (threadIdx.x == 0) atomicOr(p.status, DEV_ERR_BAD_WORK);
  return false;
}

__device__ __forceinline__ int64_t row_of(const LinReadParams& p, const int4& w, int r) {
  const int slot = r / p.Lq;
  return (static_cast<int64_t>(__ldg(p.perm + w.z + slot)) * p.H + w.y) * p.Lq + (r - slot * p.Lq);
}

// 16 bytes that nobody reads again (and that may be overwritten by whoever read
// them: not the read-only path).
__device__ __forceinline__ uint4 ld_once(const uint4* p) {
  uint4 r;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "l"(p) : "memory");
  return r;
}

// This CTA's units: an equal run of the list.
__device__ __forceinline__ void unit_range(const LinReadParams& p, int cta, int& a, int& b) {
  const int n = min(static_cast<int64_t>(__ldg(p.n_units)), p.max_units);
  a = static_cast<int>(static_cast<int64_t>(cta) * n / gridDim.x);
  b = static_cast<int>(static_cast<int64_t>(cta + 1) * n / gridDim.x);
}

// out = scale x S (or x S^T).  The state's bf16 image lies in shared memory, [inner
// element][column], columns in the order that leaves each lane eight consecutive
// ones of a row: column 32 m + 8 t + 2 i + e at 32 m + 8 i + 2 t + e.  A lane loads
// its rows in 16-byte pieces, which the inner order of the products follows: slot k
// of step 2 j + f is element 32 j + 8 ((k & 7) >> 1) + 4 f + 2 (k >> 3) + (k & 1).
struct ReadRows {
  uint4 x[2][4];  // rows g and g + 8 of the warp's 16, element 32 j + 8 t of piece j
  int64_t at[2];  // their places, -1: not there
};

__global__ void __launch_bounds__(RD_THREADS, 2) lin_read_kernel(const __grid_constant__ LinReadParams p) {
  __shared__ __align__(128) uint8_t st[LIN_STATE * 2];
  const uint32_t base = smem_u32(st);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  int a, b;
  unit_range(p, static_cast<int>(blockIdx.x), a, b);
  int held = -1;  // (user, head) of the state in shared memory
  const int slot = lane & 15;
  const uint32_t inner = static_cast<uint32_t>(8 * ((slot & 7) >> 1) + 2 * (slot >> 3) + (slot & 1));  // of f = 0, without 32 j
  int4 w = make_int4(0, 0, 0, 0);
  ReadRows now;
  const auto fetch = [&](int i, int4& w, ReadRows& r) {
    if (!read_unit(p, i, w)) w.w = 0;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int row = 16 * warp + g + 8 * e;
      r.at[e] = row < w.w * p.Lq ? row_of(p, w, row) : -1;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        r.x[e][j] = r.at[e] >= 0 ? ld_once(reinterpret_cast<const uint4*>(p.x + r.at[e] * LIN_D + 32 * j + 8 * t)) : uint4{};
    }
  };
  if (a < b) fetch(a, w, now);
#pragma unroll 1
  for (int i = a; i < b; ++i) {
    int4 w_next = make_int4(0, 0, 0, 0);
    ReadRows next;
    if (i + 1 < b) fetch(i + 1, w_next, next);  // on its way meanwhile
    if (w.w > 0 && w.x * p.H + w.y != held) {
      __syncthreads();
      held = w.x * p.H + w.y;
      const float* s = p.state + static_cast<int64_t>(held) * LIN_STATE;
      if (!p.turned) {  // rows of the state are the inner elements; a thread takes two columns
#pragma unroll 8
        for (int k = 0; k < LIN_STATE / 2 / RD_THREADS; ++k) {
          const int e = k * RD_THREADS + tid, row = e >> 6, c = (e & 63) * 2;
          const float2 v = __ldg(reinterpret_cast<const float2*>(s) + e);
          const int at = (c & 96) + 8 * ((c >> 1) & 3) + 2 * ((c >> 3) & 3);
          *reinterpret_cast<uint32_t*>(st + row * 256 + (((at >> 3) ^ (row & 7)) << 4) + (at & 7) * 2) = pack_bf16x2(v.x, v.y);
        }
      } else {  // rows of the state are the columns: two of them, four inner elements
#pragma unroll 2
        for (int k = 0; k < LIN_STATE / 8 / RD_THREADS; ++k) {
          const int e = k * RD_THREADS + tid, c = (e >> 5) * 2, row = (e & 31) * 4;
          const float4 v = __ldg(reinterpret_cast<const float4*>(s + c * LIN_D + row));
          const float4 n = __ldg(reinterpret_cast<const float4*>(s + (c + 1) * LIN_D + row));
          const int at = (c & 96) + 8 * ((c >> 1) & 3) + 2 * ((c >> 3) & 3);
          const float lo[4] = {v.x, v.y, v.z, v.w}, hi[4] = {n.x, n.y, n.z, n.w};
#pragma unroll
          for (int d = 0; d < 4; ++d)
            *reinterpret_cast<uint32_t*>(st + (row + d) * 256 + (((at >> 3) ^ ((row + d) & 7)) << 4) + (at & 7) * 2) = pack_bf16x2(lo[d], hi[d]);
        }
      }
      __syncthreads();
    }
    if (16 * warp < w.w * p.Lq) {
#pragma unroll
      for (int half = 0; half < 2; ++half) {  // of the columns
        float o[8][4] = {};
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int f = 0; f < 2; ++f) {
            const uint32_t af[4] = {f ? now.x[0][j].z : now.x[0][j].x, f ? now.x[1][j].z : now.x[1][j].x, f ? now.x[0][j].w : now.x[0][j].y,
                                    f ? now.x[1][j].w : now.x[1][j].y};
            const uint32_t row = 32 * j + 4 * f + inner;
#pragma unroll
            for (int n = 0; n < 4; ++n) {
              uint32_t bf[4];
              ldsm4_t(bf, base + row * 256 + (((8 * half + 2 * n + (lane >> 4)) ^ (row & 7)) << 4));
              mma_16816(o[2 * n], af, bf[0], bf[1]);
              mma_16816(o[2 * n + 1], af, bf[2], bf[3]);
            }
          }
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            if (now.at[k] < 0) continue;
            uint32_t v[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) v[q] = pack_bf16x2(o[4 * m + q][2 * k] * p.scale, o[4 * m + q][2 * k + 1] * p.scale);
            *reinterpret_cast<uint4*>(p.out + now.at[k] * LIN_D + 64 * half + 32 * m + 8 * t) = make_uint4(v[0], v[1], v[2], v[3]);
          }
      }
    }
    w = w_next;
    now = next;
  }
}

// dS, unit by unit: a warp has 16 of the state's rows, all columns, in registers
// over the units of a (user, head).  A CTA's first and last (user, head) may have
// units of other CTAs too: those sums go to the CTA's two places of the workspace.
__global__ void __launch_bounds__(RD_THREADS, 1) lin_read_state_kernel(const __grid_constant__ LinReadParams p) {
  extern __shared__ __align__(128) uint8_t rd_sm[];
  const uint32_t base = smem_u32(rd_sm);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  int a, b;
  unit_range(p, static_cast<int>(blockIdx.x), a, b);
  const int n = min(static_cast<int64_t>(__ldg(p.n_units)), p.max_units);
  // users without candidates: zero
  for (int64_t uh = blockIdx.x; uh < static_cast<int64_t>(p.n_users) * p.H; uh += gridDim.x) {
    const int u = static_cast<int>(uh / p.H);
    if (__ldg(p.offsets + u + 1) > __ldg(p.offsets + u)) continue;
    for (int e = tid; e < LIN_STATE / 4; e += RD_THREADS)
      reinterpret_cast<float4*>(p.d_state + uh * LIN_STATE)[e] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  const auto load = [&](int i, int stage) {
    int4 w;
    if (!read_unit(p, i, w)) w = make_int4(0, 0, 0, 0);
    const int rows = w.w * p.Lq;
#pragma unroll
    for (int k = 0; k < RD_TILE / 16 / RD_THREADS; ++k) {
      const int r = k * (RD_THREADS / 16) + (tid >> 4), c = tid & 15;
      const int64_t at = r < rows ? row_of(p, w, r) * LIN_D + 8 * c : -1;
      const uint32_t dst = base + stage * 2 * RD_TILE + r * 256 + ((c ^ (r & 7)) << 4);
      copy16(dst, p.q + max(at, int64_t{0}), at >= 0);
      copy16(dst + RD_TILE, p.x + max(at, int64_t{0}), at >= 0);
    }
  };
  if (a < b) load(a, 0);
  copies_commit();
  float s[16][4] = {};
#pragma unroll 1
  for (int i = a; i < b; ++i) {
    if (i + 1 < b) load(i + 1, (i + 1 - a) & 1);
    copies_commit();
    copies_wait<1>();
    __syncthreads();
    const uint32_t q_at = base + ((i - a) & 1) * 2 * RD_TILE, o_at = q_at + RD_TILE;
    int4 w;
    if (!read_unit(p, i, w)) {
      __syncthreads();
      continue;
    }
    const int steps = (w.w * p.Lq + 15) >> 4;
#pragma unroll 1
    for (int kb = 0; kb < steps; ++kb) {
      uint32_t af[4];
      int r = 16 * kb + (lane & 7) + 8 * (lane >> 4);
      ldsm4_t(af, q_at + r * 256 + (((2 * warp + ((lane >> 3) & 1)) ^ (r & 7)) << 4));
      r = 16 * kb + (lane & 15);
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        uint32_t bf[4];
        ldsm4_t(bf, o_at + r * 256 + (((2 * c + (lane >> 4)) ^ (r & 7)) << 4));
        mma_16816(s[2 * c], af, bf[0], bf[1]);
        mma_16816(s[2 * c + 1], af, bf[2], bf[3]);
      }
    }
    __syncthreads();
    // the (user, head) ends here, or the CTA's units do
    const int4 next = i + 1 < n ? __ldg(reinterpret_cast<const int4*>(p.work) + i + 1) : make_int4(-1, -1, 0, 0);
    const bool ends = next.x != w.x || next.y != w.y;
    if (!ends && i + 1 < b) continue;
    bool begun = true;  // within this CTA
    if (a > 0) {
      const int4 before = __ldg(reinterpret_cast<const int4*>(p.work) + a - 1);
      begun = before.x != w.x || before.y != w.y;
    }
    const bool whole = begun && ends;
    float* to = whole ? p.d_state + (static_cast<int64_t>(w.x) * p.H + w.y) * LIN_STATE
                      : p.part + (2 * static_cast<int64_t>(blockIdx.x) + (begun ? 1 : 0)) * LIN_STATE;
    const float f = whole ? p.scale : 1.f;
#pragma unroll
    for (int c = 0; c < 16; ++c)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        *reinterpret_cast<float2*>(to + (16 * warp + g + 8 * k) * LIN_D + 8 * c + 2 * t) = make_float2(s[c][2 * k] * f, s[c][2 * k + 1] * f);
        s[c][2 * k] = s[c][2 * k + 1] = 0.f;
      }
  }
}

// Adds the parts of each (user, head) whose units several CTAs had, in order:
// block c those of the one that begins in CTA c and goes on in the next.
__global__ void __launch_bounds__(RD_THREADS) lin_read_join_kernel(const __grid_constant__ LinReadParams p) {
  const int c = static_cast<int>(blockIdx.x);
  const int n = min(static_cast<int64_t>(__ldg(p.n_units)), p.max_units);
  const int4* work = reinterpret_cast<const int4*>(p.work);
  const auto same = [&](int i, int j) {
    const int4 x = __ldg(work + i), y = __ldg(work + j);
    return x.x == y.x && x.y == y.y;
  };
  int a, b;
  unit_range(p, c, a, b);
  if (a >= b || b >= n || !same(b - 1, b)) return;  // nothing, or its last one ends here
  if (a > 0 && same(a - 1, a) && same(a, b - 1)) return;  // begins in a CTA before
  const int4 w = __ldg(work + b - 1);
  int last = c;  // the CTA where it ends
  for (int end = b; end < n && same(b - 1, end);) {
    int x, y;
    unit_range(p, ++last, x, y);
    end = y;
    if (y > x && !same(b - 1, y - 1)) break;
  }
  float* to = p.d_state + (static_cast<int64_t>(w.x) * p.H + w.y) * LIN_STATE;
  const int per = LIN_STATE / 4 / gridDim.y, e0 = static_cast<int>(blockIdx.y) * per;
  for (int e = e0 + threadIdx.x; e < e0 + per; e += RD_THREADS) {
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int k = c; k <= last; ++k) {
      int x, y;
      unit_range(p, k, x, y);
      if (x >= y) continue;  // a CTA without units has left nothing
      const float4 v = __ldcg(reinterpret_cast<const float4*>(p.part + (2 * static_cast<int64_t>(k) + (k == c ? 1 : 0)) * LIN_STATE) + e);
      s.x += v.x;
      s.y += v.y;
      s.z += v.z;
      s.w += v.w;
    }
    reinterpret_cast<float4*>(to)[e] = make_float4(s.x * p.scale, s.y * p.scale, s.z * p.scale, s.w * p.scale);
  }
}

}  // namespace

int lin_read_ctas(int num_sms) { return num_sms; }

cudaError_t launch_lin_read(const LinReadParams& p, int num_sms, cudaStream_t s) {
  const int64_t ctas = p.max_units < 2 * static_cast<int64_t>(num_sms) ? p.max_units : 2 * static_cast<int64_t>(num_sms);
  lin_read_kernel<<<static_cast<unsigned>(ctas), RD_THREADS, 0, s>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_lin_read_state(const LinReadParams& p, int num_sms, cudaStream_t s) {
  constexpr int smem = 4 * RD_TILE;
  cudaError_t e = cudaFuncSetAttribute(lin_read_state_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  const unsigned ctas = static_cast<unsigned>(lin_read_ctas(num_sms));
  lin_read_state_kernel<<<ctas, RD_THREADS, smem, s>>>(p);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  lin_read_join_kernel<<<dim3(ctas, 8), RD_THREADS, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace ikbo
