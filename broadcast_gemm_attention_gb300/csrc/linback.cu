// linback.cu -- the gradient of linear attention for a few rows a user, in one pass:
// each state is read once and each gradient written once (three scans, as longer
// histories have them, read the last state's gradient twice and start three CTAs).
//
// For a block of rows 0 .. n - 1, S the state before it and R the gradient of the
// state behind it,
//   dq_t = scale ( decay^(t+1) S do_t + sum_{j <= t} decay^(t-j) (do_t.v_j) k_j )
//   dk_t = decay^(n-1-t) R v_t   + scale sum_{i >= t} decay^(i-t) (v_t.do_i) q_i
//   dv_t = decay^(n-1-t) R^T k_t + scale sum_{i >= t} decay^(i-t) (k_t.q_i) do_i
//   S <- decay^n S + sum_j decay^(n-1-j) k_j v_j^T
//   R <- decay^n R + scale sum_i decay^(i+1) q_i do_i^T
// S goes from the first block to the last, then R from the last to the first.
//
// A CTA has one (user, head), a warp 16 of the state's rows as accumulators of 16x8x16
// products in fp32.  Rounded to bf16 they are the B operand of S do_t and R v_t as they
// lie, and turned by 8x8 blocks that of R^T k_t, whose sums over the warps' rows go
// through shared memory.  What is added to a state goes in as two bf16 parts (2^-17).
// Columns are taken in an order in which a lane's are four neighbours (16 bytes of a
// row): the order of the inner dimension is free, and v and do lie in it too.
// What rows read of each other is rounded to bf16, with its decay, as the longer
// histories' is; sums and states are fp32.
//
// Bound: memory, with two CTAs on an SM whose chains (5.4 us alone) take turns.
// 400 users, 8 heads: 16 rows 153 us, 4.4 TB/s (three scans in registers 348), one row
// 132 (334); 15 users of 16 rows 8.7 us (14.6).  With the vector units and one row after
// the other one row took 93, 4 rows 113 (for 134), 8 rows 171 (138), 16 rows 346.
#include <cuda_bf16.h>

#include "launch.cuh"
#include "linattn_internal.h"
#include "mma_common.cuh"

namespace ikbo {
namespace {

constexpr int LB_THREADS = 256;
constexpr int LB_ROWS = 16;                       // of a block
constexpr int LB_TILE = LB_ROWS * LIN_D * 2;      // bytes of a block of q, k, v or do
constexpr int LB_ASK = 128;                       // rows asked for at once
constexpr int LB_SUM = LIN_D + 8;                 // (rows of sums eight banks apart)
enum { LB_Q, LB_K, LB_V, LB_DO };

struct BackShared {
  uint8_t rows[4][LB_TILE];
  float sums[8][LB_ROWS][LB_SUM];  // R^T k_t over a warp's rows
  float power[LB_ROWS + 1];        // decay^n
  int odd;                         // some row so far holds an infinity or NaN
};

__device__ __forceinline__ uint32_t place(int r, int c) { return static_cast<uint32_t>(r * 256 + ((c ^ (r & 7)) << 4)); }

__device__ __forceinline__ int user_rows(const LinBackParams& p, int u, int& first) {
  if (!p.offsets) {
    const int each = p.n_rows / p.n_users;
    first = u * each;
    return each;
  }
  const int a = __ldcg(p.offsets + u), b = __ldcg(p.offsets + u + 1);
  first = a;
  if (a >= 0 && b >= a && b <= p.n_rows && b - a <= p.max_len) return b - a;
  if (threadIdx.x == 0) atomicOr(p.status, DEV_ERR_CACHE);
  first = 0;
  return 0;
}

// Rows first .. first + n - 1 of the four, zeros behind them.  v's and do's pairs of each 16
// columns: 0 2 4 6 1 3 5 7.  Notes where one holds an infinity or NaN.
__device__ __forceinline__ void load_rows(const LinBackParams& p, BackShared& sh, int64_t first, int n, int h) {
  uint32_t odd = 0;  // 0 times all of them
#pragma unroll
  for (int i = threadIdx.x; i < 4 * LB_ROWS * 8; i += LB_THREADS) {
    const int t = i >> 7, r = (i >> 3) & 15, c = i & 7;
    const uint16_t* src = t == LB_Q ? p.q : (t == LB_K ? p.k : (t == LB_V ? p.v : p.d_o));
    const int64_t stride = t == LB_Q ? p.qs : (t == LB_K ? p.ks : (t == LB_V ? p.vs : p.d_os));
    uint4 a = {}, b = {};
    if (r < n) {
      const uint4* from = reinterpret_cast<const uint4*>(src + (first + r) * stride + h * LIN_D) + 2 * c;
      a = __ldcg(from);
      b = __ldcg(from + 1);
    }
    odd |= times_zero(a) | times_zero(b);
    const bool mixed = t >= LB_V;
    *reinterpret_cast<uint4*>(sh.rows[t] + place(r, 2 * c)) = mixed ? make_uint4(a.x, a.z, b.x, b.z) : a;
    *reinterpret_cast<uint4*>(sh.rows[t] + place(r, 2 * c + 1)) = mixed ? make_uint4(a.y, a.w, b.y, b.w) : b;
  }
  if (odd & 0x7fff7fffu) sh.odd = 1;
}

// s[2 i], s[2 i + 1]: a lane's rows 16 warp + g (+ 8), columns 16 i + 4 t .. + 3.
__device__ __forceinline__ void load_state(float (&s)[16][4], const float* from, int row, int t) {
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      if (from) v = __ldcg(reinterpret_cast<const float4*>(from + (row + 8 * k) * LIN_D + 16 * i + 4 * t));
      s[2 * i][2 * k] = v.x;
      s[2 * i][2 * k + 1] = v.y;
      s[2 * i + 1][2 * k] = v.z;
      s[2 * i + 1][2 * k + 1] = v.w;
    }
}

// s <- down s + sum_r w_r a_r b_r^T
__device__ __forceinline__ void add_rows(float (&s)[16][4], uint32_t a_at, uint32_t b_at, float down, const float (&w)[4], int warp, int lane) {
#pragma unroll
  for (int i = 0; i < 16; ++i)
#pragma unroll
    for (int k = 0; k < 4; ++k) s[i][k] *= down;
  uint32_t a[4], hi[4], lo[4];
  ldsm4_t(a, a_at + place((lane & 7) + 8 * (lane >> 4), 2 * warp + ((lane >> 3) & 1)));
#pragma unroll
  for (int k = 0; k < 4; ++k) split_bf16x2(bf16_lo(a[k]) * w[k & 2], bf16_hi(a[k]) * w[(k & 2) + 1], hi[k], lo[k]);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    uint32_t b[4];
    ldsm4_t(b, b_at + place(lane & 15, 2 * i + (lane >> 4)));
    mma_16816(s[2 * i], hi, b[0], b[1]);
    mma_16816(s[2 * i + 1], hi, b[2], b[3]);
    mma_16816(s[2 * i], lo, b[0], b[1]);
    mma_16816(s[2 * i + 1], lo, b[2], b[3]);
  }
}

// c = X S^T for the warp's 16 columns (rows of the state), d = X Y^T.
__device__ __forceinline__ void times(float (&c)[2][4], float (&d)[2][4], const float (&s)[16][4], uint32_t x_at, uint32_t y_at, int lane) {
#pragma unroll
  for (int kk = 0; kk < 8; ++kk) {
    uint32_t x[4], y[4];
    ldsm4(x, x_at + place(lane & 15, 2 * kk + (lane >> 4)));
    ldsm4(y, y_at + place((lane & 7) + 8 * (lane >> 4), 2 * kk + ((lane >> 3) & 1)));
    mma_16816(c[0], x, pack_bf16x2(s[2 * kk][0], s[2 * kk][1]), pack_bf16x2(s[2 * kk + 1][0], s[2 * kk + 1][1]));
    mma_16816(c[1], x, pack_bf16x2(s[2 * kk][2], s[2 * kk][3]), pack_bf16x2(s[2 * kk + 1][2], s[2 * kk + 1][3]));
    mma_16816(d[0], x, y[0], y[1]);
    mma_16816(d[1], x, y[2], y[3]);
  }
}

// c <- w c + P Y for the warp's 16 columns of Y, P = scale d with its rows' decays to each other, rounded to bf16:
// row t reads rows up to t, or (later) from t on.  odd: Y may hold infinities and NaN, which in the product would reach rows
// that do not read them, as 0 times infinity.  They stay out of it, a second product counts how many of them each
// row reads, and where that is any the result is NaN.  (Looking for them where rows are loaded takes 1 to 2%: 400 users' 16 rows
// 151.2 -> 152.8 us, 64 rows 418 -> 425; where each product takes them 6%.)
__device__ __forceinline__ void among(float (&c)[2][4], const float (&d)[2][4], const float* power, float w0, float w1, float scale, bool later,
                                      uint32_t y_at, int piece, int lane, bool odd) {
  const int g = lane >> 2, t = lane & 3;
  uint32_t pr[4], y[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {  // rows g, g + 8 (k odd), columns 8 (k / 2) + 2 t ..
    const int row = g + 8 * (k & 1), col = 8 * (k >> 1) + 2 * t, gap = later ? col - row : row - col, next = later ? gap + 1 : gap - 1;
    pr[k] = pack_bf16x2(gap >= 0 ? d[k >> 1][2 * (k & 1)] * power[gap] * scale : 0.f,
                        next >= 0 ? d[k >> 1][2 * (k & 1) + 1] * power[next] * scale : 0.f);
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    c[i][0] *= w0;
    c[i][1] *= w0;
    c[i][2] *= w1;
    c[i][3] *= w1;
  }
  ldsm4_t(y, y_at + place(lane & 15, piece + (lane >> 4)));
  if (!odd) {
    mma_16816(c[0], pr, y[0], y[1]);
    mma_16816(c[1], pr, y[2], y[3]);
    return;
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    float bad[4] = {};
    uint32_t reads[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int row = g + 8 * (k & 1), col = 8 * (k >> 1) + 2 * t, gap = later ? col - row : row - col, next = later ? gap + 1 : gap - 1;
      reads[k] = (gap >= 0 ? 0x3f80u : 0u) | (next >= 0 ? 0x3f800000u : 0u);
    }
    mma_16816(bad, reads, odd_ones(y[2 * i]), odd_ones(y[2 * i + 1]));
    mma_16816(c[i], pr, finite_part(y[2 * i]), finite_part(y[2 * i + 1]));
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (bad[k] > 0.f) c[i][k] = __int_as_float(0x7fffffff);
  }
}

// Asks for a state in L2.
__device__ __forceinline__ void ask(const float* state) {
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(state), "n"(LIN_STATE * 4) : "memory");
}

__global__ void __launch_bounds__(LB_THREADS, 2) lin_back_kernel(const __grid_constant__ LinBackParams p) {
  wait_for_launch_before();
  extern __shared__ __align__(128) uint8_t raw[];
  BackShared& sh = *reinterpret_cast<BackShared*>(raw);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int u = static_cast<int>(blockIdx.x) / p.H, h = static_cast<int>(blockIdx.x) - u * p.H;
  const uint32_t q_at = smem_u32(sh.rows[LB_Q]), k_at = smem_u32(sh.rows[LB_K]), v_at = smem_u32(sh.rows[LB_V]), do_at = smem_u32(sh.rows[LB_DO]);
  const int64_t state = (static_cast<int64_t>(u) * p.H + h) * LIN_STATE;
  float s[16][4];
  if (p.dq) load_state(s, p.s_in ? p.s_in + state : nullptr, 16 * warp + g, t);
  int first;
  const int len = user_rows(p, u, first);
  const bool behind = p.dk || p.dv || p.ds_in, before = p.dq && len > 0;
  // on their way to L2: this scan's other state, and the first of one that begins later (400 users' 16 rows
  // 157 -> 150 us; of the one after that 153)
  if (before && behind && p.ds_out && tid == 0) ask(p.ds_out + state);
  const int64_t later = static_cast<int64_t>(blockIdx.x) + p.ahead;
  const float* start = p.dq ? p.s_in : p.ds_out;
  if (start && later < static_cast<int64_t>(p.n_users) * p.H && tid == 32) ask(start + later * LIN_STATE);
  // later blocks' rows too, a 128-byte line a thread (400 users' 24 rows 246 -> 229 us, 64 rows 428 -> 417)
  for (int i = LB_ROWS * 8 + tid; i < min(len, LB_ASK) * 8; i += LB_THREADS) {
    const int of = (i >> 1) & 3;
    const uint16_t* src = of == LB_Q ? p.q : (of == LB_K ? p.k : (of == LB_V ? p.v : p.d_o));
    const int64_t stride = of == LB_Q ? p.qs : (of == LB_K ? p.ks : (of == LB_V ? p.vs : p.d_os));
    asm volatile("prefetch.global.L2 [%0];" ::"l"(src + (static_cast<int64_t>(first) + (i >> 3)) * stride + h * LIN_D + 64 * (i & 1)) : "memory");
  }
  const float decay = __ldcg(p.decay + h);
  if (tid == 0) sh.odd = 0;
  __syncthreads();
  const float log2_decay = log2f(decay);
  if (tid <= LB_ROWS) sh.power[tid] = tid == 0 ? 1.f : exp2f(static_cast<float>(tid) * log2_decay);
  const auto power = [&](int n) { return n >= 0 ? sh.power[n] : 0.f; };
#pragma unroll 1
  for (int r0 = 0; r0 < len && before; r0 += LB_ROWS) {
    const int n = min(LB_ROWS, len - r0);
    load_rows(p, sh, static_cast<int64_t>(first) + r0, n, h);
    __syncthreads();
    const bool odd = sh.odd != 0;
    float c[2][4] = {}, d[2][4] = {};
    times(c, d, s, do_at, v_at, lane);
    among(c, d, sh.power, sh.power[g + 1] * p.scale, sh.power[g + 9] * p.scale, p.scale, false, k_at, 2 * warp, lane, odd);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      if (g + 8 * k >= n) continue;
      uint16_t* dst = p.dq + (static_cast<int64_t>(first) + r0 + g + 8 * k) * p.dqs + h * LIN_D + 16 * warp + 2 * t;
      *reinterpret_cast<uint32_t*>(dst) = pack_bf16x2(c[0][2 * k], c[0][2 * k + 1]);
      *reinterpret_cast<uint32_t*>(dst + 8) = pack_bf16x2(c[1][2 * k], c[1][2 * k + 1]);
    }
    if (r0 + n < len) {
      const int j = n - 1 - 2 * t;
      add_rows(s, k_at, v_at, sh.power[n], {power(j), power(j - 1), power(j - 8), power(j - 9)}, warp, lane);
      __syncthreads();
    }
  }
  if (!behind) return;
  load_state(s, p.ds_out ? p.ds_out + state : nullptr, 16 * warp + g, t);
#pragma unroll 1
  for (int r0 = (len - 1) / LB_ROWS * LB_ROWS; r0 >= 0 && len > 0; r0 -= LB_ROWS) {
    const int n = min(LB_ROWS, len - r0);
    const int64_t row0 = static_cast<int64_t>(first) + r0;
    __syncthreads();
    if (!before || len > LB_ROWS) {
      load_rows(p, sh, row0, n, h);
      __syncthreads();
    }
    const bool odd = sh.odd != 0;
    const float w0 = power(n - 1 - g), w1 = power(n - 9 - g);
    if (p.dk) {
      float c[2][4] = {}, d[2][4] = {};
      times(c, d, s, v_at, do_at, lane);
      among(c, d, sh.power, w0, w1, p.scale, true, q_at, 2 * warp, lane, odd);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        if (g + 8 * k >= n) continue;
        uint16_t* dst = p.dk + (row0 + g + 8 * k) * p.dks + h * LIN_D + 16 * warp + 2 * t;
        *reinterpret_cast<uint32_t*>(dst) = pack_bf16x2(c[0][2 * k], c[0][2 * k + 1]);
        *reinterpret_cast<uint32_t*>(dst + 8) = pack_bf16x2(c[1][2 * k], c[1][2 * k + 1]);
      }
    }
    if (p.dv) {
      uint32_t kf[4];
      ldsm4(kf, k_at + place(lane & 15, 2 * warp + (lane >> 4)));
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        float c[4] = {};
        mma_16816(c, kf, turn8x8(pack_bf16x2(s[i][0], s[i][1])), turn8x8(pack_bf16x2(s[i][2], s[i][3])));
        *reinterpret_cast<float2*>(&sh.sums[warp][g][8 * i + 2 * t]) = make_float2(c[0], c[1]);
        if (n > 8) *reinterpret_cast<float2*>(&sh.sums[warp][g + 8][8 * i + 2 * t]) = make_float2(c[2], c[3]);
      }
      __syncthreads();
      float c[2][4] = {}, d[2][4] = {};
#pragma unroll
      for (int kk = 0; kk < 8; ++kk) {
        uint32_t x[4], y[4];
        ldsm4(x, k_at + place(lane & 15, 2 * kk + (lane >> 4)));
        ldsm4(y, q_at + place((lane & 7) + 8 * (lane >> 4), 2 * kk + ((lane >> 3) & 1)));
        mma_16816(d[0], x, y[0], y[1]);
        mma_16816(d[1], x, y[2], y[3]);
      }
#pragma unroll
      for (int w = 0; w < 8; ++w)
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            if (8 * k >= n) continue;
            const float2 v = *reinterpret_cast<const float2*>(&sh.sums[w][g + 8 * k][16 * warp + 8 * i + 2 * t]);
            c[i][2 * k] += v.x;
            c[i][2 * k + 1] += v.y;
          }
      among(c, d, sh.power, w0, w1, p.scale, true, do_at, 2 * warp, lane, odd);
#pragma unroll
      for (int k = 0; k < 2; ++k)
        if (g + 8 * k < n)
          *reinterpret_cast<uint2*>(p.dv + (row0 + g + 8 * k) * p.dvs + h * LIN_D + 16 * warp + 4 * t) =
              make_uint2(pack_bf16x2(c[0][2 * k], c[0][2 * k + 1]), pack_bf16x2(c[1][2 * k], c[1][2 * k + 1]));
    }
    if (r0 > 0 || p.ds_in) {
      const auto weight = [&](int i) { return i < n ? sh.power[i + 1] * p.scale : 0.f; };
      add_rows(s, q_at, do_at, sh.power[n], {weight(2 * t), weight(2 * t + 1), weight(2 * t + 8), weight(2 * t + 9)}, warp, lane);
    }
  }
  if (!p.ds_in) return;
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int k = 0; k < 2; ++k)
      *reinterpret_cast<float4*>(p.ds_in + state + (16 * warp + g + 8 * k) * LIN_D + 16 * i + 4 * t) =
          make_float4(s[2 * i][2 * k], s[2 * i][2 * k + 1], s[2 * i + 1][2 * k], s[2 * i + 1][2 * k + 1]);
}

}  // namespace

cudaError_t launch_linattn_back(LinBackParams p, int num_sms, cudaStream_t s) {
  p.ahead = num_sms;
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = allow_smem(lin_back_kernel, sizeof(BackShared), done);
  if (e != cudaSuccess) return e;
  return launch_behind(lin_back_kernel, dim3(static_cast<unsigned>(p.n_users * p.H)), LB_THREADS, sizeof(BackShared), s, p);
}

}  // namespace ikbo
