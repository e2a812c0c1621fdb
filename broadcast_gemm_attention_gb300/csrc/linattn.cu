// linattn.cu -- linear attention with a decay for each head: whole histories
// in chunks, single tokens, and the gradient.
//
//   S_t = decay S_{t-1} + k_t v_t^T,   o_t = scale q_t S_t
//
// In chunks of C rows (S the state before the chunk, i and j counted in it):
//   o_i = scale ( sum_{j <= i} decay^(i-j) (q_i.k_j) v_j + decay^(i+1) q_i S )
//   S  <- decay^n S + sum_j decay^(n-1-j) k_j v_j^T        (n rows in the chunk)
//
// The gradient of more than a few rows (of those: linback.cu) is three scans of the same kind.  With
//   R_t = sum_{i >= t} decay^(i-t) scale q_i do_i^T + decay^(T-t) dS_T,
//   dq_t = scale S_t do_t     a scan with queries do, keys v, values k,
//   dk_t = R_t v_t            from the last row on: queries v, keys do, values q,
//   dv_t = R_t^T k_t          from the last row on: queries k, keys q, values do,
// and the gradient of the first state is decay R_1, the last one's end.  So the
// kernel of lintile.cu does all of it, three jobs a launch; nothing but the inputs
// is kept from the forward pass.
#include <cuda_bf16.h>

#include <type_traits>

#include "launch.cuh"
#include "linattn_internal.h"
#include "mma_common.cuh"
#include "tile_common.cuh"

namespace ikbo {
namespace {

constexpr int LIN_CHUNK = 64;
constexpr int LIN_THREADS = 256;
constexpr int LIN_TILE = LIN_CHUNK * LIN_D * 2;  // bytes of a chunk of x, y or z
constexpr int LIN_STAGES = 2;

// decay^n, n >= 0 (decay^0 = 1 for any decay).
__device__ __forceinline__ float lin_power(float log2_decay, int n) {
  return n == 0 ? 1.f : exp2f(static_cast<float>(n) * log2_decay);
}

// The rows of user u; none, and a report, where the offsets are out of range.
__device__ __forceinline__ int lin_rows(const LinParams& p, int u, int& first) {
  if (!p.offsets) {
    const int each = p.n_rows / p.n_users;
    first = u * each;
    return each;
  }
  const int a = __ldcg(p.offsets + u), b = __ldcg(p.offsets + u + 1);
  if (a < 0 || b < a || b > p.n_rows || b - a > p.max_len) {
    if (threadIdx.x == 0) atomicOr(p.status, DEV_ERR_CACHE);
    first = 0;
    return 0;
  }
  first = a;
  return b - a;
}

// Place of 16-byte piece c of row r in a tile of 256-byte rows: eight rows' same
// pieces lie in different banks.
__device__ __forceinline__ uint32_t tile_at(int r, int c) { return static_cast<uint32_t>(r * 256 + ((c ^ (r & 7)) << 4)); }

struct LinShared {
  float power[LIN_CHUNK + 1];  // decay^n
};

// o += the rows' weights of z's rows that they read, without the matrix instruction: o's rows are `row` and row + 8, its
// columns 16 warp + 8 e + 2 t (+ 1); z's rows are those below `rows`.
__device__ __forceinline__ void one_by_one(float (&o)[2][4], uint32_t probs, uint32_t z_at, int row, int rows, int warp, int t) {
#pragma unroll 1
  for (int j = 0; j < rows; ++j) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int r = row + 8 * k;
      if (r < j) continue;
      uint16_t p;
      asm volatile("ld.shared.u16 %0, [%1];" : "=h"(p) : "r"(probs + r * 128 + (((j >> 3) ^ (r & 7)) << 4) + 2 * (j & 7)) : "memory");
      const float w = __uint_as_float(static_cast<uint32_t>(p) << 16);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        uint32_t z;
        asm volatile("ld.shared.b32 %0, [%1];" : "=r"(z) : "r"(z_at + tile_at(j, 2 * warp + e) + 4 * t) : "memory");
        o[e][2 * k] = fmaf(w, bf16_lo(z), o[e][2 * k]);
        o[e][2 * k + 1] = fmaf(w, bf16_hi(z), o[e][2 * k + 1]);
      }
    }
  }
}

// The scan in registers, for histories of a few chunks: 16x8x16 products, a CTA a scan,
// the turned state as accumulators (their layout is the next product's B operand).
// Bound: those products (603 TFLOP/s at most on this part, 117 kFLOP a row and head with
// queries) and each chunk's chain; no state to set up in tensor memory, so the shorter
// histories are its own.  Measured: the states of 15 users' 0 to 24 new rows, 8 heads,
// 5.5 us; 15 histories of 1200 to 2048 rows 142 us (lintile.cu: 52).
//
// kOutputs: with queries; else the states alone.
template <bool kOutputs>
__global__ void __launch_bounds__(LIN_THREADS, kOutputs ? 1 : 2) lin_chunk_kernel(const __grid_constant__ LinParams p) {
  wait_for_launch_before();
  extern __shared__ __align__(128) uint8_t lin_sm[];
  __shared__ LinShared sh;
  constexpr int kTiles = kOutputs ? 3 : 2;  // y, z, x
  constexpr int kStage = kTiles * LIN_TILE;
  const uint32_t base = smem_u32(lin_sm), probs = base + LIN_STAGES * kStage;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int u = static_cast<int>(blockIdx.x) / p.H, h = static_cast<int>(blockIdx.x) - u * p.H;
  const LinJob& job = p.job[0];

  int first_row;
  const int n = lin_rows(p, u, first_row);
  const float log2_decay = log2f(__ldcg(p.decay + h));
  if (tid <= LIN_CHUNK) sh.power[tid] = lin_power(log2_decay, tid);

  const int64_t row_at = first_row;
  const auto load_tile = [&](const uint16_t* src, int64_t stride, uint32_t dst, int c0) {
#pragma unroll
    for (int k = 0; k < LIN_TILE / 16 / LIN_THREADS; ++k) {
      const int i = k * LIN_THREADS + tid, r = i >> 4, c = i & 15;
      const bool there = c0 + r < n;
      copy16(dst + tile_at(r, c), there ? src + (row_at + c0 + r) * stride + h * LIN_D + c * 8 : src, there);
    }
  };
  const auto load_stage = [&](int stage, int c0) {
    const uint32_t at = base + stage * kStage;
    load_tile(job.y, job.ys, at, c0);
    load_tile(job.z, job.zs, at + LIN_TILE, c0);
    if (kOutputs) load_tile(job.x, job.xs, at + 2 * LIN_TILE, c0);
  };
  const int chunks = (n + LIN_CHUNK - 1) / LIN_CHUNK;
  if (chunks > 0) load_stage(0, 0);
  copies_commit();

  // the state, turned: row m of s[i] is z's element 16 warp + m, columns y's 8 i ..
  float s[16][4];
  const int64_t state = (static_cast<int64_t>(u) * p.H + h) * LIN_STATE;
  const float* from = job.s_in ? job.s_in + state : nullptr;
  // the start of a scan that begins when this one ends, to L2 (400 users of 24 rows 150 -> 130 us, of 64 191 -> 165)
  const int64_t later = static_cast<int64_t>(blockIdx.x) + p.ahead;
  if (job.s_in && tid == 0 && later < static_cast<int64_t>(p.n_users) * p.H)
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(job.s_in + later * LIN_STATE), "n"(LIN_STATE * 4) : "memory");
  const int e0 = 16 * warp + g;
#pragma unroll
  for (int i = 0; i < 16; ++i)
#pragma unroll
    for (int k = 0; k < 4; ++k) s[i][k] = from ? __ldcg(from + (8 * i + 2 * t + (k & 1)) * LIN_D + e0 + 8 * (k >> 1)) : 0.f;

#pragma unroll 1
  for (int ch = 0; ch < chunks; ++ch) {
    const int c0 = ch * LIN_CHUNK, rows = min(LIN_CHUNK, n - c0);
    if (ch + 1 < chunks) load_stage((ch + 1) & 1, c0 + LIN_CHUNK);
    copies_commit();
    copies_wait<1>();
    __syncthreads();
    const uint32_t y_at = base + (ch & 1) * kStage, z_at = y_at + LIN_TILE, x_at = y_at + 2 * LIN_TILE;
    if (kOutputs) {
      // A = x y^T with decay^(i-j), rows 16 (warp / 2) .., columns 32 (warp % 2) .., to shared memory
      const int rb = 16 * (warp >> 1), cb = 32 * (warp & 1);
      if (cb <= rb + 15) {
        float a[4][4] = {};
#pragma unroll
        for (int kk = 0; kk < 8; ++kk) {
          uint32_t xf[4];
          ldsm4(xf, x_at + tile_at(rb + (lane & 15), 2 * kk + (lane >> 4)));
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            uint32_t yf[4];
            ldsm4(yf, y_at + tile_at(cb + 16 * half + (lane & 7) + 8 * (lane >> 4), 2 * kk + ((lane >> 3) & 1)));
            mma_16816(a[2 * half], xf, yf[0], yf[1]);
            mma_16816(a[2 * half + 1], xf, yf[2], yf[3]);
          }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const int row = rb + g + 8 * k, gap = row - (cb + 8 * i + 2 * t);
            const float w0 = gap >= 0 ? a[i][2 * k] * sh.power[gap] : 0.f;
            const float w1 = gap >= 1 ? a[i][2 * k + 1] * sh.power[gap - 1] : 0.f;
            const int piece = (cb >> 3) + i;
            asm volatile("st.shared.b32 [%0], %1;" ::"r"(probs + row * 128 + ((piece ^ (row & 7)) << 4) + 4 * t), "r"(pack_bf16x2(w0, w1))
                         : "memory");
          }
      }
      __syncthreads();
    }
    // z's columns 16 warp .. of 16 rows each: A of the state's product, B of the outputs'
    uint32_t zf[4][4];
#pragma unroll
    for (int kb = 0; kb < 4; ++kb)  // matrices: (columns 0-7, rows 0-7), (8-15, 0-7), (0-7, 8-15), (8-15, 8-15)
      ldsm4_t(zf[kb], z_at + tile_at(16 * kb + (lane & 7) + 8 * (lane >> 4), 2 * warp + ((lane >> 3) & 1)));
    if (kOutputs) {
      // z's infinities and NaN would reach rows that do not read them in the product, as 0 times infinity: such chunks go
      // without it.  (Looking for them, 400 users' 24 rows 129.5 -> 131.5 us, 128 rows 245 -> 249; a branch at each product 251.)
      uint32_t odd = 0;
#pragma unroll
      for (int kb = 0; kb < 4; ++kb) odd |= times_zero(zf[kb]);
      const bool any_odd = __any_sync(0xffffffffu, (odd & 0x7fff7fffu) != 0);
      uint32_t sb[16][2];
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        sb[i][0] = pack_bf16x2(s[i][0], s[i][1]);
        sb[i][1] = pack_bf16x2(s[i][2], s[i][3]);
      }
      const auto outputs = [&](auto kOdd) {
#pragma unroll
        for (int mt = 0; mt < 4; ++mt) {
          if (16 * mt >= rows) break;
          float o[2][4] = {};
#pragma unroll
          for (int kk = 0; kk < 8; ++kk) {
            uint32_t xf[4];
            ldsm4(xf, x_at + tile_at(16 * mt + (lane & 15), 2 * kk + (lane >> 4)));
            mma_16816(o[0], xf, sb[2 * kk][0], sb[2 * kk + 1][0]);
            mma_16816(o[1], xf, sb[2 * kk][1], sb[2 * kk + 1][1]);
          }
          const int row = 16 * mt + g;
          const float w0 = sh.power[row + 1], w1 = sh.power[row + 9];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            o[e][0] *= w0;
            o[e][1] *= w0;
            o[e][2] *= w1;
            o[e][3] *= w1;
          }
          if constexpr (kOdd.value) {
            one_by_one(o, probs, z_at, row, min(rows, 16 * mt + 16), warp, t);
          } else {
#pragma unroll
            for (int kb = 0; kb <= mt; ++kb) {
              uint32_t pf[4];
              const int r = 16 * mt + (lane & 15);
              ldsm4(pf, probs + r * 128 + (((2 * kb + (lane >> 4)) ^ (r & 7)) << 4));
              mma_16816(o[0], pf, zf[kb][0], zf[kb][2]);
              mma_16816(o[1], pf, zf[kb][1], zf[kb][3]);
            }
          }
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const int r = row + 8 * k;
            if (r >= rows) continue;
            uint16_t* dst = job.out + (row_at + c0 + r) * job.os + h * LIN_D + 16 * warp + 2 * t;
            *reinterpret_cast<uint32_t*>(dst) = pack_bf16x2(o[0][2 * k] * p.scale, o[0][2 * k + 1] * p.scale);
            *reinterpret_cast<uint32_t*>(dst + 8) = pack_bf16x2(o[1][2 * k] * p.scale, o[1][2 * k + 1] * p.scale);
          }
        }
      };
      if (any_odd) outputs(std::true_type());
      else outputs(std::false_type());
    }
    // the state: decayed, and z^T y with each row's decay on z, to 16 bits of mantissa
    const float down = sh.power[rows];
#pragma unroll
    for (int i = 0; i < 16; ++i)
#pragma unroll
      for (int k = 0; k < 4; ++k) s[i][k] *= down;
#pragma unroll
    for (int kb = 0; kb < 4; ++kb) {
      if (16 * kb >= rows) break;
      uint32_t hi[4], lo[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int j = rows - 1 - (16 * kb + 2 * t + 8 * (k >> 1));
        split_bf16x2(bf16_lo(zf[kb][k]) * sh.power[max(j, 0)], bf16_hi(zf[kb][k]) * sh.power[max(j - 1, 0)], hi[k], lo[k]);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        uint32_t yf[4];
        ldsm4_t(yf, y_at + tile_at(16 * kb + (lane & 15), 2 * i + (lane >> 4)));
        mma_16816(s[2 * i], hi, yf[0], yf[1]);
        mma_16816(s[2 * i + 1], hi, yf[2], yf[3]);
        mma_16816(s[2 * i], lo, yf[0], yf[1]);
        mma_16816(s[2 * i + 1], lo, yf[2], yf[3]);
      }
    }
    __syncthreads();  // the stage is loaded again
  }

  float* to = job.s_out ? job.s_out + state : nullptr;
  if (!to) return;
#pragma unroll
  for (int i = 0; i < 16; ++i)
#pragma unroll
    for (int k = 0; k < 4; ++k) to[(8 * i + 2 * t + (k & 1)) * LIN_D + e0 + 8 * (k >> 1)] = s[i][k];
}

constexpr int JOIN_AHEAD = 32;  // parts on their way at a time

// The states at the segments' ends, from the segments' own parts (in the last
// one's place, which has no part, the start).  Bound: latency; a user's parts are
// on their way together (by eights two users' 20000 and 30001 rows, 4 heads, 83.9 us, so 82.9).
__global__ void __launch_bounds__(256) lin_join_kernel(const __grid_constant__ LinParams p) {
  wait_for_launch_before();
  constexpr int kParts = LIN_STATE / 256;
  const int item = static_cast<int>(blockIdx.x) / kParts;
  const int u = item / p.H, h = item - u * p.H;
  const LinJob& job = p.job[blockIdx.y];
  int first;
  const int len = lin_rows(p, u, first);
  const int segs = max(1, (len + p.seg_len - 1) / p.seg_len);
  if (segs == 1) return;
  const int e = (static_cast<int>(blockIdx.x) - item * kParts) * 256 + threadIdx.x;
  const int64_t state = (static_cast<int64_t>(u) * p.H + h) * LIN_STATE;
  float* ws = p.ws + ((static_cast<int64_t>(blockIdx.y) * p.n_users + u) * p.H + h) * p.segs * LIN_STATE + e;
  float s = 0.f;
  if (job.s_in) s = job.s_in[state + (job.s_in_turned ? (e % LIN_D) * LIN_D + e / LIN_D : e)];
  ws[static_cast<int64_t>(segs - 1) * LIN_STATE] = s;
  const float log2_decay = log2f(__ldcg(p.decay + h));
  const float down = lin_power(log2_decay, p.seg_len);
  s *= job.reverse ? lin_power(log2_decay, p.seg_len - 1) : down;
#pragma unroll 1
  for (int k0 = 0; k0 + 1 < segs; k0 += JOIN_AHEAD) {
    float part[JOIN_AHEAD];
#pragma unroll
    for (int k = 0; k < JOIN_AHEAD; ++k) part[k] = k0 + k + 1 < segs ? __ldcg(ws + static_cast<int64_t>(k0 + k) * LIN_STATE) : 0.f;
#pragma unroll
    for (int k = 0; k < JOIN_AHEAD; ++k) {
      if (k0 + k + 1 >= segs) break;
      s += part[k];
      ws[static_cast<int64_t>(k0 + k) * LIN_STATE] = s;
      s *= down;
    }
  }
}

// Few rows a user: the state through registers once, a row at a time.  A warp
// has 16 of the state's rows (y's elements), a lane 4 of its columns; x, y and z
// come as fp32 through shared memory, 16 rows of them at a time.
// Bound: memory, the state read and written.  One row for each of 256 users, 8 heads:
// 41.9 us, 6.4 TB/s, 0.97 of a plain copy's rate.
constexpr int STEP_ROWS = 16;

template <bool kOutputs>
__global__ void __launch_bounds__(LIN_THREADS) lin_step_kernel(const __grid_constant__ LinParams p) {
  wait_for_launch_before();
  __shared__ float4 rows[kOutputs ? 3 : 2][STEP_ROWS][LIN_D / 4];  // y, z, x
  __shared__ float part[2][8][LIN_D];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int u = static_cast<int>(blockIdx.x) / p.H, h = static_cast<int>(blockIdx.x) - u * p.H;
  const LinJob& job = p.job[0];
  int first;
  const int len = lin_rows(p, u, first);
  const int64_t state = (static_cast<int64_t>(u) * p.H + h) * LIN_STATE;
  float* to = job.s_out ? job.s_out + state : nullptr;
  const float* from = job.s_in ? job.s_in + state : nullptr;
  if (len == 0 && (!to || to == from)) return;
  float4 s[16];
#pragma unroll
  for (int k = 0; k < 16; ++k)
    s[k] = from ? __ldcg(reinterpret_cast<const float4*>(from) + (16 * warp + k) * 32 + lane) : make_float4(0.f, 0.f, 0.f, 0.f);
  const float decay = __ldcg(p.decay + h);
#pragma unroll 1
  for (int r0 = 0; r0 < len; r0 += STEP_ROWS) {
    const int n = min(STEP_ROWS, len - r0);
    if (r0 > 0) __syncthreads();
    for (int i = tid; i < n * 16 * (kOutputs ? 3 : 2); i += LIN_THREADS) {  // 16-byte pieces
      const int t = i / (16 * n), r = (i - t * 16 * n) >> 4, c = i & 15;
      const uint16_t* src = t == 0 ? job.y : (t == 1 ? job.z : job.x);
      const int64_t stride = t == 0 ? job.ys : (t == 1 ? job.zs : job.xs);
      const uint4 v = *reinterpret_cast<const uint4*>(src + (static_cast<int64_t>(first) + r0 + r) * stride + h * LIN_D + 8 * c);
      rows[t][r][2 * c] = make_float4(bf16_lo(v.x), bf16_hi(v.x), bf16_lo(v.y), bf16_hi(v.y));
      rows[t][r][2 * c + 1] = make_float4(bf16_lo(v.z), bf16_hi(v.z), bf16_lo(v.w), bf16_hi(v.w));
    }
    __syncthreads();
#pragma unroll 1
    for (int r = 0; r < n; ++r) {
      const float4 z = rows[1][r][lane];
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float4 yv = rows[0][r][4 * warp + q], xv = kOutputs ? rows[kOutputs ? 2 : 0][r][4 * warp + q] : yv;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float y = e == 0 ? yv.x : (e == 1 ? yv.y : (e == 2 ? yv.z : yv.w));
          float4& v = s[4 * q + e];
          mul2(v.x, v.y, v.x, v.y, decay, decay);
          mul2(v.z, v.w, v.z, v.w, decay, decay);
          fma2v(v.x, v.y, z.x, z.y, y, v.x, v.y);
          fma2v(v.z, v.w, z.z, z.w, y, v.z, v.w);
          if (kOutputs) {
            const float x = e == 0 ? xv.x : (e == 1 ? xv.y : (e == 2 ? xv.z : xv.w));
            fma2v(o.x, o.y, v.x, v.y, x, o.x, o.y);
            fma2v(o.z, o.w, v.z, v.w, x, o.z, o.w);
          }
        }
      }
      if (kOutputs) {
        reinterpret_cast<float4*>(part[r & 1][warp])[lane] = o;
        __syncthreads();  // (the other half is written next)
        if (tid < LIN_D) {
          float sum = 0.f;
#pragma unroll
          for (int w = 0; w < 8; ++w) sum += part[r & 1][w][tid];
          reinterpret_cast<__nv_bfloat16*>(job.out)[(static_cast<int64_t>(first) + r0 + r) * job.os + h * LIN_D + tid] =
              __float2bfloat16_rn(sum * p.scale);
        }
      }
    }
  }
  if (!to) return;
#pragma unroll
  for (int k = 0; k < 16; ++k) reinterpret_cast<float4*>(to)[(16 * warp + k) * 32 + lane] = s[k];
}

template <bool kOutputs>
cudaError_t launch_chunks(const LinParams& p, cudaStream_t s) {
  constexpr int smem = LIN_STAGES * (kOutputs ? 3 : 2) * LIN_TILE + (kOutputs ? LIN_CHUNK * LIN_CHUNK * 2 : 0);
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = allow_smem(lin_chunk_kernel<kOutputs>, smem, done);
  if (e != cudaSuccess) return e;
  return launch_behind(lin_chunk_kernel<kOutputs>, dim3(static_cast<unsigned>(p.n_users * p.H)), LIN_THREADS, smem, s, p);
}

}  // namespace

cudaError_t launch_lin_tiles(const LinParams& p, bool local, int num_sms, cudaStream_t s);

// Launches: one, or three where histories are cut into segments (two users' 20000
// and 30001 rows 84.6 us).
cudaError_t launch_linattn(const LinParams& p, int num_sms, cudaStream_t s, int* launches) {
  *launches = 0;
  const bool outputs = p.job[0].x != nullptr;
  cudaError_t e;
  if (p.steps) {
    const unsigned grid = static_cast<unsigned>(p.n_users * p.H);
    *launches = 1;
    return outputs ? launch_behind(lin_step_kernel<true>, dim3(grid), LIN_THREADS, 0, s, p)
                   : launch_behind(lin_step_kernel<false>, dim3(grid), LIN_THREADS, 0, s, p);
  }
  if (p.segs > 1) {
    e = launch_lin_tiles(p, true, num_sms, s);
    if (e != cudaSuccess) return e;
    const dim3 grid(static_cast<unsigned>(LIN_STATE / 256 * p.n_users * p.H), static_cast<unsigned>(p.n_jobs));
    e = launch_behind(lin_join_kernel, grid, 256, 0, s, p);
    if (e != cudaSuccess) return e;
    *launches += 2;
  }
  if (p.tiles) e = launch_lin_tiles(p, false, num_sms, s);
  else e = outputs ? launch_chunks<true>(p, s) : launch_chunks<false>(p, s);
  *launches += e == cudaSuccess;
  return e;
}

}  // namespace ikbo
