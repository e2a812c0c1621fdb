// rope.cu -- rotary positions, forward and backward.
//
// Pair j of row (i, h, l) is turned by the angle pos * f_j, pos = start + l:
//   (x, y) -> m (x cos - y sin, y cos + x sin),
// and the gradient is the transpose, the same with the sine negated.  The
// start of a candidate's queries is its user's, read through the map, so
// positions stay at the user batch like the rest of the request.
//
// The angle.  A float product pos * f_j loses pos * 2^-24 radians (0.06 at a
// position of a million).  Here f_j is held as turns per position in 64-bit
// fixed point (2^64 = one turn): pos * turn[j] modulo 2^64 drops whole turns
// exactly, its top 32 bits are the angle to 2^-32 of a turn, at any position,
// for one 64-bit integer product per pair.  As a float for the sine and cosine it
// keeps 24 bits (2^-26 of a turn, 9.4e-8 radians: less than the results' own
// rounding to fp32 where x and y are of one size).
//
// Bound: memory, one read and one write of X.  A thread keeps the cosines
// and sines of eight pairs (16 elements of a row) and runs them over the
// heads of its token, so the transcendental work is shared by the heads and
// each head costs two 16-byte loads, 32 FMAs and two 16-byte stores (fp32:
// twice the loads).  Several heads' loads are issued before the first is used.
// Measured (among other calls, warm): the queries of 1024 candidates, 8 heads x 32
// tokens x 128 in bf16, 21.4 us, 6.3 TB/s; 32768 rows x 8 heads in fp32, half of
// the head turned, 44.5 us, 6.0 TB/s; one token 2.3 us.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "qcache_internal.h"

namespace ikbo {
namespace {

constexpr int ROPE_THREADS = 128;  // (256: 22.3 us for the 70:1 queries, against 21.3)

template <typename T>
struct Num;
template <>
struct Num<__nv_bfloat16> {
  static __device__ __forceinline__ float up(__nv_bfloat16 x) { return __bfloat162float(x); }
  static __device__ __forceinline__ __nv_bfloat16 down(float x) { return __float2bfloat16_rn(x); }
};
template <>
struct Num<__half> {
  static __device__ __forceinline__ float up(__half x) { return __half2float(x); }
  static __device__ __forceinline__ __half down(float x) { return __float2half_rn(x); }
};
template <>
struct Num<float> {
  static __device__ __forceinline__ float up(float x) { return x; }
  static __device__ __forceinline__ float down(float x) { return x; }
};

// Position of token l of item i; false for a candidate whose user is out of range.
__device__ __forceinline__ bool position(const RopeParams& p, int i, int l, int64_t* pos) {
  int src = i;
  if (p.map) {
    src = __ldg(p.map + i);
    if (src < 0 || src >= p.n_users) {
      atomicOr(p.status, DEV_ERR_MAP_RANGE);
      return false;
    }
  }
  *pos = (p.start ? static_cast<int64_t>(__ldg(p.start + src)) : 0) + l;
  return true;
}

// Cosine and sine of pair j's angle, times the factor.  32-bit types take the
// exact functions; for 16-bit ones the hardware's (2^-20.5 absolute on this
// range) are far below the rounding of the result, and a token with few heads
// is bound by them (one head of 200000 rows: 52 us with sincospi).
template <typename T>
__device__ __forceinline__ void turn_of(const RopeParams& p, int64_t pos, int j, float* cs, float* sn) {
  const uint64_t t = static_cast<uint64_t>(pos) * p.turn[j] + 0x80000000ull;
  const float signed_turns = static_cast<float>(static_cast<int32_t>(t >> 32));  // 2^32: one turn
  float s, c;
  if (sizeof(T) == 4) {
    sincospif(signed_turns * 4.656612873077393e-10f, &s, &c);  // 2^-31: half turns
  } else {
    const float radians = signed_turns * 1.4629180792671596e-9f;  // 2 pi 2^-32
    s = __sinf(radians);
    c = __cosf(radians);
  }
  *cs = c * p.magnitude;
  *sn = (p.backward ? -s : s) * p.magnitude;
}

// Eight elements, moved as 16-byte pieces.
template <typename T>
struct alignas(16) Vec8 {
  T v[8];
};

template <typename T>
__device__ __forceinline__ Vec8<T> load8(const T* p) {
  Vec8<T> r;
  constexpr int n = sizeof(Vec8<T>) / 16;
#pragma unroll
  for (int i = 0; i < n; ++i) reinterpret_cast<uint4*>(&r)[i] = reinterpret_cast<const uint4*>(p)[i];
  return r;
}

template <typename T>
__device__ __forceinline__ void store8(T* p, const Vec8<T>& r) {
  constexpr int n = sizeof(Vec8<T>) / 16;
#pragma unroll
  for (int i = 0; i < n; ++i) reinterpret_cast<uint4*>(p)[i] = reinterpret_cast<const uint4*>(&r)[i];
}

// Rows of 16-element pieces: rot / 16 that turn, then the rest of the head.
// rot % 16 == 0, d % 8 == 0, pointers and strides multiples of 8 elements and
// 16 bytes.
// kAhead: heads whose loads are in flight together.
template <typename T, bool kInterleaved, int kAhead>
__global__ void __launch_bounds__(ROPE_THREADS) rope_vec_kernel(const __grid_constant__ RopeParams p) {
  const int turning = p.rot >> 4;
  const int pieces = turning + (p.copy_rest ? (p.d - p.rot + 15) >> 4 : 0);
  const int rows_per_cta = ROPE_THREADS / pieces;
  const int r = static_cast<int>(threadIdx.x) / pieces;
  const int piece = static_cast<int>(threadIdx.x) - r * pieces;
  const int64_t row64 = static_cast<int64_t>(blockIdx.x) * rows_per_cta + r;
  if (r >= rows_per_cta || row64 >= static_cast<int64_t>(p.n) * p.L) return;
  const int row = static_cast<int>(row64);  // n * L is below 2^31
  const int i = row / p.L, l = row - i * p.L;
  int64_t pos;
  if (!position(p, i, l, &pos)) return;
  const int h0 = static_cast<int>(blockIdx.y) * p.heads_per_cta;
  const int h1 = min(p.H, h0 + p.heads_per_cta);
  const T* x = static_cast<const T*>(p.X) + i * p.xs[0] + l * p.xs[2] + h0 * p.xs[1];
  T* y = static_cast<T*>(p.Y) + i * p.ys[0] + l * p.ys[2] + h0 * p.ys[1];
  // the piece's two groups of eight: both members of pairs 8c .. 8c + 7
  int a = piece * 8, b = a + (p.rot >> 1);
  if (kInterleaved) a = piece * 16, b = a + 8;
  const bool turn = piece < turning;
  bool second = true;
  if (!turn) {
    a = p.rot + (piece - turning) * 16;
    b = a + 8;
    second = b < p.d;
    if (!second) b = a;
  }
  Vec8<T> va[kAhead], vb[kAhead];
  const auto fetch = [&](int h) {
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
      if (h + k < h1) {
        va[k] = load8(x + k * p.xs[1] + a);
        vb[k] = load8(x + k * p.xs[1] + b);
      }
  };
  fetch(h0);  // on their way while the angles are formed
  float cs[8], sn[8];
  if (turn) {
#pragma unroll
    for (int j = 0; j < 8; ++j) turn_of<T>(p, pos, piece * 8 + j, &cs[j], &sn[j]);
  }
  for (int h = h0; h < h1; h += kAhead) {
    if (h > h0) fetch(h);
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
      if (h + k < h1) {
        if (turn) {
          if (kInterleaved) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float x0 = Num<T>::up(va[k].v[2 * j]), y0 = Num<T>::up(va[k].v[2 * j + 1]);
              va[k].v[2 * j] = Num<T>::down(x0 * cs[j] - y0 * sn[j]);
              va[k].v[2 * j + 1] = Num<T>::down(y0 * cs[j] + x0 * sn[j]);
              const float x1 = Num<T>::up(vb[k].v[2 * j]), y1 = Num<T>::up(vb[k].v[2 * j + 1]);
              vb[k].v[2 * j] = Num<T>::down(x1 * cs[4 + j] - y1 * sn[4 + j]);
              vb[k].v[2 * j + 1] = Num<T>::down(y1 * cs[4 + j] + x1 * sn[4 + j]);
            }
          } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const float x0 = Num<T>::up(va[k].v[j]), y0 = Num<T>::up(vb[k].v[j]);
              va[k].v[j] = Num<T>::down(x0 * cs[j] - y0 * sn[j]);
              vb[k].v[j] = Num<T>::down(y0 * cs[j] + x0 * sn[j]);
            }
          }
        }
        store8(y + k * p.ys[1] + a, va[k]);
        if (second) store8(y + k * p.ys[1] + b, vb[k]);
      }
    x += kAhead * p.xs[1];
    y += kAhead * p.ys[1];
  }
}

// Any sizes and strides: a thread per pair (or element behind the rotated
// ones) of a token, over its heads.
template <typename T>
__global__ void __launch_bounds__(ROPE_THREADS) rope_any_kernel(const __grid_constant__ RopeParams p) {
  const int half = p.rot >> 1;
  const int pieces = half + (p.copy_rest ? p.d - p.rot : 0);
  const int64_t total = static_cast<int64_t>(p.n) * p.L * pieces;
  const int64_t step = static_cast<int64_t>(gridDim.x) * ROPE_THREADS;
  for (int64_t e = static_cast<int64_t>(blockIdx.x) * ROPE_THREADS + threadIdx.x; e < total; e += step) {
    const int64_t row = e / pieces;
    const int piece = static_cast<int>(e - row * pieces);
    const int i = static_cast<int>(row / p.L), l = static_cast<int>(row - static_cast<int64_t>(i) * p.L);
    int64_t pos;
    if (!position(p, i, l, &pos)) continue;
    const T* x = static_cast<const T*>(p.X) + i * p.xs[0] + l * p.xs[2];
    T* y = static_cast<T*>(p.Y) + i * p.ys[0] + l * p.ys[2];
    const int h0 = static_cast<int>(blockIdx.y) * p.heads_per_cta;
    const int h1 = min(p.H, h0 + p.heads_per_cta);
    if (piece >= half) {
      const int k = p.rot + piece - half;
      for (int h = h0; h < h1; ++h) y[h * p.ys[1] + k] = x[h * p.xs[1] + k];
      continue;
    }
    float cs, sn;
    turn_of<T>(p, pos, piece, &cs, &sn);
    const int a = p.interleaved ? 2 * piece : piece, b = p.interleaved ? a + 1 : a + half;
    for (int h = h0; h < h1; ++h) {
      const float x0 = Num<T>::up(x[h * p.xs[1] + a]), y0 = Num<T>::up(x[h * p.xs[1] + b]);
      y[h * p.ys[1] + a] = Num<T>::down(x0 * cs - y0 * sn);
      y[h * p.ys[1] + b] = Num<T>::down(y0 * cs + x0 * sn);
    }
  }
}

// Loads in flight per thread against threads per SM: one head at a time where a
// thread has only one (200000 rows of one bf16 head: 32 us, against 49 with the
// registers of four), else as many as their registers pay for (the 70:1 queries:
// 22.3 us with four, 22.8 with two, 26.2 with eight).
template <typename T, bool kInterleaved>
void launch_vec(const RopeParams& p, dim3 grid, cudaStream_t s) {
  constexpr int kMost = sizeof(T) == 4 ? 2 : 4;
  if (p.heads_per_cta == 1) rope_vec_kernel<T, kInterleaved, 1><<<grid, ROPE_THREADS, 0, s>>>(p);
  else rope_vec_kernel<T, kInterleaved, kMost><<<grid, ROPE_THREADS, 0, s>>>(p);
}

template <typename T>
cudaError_t launch(RopeParams p, bool vec, int num_sms, cudaStream_t s) {
  const int64_t rows = static_cast<int64_t>(p.n) * p.L;
  int64_t ctas;
  if (vec) {
    const int pieces = (p.rot >> 4) + (p.copy_rest ? (p.d - p.rot + 15) >> 4 : 0);
    const int per = ROPE_THREADS / pieces;
    ctas = (rows + per - 1) / per;
  } else {
    const int pieces = (p.rot >> 1) + (p.copy_rest ? p.d - p.rot : 0);
    ctas = (rows * pieces + ROPE_THREADS - 1) / ROPE_THREADS;
    if (ctas > 32 * static_cast<int64_t>(num_sms)) ctas = 32 * static_cast<int64_t>(num_sms);
  }
  if (ctas > 0x7fffffff) return cudaErrorInvalidValue;
  // one CTA takes all heads of its tokens (their angles are formed once)
  // unless that leaves SMs without work
  int parts = 1;
  while (parts < p.H && parts < 32 && ctas * parts < 4 * static_cast<int64_t>(num_sms)) parts *= 2;
  if (parts > p.H) parts = p.H;
  p.heads_per_cta = (p.H + parts - 1) / parts;
  const dim3 grid(static_cast<unsigned>(ctas), static_cast<unsigned>((p.H + p.heads_per_cta - 1) / p.heads_per_cta));
  if (!vec) rope_any_kernel<T><<<grid, ROPE_THREADS, 0, s>>>(p);
  else if (p.interleaved) launch_vec<T, true>(p, grid, s);
  else launch_vec<T, false>(p, grid, s);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rope(const RopeParams& p, int dtype, int num_sms, cudaStream_t s) {
  const int64_t elt = dtype == 2 ? 4 : 2;
  bool vec = p.rot % 16 == 0 && p.d % 8 == 0;
  for (int k = 0; k < 3; ++k) vec = vec && p.xs[k] * elt % 16 == 0 && p.ys[k] * elt % 16 == 0;
  vec = vec && reinterpret_cast<uintptr_t>(p.X) % 16 == 0 && reinterpret_cast<uintptr_t>(p.Y) % 16 == 0;
  if (dtype == 0) return launch<__nv_bfloat16>(p, vec, num_sms, s);
  if (dtype == 1) return launch<__half>(p, vec, num_sms, s);
  return launch<float>(p, vec, num_sms, s);
}

}  // namespace ikbo
