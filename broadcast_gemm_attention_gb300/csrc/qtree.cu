// qtree.cu -- the drafted rows' part of attention over a tree of drafted tokens.
//
// Row l of candidate i's draft reads its user's history, its ancestors in the
// draft and itself.  The history's part is the cache attention's
// (ikbo_attn_qcache_forward), whose O and log-sum-exp this kernel goes on from:
// with m the running maximum, a row begins at
//   m = lse_history,  l = 1,  o = O_history        (l = 0, o = 0 without a history)
// and takes the draft's keys in as any softmax in one pass does,
//   m' = max(m, s_j),  l = l 2^(m-m') + sum 2^(s_j-m'),  o = o 2^(m-m') + sum 2^(s_j-m') v_j,
// so that joining the parts costs no pass of its own.  O_history has been
// rounded to bf16 (2^-9 of it, once more than O): an fp32 image of it would be
// a quarter of this kernel's bytes at a request's sizes.
//
// The draft's K and V are a few rows of bf16, read once per 16 query rows (or, above 16, once a CTA), and
// the products are small: bound by memory and latency.  Measured: 1024 drafts of 16
// rows, 8 heads, 31 us, 5.4 TB/s (three CTAs an SM, whose registers spill: 7 us more);
// 64 of 32 rows 12 us; one of 8 rows 5.8 us.
//
// A warp takes 16 rows of one K/V head by itself:
// the inner order of Q K^T is free, so queries and keys are loaded as 16-byte
// pieces (element 32 j + 8 t + 4 f + .. for lane t), and so is the order of V's
// columns, so that V is loaded the same way, turned by 8x8 transposes, and every
// lane ends up with whole 16-byte pieces of O.
#include <cuda_bf16.h>

#include "launch.cuh"
#include "mma_common.cuh"
#include "qcache_internal.h"

namespace ikbo {
namespace {

constexpr int TR_THREADS = 128;
constexpr int TR_MOST = 128;  // rows of a draft
constexpr int TR_SHARED_CTAS = 3;  // an SM

__device__ __forceinline__ uint32_t word(const uint4& x, int i) { return i == 0 ? x.x : (i == 1 ? x.y : (i == 2 ? x.z : x.w)); }

struct Tree {
  uint4 sees[TR_MOST];  // rows that a row reads, itself among them
  int up[2][TR_MOST];   // the row above, -1: none, -2: the row is not there
};

__device__ __forceinline__ int parent(const QcTreeParams& p, int cand, int l) {
  const int up = p.parents ? __ldg(p.parents + static_cast<int64_t>(cand) * p.Lq + l) : l - 1;
  if (up >= l) atomicOr(p.status, DEV_ERR_CACHE);
  return up >= l || up < -1 ? -2 : up;
}

// Which rows of a draft of up to 32 each row reads, by doubling the way up: every warp
// for itself, a lane a row.
__device__ __forceinline__ uint32_t small_tree(const QcTreeParams& p, int up, int lane) {
  uint32_t m = 1u << lane;
#pragma unroll 1
  for (int reach = 1; reach < p.Lq; reach <<= 1) {
    const int at = up >= 0 ? up : lane;
    const uint32_t more = __shfl_sync(0xffffffffu, m, at);
    const int next = __shfl_sync(0xffffffffu, up, at);
    if (up < 0) continue;
    if (next == -2) atomicOr(p.status, DEV_ERR_CACHE);  // below a row that is not there
    up = next;
    m |= more;
  }
  return up == -2 ? 0u : m;
}

// The same for up to 128, by the whole CTA.
__device__ void large_tree(const QcTreeParams& p, int cand, Tree& tr) {
  const int l = threadIdx.x, L = p.Lq;  // TR_THREADS >= Lq
  uint32_t m[4] = {};
  int up = -1;
  if (l < L) {
    up = parent(p, cand, l);
#pragma unroll
    for (int w = 0; w < 4; ++w) m[w] = (l >> 5) == w ? 1u << (l & 31) : 0u;
    tr.sees[l] = make_uint4(m[0], m[1], m[2], m[3]);
    tr.up[0][l] = up;
  }
  __syncthreads();
  int from = 0;
#pragma unroll 1
  for (int reach = 1; reach < L; reach <<= 1, from ^= 1) {
    uint4 more = {};
    int next = up;
    if (l < L && up >= 0) {
      more = tr.sees[up];
      next = tr.up[from][up];
    }
    __syncthreads();
    if (l < L) {
      if (up >= 0 && next == -2) atomicOr(p.status, DEV_ERR_CACHE);  // below a row that is not there
      up = next;
      m[0] |= more.x;
      m[1] |= more.y;
      m[2] |= more.z;
      m[3] |= more.w;
      tr.sees[l] = make_uint4(m[0], m[1], m[2], m[3]);
      tr.up[from ^ 1][l] = up;
    }
    __syncthreads();
  }
  if (l < L && up == -2) tr.sees[l] = make_uint4(0, 0, 0, 0);
  __syncthreads();
}

// Place of 16-byte piece c of row r of a draft's keys or values in shared memory: a quarter
// warp reads four pieces of two rows, which lie in different halves of the banks.
__device__ __forceinline__ uint32_t piece_at(int r, int c) { return static_cast<uint32_t>(r * 256 + ((c ^ ((r & 1) << 2)) << 4)); }

// kShared: a CTA has one K/V head of a draft, whose keys and values are in shared memory, for drafts
// of more than 16 rows (whose warps wait for one block of 16 after the other else: 60 drafts of 128 rows,
// 32 heads over 8, 156 us with the history for 193, 335 of 64 rows 92 for 106, 216 of 24 65 for 70).  By
// turned 8x8 loads of words laid out for them, and 2, 4 CTAs an SM, no faster.
template <bool kShared>
__global__ void __launch_bounds__(TR_THREADS, kShared ? TR_SHARED_CTAS : 2) qtree_kernel(const QcTreeParams p) {
  __shared__ Tree tr;
  extern __shared__ __align__(128) uint8_t kv[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int cand = static_cast<int>(blockIdx.x);
  const int u = __ldg(p.map + cand);
  if (u < 0 || u >= p.n_users) {  // (reported by the plan)
    wait_for_launch_before();
    return;
  }
  const int rows = p.group * p.Lq, tiles = (rows + 15) >> 4, items = kShared ? tiles : tiles * p.H_kv;
  const int parts = kShared ? static_cast<int>(gridDim.y) / p.H_kv : static_cast<int>(gridDim.y);
  const int head = kShared ? static_cast<int>(blockIdx.y) / parts : 0, part = static_cast<int>(blockIdx.y) - head * parts;
  const int padded = (p.Lq + 15) & ~15;
  if (kShared) {
    for (int i = threadIdx.x; i < padded * 32; i += TR_THREADS) {
      const int of = i >= padded * 16 ? 1 : 0, e = i - of * padded * 16, row = e >> 4, c = e & 15;
      const uint16_t* from = (of ? p.V : p.K) + static_cast<int64_t>(cand) * p.cand_stride + head * QC_D + 8 * c;
      copy16(smem_u32(kv) + of * padded * 256 + piece_at(row, c), row < p.Lq ? from + row * p.row_stride : from, row < p.Lq);
    }
    copies_commit();
  }
  const bool small = p.Lq <= 32;
  const int up = small && lane < p.Lq ? parent(p, cand, lane) : -1;
  uint32_t line = 0;
  bool built = false;
#pragma unroll 1
  for (int first = part * 4; first < items; first += parts * 4) {
    const int item = min(first + warp, items - 1);  // (the last item's warps again: they store nothing)
    const int hk = kShared ? head : item / tiles, tile = kShared ? item : item - hk * tiles;
    const int64_t row0 = (static_cast<int64_t>(cand) * p.H + hk * p.group) * p.Lq + 16 * tile;
    const int r0 = 16 * tile + g;
    const bool here[2] = {r0 < rows, r0 + 8 < rows};
    const uint16_t* kp = p.K + static_cast<int64_t>(cand) * p.cand_stride + hk * QC_D + 8 * t;
    const uint16_t* vp = p.V + static_cast<int64_t>(cand) * p.cand_stride + hk * QC_D + 8 * t;
    uint4 k[2][4], v[2][4];
    const auto fetch = [&](const uint16_t* from, int k0, uint4 (&to)[2][4]) {
      const uint8_t* at = kv + (from == vp ? padded * 256 : 0);
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int row = k0 + 8 * n + g;
          if (kShared) to[n][j] = *reinterpret_cast<const uint4*>(at + piece_at(row, 4 * j + t));
          else to[n][j] = row < p.Lq ? __ldg(reinterpret_cast<const uint4*>(from + row * p.row_stride + 32 * j)) : uint4{};
        }
    };
    if (!kShared) {
      fetch(kp, 0, k);
      fetch(vp, 0, v);
    }
    uint4 q[2][4] = {};
#pragma unroll
    for (int e = 0; e < 2; ++e)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (here[e]) q[e][j] = __ldg(reinterpret_cast<const uint4*>(p.Q + (row0 + g + 8 * e) * QC_D + 32 * j + 8 * t));
    wait_for_launch_before();  // for O and the log-sum-exp
    float o[16][4], m[2], l[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int64_t row = row0 + g + 8 * e;
      float lse = -INFINITY;
      if (here[e]) lse = __ldcg(p.hist_lse + row);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        uint4 h = {};
        if (here[e]) h = *reinterpret_cast<const uint4*>(p.O + row * QC_D + 32 * j + 8 * t);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          o[4 * j + i][2 * e] = bf16_lo(word(h, i));
          o[4 * j + i][2 * e + 1] = bf16_hi(word(h, i));
        }
      }
      m[e] = lse * 1.4426950408889634f;
      l[e] = lse == -INFINITY ? 0.f : 1.f;
    }
    if (!built) {
      if (small) line = small_tree(p, up, lane);
      else large_tree(p, cand, tr);
    }
    if (kShared && !built) {
      copies_wait<0>();
      __syncthreads();
    }
    built = true;
    const int l0 = r0 % p.Lq, l1 = (r0 + 8) % p.Lq;
    uint4 sees[2] = {};
    if (small) {
      const uint32_t s0 = __shfl_sync(0xffffffffu, line, l0), s1 = __shfl_sync(0xffffffffu, line, l1);
      sees[0].x = here[0] ? s0 : 0u;
      sees[1].x = here[1] ? s1 : 0u;
    } else {
      if (here[0]) sees[0] = tr.sees[l0];
      if (here[1]) sees[1] = tr.sees[l1];
    }
    const int n_keys = min(p.Lq, 16 * tile % p.Lq + 16);  // up to the tile's last row (all, where it goes on in the next head)
#pragma unroll 1
    for (int k0 = 0; k0 < n_keys; k0 += 16) {
      if (kShared || k0 > 0) {
        fetch(kp, k0, k);
        if (!kShared) fetch(vp, k0, v);
      }
      float s[2][4] = {};
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int f = 0; f < 2; ++f) {
          const uint32_t a[4] = {word(q[0][j], 2 * f), word(q[1][j], 2 * f), word(q[0][j], 2 * f + 1), word(q[1][j], 2 * f + 1)};
#pragma unroll
          for (int n = 0; n < 2; ++n) mma_16816(s[n], a, word(k[n][j], 2 * f), word(k[n][j], 2 * f + 1));
        }
      // the tree's rows, one pass of the softmax
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const uint32_t bits = word(sees[e], k0 >> 5) >> (k0 & 31);
        float top_s = -INFINITY;
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            float& x = s[n][2 * e + c];
            x = (bits >> (8 * n + 2 * t + c)) & 1u ? x * p.scale_log2 : -INFINITY;
            top_s = fmaxf(top_s, x);
          }
        top_s = fmaxf(top_s, __shfl_xor_sync(0xffffffffu, top_s, 1));
        top_s = fmaxf(top_s, __shfl_xor_sync(0xffffffffu, top_s, 2));
        const float to = fmaxf(m[e], top_s), ref = to == -INFINITY ? 0.f : to;
        const float keep = m[e] == -INFINITY ? 0.f : ex2(m[e] - ref);
        m[e] = to;
        l[e] *= keep;
        float sum = 0.f;
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            float& x = s[n][2 * e + c];
            x = (bits >> (8 * n + 2 * t + c)) & 1u ? ex2(x - ref) : 0.f;
            sum += x;
          }
        sum += __shfl_xor_sync(0xffffffffu, sum, 1);
        sum += __shfl_xor_sync(0xffffffffu, sum, 2);
        l[e] += sum;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          o[i][2 * e] *= keep;
          o[i][2 * e + 1] *= keep;
        }
      }
      if (kShared) fetch(vp, k0, v);
      // rows of V with an infinity or NaN stay out of the product, where they would
      // reach rows that do not read them (0 times infinity), and are added after it
      uint32_t odd[2];
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        const uint32_t x = not_finite(v[n][0]) | not_finite(v[n][1]) | not_finite(v[n][2]) | not_finite(v[n][3]);
        odd[n] = __ballot_sync(0xffffffffu, (x & 0x80008000u) != 0);
        if ((odd[n] >> (4 * g)) & 15u) {
#pragma unroll
          for (int j = 0; j < 4; ++j) v[n][j] = uint4{};
        }
      }
      const uint32_t pr[4] = {pack_bf16x2(s[0][0], s[0][1]), pack_bf16x2(s[0][2], s[0][3]), pack_bf16x2(s[1][0], s[1][1]),
                              pack_bf16x2(s[1][2], s[1][3])};
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) mma_16816(o[4 * j + i], pr, turn8x8(word(v[0][j], i)), turn8x8(word(v[1][j], i)));
      if (odd[0] | odd[1]) {
#pragma unroll 1
        for (int key = 0; key < 16; ++key) {
          if (!(((key < 8 ? odd[0] : odd[1]) >> (4 * (key & 7))) & 15u)) continue;
          float w[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float a = key < 8 ? s[0][2 * e] : s[1][2 * e], b = key < 8 ? s[0][2 * e + 1] : s[1][2 * e + 1];
            w[e] = __shfl_sync(0xffffffffu, key & 1 ? b : a, (lane & ~3) | ((key & 7) >> 1));
          }
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint4 x = __ldg(reinterpret_cast<const uint4*>(vp + (k0 + key) * p.row_stride + 32 * j));
#pragma unroll
            for (int e = 0; e < 2; ++e)
              if ((word(sees[e], k0 >> 5) >> ((k0 & 31) + key)) & 1u) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  o[4 * j + i][2 * e] = fmaf(w[e], bf16_lo(word(x, i)), o[4 * j + i][2 * e]);
                  o[4 * j + i][2 * e + 1] = fmaf(w[e], bf16_hi(word(x, i)), o[4 * j + i][2 * e + 1]);
                }
              }
          }
        }
      }
    }
    if (first + warp >= items) continue;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      if (!here[e]) continue;
      const bool there = (sees[e].x | sees[e].y | sees[e].z | sees[e].w) != 0;
      const int64_t row = row0 + g + 8 * e;
      const float inv = l[e] > 0.f ? 1.0f / l[e] : (l[e] == 0.f ? 0.f : l[e]);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        uint32_t x[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = there ? pack_bf16x2(o[4 * j + i][2 * e] * inv, o[4 * j + i][2 * e + 1] * inv) : 0u;
        *reinterpret_cast<uint4*>(p.O + row * QC_D + 32 * j + 8 * t) = make_uint4(x[0], x[1], x[2], x[3]);
      }
      if (p.lse && t == 0)
        p.lse[row] = !there ? -INFINITY : (l[e] > 0.f ? (m[e] + __log2f(l[e])) * 0.69314718055994531f : (l[e] == 0.f ? -INFINITY : l[e]));
    }
  }
}

}  // namespace

// The kernel reads the map, the parents and Q, K and V ahead of its wait, by the read-only path.  That is sound because
// the launch before it in the stream is the history's, an ordinary one that writes none of these: it has begun when
// all before it had ended and could be seen.  Behind a kernel that is itself set up early (launch_behind), or one
// that writes one of these, every load has to move behind the wait.
cudaError_t launch_qtree(const QcTreeParams& p, int num_sms, cudaStream_t s) {
  const bool shared = p.Lq > 16;
  const int heads = shared ? p.H_kv : 1, items = ((p.group * p.Lq + 15) / 16) * (shared ? 1 : p.H_kv);
  // a CTA takes four items of a candidate (of one K/V head), more where there are CTAs enough (1024 drafts of 8 items
  // 177.6 us, with the history, for 179.7: the tree is found once); set up while the history's last CTAs end (85.9 -> 83.9,
  // 177.1 -> 174.5)
  int parts = (items + 3) / 4;
  while (parts > 1 && static_cast<int64_t>(parts / 2) * heads * p.n_cand >= 4 * static_cast<int64_t>(num_sms)) parts = (parts + 1) / 2;
  const dim3 grid(static_cast<unsigned>(p.n_cand), static_cast<unsigned>(parts * heads));
  if (!shared) return launch_behind(qtree_kernel<false>, grid, TR_THREADS, 0, s, p);
  static std::atomic<uint64_t> done{0};
  const int bytes = 2 * ((p.Lq + 15) / 16 * 16) * QC_D * 2;
  const cudaError_t e = allow_smem(qtree_kernel<true>, 2 * TR_MOST * QC_D * 2, done);
  if (e != cudaSuccess) return e;
  return launch_behind(qtree_kernel<true>, grid, TR_THREADS, bytes, s, p);
}

}  // namespace ikbo
