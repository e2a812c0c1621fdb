// qcache_internal.h -- parameter blocks and shared device code of the rotary
// positions (rope.cu), the 4-bit cache (qcache.cu) and the attention that
// reads it (qattn.cu).  Not part of the public ABI.
#pragma once
#include <vector_types.h>

#include "ikbo_internal.h"

namespace ikbo {

// --------------------------------------------------------------- rotation
constexpr int ROPE_MAX_DIM = 512;

struct RopeParams {
  const void* X;
  void* Y;
  const int32_t* start;  // [n], or [n_users] read through map; null: 0
  const int32_t* map;    // null: item i reads start[i]
  uint32_t* status;
  int64_t xs[3], ys[3];  // element strides of item, head, token
  int n, n_users, H, L, d;
  int heads_per_cta;
  int rot, interleaved, backward, copy_rest;  // copy_rest: elements from rot on are written (not in place)
  float magnitude;
  uint64_t turn[ROPE_MAX_DIM / 2];  // turns per position, 2^64 = one turn
};

// ------------------------------------------------------------ 4-bit cache
constexpr int QC_D = 128;              // head dimension
constexpr int QC_ROWS = 16;            // tokens of a block
constexpr int QC_BLOCK_BYTES = 2560;   // 16 tokens of one head: keys, then values
constexpr int QC_HALF_BYTES = 1280;    // keys' or values' codes and pairs
constexpr int QC_CODE_BYTES = 1024;    // 16 x 64 bytes of codes, then 16 x 4 pairs (s, z) of two bf16
constexpr int QC_MAX_PAGE = 1024;

// Histories are split so that the longest CTA's share is short: QA_ROUNDS
// lengths of a split are compared, aiming at 1, 2, 4 .. items per CTA; the
// splits of a launch are at most QA_MOST_SPLITS per CTA.
constexpr int QA_ROUNDS = 4;
constexpr int QA_MOST_SPLITS = 1 << (QA_ROUNDS - 1);

struct QcResizeParams {
  int32_t* lens;
  const int32_t* new_lens;
  int32_t* table;
  int32_t* free_pages;
  int32_t* n_free;
  int32_t* slots;
  int32_t* offsets;
  int32_t* positions;
  uint32_t* status;
  int n_users, max_blocks, page_log2, n_pages, max_new;
};

struct QcAppendParams {
  const uint16_t* K;
  const uint16_t* V;
  const int32_t* slots;
  uint8_t* data;
  uint32_t* status;
  int64_t row_stride;
  int n_rows, H, heads_per_cta;
  int blocks_log2;      // log2(page / 16)
  int64_t n_slots;
};

struct QcLoadParams {
  const uint8_t* data;
  const int32_t* table;
  const int32_t* lens;
  const int32_t* kv_offsets;  // rows given by the caller, or null: packed at multiples of 128 rows
  int32_t* ranges;            // packed: [n_users] first row, [n_users] length (written)
  uint16_t* K;
  uint16_t* V;
  uint32_t* status;
  int64_t n_rows;             // rows of K and V
  int64_t bound;              // packed: the caller's bound on the sum of the lengths
  int n_users, max_blocks, n_pages, blocks_log2, H;
};

struct QcAttnParams {
  const uint16_t* Q;
  uint16_t* O;
  float* lse;
  const uint8_t* data;
  const int32_t* table;
  const int32_t* lens;
  const int32_t* offsets;  // the plan's segments
  const int32_t* perm;
  float* part;             // [QA_MOST_SPLITS * ctas] splits' partial rows: unnormalised O, reference and sums
  uint32_t* tickets;       // one per slot of part (tiles of 128 rows: 8 each)
  int4* list;              // tiles of 128 rows: the work list, three per item
  int64_t max_items;
  uint32_t* status;
  int64_t bound;
  int n_cand, n_users, H, H_kv, group, Lq;
  int n_pages, max_blocks, blocks_log2;
  int ctas;                // of the launch
  float scale_log2;
  uint32_t sixteen;        // QC_SIXTEEN
  uint64_t timeout_ns;
};

#ifdef __CUDACC__
// A length of the cache, or 0 for one outside [0, max_blocks * page] (reported).
__device__ __forceinline__ int qc_length(const int32_t* lens, int u, int64_t most, bool& bad) {
  const int n = __ldg(lens + u);
  if (n < 0 || n > most) {
    bad = true;
    return 0;
  }
  return n;
}

// The last u in [0, n) with base[u] <= x (base ascending, base[0] <= x): the
// user whose range of a flattened index holds x (empty ranges are skipped).
__device__ __forceinline__ int qc_find(const int32_t* base, int n, int x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (base[mid] <= x) lo = mid;
    else hi = mid;
  }
  return lo;
}

// Splits of a history of `units` (blocks or key tiles) into at most `chunk` each.
__device__ __forceinline__ int qc_splits(int units, int chunk) {
  return units <= chunk ? 1 : (units + chunk - 1) / chunk;
}

// First unit of split i of n of `units` (the first units % n are one longer).
__device__ __forceinline__ int qc_split_start(int units, int n, int i) {
  const int q = units / n, rest = units - q * n;
  return q * i + min(i, rest);
}

// Sums (scan: exclusive prefixes) of N values over the CTA's threads, or with
// `warp` over each warp's lanes, where every warp holds the same values.
// red: [N][the CTA's warps].
template <int N, int kThreads>
__device__ __forceinline__ void qc_sum(int64_t (&v)[N], int64_t (*red)[kThreads / 32], bool warp) {
#pragma unroll
  for (int k = 0; k < N; ++k) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
    if (!warp && (threadIdx.x & 31) == 0) red[k][threadIdx.x >> 5] = v[k];
  }
  if (warp) return;
  __syncthreads();
#pragma unroll
  for (int k = 0; k < N; ++k) {
    v[k] = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) v[k] += red[k][w];
  }
  __syncthreads();
}

template <int N, int kThreads>
__device__ __forceinline__ void qc_scan(int64_t (&v)[N], int64_t (&total)[N], int64_t (*red)[kThreads / 32], bool warp) {
  const int lane = threadIdx.x & 31, w0 = threadIdx.x >> 5;
  int64_t incl[N];
#pragma unroll
  for (int k = 0; k < N; ++k) {
    incl[k] = v[k];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, incl[k], o);
      if (lane >= o) incl[k] += y;
    }
    if (!warp && lane == 31) red[k][w0] = incl[k];
    total[k] = __shfl_sync(0xffffffffu, incl[k], 31);
    v[k] = incl[k] - v[k];
  }
  if (warp) return;
  __syncthreads();
#pragma unroll
  for (int k = 0; k < N; ++k) {
    total[k] = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
      v[k] += w < w0 ? red[k][w] : 0;
      total[k] += red[k][w];
    }
  }
  __syncthreads();
}

// The list of items that every CTA of an attention launch works out for
// itself: item0[u], part0[u] = items and partial slots before user u; an item
// is (user, K/V head, split, tile) in that order, slots only where a history
// has several splits.  work(u, bad) gives a user's tiles per head, units
// (blocks or key tiles) and length.  With up to 32 users every warp does it by
// itself.  Lengths of a split are compared by the CTAs' largest share: its
// items' units, kItem beside each and kJoin for each split of a tile.
struct QcUserWork {
  int tiles, units, len;
};
struct QcItems {
  int64_t items, slots;
  int chunk;  // units of a split, at most
};

template <int kThreads, int kMin, int kItem, int kJoin, typename Work>
__device__ __forceinline__ QcItems qc_items(const QcAttnParams& p, const Work& work, int32_t* item0, int32_t* part0,
                                            int64_t (*red)[kThreads / 32]) {
  const int n = p.n_users;
  const bool few = n <= 32;
  const int me = few ? static_cast<int>(threadIdx.x & 31) : static_cast<int>(threadIdx.x);
  const int per = few ? 1 : (n + kThreads - 1) / kThreads;
  const int lo = min(me * per, n), hi = min(lo + per, n);
  bool bad = false, ignored = false;
  QcUserWork one = {};  // this thread's user where it has only one
  if (per == 1 && lo < n) one = work(lo, bad);
  const auto get = [&](int u) { return per == 1 ? one : work(u, ignored); };
  int64_t sums[3] = {0, 0, 0};
  int longest = 0;
  for (int u = lo; u < hi; ++u) {
    const QcUserWork w = per == 1 ? one : work(u, bad);
    sums[0] += static_cast<int64_t>(w.tiles) * w.units;
    sums[1] += w.len;
    sums[2] += w.tiles;
    if (w.tiles > 0) longest = max(longest, w.units);
  }
  qc_sum<3, kThreads>(sums, red, few);
  longest = __reduce_max_sync(0xffffffffu, longest);
  if (!few) {
    if ((threadIdx.x & 31) == 0) red[0][threadIdx.x >> 5] = longest;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) longest = max(longest, static_cast<int>(red[0][w]));
    __syncthreads();
  }
  if (sums[1] > p.bound) bad = true;
  if (bad && blockIdx.x == 0) atomicOr(p.status, DEV_ERR_CACHE);
  // r CTAs' worth of items: a tile's splits are rounded up, hence the tiles
  // taken off; too few to split anything: one item per tile
  // (fp32 quotients, rounded up by more than their error: 64-bit divisions are
  // the slowest part of a small launch)
  const int64_t work_all = sums[0] * p.H_kv, tiles_all = sums[2] * p.H_kv;
  int chunks[QA_ROUNDS];
  int64_t counts[QA_ROUNDS];
#pragma unroll
  for (int r = 0; r < QA_ROUNDS; ++r) {
    const int64_t room = (static_cast<int64_t>(p.ctas) << r) - tiles_all;
    const float c = static_cast<float>(work_all) / static_cast<float>(room) * 1.00001f + 1.f;
    chunks[r] = room > 0 ? max(static_cast<int>(fminf(c, 1e8f)), kMin) : max(longest, 1);
    counts[r] = 0;
  }
  for (int u = lo; u < hi; ++u) {
    const QcUserWork w = get(u);
#pragma unroll
    for (int r = 0; r < QA_ROUNDS; ++r) counts[r] += static_cast<int64_t>(w.tiles) * qc_splits(w.units, chunks[r]);
  }
  qc_sum<QA_ROUNDS, kThreads>(counts, red, few);
  QcItems it;
  it.chunk = chunks[0];
  float best = 0.f;
#pragma unroll
  for (int r = 0; r < QA_ROUNDS; ++r) {
    const int ns = qc_splits(longest, chunks[r]);
    const float share = ceilf(static_cast<float>(counts[r] * p.H_kv) / static_cast<float>(p.ctas)) *
                            static_cast<float>((longest + ns - 1) / ns + kItem) +
                        (ns > 1 ? static_cast<float>(ns * kJoin) : 0.f);
    if (r == 0 || share < best) {
      best = share;
      it.chunk = chunks[r];
    }
  }
  int64_t v[2] = {0, 0}, total[2];
  for (int u = lo; u < hi; ++u) {
    const QcUserWork w = get(u);
    const int ns = qc_splits(w.units, it.chunk);
    const int64_t items = static_cast<int64_t>(w.tiles) * p.H_kv * ns;
    v[0] += items;
    v[1] += ns > 1 ? items : 0;
  }
  qc_scan<2, kThreads>(v, total, red, few);
  for (int u = lo; u < hi; ++u) {
    const QcUserWork w = get(u);
    const int ns = qc_splits(w.units, it.chunk);
    const int64_t items = static_cast<int64_t>(w.tiles) * p.H_kv * ns;
    item0[u] = static_cast<int32_t>(v[0]);
    part0[u] = static_cast<int32_t>(v[1]);
    v[0] += items;
    v[1] += ns > 1 ? items : 0;
  }
  __syncthreads();
  it.items = total[0];
  it.slots = total[1];
  return it;
}

// Two bf16 values from nibbles at bits SHIFT .. of each half of w:
// z + (16 + c) s in one rounding.  The nibble lands in the top four mantissa
// bits of 16.0, which makes the operand 16 + c exactly.  sixteen: QC_SIXTEEN, by
// way of the launch's parameters: of two constants that it can see the compiler
// makes two instructions (an AND and an OR take one, with one constant in a
// register), a quarter of the tile kernel's integer work.
constexpr uint32_t QC_SIXTEEN = 0x41804180u;
template <int kNibble>
__device__ __forceinline__ uint32_t qc_decode(uint32_t w, uint32_t s2, uint32_t z2, uint32_t sixteen = QC_SIXTEEN) {
  constexpr int kShift = 3 - 4 * kNibble;
  uint32_t c;
  if (kShift >= 0) c = w << (kShift >= 0 ? kShift : 0);
  else c = w >> (kShift < 0 ? -kShift : 0);
  c = (c & 0x00780078u) | sixteen;
  uint32_t r;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(c), "r"(s2), "r"(z2));
  return r;
}
#endif

}  // namespace ikbo
