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

// Splits of a history of `units` (blocks or key tiles) into about `chunk` each:
// the quotient rounded up, in fp32 and so that an error of its last bits adds
// no split (a split may be 1/100000 longer than `chunk`).  The same in every
// place that asks.
__device__ __forceinline__ int qc_splits(int units, int chunk) {
  const float q = __fmul_rn(__fdividef(static_cast<float>(units), static_cast<float>(chunk)), 0.99999f);
  return units <= chunk ? 1 : static_cast<int>(ceilf(q));
}

// First unit of split i of n of `units` (the first units % n are one longer).
__device__ __forceinline__ int qc_split_start(int units, int n, int i) {
  const int q = units / n, rest = units - q * n;
  return q * i + min(i, rest);
}

// Sums over the CTA's threads, or with `warp` over one warp that is alone here;
// red: a word per warp.
template <int kThreads>
__device__ __forceinline__ uint32_t qc_sum(uint32_t v, uint32_t* red, bool warp) {
  v = __reduce_add_sync(0xffffffffu, v);
  if (warp) return v;
  const int lane = threadIdx.x & 31;
  __syncthreads();  // red has been read
  if (lane == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  return __reduce_add_sync(0xffffffffu, lane < kThreads / 32 ? red[lane] : 0u);
}

__device__ __forceinline__ float qc_warp_sum(float v) {
#pragma unroll 1
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Exclusive prefixes of a warp's lanes.
__device__ __forceinline__ uint32_t qc_warp_scan(uint32_t v) {
  uint32_t x = v;
#pragma unroll 1
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, x, o);
    if (static_cast<int>(threadIdx.x & 31) >= o) x += y;
  }
  return x - v;
}

// The list of items that every CTA of an attention launch works out for
// itself: item0[u], part0[u] = items and partial slots before user u; an item
// is (user, K/V head, split, tile) in that order, slots only where a history
// has several splits.  work(u, bad) gives a user's tiles per head, units
// (blocks or key tiles) and length.  With up to 32 users one warp does it
// alone.  Lengths of a split are compared by the CTAs' largest share: its
// items' units, kItem beside each and kJoin for each split of a tile.
//
// A CTA runs this once, from instructions that no cache holds yet (a small
// launch spends more time here than on its products), so it is written for few
// instructions: loops stay loops, 32-bit and fp32 numbers, no integer division.
// (All items and tiles fit in 31 bits: checked on the host.)
struct QcUserWork {
  int tiles, units, len;
};
struct QcItems {
  uint32_t items, slots;
  int chunk;  // units of a split, at most
};
struct QcItemsShared {
  uint32_t red[32];
  QcItems it;
};

template <int kThreads, int kMin, int kItem, int kJoin, typename Work>
__device__ __forceinline__ QcItems qc_items(const QcAttnParams& p, const Work& work, int32_t* item0, int32_t* part0,
                                            QcItemsShared& sh) {
  static_assert(kThreads <= 1024, "a word of red per warp");
  const int n = p.n_users;
  const bool few = n <= 32;
  const int tid = static_cast<int>(threadIdx.x), lane = tid & 31, warp = tid >> 5;
  if (!few || warp == 0) {
    const int per = few ? 1 : (n + kThreads - 1) / kThreads;
    const int lo = min(tid * per, n), hi = min(lo + per, n);
    bool bad = false, ignored = false;
    QcUserWork one = {};  // this thread's user where it has only one
    if (per == 1 && lo < n) one = work(lo, bad);
    const auto get = [&](int u) { return per == 1 ? one : work(u, ignored); };
    float sum = 0.f;  // of tiles x units: a bound with a margin for its rounding is made of it
    int64_t lens = 0;
    uint32_t tiles = 0;
    int longest = 0;
    for (int u = lo; u < hi; ++u) {
      const QcUserWork w = per == 1 ? one : work(u, bad);
      sum += static_cast<float>(w.tiles) * static_cast<float>(w.units);
      lens += w.len;
      tiles += static_cast<uint32_t>(w.tiles);
      if (w.tiles > 0) longest = max(longest, w.units);
    }
    sum = qc_warp_sum(sum);
    longest = static_cast<int>(__reduce_max_sync(0xffffffffu, static_cast<unsigned>(longest)));
    if (!few) {
      if (lane == 0) {
        sh.red[warp] = __float_as_uint(sum);
        item0[warp] = longest;  // (there are more users than warps)
      }
      __syncthreads();
      sum = qc_warp_sum(lane < kThreads / 32 ? __uint_as_float(sh.red[lane]) : 0.f);
      longest = static_cast<int>(__reduce_max_sync(0xffffffffu, lane < kThreads / 32 ? static_cast<unsigned>(item0[lane]) : 0u));
    }
    tiles = qc_sum<kThreads>(tiles, sh.red, few);
    // 24 bits and the rest: neither sum leaves 32 bits
    const uint32_t l0 = qc_sum<kThreads>(static_cast<uint32_t>(lens & 0xFFFFFF), sh.red, few);
    const uint32_t l1 = qc_sum<kThreads>(static_cast<uint32_t>(lens >> 24), sh.red, few);
    if ((static_cast<int64_t>(l1) << 24) + l0 > p.bound) bad = true;
    if (bad && blockIdx.x == 0) atomicOr(p.status, DEV_ERR_CACHE);
    // r: 2^r items per CTA aimed at (a tile's splits are rounded up, hence the
    // tiles taken off); too few to split anything: one item per tile
    const float work_all = sum * static_cast<float>(p.H_kv) * 1.0001f;
    const int64_t tiles_all = static_cast<int64_t>(tiles) * p.H_kv;
    QcItems it = {0, 0, 1};
    float best = 0.f;
#pragma unroll 1
    for (int r = 0; r < QA_ROUNDS; ++r) {
      const int64_t room = (static_cast<int64_t>(p.ctas) << r) - tiles_all;
      int chunk = max(longest, 1);
      if (room > 0) chunk = max(static_cast<int>(fminf(__fdividef(work_all, static_cast<float>(room)) + 1.f, 1e8f)), kMin);
      uint32_t count = 0;
      for (int u = lo; u < hi; ++u) {
        const QcUserWork w = get(u);
        count += static_cast<uint32_t>(w.tiles * qc_splits(w.units, chunk));
      }
      count = qc_sum<kThreads>(count, sh.red, few) * static_cast<uint32_t>(p.H_kv);
      const int ns = qc_splits(longest, chunk);
      const float share = ceilf(static_cast<float>(count) / static_cast<float>(p.ctas)) *
                              (ceilf(__fdividef(static_cast<float>(longest), static_cast<float>(ns))) + kItem) +
                          (ns > 1 ? static_cast<float>(ns * kJoin) : 0.f);
      if (r == 0 || share < best) {
        best = share;
        it.chunk = chunk;
      }
      if (room > 0 && chunk == kMin) break;  // shorter splits there are not
    }
    uint32_t items = 0, slots = 0;
    for (int u = lo; u < hi; ++u) {
      const QcUserWork w = get(u);
      const int ns = qc_splits(w.units, it.chunk);
      const uint32_t k = static_cast<uint32_t>(w.tiles) * static_cast<uint32_t>(p.H_kv * ns);
      items += k;
      slots += ns > 1 ? k : 0u;
    }
    uint32_t v0 = qc_warp_scan(items), v1 = qc_warp_scan(slots);
    it.items = qc_sum<kThreads>(items, sh.red, few);
    if (!few) {  // red holds the warps' sums
      uint32_t before = qc_warp_scan(lane < kThreads / 32 ? sh.red[lane] : 0u);
      v0 += __shfl_sync(0xffffffffu, before, warp);
      it.slots = qc_sum<kThreads>(slots, sh.red, few);
      before = qc_warp_scan(lane < kThreads / 32 ? sh.red[lane] : 0u);
      v1 += __shfl_sync(0xffffffffu, before, warp);
    } else {
      it.slots = qc_sum<kThreads>(slots, sh.red, few);
    }
    for (int u = lo; u < hi; ++u) {
      const QcUserWork w = get(u);
      const int ns = qc_splits(w.units, it.chunk);
      const uint32_t k = static_cast<uint32_t>(w.tiles) * static_cast<uint32_t>(p.H_kv * ns);
      item0[u] = static_cast<int32_t>(v0);
      part0[u] = static_cast<int32_t>(v1);
      v0 += k;
      v1 += ns > 1 ? k : 0u;
    }
    if (tid == 0) sh.it = it;
  }
  __syncthreads();
  return sh.it;
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
