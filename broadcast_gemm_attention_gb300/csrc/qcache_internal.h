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

// Slots for partial rows per worker (CTA or warp) of an attention launch: its
// share of the work begins and ends within an item.
constexpr int QA_SLOTS = 2;

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
  float* part;             // [QA_SLOTS * workers] parts' rows: unnormalised O, reference and sums
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
  uint32_t debug;          // the plan's switches
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
template <typename T>
__device__ __forceinline__ int qc_find(const T* base, int n, T x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (base[mid] <= x) lo = mid;
    else hi = mid;
  }
  return lo;
}

// The sum of a warp's lanes (none below 0), 24 bits at a time.
__device__ __forceinline__ int64_t qc_warp_sum(int64_t v) {
  const int64_t x = v;
  const uint32_t lo = __reduce_add_sync(0xffffffffu, static_cast<uint32_t>(x) & 0xFFFFFFu);
  const uint32_t mid = __reduce_add_sync(0xffffffffu, static_cast<uint32_t>(x >> 24) & 0xFFFFFFu);
  const uint32_t hi = __reduce_add_sync(0xffffffffu, static_cast<uint32_t>(x >> 48));
  return (static_cast<int64_t>(hi) << 48) + (static_cast<int64_t>(mid) << 24) + lo;
}

// x / c for 0 <= x, 1 <= c: an estimate, put right.
__device__ __forceinline__ int64_t qc_div(int64_t x, int c) {
  int64_t q = static_cast<int64_t>(__fdividef(static_cast<float>(x), static_cast<float>(c)));
#pragma unroll 1
  while (q * c > x) --q;
#pragma unroll 1
  while ((q + 1) * c <= x) ++q;
  return q;
}

// Inclusive prefixes of a warp's lanes.
template <typename T>
__device__ __forceinline__ T qc_warp_scan(T x) {
#pragma unroll 1
  for (int o = 1; o < 32; o <<= 1) {
    const T y = __shfl_up_sync(0xffffffffu, x, o);
    if (static_cast<int>(threadIdx.x & 31) >= o) x += y;
  }
  return x;
}

// ---- how the CTAs of an attention launch share the work
// An item is (user, K/V head, tile of query rows), in that order; its length is
// the history's units (blocks or key tiles), and its cost that and `overhead`
// units more (1 where there are no tokens).  All items' costs in a row are cut
// into as many equal shares as there are workers (CTAs, or single warps), so each has a run of items,
// of which the first and the last may be parts: every worker has the same to do
// (to the rows that a tile lacks), there are no more parts than items and
// workers, and parts of one item always lie with consecutive workers.  (Whole items dealt out
// in turn, with histories cut to one length that fills the CTAs best, took 10%
// to 25% longer where histories differ.)
//
// A request too small for shares of an item's overhead and kMin units is cut
// evenly instead, each item into parts of about `chunk` units, one for a CTA: an
// item's cost is then its parts, and a share 1.
struct QcUserWork {
  int tiles, units, len;
};
struct QcShares {
  int64_t base;         // start(b) = b base + b rest / parts
  int parts, rest;      // shares (at most the launch's workers), items' costs beside base parts
  int overhead, chunk;  // chunk > 0: even parts
  __device__ __forceinline__ int64_t start(int b) const {
    const int x = b * rest;  // (both below parts, of which there are at most a few thousand)
    int q = static_cast<int>(__fdividef(static_cast<float>(x), static_cast<float>(parts)));
    q += (q + 1) * parts <= x ? 1 : (q * parts > x ? -1 : 0);
    return b * base + q;
  }
  __device__ __forceinline__ int item_cost(int units) const;
};
struct QcSharesScratch {
  int64_t red[3][32];
  QcShares shares;
};
// A CTA's part of an item.
struct QcPart {
  int t0, nt;       // units t0 .. t0 + nt - 1
  int ns;           // parts of the item that are not empty; if above 1:
  int slot, first;  // this part's slot for partial rows, the first part's
};
__device__ __forceinline__ int QcShares::item_cost(int units) const {
  if (units == 0) return 1;
  // parts of at most `chunk`, but for the quotient's last bits
  return chunk > 0 ? static_cast<int>(ceilf(__fmul_rn(__fdividef(static_cast<float>(units), static_cast<float>(chunk)), 0.99999f)))
                   : units + overhead;
}
// The k-th part's slot (the first part ends its CTA's share, the others begin one).
__device__ __forceinline__ int qc_slot(int first, int k) { return k == 0 ? first : (first & ~1) + 2 * k; }

// Works out the shares, and where each user's items begin: cost0[u] in costs,
// item0[u] (if not null) counted.  work(u, bad) gives a user's tiles per head,
// units and length.  With up to 32 users one warp does it alone.
//
// A CTA runs this once, from instructions that no cache holds yet (a small
// launch spends more time here than on its products), so it is written for few
// instructions: loops stay loops, and no integer division.  (All items fit in 31
// bits: checked on the host.)
template <int kThreads, int kMin, int kOverhead, typename Work>
__device__ __forceinline__ QcShares qc_shares(const QcAttnParams& p, int workers, const Work& work, int64_t* cost0,
                                              int32_t* item0, QcSharesScratch& sh) {
  constexpr int kWarps = kThreads / 32;
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
    // three sums: the units of all items, tokens, and items with units (low half) and without
    int64_t v[3] = {0, 0, 0};
    for (int u = lo; u < hi; ++u) {
      const QcUserWork w = per == 1 ? one : work(u, bad);
      const int64_t items = static_cast<int64_t>(w.tiles) * p.H_kv;
      v[0] += items * w.units;
      v[1] += w.len;
      v[2] += w.units > 0 ? items : items << 32;
    }
#pragma unroll 1
    for (int k = 0; k < 3; ++k) {
      const int64_t x = qc_warp_sum(v[0]);
      v[0] = v[1], v[1] = v[2], v[2] = x;
      if (!few && lane == 0) sh.red[k][warp] = x;
    }
    if (!few) {
      __syncthreads();
#pragma unroll 1
      for (int k = 0; k < 3; ++k) {
        const int64_t x = qc_warp_sum(lane < kWarps ? sh.red[k][lane] : int64_t{0});
        v[0] = v[1], v[1] = v[2], v[2] = x;
      }
      __syncthreads();  // red has been read
    }
    if (v[1] > p.bound) bad = true;
    if (bad && blockIdx.x == 0) atomicOr(p.status, DEV_ERR_CACHE);
    const int64_t with = v[2] & 0xFFFFFFFF, without = v[2] >> 32, items_all = with + without;
    int64_t total = v[0] + with * kOverhead + without;
    QcShares r = {0, workers, 0, kOverhead, 0};
    if (total < static_cast<int64_t>(kMin + kOverhead) * workers) {
      if (items_all < workers)  // (each item's parts are rounded up, hence the items taken off)
        r.chunk = max(kMin, static_cast<int>(__fdividef(static_cast<float>(v[0]), static_cast<float>(workers - items_all)) * 1.0001f) + 1);
      else
        r.parts = max(1, static_cast<int>(total) / (kMin + kOverhead));
    }
    int64_t cost = 0;
    uint32_t items = 0;
    const auto add = [&](const QcUserWork& w) {
      const int64_t k = static_cast<int64_t>(w.tiles) * p.H_kv;
      cost += k * r.item_cost(w.units);
      items += static_cast<uint32_t>(k);
    };
    for (int u = lo; u < hi; ++u) add(get(u));
    const int64_t mine = cost;
    const uint32_t mine_items = items;
#pragma unroll 1
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t x = __shfl_up_sync(0xffffffffu, cost, o);
      const uint32_t y = __shfl_up_sync(0xffffffffu, items, o);
      if (lane >= o) cost += x, items += y;
    }
    if (!few) {  // and the warps before
      if (lane == 31) {
        sh.red[0][warp] = cost;
        sh.red[1][warp] = items;
      }
      __syncthreads();
      cost += qc_warp_sum(lane < warp ? sh.red[0][lane] : int64_t{0});
      items += __reduce_add_sync(0xffffffffu, lane < warp ? static_cast<uint32_t>(sh.red[1][lane]) : 0u);
    }
    if (tid == (few ? 31 : kThreads - 1)) {  // has all costs
      if (r.chunk > 0) {
        total = cost;
        r.parts = max(1, static_cast<int>(cost));
      }
      r.base = qc_div(total, r.parts);
      r.rest = static_cast<int>(total - r.base * r.parts);
      sh.shares = r;
    }
    cost -= mine;
    items -= mine_items;
    for (int u = lo; u < hi; ++u) {
      cost0[u] = cost;
      if (item0) item0[u] = static_cast<int32_t>(items);
      add(get(u));
    }
  }
  __syncthreads();
  return sh.shares;
}

// The part of the item at `pos` (of a user's work w) that belongs to worker cta,
// whose share overlaps it.  Cuts that would leave a part of fewer than kMin
// units move to the item's end, the same way for the CTAs on both sides.
template <int kMin>
__device__ __forceinline__ QcPart qc_part(const QcShares& sh, int cta, const QcUserWork& w, int64_t pos) {
  QcPart r = {0, w.units, 1, 0, 0};
  const int cost = sh.item_cost(w.units);
  const int64_t start = sh.start(cta), end = sh.start(cta + 1);
  if (w.units == 0 || (pos >= start && pos + cost <= end)) return r;
  const auto cut = [&](int64_t at) {  // a cut at cost `at`, in units
    const int x = static_cast<int>(at - pos);
    if (sh.chunk > 0) return static_cast<int>(static_cast<uint32_t>(x) * static_cast<uint32_t>(w.units) / static_cast<uint32_t>(cost));
    const int t = x - sh.overhead;
    return t < kMin ? 0 : (t > w.units - kMin ? w.units : t);
  };
  // the CTAs whose shares the item lies in: at least so many, then the others
  const uint32_t most = static_cast<uint32_t>(min(sh.base + (sh.rest > 0), int64_t{0x7fffffff}));  // of a share
  int first = cta, last = cta;
  if (pos < start) first -= static_cast<int>(static_cast<uint32_t>(start - pos) / most);
  if (pos + cost > end) last += static_cast<int>(static_cast<uint32_t>(pos + cost - end) / most);
#pragma unroll 1
  while (sh.start(first) > pos) --first;
#pragma unroll 1
  while (sh.start(last + 1) < pos + cost) ++last;
  r.t0 = first < cta ? cut(start) : 0;
  r.nt = (cta < last ? cut(end) : w.units) - r.t0;
  // a share is at least kMin and the overhead, so only the first and the last part can be empty
  const int headless = cut(sh.start(first + 1)) == 0;
  const int tailless = cut(sh.start(last)) == w.units;
  r.ns = last - first + 1 - headless - tailless;
  r.first = 2 * (first + headless) + (headless ? 0 : 1);
  r.slot = 2 * cta + (first < cta ? 0 : 1);
  return r;
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
