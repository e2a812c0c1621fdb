// qcache_internal.h -- parameter blocks and shared device code of the rotary
// positions (rope.cu), the 4-bit cache (qcache.cu) and the attention that
// reads it (qattn.cu).  Not part of the public ABI.
#pragma once
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

// Up to this many query rows per user and K/V head (on average) the attention
// reads the 4-bit blocks directly.
constexpr int QATTN_FEW_ROWS = 160;

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
  int n_rows, H;
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
  float* part;             // [2 * target][rows * (128 + 2)] unnormalised O, then m and l of each row
  uint32_t* tickets;       // [2 * target]
  uint32_t* status;
  int64_t bound;
  int n_cand, n_users, H, H_kv, group, Lq;
  int n_pages, max_blocks, blocks_log2;
  int target;              // items the histories are split into, at most (besides one per tile)
  float scale_log2;
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

// Two bf16 values from nibbles at bits SHIFT .. of each half of w:
// z + (16 + c) s in one rounding.  The nibble lands in the top four mantissa
// bits of 16.0, which makes the operand 16 + c exactly.
template <int kNibble>
__device__ __forceinline__ uint32_t qc_decode(uint32_t w, uint32_t s2, uint32_t z2) {
  constexpr int kShift = 3 - 4 * kNibble;
  uint32_t c;
  if (kShift >= 0) c = w << (kShift >= 0 ? kShift : 0);
  else c = w >> (kShift < 0 ? -kShift : 0);
  c = (c & 0x00780078u) | 0x41804180u;
  uint32_t r;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(c), "r"(s2), "r"(z2));
  return r;
}
#endif

}  // namespace ikbo
