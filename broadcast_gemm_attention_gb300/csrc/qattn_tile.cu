// qattn_tile.cu -- broadcast attention from the 4-bit cache on the 5th-gen
// tensor cores, for more query rows per user and K/V head than a few.
//
//   O[i,h] = softmax(Q[i,h] K[map[i],g]^T * scale) V[map[i],g]
//
// A tile is 128 rows of one (user u, K/V head g): the queries of u's
// candidates, of all heads that share g, in order.  The history never exists
// as bf16 outside shared memory: eight warps decode each 128-token tile of
// codes into the operand tiles of the products while the tile before is
// multiplied, so the tile's 128 rows share one decode.  The rest follows
// attn.cu: S and P.V issuers, two softmax groups that take turns at the key
// tiles, and a chain of reference maxima between them.
//
// Per CTA (persistent, one per SM, 20 warps):
//   warp 0       asks for the codes of the tiles ahead in L2
//   warp 1       S issuer and TMEM owner;  warp 2  P.V issuer
//   warp 3       Q: 128 gathered rows by 16-byte asynchronous copies
//   warps 4-11   softmax and epilogue (as in attn.cu)
//   warps 12-19  decode: one AND-OR and one FMA for two elements.  A word's
//                codes come out as elements (0,4) (1,5) (2,6) (3,7); instead of
//                putting them in order, Q's elements are put in the same order
//                once per tile (an inner product does not care), and V's
//                columns are, which the epilogue undoes by its choice of names.
//
// Work: each CTA takes an equal share of all tiles' histories, in a row, and
// lists it for itself (a scan over the users); a history is split where one
// CTA's share ends and the next one's begins.  A split leaves its unnormalised O, [column][row], with
// each row's reference and sum; the last warp to finish a 32-row, 64-column
// piece of a tile adds that piece's splits in order, so results repeat bit for
// bit whichever CTA that is.
//
// What bounds it: not the products (1024 cycles of the tensor pipe per key
// tile, 46% busy) and hardly the decode (without three quarters of its
// arithmetic, on wrong results, 7% less time), but each softmax group's chain
// through its tile, which two groups share: about 1850 cycles per key tile, the
// pace of attn.cu.  152 tiles of 128 rows over 64 key tiles each (19 histories of
// 8192, 8 heads): 78.5 us, 1040 TFLOP/s; with 4 key tiles each 21 us, of which the
// work list, the cold instructions and the first loads are about 15.
// Measured slower: one pass that makes P with the last reference and corrects it
// where the chain says otherwise, with P beside S in TMEM (89 us: P.V has to be
// through before the group's next P); codes through shared memory by bulk copies
// (over a thousand cycles of a producer warp a tile); the epilogue's code copied
// into five places (ten candidates for 102 users: 207 us against 176).
#include <cuda_bf16.h>

#include "attn_common.cuh"
#include "qcache_internal.h"

namespace ikbo {
namespace {

constexpr int TL_THREADS = 640;
constexpr int SOFTMAX_WARP0 = 4, DECODE_WARP0 = 12;
constexpr int SOFTMAX_THREADS = 256, GROUP_THREADS = 128;
constexpr int DECODE_WARPS = 4;  // of each kind
constexpr int CTRL_REGS = 56, SOFTMAX_REGS = 136, DECODE_REGS = 72;
constexpr int LAUNCH_REGS = 96;  // 65536 / 640, in eights
static_assert(128 * CTRL_REGS + SOFTMAX_THREADS * SOFTMAX_REGS + 64 * DECODE_WARPS * DECODE_REGS <= TL_THREADS * LAUNCH_REGS,
              "register split exceeds the launch's registers");
constexpr float RESCALE_THRESHOLD = 8.0f;  // log2 units
constexpr int TL_ITEM_TILES = 3;           // what an item costs beside its key tiles, in key tiles
constexpr int TL_MIN_TILES = 4;            // key tiles of a split, at least
constexpr int TL_PART = ATT_BM * ATT_D + 4 * ATT_BM;  // floats of a split's partial rows: O, and m and l per half
constexpr int S_BUFS = 3;
constexpr uint32_t TM_S = 0, TM_O = 384;  // S_b at TM_S + 128 b, its P in its first 64 columns

constexpr int STAGE_BYTES = 1024;  // of O, per softmax warp: 32 rows x 16 elements
constexpr uint32_t K_AT = 2 * ATT_Q_TILE_BYTES, V_AT = K_AT + 2 * ATT_KV_STAGE_BYTES;
constexpr uint32_t OUT_AT = V_AT + 2 * ATT_KV_STAGE_BYTES;
constexpr uint32_t AUX_AT = OUT_AT + 8 * STAGE_BYTES;
constexpr int NUM_BARS = 6 + 3 * S_BUFS + 8 + 2 + 2;

constexpr int LIST_NEAR = 64;  // of a CTA's items, kept in shared memory

struct Aux {
  int4 list[3 * LIST_NEAR];
  uint64_t bars[NUM_BARS];
  float2 fin[2][2][ATT_BM];  // [item parity][group][row]: reference and sum of a finished item
  uint32_t chain[ATT_BM];
  QcSharesScratch shares;
  uint32_t tmem_slot, abort, n_tiles;
  int n_items;
  uint32_t decoded;  // key tile that the decode is at
};
constexpr uint32_t SMEM_USED = AUX_AT + sizeof(Aux);
constexpr uint32_t SMEM_ALLOC = 227 * 1024;
static_assert(SMEM_USED <= SMEM_ALLOC, "tiles do not fit in shared memory");
static_assert((sizeof(int64_t) + sizeof(int32_t)) * SEG_MAX_USERS <= AUX_AT, "the users' prefixes do not fit");

struct Smem {
  uint8_t *q, *k, *v, *out;
  uint64_t *q_full, *q_empty, *s_full, *p_full, *pv_done, *o_full, *o_empty, *k_full, *k_empty, *v_full,
      *v_empty, *fin_full, *drain;
  Aux* x;
};

__device__ __forceinline__ Smem carve(uint8_t* base) {
  Smem s;
  s.q = base;
  s.k = base + K_AT;
  s.v = base + V_AT;
  s.out = base + OUT_AT;
  s.x = reinterpret_cast<Aux*>(base + AUX_AT);
  uint64_t* b = s.x->bars;
  s.q_full = b;
  s.q_empty = b + 2;
  s.o_full = b + 4;
  s.o_empty = b + 5;
  s.s_full = b + 6;
  s.p_full = s.s_full + S_BUFS;
  s.pv_done = s.p_full + S_BUFS;
  s.k_full = s.pv_done + S_BUFS;
  s.k_empty = s.k_full + 2;
  s.v_full = s.k_empty + 2;
  s.v_empty = s.v_full + 2;
  s.fin_full = s.v_empty + 2;
  s.drain = s.fin_full + 2;
  return s;
}

// ------------------------------------------------------------------- items
// An item of the list (48 bytes).
struct Item {
  int u, hk, seg, n_rows;     // user, K/V head, the user's first place in perm, rows that read this history
  int row0, len, t0, nt;      // the tile's first row; tokens of the history; the split's key tiles t0 .. t0 + nt - 1
  int ns, slot, first, pad;  // splits of the tile; this split's slot for partial rows, the first split's
};

__device__ __forceinline__ int4 ld_int4(const int4* p) {  // written by this CTA in this launch: not the read-only path
  int4 r;
  asm volatile("ld.global.v4.s32 {%0,%1,%2,%3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "l"(p) : "memory");
  return r;
}

// This CTA's items: the first ones in shared memory, the others in its part of
// the list.
struct List {
  const int4* near;
  const int4* far;
  int count;
};
__device__ __forceinline__ int4 item_part(const List& l, int k, int i) {
  return k < LIST_NEAR ? l.near[3 * k + i] : ld_int4(l.far + 3 * static_cast<int64_t>(k) + i);
}
__device__ __forceinline__ int item_tiles(const List& l, int k) { return item_part(l, k, 1).w; }
__device__ __forceinline__ Item load_item(const List& l, int k) {
  const int4 a = item_part(l, k, 0), b = item_part(l, k, 1), c = item_part(l, k, 2);
  return {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w, c.x, c.y, c.z, c.w};
}

__device__ __forceinline__ QcUserWork user_work(const QcAttnParams& p, int u, int64_t most, bool& bad) {
  QcUserWork w;
  const int count = __ldg(p.offsets + u + 1) - __ldg(p.offsets + u);
  w.len = qc_length(p.lens, u, most, bad);
  w.tiles = static_cast<int>((static_cast<int64_t>(count) * p.group * p.Lq + ATT_BM - 1) / ATT_BM);
  w.units = static_cast<int>((static_cast<uint32_t>(w.len) + ATT_BN - 1) / ATT_BN);
  return w;
}

// Lists this CTA's items; sm: 12 bytes of scratch per user.
__device__ List make_list(const QcAttnParams& p, uint8_t* sm, Aux& x) {
  const int tid = threadIdx.x, n = p.n_users;
  int64_t* cost0 = reinterpret_cast<int64_t*>(sm);
  int32_t* item0 = reinterpret_cast<int32_t*>(cost0 + n);
  const int64_t most = (static_cast<int64_t>(p.max_blocks) << p.blocks_log2) * QC_ROWS;
  const QcShares sh = qc_shares<TL_THREADS, TL_MIN_TILES, TL_ITEM_TILES>(
      p, p.ctas, [&](int u, bool& bad) { return user_work(p, u, most, bad); }, cost0, item0, x.shares);
  List l = {x.list, p.list, 0};
  bool ignored = false;
  const int cta = static_cast<int>(blockIdx.x);
  const int64_t end = cta < sh.parts ? sh.start(cta + 1) : 0;
  if (cta < sh.parts && sh.start(cta) < end) {
    int u = qc_find(cost0, n, sh.start(cta));
    QcUserWork w = user_work(p, u, most, ignored);
    const int i0 = item0[u] + static_cast<int>(qc_div(sh.start(cta) - cost0[u], sh.item_cost(w.units)));
    l.far += 3 * (static_cast<int64_t>(i0) + cta);  // a CTA's first item may be the last of the one before
    int tiles = 0, k = tid;
    for (;; k += TL_THREADS) {
      if (k > 0) {
        u = qc_find(item0, n, i0 + k);
        w = user_work(p, u, most, ignored);
      }
      const int local = i0 + k - item0[u];
      const int64_t pos = cost0[u] + static_cast<int64_t>(local) * sh.item_cost(w.units);
      if (pos >= end) break;
      if (static_cast<int64_t>(i0) + cta + k >= p.max_items) {  // cannot be: the host counts them the same way
        atomicOr(p.status, DEV_ERR_BAD_WORK);
        break;
      }
      const QcPart part = qc_part<TL_MIN_TILES>(sh, cta, w, pos);
      const int hk = static_cast<int>(static_cast<uint32_t>(local) / static_cast<uint32_t>(w.tiles));
      const int seg = __ldg(p.offsets + u);
      int rows = (__ldg(p.offsets + u + 1) - seg) * p.group * p.Lq;
      if (w.units > 0 && part.nt == 0) rows = 0;  // an empty part of an item
      int4* e = k < LIST_NEAR ? x.list + 3 * k : const_cast<int4*>(l.far) + 3 * static_cast<int64_t>(k);
      e[0] = make_int4(u, hk, seg, rows);
      e[1] = make_int4((local - hk * w.tiles) * ATT_BM, w.len, part.t0, part.nt);
      e[2] = make_int4(part.ns, part.slot, part.first, 0);
      tiles += part.nt;
    }
    // the threads' first places behind the end: the least is the number of items
    if (tiles) atomicAdd(&x.n_tiles, static_cast<uint32_t>(tiles));
    atomicMin(&x.n_items, k);
  }
  __syncthreads();  // the entries are visible to the CTA, the scratch is free
  l.count = x.n_items == 0x7fffffff ? 0 : x.n_items;
  return l;
}

// A wait taken by a whole warp: the lanes agree on its outcome, so that a limit
// that expires while the barrier completes never splits the warp before its next
// warp-wide instruction.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, const Smem& s, const QcAttnParams& p) {
  const bool ok = mbar_wait(bar, parity, &s.x->abort, p.timeout_ns, 1);
  return __all_sync(0xffffffffu, ok);
}

// ------------------------------------------------------------------ decode
// Place in the CTA's sequence of key tiles.
struct Cursor {
  int k, t, nt, t0, len;
  const int32_t* table;
  const uint8_t* data;  // the cache, at the item's K/V head and the warp's half
  int page;             // of block lane & 1 (of the warp's two) of tile (t & ~15) + lane / 2
};

// To the first tile of the next item with any; k == count: the end.
__device__ __forceinline__ void cursor_item(const QcAttnParams& p, const List& l, Cursor& c, int half) {
  for (; c.k < l.count; ++c.k) {
    const int4 b = item_part(l, c.k, 1);
    if (b.w == 0) continue;
    const int4 a = item_part(l, c.k, 0);
    c.table = p.table + static_cast<int64_t>(a.x) * p.max_blocks;
    c.data = p.data + ((static_cast<int64_t>(a.y) << p.blocks_log2) * QC_BLOCK_BYTES + half);
    c.len = b.y;
    c.t0 = b.z;
    c.nt = b.w;
    c.t = 0;
    return;
  }
}

// A warp's share of a half tile, in registers: 2 blocks of 16 tokens, of which
// a lane has 4 chunks of 16 code bytes (one token's group of 32 elements) with
// their pairs.  A zero pair makes a chunk of zeros, whatever its codes.
struct Raw {
  uint4 c[4];
  uint32_t sz[4];
};

// Four warps turn the keys' half tiles, four the values', so that one kind's
// waits lie beside the other's work.  The codes come straight from global
// memory into registers, a warp reading 512 contiguous bytes, and each chunk's
// registers are loaded again (for the next tile) as soon as it is decoded.  (Codes that passed
// through shared memory by bulk copies cost a producer warp over a thousand
// cycles a tile to issue.)  A quarter warp's 16-byte stores (2 tokens x 4
// groups) hit all banks because the second 64 elements' pieces lie two places
// further (place ^ 2): like the order within a piece, Q's elements and the
// epilogue follow that.
__device__ void decode_warps(const QcAttnParams& p, const Smem& s, const List& l) {
  const bool values = threadIdx.x >= 32 * (DECODE_WARP0 + DECODE_WARPS);  // one code for both kinds
  const int lane = static_cast<int>(lane_id()), dw = static_cast<int>(threadIdx.x >> 5) & (DECODE_WARPS - 1);
  const int grp = lane & 3, tok8 = lane >> 2;
  uint8_t* const ring = (values ? s.v : s.k) + (dw * 32 + tok8) * 128;
  uint64_t* const full = values ? s.v_full : s.k_full;
  uint64_t* const empty = values ? s.v_empty : s.k_empty;
  const int half = values ? QC_HALF_BYTES : 0;
  uint32_t place[4];  // of the group's four pieces in a row of the tile
#pragma unroll
  for (int k = 0; k < 4; ++k)
    place[k] = (grp >> 1) * HALF_TILE + (((((grp & 1) * 4 + k) ^ (grp & 2)) ^ tok8) << 4);
  const uint32_t tiles = s.x->n_tiles, sixteen = p.sixteen;
  const int64_t page_bytes = (static_cast<int64_t>(p.H_kv) << p.blocks_log2) * QC_BLOCK_BYTES;

  Cursor c = {};
  cursor_item(p, l, c, half);
  Raw raw;
  const uint8_t* src[2];  // the warp's two blocks of the cursor's tile
  int left = 0;           // tokens of the history from the warp's first one on
  // the cursor's tile becomes the one that fetch() reads, and the cursor moves on
  const auto point = [&]() {
    if ((c.t & 15) == 0) {
      const int blk = (c.t0 + c.t + (lane >> 1)) * 8 + dw * 2 + (lane & 1);
      c.page = 0;
      if (c.t + (lane >> 1) < c.nt && blk * QC_ROWS < c.len) {
        c.page = __ldg(c.table + (blk >> p.blocks_log2));
        if (c.page < 0 || c.page >= p.n_pages) {
          atomicOr(p.status, DEV_ERR_CACHE);
          c.page = 0;
        }
      }
    }
    const int blk = (c.t0 + c.t) * 8 + dw * 2;
    left = c.len - blk * QC_ROWS;
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      const int page = __shfl_sync(0xffffffffu, c.page, ((c.t & 15) << 1) | b);
      src[b] = c.data + page * page_bytes + ((blk + b) & ((1 << p.blocks_log2) - 1)) * QC_BLOCK_BYTES;
    }
    if (++c.t == c.nt) {
      ++c.k;
      cursor_item(p, l, c, half);
    }
  };
  // Unconditional (blocks that do not exist have page 0's address), so that the
  // loads stay in flight: nothing touches their registers before the next tile.
  const auto fetch = [&](int i) {
    const uint8_t* blk = src[i >> 1];
    raw.c[i] = __ldg(reinterpret_cast<const uint4*>(blk) + ((i & 1) * 32 + lane));
    raw.sz[i] = __ldg(reinterpret_cast<const uint32_t*>(blk + QC_CODE_BYTES) + ((i & 1) * 32 + lane));
  };
  if (tiles > 0) {
    point();
#pragma unroll
    for (int i = 0; i < 4; ++i) fetch(i);
  }
#pragma unroll 1
  for (uint32_t g = 0; g < tiles; ++g) {
    const int valid = left - tok8;  // > 8 i: the lane's token of chunk i exists
    if (g + 1 < tiles) point();
    if (!values && dw == 0 && lane == 0) *const_cast<volatile uint32_t*>(&s.x->decoded) = g;
    if (!warp_wait(empty + (g & 1u), ((g >> 1) & 1u) ^ 1u, s, p)) return;
    uint8_t* dst = ring + (g & 1u) * ATT_KV_STAGE_BYTES;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t sz = valid > 8 * i ? raw.sz[i] : 0u;
      const uint32_t s2 = __byte_perm(sz, 0, 0x1010), z2 = __byte_perm(sz, 0, 0x3232);
      const uint32_t w[4] = {raw.c[i].x, raw.c[i].y, raw.c[i].z, raw.c[i].w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint4 o = make_uint4(qc_decode<0>(w[k], s2, z2, sixteen), qc_decode<1>(w[k], s2, z2, sixteen),
                                   qc_decode<2>(w[k], s2, z2, sixteen), qc_decode<3>(w[k], s2, z2, sixteen));
        *reinterpret_cast<uint4*>(dst + i * 1024 + place[k]) = o;
      }
      fetch(i);
    }
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(full + (g & 1u));
  }
}

// Asks for the codes of the tiles ahead in L2, four tiles at a time (a lane per
// block of keys and values), as soon as they are AHEAD tiles past the one being
// decoded; across items.
constexpr uint32_t AHEAD = 3;

__device__ void prefetcher(const QcAttnParams& p, const Smem& s, const List& l) {
  const int lane = static_cast<int>(lane_id());
  const int64_t page_bytes = (static_cast<int64_t>(p.H_kv) << p.blocks_log2) * QC_BLOCK_BYTES;
  uint32_t g = 0;
  Cursor c = {};
#pragma unroll 1
  for (cursor_item(p, l, c, 0); c.k < l.count; ++c.k, cursor_item(p, l, c, 0)) {
#pragma unroll 1
    for (int t = 0; t < c.nt; t += 4, g += 4) {
      const int blk = (c.t0 + t) * 8 + lane;
      const bool there = t + (lane >> 3) < c.nt && blk * QC_ROWS < c.len;
      const int page = there ? __ldg(c.table + (blk >> p.blocks_log2)) : -1;
      const uint64_t t_0 = globaltimer_ns();
      // bounded like every wait here, though nothing depends on this warp
      while (!__any_sync(0xffffffffu, g <= *const_cast<volatile uint32_t*>(&s.x->decoded) + AHEAD)) {
        __nanosleep(200);
        if (__any_sync(0xffffffffu, *const_cast<volatile uint32_t*>(&s.x->abort) || globaltimer_ns() - t_0 > p.timeout_ns)) return;
      }
      if (page >= 0 && page < p.n_pages) {
        const uint8_t* block = c.data + page * page_bytes + (blk & ((1 << p.blocks_log2) - 1)) * QC_BLOCK_BYTES;
        asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(block), "n"(QC_BLOCK_BYTES) : "memory");
      }
      __syncwarp();
    }
    g -= (4 - (c.nt & 3)) & 3;  // the last four were fewer
  }
}

// ---------------------------------------------------------------- Q loader
// Rows of the tile into a Q buffer: asynchronous copies (rows behind the last
// become zeros), then each eight elements into the decoded codes' order.
__device__ __forceinline__ int64_t row_index(const QcAttnParams& p, const Item& x, int r, int rows_per_cand) {
  const int slot = r / rows_per_cand;
  return (static_cast<int64_t>(__ldg(p.perm + x.seg + slot)) * p.H + x.hk * p.group) * p.Lq + (r - slot * rows_per_cand);
}

__device__ void q_loader(const QcAttnParams& p, const Smem& s, const List& l) {
  const int lane = static_cast<int>(lane_id());
  const int rows_per_cand = p.group * p.Lq;
  uint32_t qc = 0;
  for (int k = 0; k < l.count; ++k) {
    const Item x = load_item(l, k);
    if (x.nt == 0) continue;
    int64_t at[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = x.row0 + i * 32 + lane;
      at[i] = r < x.n_rows ? row_index(p, x, r, rows_per_cand) * ATT_D : -1;
    }
    const uint32_t qb = qc & 1u;
    if (!warp_wait(&s.q_empty[qb], ((qc >> 1) & 1u) ^ 1u, s, p)) return;
    ++qc;
    uint8_t* q = s.q + qb * ATT_Q_TILE_BYTES;
    const int chunk = lane & 15;
    const uint32_t col = static_cast<uint32_t>((chunk >> 3) * HALF_TILE);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll 4
      for (int j = 0; j < 16; ++j) {
        const int r = 2 * j + (lane >> 4);
        const int64_t a = __shfl_sync(0xffffffffu, at[i], r);
        const uint32_t dst = smem_u32(q) + col + (i * 32 + r) * 128 + (((chunk & 7) ^ (r & 7)) << 4);
        const uint16_t* src = p.Q + (a < 0 ? 0 : a + (chunk ^ ((chunk >> 2) & 2)) * 8);  // places 8.. of a row: ^ 2
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(a < 0 ? 0 : 16) : "memory");
      }
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncwarp();
#pragma unroll 8
    for (int j = 0; j < 64; ++j) {  // any order of the tile's 2048 pieces
      uint4* at16 = reinterpret_cast<uint4*>(q) + j * 32 + lane;
      const uint4 v = *at16;
      *at16 = make_uint4(__byte_perm(v.x, v.z, 0x5410), __byte_perm(v.x, v.z, 0x7632), __byte_perm(v.y, v.w, 0x5410),
                         __byte_perm(v.y, v.w, 0x7632));
    }
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(&s.q_full[qb]);
  }
}

// ----------------------------------------------------------------- issuers
__device__ void s_issuer(const QcAttnParams& p, const Smem& s, uint32_t tmem, const List& l) {
  uint32_t g = 0, qu = 0;
  for (int k = 0; k < l.count; ++k) {
    const int nt = item_tiles(l, k);
    if (nt == 0) continue;
    const uint32_t qb = qu & 1u;
    const uint32_t q_base = smem_u32(s.q + qb * ATT_Q_TILE_BYTES);
    for (int jt = 0; jt < nt; ++jt, ++g) {
      const uint32_t b = g & 1u, sb = g % S_BUFS;
      if (!warp_wait(&s.k_full[b], (g >> 1) & 1u, s, p)) return;
      if (g >= S_BUFS && !warp_wait(&s.pv_done[sb], (g / S_BUFS - 1) & 1u, s, p)) return;
      if (jt == 0 && !warp_wait(&s.q_full[qb], (qu >> 1) & 1u, s, p)) return;
      tc_fence_after();
      if (elect_one()) {
        issue_qk_ss(tmem + TM_S + sb * 128, q_base, smem_u32(s.k + b * ATT_KV_STAGE_BYTES));
        mma_commit(&s.s_full[sb]);
        mma_commit(&s.k_empty[b]);
        if (jt + 1 == nt) mma_commit(&s.q_empty[qb]);
      }
      __syncwarp();
    }
    ++qu;
  }
}

__device__ void pv_issuer(const QcAttnParams& p, const Smem& s, uint32_t tmem, const List& l) {
  uint32_t g = 0, ou = 0;
  for (int k = 0; k < l.count; ++k) {
    const int nt = item_tiles(l, k);
    for (int jt = 0; jt < nt; ++jt, ++g) {
      const uint32_t b = g & 1u, sb = g % S_BUFS;
      if (!warp_wait(&s.p_full[sb], (g / S_BUFS) & 1u, s, p)) return;
      if (!warp_wait(&s.v_full[b], (g >> 1) & 1u, s, p)) return;
      if (jt == 0 && !warp_wait(s.o_empty, (ou & 1u) ^ 1u, s, p)) return;
      tc_fence_after();
      if (elect_one()) {
        issue_pv(tmem + TM_O, tmem + TM_S + sb * 128, smem_u32(s.v + b * ATT_KV_STAGE_BYTES), jt > 0);
        mma_commit(&s.pv_done[sb]);
        mma_commit(&s.v_empty[b]);
        if (jt + 1 == nt) mma_commit(s.o_full);
      }
      __syncwarp();
      if (jt + 1 == nt) ++ou;
    }
  }
}

// An issuer leaves when its products in flight have ended (they need nothing
// more), or a second is over: whichever warp's wait ran out, the CTA does not free
// their memory before.  (Only where a wait ran out does anything remain in
// flight here.  Asked for by a flag behind the roles' last barrier instead, the
// drain cost 2% of the kernel.)
__device__ void drain(uint64_t* bar) {
  __syncwarp();
  if (elect_one()) mma_commit(bar);
  __syncwarp();
  const uint64_t t0 = globaltimer_ns();
  while (!mbar_try_wait(bar, 0) && globaltimer_ns() - t0 < 1000000000ull) {}
  __syncwarp();
}

// ---------------------------------------------------- softmax and epilogue
struct Lane {
  int quarter, half, r;  // half: the warp's group (its key tiles) and its d half of O
};

// The chain of reference maxima through the tiles of both groups (attn.cu
// describes it): the high 30 bits of the value, the tile's tag below (a reader finds
// the word it waits for or the one before).  A score may lie above its reference by
// what the cut bits are worth, 2^-21 of it, and P then by two to that power: in range
// for scores up to 2^27 in magnitude.
constexpr uint32_t CHAIN_TAG = 3u;
__device__ __forceinline__ float chain_value(float m) { return __uint_as_float(__float_as_uint(m) & ~CHAIN_TAG); }
__device__ __forceinline__ void chain_post(const Smem& s, int r, uint32_t tag, float m) {
  const uint32_t w = (__float_as_uint(m) & ~CHAIN_TAG) | (tag & CHAIN_TAG);
  asm volatile("st.volatile.shared.b32 [%0], %1;" ::"r"(smem_u32(s.x->chain + r)), "r"(w) : "memory");
}
__device__ __forceinline__ uint32_t chain_load(const Smem& s, int r) {
  uint32_t w;
  asm volatile("ld.volatile.shared.b32 %0, [%1];" : "=r"(w) : "r"(smem_u32(s.x->chain + r)) : "memory");
  return w;
}
// The softmax warps' waits for barriers are taken lane by lane, without a vote
// (which cost up to 4% of the kernel), and a lane whose wait ran out does not
// leave: it goes on with whatever it finds, as the abort flag has made the call's
// results worthless (no address comes from that, the tensor memory stays allocated
// until the products have ended, and barriers still count whole warps), until the
// warp leaves as one at the chain, where it votes in any case: the tag that such a
// lane wants there is one that no word has (those hold g or g - 1), so that it looks
// at the flag.
__device__ __forceinline__ uint32_t tag_wanted(uint32_t g, bool there) { return (g + (there ? 0u : 2u)) & CHAIN_TAG; }
__device__ __forceinline__ bool chain_wait(const QcAttnParams& p, const Smem& s, int r, uint32_t tag, float& m) {
  uint32_t w = chain_load(s, r);
  bool ok = true;
  if ((w & CHAIN_TAG) != tag) {
    const uint64_t t0 = globaltimer_ns();
    for (uint32_t it = 1;; ++it) {
      w = chain_load(s, r);
      if ((w & CHAIN_TAG) == tag) break;
      if ((it & 63u) == 0) {
        volatile uint32_t* abort = &s.x->abort;
        if (*abort) {
          ok = false;
          break;
        }
        if (globaltimer_ns() - t0 > p.timeout_ns) {
          *abort = 1;
          ok = false;
          break;
        }
      }
    }
  }
  m = __uint_as_float(w & ~CHAIN_TAG);
  return __all_sync(0xffffffffu, ok);
}

// Scores of columns from n on: none.
__device__ __forceinline__ void mask_columns(uint32_t (&v)[32], int n) {
#pragma unroll
  for (int j = 0; j < 32; ++j)
    if (j >= n) v[j] = __float_as_uint(-INFINITY);
}

// The running maximum of 32 columns' scores.
__device__ __forceinline__ void row_max(const uint32_t (&v)[32], float& mx) {
  float mx0 = mx, mx1 = -INFINITY;
#pragma unroll
  for (int j = 0; j < 32; j += 4) {
    mx0 = fmax3(mx0, __uint_as_float(v[j]), __uint_as_float(v[j + 1]));
    mx1 = fmax3(mx1, __uint_as_float(v[j + 2]), __uint_as_float(v[j + 3]));
  }
  mx = fmaxf(mx0, mx1);
}

// p = 2^(s sl - m) of 32 columns, summed into l0, l1, and as bf16 pairs to TMEM.
__device__ __forceinline__ void row_exp(const uint32_t (&v)[32], float sl, float m, float& l0, float& l1, uint32_t to) {
  uint32_t pk[16];
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    float t0, t1;
    fma2(t0, t1, __uint_as_float(v[2 * j]), __uint_as_float(v[2 * j + 1]), sl, -m);
    const float p0 = ex2(t0);
    const float p1 = ex2(t1);
    add2(l0, l1, p0, p1);
    pk[j] = pack_bf16x2(p0, p1);
  }
  tmem_st16(to, pk);
}

// A finished item whose O has not been read out yet: its place in the list
// (-1: none), and what this thread read of it early.
struct Done {
  int k;
  int cand;  // the candidate of this thread's row, if the row exists
};

// Packs 16 columns of finished rows, scaled, in element order: column 8k + j
// holds element 8 (k ^ 2 half) + (j >> 1) + 4 (j & 1) of the warp's half.
__device__ __forceinline__ void pack_columns(const float* o, float inv, uint32_t* w) {
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const float* e = o + 8 * k;
    w[4 * k + 0] = pack_bf16x2(e[0] * inv, e[2] * inv);
    w[4 * k + 1] = pack_bf16x2(e[4] * inv, e[6] * inv);
    w[4 * k + 2] = pack_bf16x2(e[1] * inv, e[3] * inv);
    w[4 * k + 3] = pack_bf16x2(e[5] * inv, e[7] * inv);
  }
}

// The c-th 16 packed columns of the warp's 64 to global memory: through 1 KB of
// shared memory, so that every store fills whole 32-byte sectors.
__device__ __forceinline__ void store_columns(const QcAttnParams& p, uint8_t* stage, const Lane& ln, int64_t row, int c,
                                              const uint32_t* w) {
  const int lane = static_cast<int>(lane_id());
#pragma unroll
  for (int k = 0; k < 2; ++k)
    *reinterpret_cast<uint4*>(stage + lane * 32 + ((k ^ ((lane >> 2) & 1)) << 4)) =
        make_uint4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]);
  __syncwarp();
  const int piece = lane & 1;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int r = 16 * i + (lane >> 1);
    const int64_t at = __shfl_sync(0xffffffffu, row, r);
    const uint4 v = *reinterpret_cast<const uint4*>(stage + r * 32 + ((piece ^ ((r >> 2) & 1)) << 4));
    if (at >= 0) reinterpret_cast<uint4*>(p.O + at * ATT_D + ln.half * 64)[(2 * c + piece) ^ (2 * ln.half)] = v;
  }
  __syncwarp();
}

__device__ __forceinline__ float inverse(float l) { return l > 0.f ? 1.0f / l : (l == 0.f ? 0.f : l); }
__device__ __forceinline__ void store_lse(const QcAttnParams& p, int64_t row, float m, float l) {
  p.lse[row] = l > 0.f ? (m + __log2f(l)) * 0.69314718055994531f : (l == 0.f ? -INFINITY : l);
}

// How many splits of an item's tile have a piece's rows in their slots.
__device__ __forceinline__ uint32_t* ticket(const QcAttnParams& p, const Item& x, int quarter, int half) {
  return p.tickets + static_cast<int64_t>(x.first) * 8 + quarter * 2 + half;
}

// A split's piece of O (this warp's 32 rows x 64 columns) to its slot; the
// warp that completes the tile's piece adds the splits in order and stores it.
__device__ __forceinline__ void join_splits(const QcAttnParams& p, uint32_t Ot, const Item& ro, int64_t row, const Lane& ln,
                                            float mf, float l, uint8_t* stage, uint64_t* o_empty) {
  const int lane = static_cast<int>(lane_id());
  // slot: [half][64 columns][128 rows], then [half][m, l][128 rows]
  constexpr int64_t SLOT = TL_PART;
  const int64_t in = static_cast<int64_t>(ln.half) * 64 * ATT_BM + ln.r;
  const int64_t ml = 2 * 64 * ATT_BM + ln.half * 2 * ATT_BM + ln.r;
  float* mine = p.part + ro.slot * SLOT;
#pragma unroll 1
  for (int c = 0; c < 2; ++c) {
    uint32_t o[32];
    tmem_ld32(Ot + c * 32, o);
    tmem_ld_wait(o);
#pragma unroll
    for (int j = 0; j < 32; ++j) __stcg(mine + in + (c * 32 + j) * ATT_BM, __uint_as_float(o[j]));
  }
  __stcg(mine + ml, mf);
  __stcg(mine + ml + ATT_BM, l);
  tc_fence_before();
  mbar_arrive(o_empty);
  __threadfence();
  __syncwarp();
  uint32_t last = 0;
  if (lane == 0) {
    uint32_t* t = ticket(p, ro, ln.quarter, ln.half);
    last = atomicAdd(t, 1u) + 1 == static_cast<uint32_t>(ro.ns);
    if (last) *t = 0;  // zero again for the next call
  }
  last = __shfl_sync(0xffffffffu, last, 0);
  if (!last) return;
  __threadfence();
  const auto part = [&](int k) { return p.part + qc_slot(ro.first, k) * SLOT; };
  float M = -INFINITY;
  for (int k = 0; k < ro.ns; ++k) M = fmaxf(M, __ldcg(part(k) + ml));
  float L = 0.f;
  for (int k = 0; k < ro.ns; ++k) {
    const float m = __ldcg(part(k) + ml);
    L += (m == -INFINITY ? 0.f : ex2(m - M)) * __ldcg(part(k) + ml + ATT_BM);
  }
  const float inv = inverse(L);
  if (p.lse && row >= 0 && ln.half == 0) store_lse(p, row, M, L);
#pragma unroll 1
  for (int c = 0; c < 4; ++c) {
    float acc[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) acc[j] = 0.f;
#pragma unroll 2
    for (int k = 0; k < ro.ns; ++k) {
      const float* sp = part(k);
      const float m = __ldcg(sp + ml);
      const float f = m == -INFINITY ? 0.f : ex2(m - M);
      float x[16];
#pragma unroll
      for (int j = 0; j < 16; ++j) x[j] = __ldcg(sp + in + (c * 16 + j) * ATT_BM);
#pragma unroll
      for (int j = 0; j < 16; ++j) acc[j] = fmaf(x[j], f, acc[j]);
    }
    uint32_t w[8];
    pack_columns(acc, inv, w);
    store_columns(p, stage, ln, row, c, w);
  }
}

// An item's epilogue: the groups' row sums joined (both have posted theirs), O
// out of TMEM to global memory (or through the partial rows of a split item).
__device__ __forceinline__ void epilogue(const QcAttnParams& p, const Smem& s, uint32_t Ot, const List& list, const Done& done,
                                         const Lane& ln, uint32_t& ou) {
  const Item x = load_item(list, done.k);
  mbar_wait(&s.fin_full[ou & 1u], (ou >> 1) & 1u, &s.x->abort, p.timeout_ns, 1);
  const float2 f0 = s.x->fin[ou & 1u][0][ln.r], f1 = s.x->fin[ou & 1u][1][ln.r];
  mbar_wait(s.o_full, ou & 1u, &s.x->abort, p.timeout_ns, 1);
  ++ou;
  if (x.row0 + ln.quarter * 32 >= x.n_rows) {  // none of the warp's rows exists
    mbar_arrive(s.o_empty);
    return;
  }
  const float mf = fmaxf(f0.x, f1.x);
  // a group without a reference (no tile, or no score that is a number) has the sum 0, or NaN
  const float l = (f0.x == -INFINITY ? f0.y : f0.y * ex2(f0.x - mf)) + (f1.x == -INFINITY ? f1.y : f1.y * ex2(f1.x - mf));
  const int rows_per_cand = p.group * p.Lq, rr = x.row0 + ln.r;
  const int64_t row = rr < x.n_rows
      ? (static_cast<int64_t>(done.cand) * p.H + x.hk * p.group) * p.Lq + rr % rows_per_cand : -1;
  tc_fence_after();
  uint8_t* stage = s.out + (ln.quarter * 2 + ln.half) * STAGE_BYTES;
  if (x.ns > 1) {
    join_splits(p, Ot, x, row, ln, mf, l, stage, s.o_empty);
    return;
  }
  const float inv = inverse(l);
  uint32_t w[32];
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    uint32_t o[32];
    tmem_ld32(Ot + c * 32, o);
    tmem_ld_wait(o);
    pack_columns(reinterpret_cast<const float*>(o), inv, w + 16 * c);
    pack_columns(reinterpret_cast<const float*>(o) + 16, inv, w + 16 * c + 8);
  }
  tc_fence_before();
  mbar_arrive(s.o_empty);
  if (p.lse && row >= 0 && ln.half == 0) store_lse(p, row, mf, l);
#pragma unroll
  for (int c = 0; c < 4; ++c) store_columns(p, stage, ln, row, c, w + 8 * c);
}

// Returns the first item whose epilogue has not run (the list's end, unless a wait
// ran out).
__device__ int softmax_warps(const QcAttnParams& p, const Smem& s, uint32_t tmem, const List& list) {
  const int warp = threadIdx.x >> 5;
  Lane ln;
  ln.quarter = warp & 3;
  ln.half = (warp - SOFTMAX_WARP0) >> 2;
  ln.r = (ln.quarter << 5) + static_cast<int>(lane_id());
  const int grp = ln.half;
  const uint32_t lane_base = static_cast<uint32_t>(ln.quarter * 32) << 16;
  const uint32_t Oall = tmem + lane_base + TM_O;
  const uint32_t Ot = Oall + grp * 64;
  const float sl = p.scale_log2;
  const int rows_per_cand = p.group * p.Lq;
  uint32_t g0 = 0, ic = 0, ou = 0;  // tiles before the item, items finished, items read out
  Done prev = {-1, 0};

  // One turn more than there are items: the last one's epilogue.  The code of a
  // tile and of an epilogue stands once each: with the SM's 20 warps at four
  // kinds of work, what is copied into several places is fetched from behind the
  // instruction cache again and again.
  for (int k = 0; k <= list.count; ++k) {
    int nt = 0, rem = 0, cand = 0;  // rem: tokens from the split's first on
    bool rows_here = false;
    if (k < list.count) {
      const Item x = load_item(list, k);
      const int rr = x.row0 + ln.r;
      if (rr < x.n_rows) cand = __ldg(p.perm + x.seg + rr / rows_per_cand);
      rows_here = x.row0 + ln.quarter * 32 < x.n_rows;
      nt = x.nt;
      rem = x.len - x.t0 * ATT_BN;
      if (nt == 0) {  // no tokens: O = 0, LSE = -inf
        if (rr < x.n_rows) {
          const int64_t row = (static_cast<int64_t>(cand) * p.H + x.hk * p.group) * p.Lq + rr % rows_per_cand;
          const uint4 z = make_uint4(0, 0, 0, 0);
#pragma unroll
          for (int c = 0; c < 8; ++c) reinterpret_cast<uint4*>(p.O + row * ATT_D + grp * 64)[c] = z;
          if (p.lse && grp == 0) p.lse[row] = -INFINITY;
        }
        continue;
      }
    }
    bool epi = prev.k >= 0;  // the previous item's epilogue is still to come
    float mref = -INFINITY, l = 0.f;
    int jt = static_cast<int>((static_cast<uint32_t>(grp) - g0) & 1u);
    do {
      const uint32_t g = g0 + static_cast<uint32_t>(jt), sb = g % S_BUFS;
      float mprev = 0.f, mj = 0.f;
      bool rescale = false;
      if (jt < nt) {
        const uint32_t St = tmem + lane_base + TM_S + sb * 128;
        const uint32_t want = tag_wanted(g, mbar_wait(&s.s_full[sb], (g / S_BUFS) & 1u, &s.x->abort, p.timeout_ns, 1));
        tc_fence_after();
        if (!rows_here) {  // none of the warp's 32 rows exists: keep the hand-shakes in step, nothing else
          if (!chain_wait(p, s, ln.r, want, mprev)) return epi ? prev.k : k;
          chain_post(s, ln.r, g + 1, 0.f);
        } else {
          // two passes over the row, 32 columns at a time with the next ones on
          // their way from TMEM (whole rows in registers, unrolled, are too much for
          // the instruction cache); the first pass goes down so that the second
          // begins with what it ended on
          const int ncols = min(ATT_BN, rem - jt * ATT_BN);
          uint32_t va[32], vb[32];
          if (ncols < ATT_BN) {  // a history's last tile: scores behind its end become -inf where they lie
#pragma unroll 1
            for (int c = ncols >> 5; c < 4; ++c) {
              tmem_ld32p(St + 32 * c, va);
              tmem_ld_wait();
              reg_fence32(va);
              mask_columns(va, ncols - 32 * c);
              tmem_st32(St + 32 * c, va);
            }
            tmem_st_wait();
          }
          float mx = -INFINITY;
          tmem_ld32p(St + 96, va);
          tmem_ld_wait();
          reg_fence32(va);
#pragma unroll 1
          for (int h = 1; h >= 0; --h) {
            tmem_ld32p(St + 64 * h, vb);
            row_max(va, mx);
            tmem_ld_wait();
            reg_fence32(vb);
            tmem_ld32p(St + 32, va);  // (the second time of no use)
            row_max(vb, mx);
            tmem_ld_wait();
            reg_fence32(va);
          }
          mx *= sl;
          const uint32_t cw = chain_load(s, ln.r);
          mprev = __uint_as_float(cw & ~CHAIN_TAG);
          if (!__all_sync(0xffffffffu, (cw & CHAIN_TAG) == want) && !chain_wait(p, s, ln.r, want, mprev)) return epi ? prev.k : k;
          if (jt == 0) mprev = -INFINITY;
          rescale = __any_sync(0xffffffffu, mx > mprev + RESCALE_THRESHOLD);
          mj = rescale ? chain_value(fmaxf(mprev, mx)) : mprev;
          chain_post(s, ln.r, g + 1, mj);
          if (mj != mref) {
            l *= ex2(mref - mj);
            mref = mj;
          }
          float l0 = 0.f, l1 = 0.f;
          // P takes the place of the scores already read
#pragma unroll 1
          for (int h = 0; h < 2; ++h) {
            tmem_ld32p(St + 64 * h + 32, va);
            row_exp(vb, sl, mj, l0, l1, St + 32 * h);
            tmem_ld_wait();
            reg_fence32(va);
            if (h == 0) tmem_ld32p(St + 64, vb);
            row_exp(va, sl, mj, l0, l1, St + 32 * h + 16);
            tmem_ld_wait();
            reg_fence32(vb);
          }
          l += l0 + l1;
        }
      }
      // Between the group's first tile of this item and that tile's P.V, which
      // waits for O anyway.
      if (epi) epilogue(p, s, Ot, list, prev, ln, ou);
      epi = false;
      if (jt < nt) {
        if (rescale && jt > 0) {
          const uint32_t gp = g - 1;
          mbar_wait(&s.pv_done[gp % S_BUFS], (gp / S_BUFS) & 1u, &s.x->abort, p.timeout_ns, 1);
          tc_fence_after();
          const float alpha = ex2(mprev - mj);
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            uint32_t o[32];
            tmem_ld32(Oall + c * 32, o);
            tmem_ld_wait(o);
#pragma unroll
            for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * alpha);
            tmem_st32(Oall + c * 32, o);
          }
        }
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(&s.p_full[sb]);
      }
      jt += 2;
    } while (jt < nt);
    if (k < list.count) {
      g0 += static_cast<uint32_t>(nt);
      prev.k = k;
      prev.cand = cand;
      s.x->fin[ic & 1u][grp][ln.r] = make_float2(mref, l);
      mbar_arrive(&s.fin_full[ic & 1u]);
      ++ic;
    }
  }
  return list.count;
}

// A softmax warp that gave up: its tickets of the items from k on, so that every
// piece of a split tile has all of its tickets in the end, whoever gave up, and its
// count is zero again for the next call.  (What the last to finish then joins is of
// no worth.)
__device__ void abandon(const QcAttnParams& p, const List& list, int k) {
  const int warp = static_cast<int>(threadIdx.x >> 5), quarter = warp & 3, half = (warp - SOFTMAX_WARP0) >> 2;
  for (; k < list.count; ++k) {
    const Item x = load_item(list, k);
    if (x.nt == 0 || x.ns == 1 || x.row0 + quarter * 32 >= x.n_rows || lane_id() != 0) continue;
    uint32_t* t = ticket(p, x, quarter, half);
    if (atomicAdd(t, 1u) + 1 == static_cast<uint32_t>(x.ns)) *t = 0;
  }
}

__global__ void __launch_bounds__(TL_THREADS, 1) qattn_tile_kernel(const QcAttnParams p) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t pad = ((raw + 1023u) & ~1023u) - raw;
  if (pad + SMEM_USED > SMEM_ALLOC) {
    if (threadIdx.x == 0) atomicOr(p.status, DEV_ERR_SMEM_LAYOUT);
    return;
  }
  const Smem s = carve(smem_raw + pad);
  const int warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) {
    for (int i = 0; i < S_BUFS; ++i) {
      mbar_init(&s.s_full[i], 1);
      mbar_init(&s.p_full[i], GROUP_THREADS);
      mbar_init(&s.pv_done[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s.fin_full[i], SOFTMAX_THREADS);
      mbar_init(&s.drain[i], 1);
      mbar_init(&s.q_full[i], 1);
      mbar_init(&s.q_empty[i], 1);
      mbar_init(&s.k_full[i], DECODE_WARPS + ((p.debug & DEBUG_WITHHOLD_KEYS) && (blockIdx.x & 3u) == 1u ? 1 : 0));
      mbar_init(&s.k_empty[i], 1);
      mbar_init(&s.v_full[i], DECODE_WARPS);
      mbar_init(&s.v_empty[i], 1);
    }
    mbar_init(s.o_full, 1);
    mbar_init(s.o_empty, SOFTMAX_THREADS);
    for (int r = 0; r < ATT_BM; ++r) s.x->chain[r] = 0;
    s.x->abort = 0;
    s.x->n_tiles = 0;
    s.x->n_items = 0x7fffffff;
    s.x->decoded = 0;
    fence_barrier_init();
    fence_proxy_async_smem();
  }
  if (warp == 1) {
    tmem_alloc(&s.x->tmem_slot, 512);
    tmem_relinquish();
  }
  const List l = make_list(p, smem_raw + pad, *s.x);
  fence_proxy_async_smem();  // the scratch of the list lay where bulk copies go
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s.x->tmem_slot;

  if (warp < SOFTMAX_WARP0) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(CTRL_REGS));
    if (warp == 0) prefetcher(p, s, l);
    else if (warp == 1) s_issuer(p, s, tmem, l);
    else if (warp == 2) pv_issuer(p, s, tmem, l);
    else if (warp == 3) q_loader(p, s, l);
    if (warp == 1 || warp == 2) drain(&s.drain[warp - 1]);
  } else if (warp < DECODE_WARP0) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(SOFTMAX_REGS));
    const int k = softmax_warps(p, s, tmem, l);
    if (k < l.count) abandon(p, l, k);
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(DECODE_REGS));
    decode_warps(p, s, l);
  }

  tc_fence_before();
  __syncthreads();
  if (s.x->abort && threadIdx.x == 0) atomicOr(p.status, DEV_ERR_PIPE_TIMEOUT);
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

}  // namespace

size_t qattn_tile_smem() { return SMEM_ALLOC; }
size_t qattn_tile_part_elems(int num_sms) { return static_cast<size_t>(QA_SLOTS) * num_sms * TL_PART; }
// Entries of the list: one per tile, and one per CTA for a tile it shares.
int64_t qattn_tile_items(int64_t rows, int n_users, int H_kv, int num_sms) {
  return (rows / ATT_BM + n_users) * H_kv + num_sms;
}

cudaError_t launch_qattn_tile(const QcAttnParams& p, cudaStream_t s) {
  cudaError_t e = cudaFuncSetAttribute(qattn_tile_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       static_cast<int>(SMEM_ALLOC));
  if (e != cudaSuccess) return e;
  qattn_tile_kernel<<<p.ctas, TL_THREADS, SMEM_ALLOC, s>>>(p);
  return cudaGetLastError();
}

}  // namespace ikbo
