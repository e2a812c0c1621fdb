// qattn.cu -- broadcast attention straight from the 4-bit cache, for few
// query rows per user and K/V head.
//
//   O[i,h] = softmax(Q[i,h] K[map[i],g]^T * scale) V[map[i],g]
//
// The rows that read one history (user u, K/V head g) are its candidates'
// queries of the heads that share g: R = count[u] * (H / H_kv) * Lq.  With few
// of them the operator is bound by the cache's bytes (160 a token and head),
// and the work that counts besides is turning 4-bit codes into operands.
// Here that happens once per tile of 8 or 16 rows, in registers: the operand
// layout of the 16x8x16 warp-level matrix instruction lets a lane read its
// share of a block as whole 16- or 8-byte pieces of codes (the order of
// elements along a product's inner dimension is free, so Q is permuted to
// match), and one AND-OR and one FMA make two operands of two codes.  A tcgen05
// product would have to write them to shared memory first and would use 8 to
// 16 of its 128 rows.
//
// The products are S^T = K Q^T (16 tokens x 8 rows) and O^T = V^T P^T (16
// elements x 8 rows): the few rows are the instruction's short side, so that 8
// of them take half the products and registers of 16, and 12 warps fit on an SM
// instead of 8.  P^T comes out of the first product as the second one needs it
// but for a transposition of 8 x 8 pairs within the warp.
//
// Work: a tile is 8 or 16 rows of one (u, g); its history is cut into parts of
// whole blocks (16 tokens, 2560 contiguous bytes) where the CTAs' equal shares
// end.  A CTA works through its share, item by item; its four warps take every
// fourth block (with an item or more for every warp each has a share of its own
// instead, which needs no joining of warps), loading the next block's codes into the
// registers of the one just decoded (no barrier in the loop; the lines of the
// block after that are asked for in L2), and keep their own running maximum,
// sum and O in registers.  The warps are joined through shared memory; parts of
// a tile leave unnormalised rows, which the last one to finish adds in order (so
// results repeat bit for bit).
//
// Softmax in fp32 in the log2 domain.  The reference maximum moves only when
// a score exceeds it by more than 2^8 (one vote per block instead of four
// shuffles).  P is rounded to bf16 for P.V (at most 2^-8 relative, as in
// ikbo_attn_forward) and so is the sum that divides O: one more column of ones
// beside V, so that a common rounding of P cancels.  The log-sum-exp has a sum
// of its own, of the unrounded values.
//
// What bounds it: each warp's chain through a block, 360 instructions from the
// codes over two products and the vote between them to the next block, with 12
// warps on an SM to fill its gaps.  No unit is full (memory 55%, issue 55%, the
// integer pipe 54% with the codes' shifts and AND-ORs), and the instructions'
// fixed latencies are the largest stall (1.1 warps an issue, memory 0.6).  One candidate for each of 64 histories of
// 4096 tokens, 8 heads of 8 queries: 84.6 us, 3.99 TB/s of the cache (0.59 of the
// measured rate); 16 rows each 105.  Measured slower: 4 CTAs an SM 88.7 us (128
// registers), 5 CTAs 98.9; the rows as the products' long side 99.9.  For 16
// rows (histories of 1200 to 4096 tokens) that layout was the faster, 72.3 us
// against 75.1, and 77.2 with 3 CTAs an SM in 168 registers, which spill.
#include <cuda_bf16.h>

#include "ptx.cuh"
#include "qcache_internal.h"

namespace ikbo {
namespace {

constexpr int QT_WARPS = 4;
constexpr int QT_THREADS = 32 * QT_WARPS;
constexpr int QT_MIN_BLOCKS = 4 * QT_WARPS;  // blocks of a split, at least
constexpr int QT_ITEM_BLOCKS = 24;           // what an item costs beside its blocks, in blocks
constexpr int QT_SOLO_MIN_BLOCKS = 8, QT_SOLO_ITEM_BLOCKS = 4;  // the same where warps work alone
constexpr float QT_THRESHOLD = 8.0f;         // log2 units
constexpr int QT_EXTRA = 3;                  // per row besides O: reference, sum, sum of the log-sum-exp

// By rows of a tile (8 kRows8): CTAs resident on an SM, floats of a part's
// partial rows, bytes of a warp's O on its way to the others.
__host__ __device__ constexpr int qt_ctas_per_sm(int rows8) { return rows8 == 1 ? 3 : 2; }
__host__ __device__ constexpr int qt_part(int rows8) { return 8 * rows8 * (QC_D + QT_EXTRA); }
__host__ __device__ constexpr int qt_warp_bytes(int rows8) { return 8 * rows8 * QC_D * 4; }

struct QtShared {
  float m[QT_WARPS][16];
  float l[QT_WARPS][16];
  float le[QT_WARPS][16];
  QcSharesScratch shares;
  uint32_t last;
};

__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// c += the columns' sums of the bf16 matrix b (16 x 8): a product with ones, of
// which one row is kept.
__device__ __forceinline__ void mma_sums(float (&c)[2], uint32_t b0, uint32_t b1) {
  float d2, d3;
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%4,%4,%4}, {%5,%6}, {%0,%1,%7,%7};"
      : "+f"(c[0]), "+f"(c[1]), "=f"(d2), "=f"(d3)
      : "r"(0x3F803F80u), "r"(b0), "r"(b1), "f"(0.f));
}

// The 8 x 8 matrix of 16-bit elements that a warp holds, two of a row per lane.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

template <int kRows>
__device__ __forceinline__ QcUserWork user_work(const QcAttnParams& p, int u, int64_t most, bool& bad) {
  QcUserWork w;
  const int count = __ldg(p.offsets + u + 1) - __ldg(p.offsets + u);
  w.len = qc_length(p.lens, u, most, bad);
  w.tiles = static_cast<int>((static_cast<int64_t>(count) * p.group * p.Lq + kRows - 1) / kRows);
  w.units = static_cast<int>((static_cast<uint32_t>(w.len) + QC_ROWS - 1) / QC_ROWS);
  return w;
}

// Place of 16-byte piece c (of 32) of a row of a warp's staged O: pieces are
// permuted so that the lanes' stores (rows 2t, pieces 4g) spread over the banks.
__device__ __forceinline__ int o_piece(int row, int c) { return c ^ ((row >> 1) & 3); }

__device__ __forceinline__ void add_scaled(float4& a, const float4 x, float f) {
  a.x = fmaf(x.x, f, a.x);
  a.y = fmaf(x.y, f, a.y);
  a.z = fmaf(x.z, f, a.z);
  a.w = fmaf(x.w, f, a.w);
}

// A warp that works alone: its rows (lane (g, t): elements 16g .. 16g + 15 of
// rows 2t and 2t + 1 of each eight) to O, or as a part's rows to its slot, where
// the last of the parts adds them in order.
template <int kRows8>
__device__ __forceinline__ void solo_rows(const QcAttnParams& p, const QcPart& part,
                                          float (&o)[kRows8][8][4], float (&m)[kRows8][2], float (&sum)[kRows8][2],
                                          float (&le)[kRows8][2], int tile, int hk, int seg, int n_rows, int rows_per_cand) {
  constexpr int kRows = 8 * kRows8, kPart = qt_part(kRows8);
  const int lane = static_cast<int>(threadIdx.x) & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
  for (int n = 0; n < kRows8; ++n)
#pragma unroll
    for (int e = 0; e < 2; ++e)
#pragma unroll
      for (int d = 4; d < 32; d <<= 1) le[n][e] += __shfl_xor_sync(0xffffffffu, le[n][e], d);
  if (part.ns > 1) {
    float* mine = p.part + static_cast<int64_t>(part.slot) * kPart;
#pragma unroll
    for (int n = 0; n < kRows8; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = 8 * n + 2 * t + e;
#pragma unroll
        for (int quad = 0; quad < 4; ++quad)
          __stcg(reinterpret_cast<float4*>(mine) + r * 32 + 4 * g + quad,
                 make_float4(o[n][2 * quad][e], o[n][2 * quad][2 + e], o[n][2 * quad + 1][e], o[n][2 * quad + 1][2 + e]));
        if (g == 0) {
          float* ex = mine + kRows * QC_D + r;
          __stcg(ex, m[n][e]);
          __stcg(ex + kRows, sum[n][e]);
          __stcg(ex + 2 * kRows, le[n][e]);
        }
      }
    __threadfence();
    __syncwarp();
    uint32_t last = 0;
    if (lane == 0) {
      last = atomicAdd(p.tickets + part.first, 1u) + 1 == static_cast<uint32_t>(part.ns);
      if (last) p.tickets[part.first] = 0;  // zero again for the next call
    }
    if (!__shfl_sync(0xffffffffu, last, 0)) return;
    __threadfence();
    const auto rows = [&](int k) { return p.part + static_cast<int64_t>(qc_slot(part.first, k)) * kPart; };
#pragma unroll
    for (int n = 0; n < kRows8; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = 8 * n + 2 * t + e;
        float mm = -INFINITY;
#pragma unroll 4
        for (int k = 0; k < part.ns; ++k) mm = fmaxf(mm, __ldcg(rows(k) + kRows * QC_D + r));
        float ll = 0.f, ee = 0.f;
        float4 acc[4] = {};
#pragma unroll 2
        for (int k = 0; k < part.ns; ++k) {
          const float* ex = rows(k) + kRows * QC_D + r;
          const float mw = __ldcg(ex);
          const float f = mw == -INFINITY ? 0.f : ex2(mw - mm);
          ll += __ldcg(ex + kRows) * f;
          ee += __ldcg(ex + 2 * kRows) * f;
#pragma unroll
          for (int quad = 0; quad < 4; ++quad)
            add_scaled(acc[quad], __ldcg(reinterpret_cast<const float4*>(rows(k)) + r * 32 + 4 * g + quad), f);
        }
        m[n][e] = mm;
        sum[n][e] = ll;
        le[n][e] = ee;
#pragma unroll
        for (int quad = 0; quad < 4; ++quad) {
          o[n][2 * quad][e] = acc[quad].x;
          o[n][2 * quad][2 + e] = acc[quad].y;
          o[n][2 * quad + 1][e] = acc[quad].z;
          o[n][2 * quad + 1][2 + e] = acc[quad].w;
        }
      }
  }
  // normalised, to O, and the log-sum-exp.  No tokens: 0 and -inf; NaN stays NaN
#pragma unroll
  for (int n = 0; n < kRows8; ++n)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int rr = tile * kRows + 8 * n + 2 * t + e;
      if (rr >= n_rows) continue;
      const int slot = rr / rows_per_cand;
      const int64_t at =
          (static_cast<int64_t>(__ldg(p.perm + seg + slot)) * p.H + hk * p.group) * p.Lq + (rr - slot * rows_per_cand);
      const float l = sum[n][e], inv = l > 0.f ? 1.0f / l : (l == 0.f ? 0.f : l);
      uint4* dst = reinterpret_cast<uint4*>(p.O + at * QC_D + 16 * g);
#pragma unroll
      for (int h = 0; h < 2; ++h)
        dst[h] = make_uint4(pack_bf16x2(o[n][4 * h][e] * inv, o[n][4 * h][2 + e] * inv),
                            pack_bf16x2(o[n][4 * h + 1][e] * inv, o[n][4 * h + 1][2 + e] * inv),
                            pack_bf16x2(o[n][4 * h + 2][e] * inv, o[n][4 * h + 2][2 + e] * inv),
                            pack_bf16x2(o[n][4 * h + 3][e] * inv, o[n][4 * h + 3][2 + e] * inv));
      if (p.lse && g == 0)
        p.lse[at] = le[n][e] > 0.f ? (m[n][e] + __log2f(le[n][e])) * 0.69314718055994531f
                                   : (le[n][e] == 0.f ? -INFINITY : le[n][e]);
    }
}

template <int kRows8, bool kSolo>
__global__ void __launch_bounds__(QT_THREADS, qt_ctas_per_sm(kRows8)) qattn_kernel(const QcAttnParams p) {
  constexpr int kWarps = kSolo ? 1 : QT_WARPS;  // that share an item
  constexpr int kRows = 8 * kRows8, kPart = qt_part(kRows8), kWarpBytes = qt_warp_bytes(kRows8);
  extern __shared__ __align__(128) uint8_t qt_sm[];
  __shared__ QtShared s;
  int64_t* cost0 = reinterpret_cast<int64_t*>(qt_sm + (kSolo ? 0 : QT_WARPS * kWarpBytes));  // [n_users] cost of the items before a user's
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, t = lane & 3;
  const int64_t most = (static_cast<int64_t>(p.max_blocks) << p.blocks_log2) * QC_ROWS;

  constexpr int kMin = kSolo ? QT_SOLO_MIN_BLOCKS : QT_MIN_BLOCKS;
  const QcShares sh = qc_shares<QT_THREADS, kMin, kSolo ? QT_SOLO_ITEM_BLOCKS : QT_ITEM_BLOCKS>(
      p, p.ctas * (QT_WARPS / kWarps), [&](int u, bool& bad) { return user_work<kRows>(p, u, most, bad); }, cost0, nullptr, s.shares);
  bool ignored = false;
  const uint32_t sixteen = p.sixteen;
  const int rows_per_cand = p.group * p.Lq;
  const int64_t page_bytes = (static_cast<int64_t>(p.H_kv) << p.blocks_log2) * QC_BLOCK_BYTES;

  const int cta = kSolo ? static_cast<int>(blockIdx.x) * QT_WARPS + warp : static_cast<int>(blockIdx.x);
  const int64_t end = cta < sh.parts ? sh.start(cta + 1) : 0;
  for (int64_t at = cta < sh.parts ? sh.start(cta) : 0; at < end;) {
    const int u = qc_find(cost0, p.n_users, at);
    const QcUserWork uw = user_work<kRows>(p, u, most, ignored);
    const int len = uw.len;
    const int cost = sh.item_cost(uw.units);
    const int local = static_cast<int>(qc_div(at - cost0[u], cost));
    const int64_t pos = cost0[u] + static_cast<int64_t>(local) * cost;
    at = pos + cost;  // the next item
    const int hk = local / uw.tiles, tile = local - hk * uw.tiles;
    const QcPart part = qc_part<kMin>(sh, cta, uw, pos);
    if (uw.units > 0 && part.nt == 0) continue;
    const int ns = part.ns;
    const int b0 = part.t0 + (kSolo ? 0 : warp), b1 = part.t0 + part.nt;
    const int nb = b1 > b0 ? (b1 - b0 + kWarps - 1) / kWarps : 0;  // this warp's blocks
    const int seg = __ldg(p.offsets + u), count = __ldg(p.offsets + u + 1) - seg;
    const int n_rows = count * rows_per_cand;

    // addresses of this warp's next 32 blocks, one per lane (page 0's for
    // blocks that do not exist: they are loaded, and not used)
    const int32_t* table = p.table + static_cast<int64_t>(u) * p.max_blocks;
    const uint8_t* head = p.data + (static_cast<int64_t>(hk) << p.blocks_log2) * QC_BLOCK_BYTES;
    const uint8_t* mine = head;
    const auto place = [&](int j) {
      mine = head;
      if (j < nb) {
        const int b = b0 + j * kWarps;
        const int id = __ldg(table + (b >> p.blocks_log2));
        if (id >= 0 && id < p.n_pages) mine = head + id * page_bytes + (b & ((1 << p.blocks_log2) - 1)) * QC_BLOCK_BYTES;
        else atomicOr(p.status, DEV_ERR_CACHE);
      }
    };
    const auto block_at = [&](int j) {
      return reinterpret_cast<const uint8_t*>(__shfl_sync(0xffffffffu, reinterpret_cast<uint64_t>(mine), j & 31));
    };
    // a block in registers: for row g of the first product (and g + 8) lane
    // (g, t) reads token (g >> 1) + 4 (g & 1) (and 8 more), so that the inner
    // elements 2t, 2t + 1, 2t + 8, 2t + 9 of the second are tokens t, t + 4,
    // t + 8, t + 12, of which it reads elements 16g .. 16g + 15
    uint4 kc[2];
    uint32_t kp[2], vp[4];
    uint2 vc[4];
    const int ktok = (g >> 1) + 4 * (g & 1);
    const auto load_k = [&](const uint8_t* blk) {
#pragma unroll
      for (int nt = 0; nt < 2; ++nt) {
        kc[nt] = __ldg(reinterpret_cast<const uint4*>(blk + (ktok + 8 * nt) * 64 + t * 16));
        kp[nt] = __ldg(reinterpret_cast<const uint32_t*>(blk + QC_CODE_BYTES + (ktok + 8 * nt) * 16 + t * 4));
      }
    };
    const auto load_v = [&](const uint8_t* blk) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        vc[i] = __ldg(reinterpret_cast<const uint2*>(blk + QC_HALF_BYTES + (t + 4 * i) * 64 + g * 8));
        vp[i] = __ldg(reinterpret_cast<const uint32_t*>(blk + QC_HALF_BYTES + QC_CODE_BYTES + (t + 4 * i) * 16 + (g >> 1) * 4));
      }
    };
    place(lane);
    const uint8_t* cur = block_at(0);
    if (nb > 0) {
      load_k(cur);
      load_v(cur);
    }

    // Q: row g of each eight; lane t holds elements 32t .. 32t+31, in the order
    // in which a block's codes unpack (element e of a word of eight with e + 4)
    uint32_t q[kRows8][8][2];
#pragma unroll
    for (int n = 0; n < kRows8; ++n) {
      const int r = tile * kRows + g + 8 * n;
      uint4 x[4] = {};
      if (r < n_rows) {
        const int slot = r / rows_per_cand, rest = r - slot * rows_per_cand;
        const int cand = __ldg(p.perm + seg + slot);
        const int64_t row = (static_cast<int64_t>(cand) * p.H + hk * p.group) * p.Lq + rest;
        const uint4* src = reinterpret_cast<const uint4*>(p.Q + row * QC_D + t * 32);
#pragma unroll
        for (int w = 0; w < 4; ++w) x[w] = __ldg(src + w);
      }
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        q[n][2 * w][0] = __byte_perm(x[w].x, x[w].z, 0x5410);
        q[n][2 * w][1] = __byte_perm(x[w].x, x[w].z, 0x7632);
        q[n][2 * w + 1][0] = __byte_perm(x[w].y, x[w].w, 0x5410);
        q[n][2 * w + 1][1] = __byte_perm(x[w].y, x[w].w, 0x7632);
      }
    }

    // per eight rows, of which the lane has 2t and 2t + 1
    float o[kRows8][8][4] = {}, sum[kRows8][2] = {};  // sum: a row of ones beside V^T
    float m[kRows8][2], le[kRows8][2];  // reference, log-sum-exp's sums
#pragma unroll
    for (int n = 0; n < kRows8; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        m[n][e] = -INFINITY;
        le[n][e] = 0.f;
      }

#pragma unroll 1
    for (int j = 0; j < nb; ++j) {
      const int left = len - (b0 + j * kWarps) * QC_ROWS;  // tokens of the block that exist, if below 16
      if (((j + 1) & 31) == 0) place(j + 1 + lane);
      const uint8_t* next = block_at(j + 1);
      {  // the lines of the block after the next (of those whose address is at hand)
        const uint8_t* ahead = block_at(j + 2);
        if (lane < 20 && ((j + 2) & 31) >= 2 && j + 2 < nb) asm volatile("prefetch.global.L2 [%0];" ::"l"(ahead + lane * 128));
      }
      float sc[2][4] = {};  // two chains of products: of the two eights of rows, or one's even and odd steps
      {
        const uint32_t s0 = __byte_perm(kp[0], 0, 0x1010), z0 = __byte_perm(kp[0], 0, 0x3232);
        const uint32_t s1 = __byte_perm(kp[1], 0, 0x1010), z1 = __byte_perm(kp[1], 0, 0x3232);
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const uint32_t w0 = w == 0 ? kc[0].x : (w == 1 ? kc[0].y : (w == 2 ? kc[0].z : kc[0].w));
          const uint32_t w1 = w == 0 ? kc[1].x : (w == 1 ? kc[1].y : (w == 2 ? kc[1].z : kc[1].w));
          const uint32_t a[4] = {qc_decode<0>(w0, s0, z0, sixteen), qc_decode<0>(w1, s1, z1, sixteen),
                                 qc_decode<1>(w0, s0, z0, sixteen), qc_decode<1>(w1, s1, z1, sixteen)};
          const uint32_t b[4] = {qc_decode<2>(w0, s0, z0, sixteen), qc_decode<2>(w1, s1, z1, sixteen),
                                 qc_decode<3>(w0, s0, z0, sixteen), qc_decode<3>(w1, s1, z1, sixteen)};
#pragma unroll
          for (int n = 0; n < kRows8; ++n) {
            mma16816(sc[n], a, q[n][2 * w][0], q[n][2 * w][1]);
            mma16816(sc[kRows8 == 1 ? 1 : n], b, q[n][2 * w + 1][0], q[n][2 * w + 1][1]);
          }
        }
      }
      if (kRows8 == 1) {
#pragma unroll
        for (int k = 0; k < 4; ++k) sc[0][k] += sc[1][k];
      }
      if (left < QC_ROWS) {  // tokens behind the end: no score, and value 0 whatever the page holds there
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (t + 4 * i >= left) vp[i] = 0;
          if (ktok + 8 * (i >> 1) >= left) {
#pragma unroll
            for (int n = 0; n < kRows8; ++n) sc[n][i] = -INFINITY;
          }
        }
      }
      bool above = false;
#pragma unroll
      for (int n = 0; n < kRows8; ++n) {
#pragma unroll
        for (int e = 0; e < 2; ++e) above |= fmaxf(sc[n][e], sc[n][2 + e]) * p.scale_log2 > m[n][e] + QT_THRESHOLD;
      }
      if (__any_sync(0xffffffffu, above)) {
#pragma unroll
        for (int n = 0; n < kRows8; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float x = fmaxf(fmaxf(sc[n][e], sc[n][2 + e]) * p.scale_log2, m[n][e]);
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, d));
            const float f = m[n][e] == -INFINITY ? 0.f : ex2(m[n][e] - x);
            le[n][e] *= f;
            sum[n][e] *= f;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              o[n][i][e] *= f;
              o[n][i][2 + e] *= f;
            }
            m[n][e] = x;
          }
      }
      uint32_t pr[kRows8][2];  // P^T: rows of tokens, then of query rows
#pragma unroll
      for (int n = 0; n < kRows8; ++n) {
#pragma unroll
        for (int k = 0; k < 4; ++k)  // (no reference yet: 0)
          sc[n][k] = ex2(fmaf(sc[n][k], p.scale_log2, m[n][k & 1] == -INFINITY ? 0.f : -m[n][k & 1]));
#pragma unroll
        for (int h = 0; h < 2; ++h) pr[n][h] = transpose8x8(pack_bf16x2(sc[n][2 * h], sc[n][2 * h + 1]));
        if (p.lse) {
          le[n][0] += sc[n][0] + sc[n][2];
          le[n][1] += sc[n][1] + sc[n][3];
        }
        mma_sums(sum[n], pr[n][0], pr[n][1]);
      }
      if (kRows8 == 1) load_k(next);  // (later with 16 rows: they have no registers to spare)
      // O^T += V^T P^T: rows g and g + 8 of product 2 quad + c are elements 16g + 4 quad + 2c and the next
      const uint32_t sa = __byte_perm(vp[0], vp[1], 0x5410), za = __byte_perm(vp[0], vp[1], 0x7632);
      const uint32_t sb = __byte_perm(vp[2], vp[3], 0x5410), zb = __byte_perm(vp[2], vp[3], 0x7632);
#pragma unroll
      for (int quad = 0; quad < 4; ++quad) {
        const uint32_t sel = (quad & 1) ? 0x7632u : 0x5410u;
        const uint32_t a = quad < 2 ? __byte_perm(vc[0].x, vc[1].x, sel) : __byte_perm(vc[0].y, vc[1].y, sel);
        const uint32_t b = quad < 2 ? __byte_perm(vc[2].x, vc[3].x, sel) : __byte_perm(vc[2].y, vc[3].y, sel);
        const uint32_t x[4] = {qc_decode<0>(a, sa, za, sixteen), qc_decode<1>(a, sa, za, sixteen),
                               qc_decode<0>(b, sb, zb, sixteen), qc_decode<1>(b, sb, zb, sixteen)};
        const uint32_t y[4] = {qc_decode<2>(a, sa, za, sixteen), qc_decode<3>(a, sa, za, sixteen),
                               qc_decode<2>(b, sb, zb, sixteen), qc_decode<3>(b, sb, zb, sixteen)};
#pragma unroll
        for (int n = 0; n < kRows8; ++n) {
          mma16816(o[n][2 * quad], x, pr[n][0], pr[n][1]);
          mma16816(o[n][2 * quad + 1], y, pr[n][0], pr[n][1]);
        }
      }
      if (kRows8 == 2) load_k(next);
      load_v(next);
    }

    if (kSolo) {
      solo_rows<kRows8>(p, part, o, m, sum, le, tile, hk, seg, n_rows, rows_per_cand);
      continue;
    }
    // ---- join the warps: rows' sums, references and O through shared memory
#pragma unroll
    for (int n = 0; n < kRows8; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) le[n][e] += __shfl_xor_sync(0xffffffffu, le[n][e], d);
        if (g == 0) {
          s.m[warp][8 * n + 2 * t + e] = m[n][e];
          s.l[warp][8 * n + 2 * t + e] = sum[n][e];
          s.le[warp][8 * n + 2 * t + e] = le[n][e];
        }
      }
    float4* ow = reinterpret_cast<float4*>(qt_sm + warp * kWarpBytes);
#pragma unroll
    for (int n = 0; n < kRows8; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int quad = 0; quad < 4; ++quad) {
          const int r = 8 * n + 2 * t + e;
          ow[r * 32 + o_piece(r, 4 * g + quad)] =
              make_float4(o[n][2 * quad][e], o[n][2 * quad][2 + e], o[n][2 * quad + 1][e], o[n][2 * quad + 1][2 + e]);
        }
    __syncthreads();
    // a thread joins kPieces x 4 elements of a row
    constexpr int kPieces = 2 * kRows8, kPer = 32 / kPieces;
    const int r = tid / kPer, cc = tid % kPer;
    float mm = -INFINITY, ll = 0.f, ee = 0.f;
#pragma unroll
    for (int w = 0; w < QT_WARPS; ++w) mm = fmaxf(mm, s.m[w][r]);
    float4 acc[kPieces] = {};
#pragma unroll
    for (int w = 0; w < QT_WARPS; ++w) {
      const float mw = s.m[w][r];
      const float f = mw == -INFINITY ? 0.f : ex2(mw - mm);
      ll += s.l[w][r] * f;
      ee += s.le[w][r] * f;
      const float4* src = reinterpret_cast<const float4*>(qt_sm + w * kWarpBytes);
#pragma unroll
      for (int k = 0; k < kPieces; ++k) add_scaled(acc[k], src[r * 32 + o_piece(r, kPer * k + cc)], f);
    }
    bool write = ns == 1;
    if (!write) {
      // partial rows [r][128], then reference and sums
      const int first = part.first;
      float* mine = p.part + static_cast<int64_t>(part.slot) * kPart;
#pragma unroll
      for (int k = 0; k < kPieces; ++k) __stcg(reinterpret_cast<float4*>(mine) + r * 32 + kPer * k + cc, acc[k]);
      if (cc == 0) {
        float* ex = mine + kRows * QC_D + r;
        __stcg(ex, mm);
        __stcg(ex + kRows, ll);
        __stcg(ex + 2 * kRows, ee);
      }
      __threadfence();
      __syncthreads();
      if (tid == 0) {
        const uint32_t before = atomicAdd(p.tickets + first, 1u);
        s.last = before + 1 == static_cast<uint32_t>(ns) ? 1u : 0u;
        if (s.last) p.tickets[first] = 0;  // zero again for the next call
      }
      __syncthreads();
      write = s.last != 0;
      if (write) {
        __threadfence();
        const auto rows = [&](int k) { return p.part + static_cast<int64_t>(qc_slot(first, k)) * kPart; };
        const auto ex = [&](int k) { return rows(k) + kRows * QC_D + r; };
        mm = -INFINITY;
#pragma unroll 4
        for (int k = 0; k < ns; ++k) mm = fmaxf(mm, __ldcg(ex(k)));
        ll = ee = 0.f;
#pragma unroll
        for (int k = 0; k < kPieces; ++k) acc[k] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
        for (int sp = 0; sp < ns; ++sp) {
          const float mw = __ldcg(ex(sp));
          const float f = mw == -INFINITY ? 0.f : ex2(mw - mm);
          ll += __ldcg(ex(sp) + kRows) * f;
          ee += __ldcg(ex(sp) + 2 * kRows) * f;
#pragma unroll
          for (int k = 0; k < kPieces; ++k)
            add_scaled(acc[k], __ldcg(reinterpret_cast<const float4*>(rows(sp)) + r * 32 + kPer * k + cc), f);
        }
      }
    }
    // the row, normalised, to O, and its log-sum-exp.  No tokens: 0 and -inf; NaN stays NaN
    const int rr = tile * kRows + r;
    if (write && rr < n_rows) {
      const int slot = rr / rows_per_cand;
      const int64_t at =
          (static_cast<int64_t>(__ldg(p.perm + seg + slot)) * p.H + hk * p.group) * p.Lq + (rr - slot * rows_per_cand);
      const float inv = ll > 0.f ? 1.0f / ll : (ll == 0.f ? 0.f : ll);
      uint2* dst = reinterpret_cast<uint2*>(p.O + at * QC_D);
#pragma unroll
      for (int k = 0; k < kPieces; ++k)
        dst[kPer * k + cc] = make_uint2(pack_bf16x2(acc[k].x * inv, acc[k].y * inv), pack_bf16x2(acc[k].z * inv, acc[k].w * inv));
      if (p.lse && cc == 0) p.lse[at] = ee > 0.f ? (mm + __log2f(ee)) * 0.69314718055994531f : (ee == 0.f ? -INFINITY : ee);
    }
    __syncthreads();  // the next item writes the shared rows
  }
}

}  // namespace

// Rows per tile: 8 where no user has more on average.
int qattn_ctas(int num_sms, bool eight) { return num_sms * qt_ctas_per_sm(eight ? 1 : 2); }
size_t qattn_part_elems(int num_sms) {
  constexpr int a = qt_ctas_per_sm(1) * qt_part(1), b = qt_ctas_per_sm(2) * qt_part(2);
  return static_cast<size_t>(QA_SLOTS) * num_sms * QT_WARPS * (a > b ? a : b);
}
size_t qattn_tickets(int num_sms) { return static_cast<size_t>(QA_SLOTS) * num_sms * QT_WARPS * qt_ctas_per_sm(1); }

template <int kRows8, bool kSolo>
static cudaError_t launch(const QcAttnParams& p, cudaStream_t s) {
  constexpr size_t rows = kSolo ? 0 : QT_WARPS * qt_warp_bytes(kRows8);
  cudaError_t e = cudaFuncSetAttribute(qattn_kernel<kRows8, kSolo>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       static_cast<int>(rows + sizeof(int64_t) * SEG_MAX_USERS));
  if (e != cudaSuccess) return e;
  qattn_kernel<kRows8, kSolo><<<p.ctas, QT_THREADS, rows + sizeof(int64_t) * static_cast<size_t>(p.n_users), s>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_qattn(const QcAttnParams& p, bool eight, bool solo, cudaStream_t s) {
  if (solo) return eight ? launch<1, true>(p, s) : launch<2, true>(p, s);
  return eight ? launch<1, false>(p, s) : launch<2, false>(p, s);
}

}  // namespace ikbo
