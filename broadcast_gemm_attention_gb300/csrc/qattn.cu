// qattn.cu -- broadcast attention straight from the 4-bit cache, for few
// query rows per user and K/V head.
//
//   O[i,h] = softmax(Q[i,h] K[map[i],g]^T * scale) V[map[i],g]
//
// The rows that read one history (user u, K/V head g) are its candidates'
// queries of the heads that share g: R = count[u] * (H / H_kv) * Lq.  With few
// of them the operator is bound by the cache's bytes (160 a token and head),
// and the work that counts besides is turning 4-bit codes into operands.
// Here that happens once per tile of 16 rows, in registers: the operand
// layout of the 16x8x16 warp-level matrix instruction lets a lane read its
// share of a block as whole 16- or 8-byte pieces of codes (the order of
// elements along a product's inner dimension is free, so Q is permuted to
// match), and one AND-OR and one FMA make two operands of two codes.  A tcgen05
// product would have to write them to shared memory first and would use 8 to
// 16 of its 128 rows.
//
// Work: a tile is 16 rows of one (u, g); its history is cut into splits
// of whole blocks (16 tokens, 2560 contiguous bytes), sized on the device so
// that the splits of all tiles fill the GPU.  A CTA takes one (tile, split); its
// four warps take every fourth block, loading the next block's codes into the
// registers of the one just decoded (no barrier in the loop; the lines of the
// block after that are asked for in L2), and keep their own running maximum,
// sum and O in registers.  The warps are joined through shared memory; splits of
// a tile leave unnormalised partial rows, which the last split's CTA to finish
// adds in split order (so results repeat bit for bit).
//
// Softmax in fp32 in the log2 domain.  The reference maximum moves only when
// a score exceeds it by more than 2^8 (one vote per block instead of four
// shuffles).  P is rounded to bf16 for P.V (at most 2^-8 relative, as in
// ikbo_attn_forward) and so is the sum that divides O: one more column of ones
// beside V, so that a common rounding of P cancels.  The log-sum-exp has a sum
// of its own, of the unrounded values.
#include <cuda_bf16.h>

#include "ptx.cuh"
#include "qcache_internal.h"

namespace ikbo {
namespace {

constexpr int QT_WARPS = 4;
constexpr int QT_THREADS = 32 * QT_WARPS;
constexpr int QT_MIN_BLOCKS = 4 * QT_WARPS;  // blocks of a split, at least
constexpr int QT_ITEM_BLOCKS = 24;           // what an item costs beside its blocks, in blocks
constexpr float QT_THRESHOLD = 8.0f;         // log2 units
constexpr int QT_EXTRA = 3;                  // per row besides O: reference, sum, sum of the log-sum-exp

constexpr int QT_ROWS = 16;
constexpr int QT_CTAS_PER_SM = 3;
constexpr int QT_PART = QT_ROWS * (QC_D + QT_EXTRA);  // floats of a split's partial rows
constexpr int QT_WARP_BYTES = QT_ROWS * QC_D * 4;     // a warp's O on its way to the others

struct QtShared {
  float m[QT_WARPS][QT_ROWS];
  float l[QT_WARPS][QT_ROWS];
  float le[QT_WARPS][QT_ROWS];
  QcSharesScratch shares;
  uint32_t last;
};

__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ QcUserWork user_work(const QcAttnParams& p, int u, int64_t most, bool& bad) {
  QcUserWork w;
  const int count = __ldg(p.offsets + u + 1) - __ldg(p.offsets + u);
  w.len = qc_length(p.lens, u, most, bad);
  w.tiles = static_cast<int>((static_cast<int64_t>(count) * p.group * p.Lq + QT_ROWS - 1) / QT_ROWS);
  w.units = (w.len + QC_ROWS - 1) / QC_ROWS;
  return w;
}

// Place of 16-byte piece c (of 32) of a row of a warp's staged O: pieces are
// permuted so that the lanes' stores (rows g, quarters t) and the readers'
// loads spread over the banks.
__device__ __forceinline__ int o_piece(int row, int c) { return (c & ~7) | ((c & 7) ^ ((c >> 3) | ((row & 1) << 2))); }

__device__ __forceinline__ void add_scaled(float4& a, const float4 x, float f) {
  a.x = fmaf(x.x, f, a.x);
  a.y = fmaf(x.y, f, a.y);
  a.z = fmaf(x.z, f, a.z);
  a.w = fmaf(x.w, f, a.w);
}

__global__ void __launch_bounds__(QT_THREADS, QT_CTAS_PER_SM) qattn_kernel(const QcAttnParams p) {
  extern __shared__ __align__(128) uint8_t qt_sm[];
  __shared__ QtShared s;
  int64_t* cost0 = reinterpret_cast<int64_t*>(qt_sm + QT_WARPS * QT_WARP_BYTES);  // [n_users] cost of the items before a user's
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, t = lane & 3;
  const int64_t most = (static_cast<int64_t>(p.max_blocks) << p.blocks_log2) * QC_ROWS;

  const QcShares sh = qc_shares<QT_THREADS, QT_MIN_BLOCKS, QT_ITEM_BLOCKS>(
      p, [&](int u, bool& bad) { return user_work(p, u, most, bad); }, cost0, nullptr, s.shares);
  bool ignored = false;
  const int rows_per_cand = p.group * p.Lq;
  const int64_t page_bytes = (static_cast<int64_t>(p.H_kv) << p.blocks_log2) * QC_BLOCK_BYTES;

  const int cta = static_cast<int>(blockIdx.x);
  const int64_t end = cta < sh.parts ? sh.start(cta + 1) : 0;
  for (int64_t at = cta < sh.parts ? sh.start(cta) : 0; at < end;) {
    const int u = qc_find(cost0, p.n_users, at);
    const QcUserWork uw = user_work(p, u, most, ignored);
    const int len = uw.len;
    const int cost = sh.item_cost(uw.units);
    const int local = static_cast<int>(qc_div(at - cost0[u], cost));
    const int64_t pos = cost0[u] + static_cast<int64_t>(local) * cost;
    at = pos + cost;  // the next item
    const int hk = local / uw.tiles, tile = local - hk * uw.tiles;
    const QcPart part = qc_part<QT_MIN_BLOCKS>(sh, uw, pos);
    if (uw.units > 0 && part.nt == 0) continue;
    const int ns = part.ns;
    const int b0 = part.t0 + warp, b1 = part.t0 + part.nt;
    const int nb = b1 > b0 ? (b1 - b0 + QT_WARPS - 1) / QT_WARPS : 0;  // this warp's blocks
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
        const int b = b0 + j * QT_WARPS;
        const int id = __ldg(table + (b >> p.blocks_log2));
        if (id >= 0 && id < p.n_pages) mine = head + id * page_bytes + (b & ((1 << p.blocks_log2) - 1)) * QC_BLOCK_BYTES;
        else atomicOr(p.status, DEV_ERR_CACHE);
      }
    };
    const auto block_at = [&](int j) {
      return reinterpret_cast<const uint8_t*>(__shfl_sync(0xffffffffu, reinterpret_cast<uint64_t>(mine), j & 31));
    };
    // a block in registers: for column g lane (g, t) reads token
    // (g >> 1) + 4 (g & 1) + 8 nt of the keys, so that its own scores are of
    // tokens t, t + 4, t + 8, t + 12, whose values it reads
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

    // Q: rows g and g + 8; lane t holds elements 32t .. 32t+31, in the order in
    // which a block's codes unpack (element e of a word of eight with e + 4)
    uint32_t q[8][4];
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int r = tile * QT_ROWS + g + 8 * half;
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
        q[2 * w][half] = __byte_perm(x[w].x, x[w].z, 0x5410);
        q[2 * w][2 + half] = __byte_perm(x[w].x, x[w].z, 0x7632);
        q[2 * w + 1][half] = __byte_perm(x[w].y, x[w].w, 0x5410);
        q[2 * w + 1][2 + half] = __byte_perm(x[w].y, x[w].w, 0x7632);
      }
    }

    float o[16][4] = {}, sum[4] = {};                // sum: the column of ones
    float m0 = -INFINITY, m1 = -INFINITY;            // reference of rows g, g + 8
    float u0 = 0.f, u1 = 0.f, le0 = 0.f, le1 = 0.f;  // the one subtracted (0 while it is -inf), log-sum-exp's sums

#pragma unroll 1
    for (int j = 0; j < nb; ++j) {
      const int left = len - (b0 + j * QT_WARPS) * QC_ROWS;  // tokens of the block that exist, if below 16
      if (((j + 1) & 31) == 0) place(j + 1 + lane);
      const uint8_t* next = block_at(j + 1);
      {  // the lines of the block after the next (of those whose address is at hand)
        const uint8_t* ahead = block_at(j + 2);
        if (lane < 20 && ((j + 2) & 31) >= 2 && j + 2 < nb) asm volatile("prefetch.global.L2 [%0];" ::"l"(ahead + lane * 128));
      }
      // four chains of products, two per eight tokens
      float sc[2][4] = {}, sd[2][4] = {};
#pragma unroll
      for (int w = 0; w < 4; ++w)
#pragma unroll
        for (int nt = 0; nt < 2; ++nt) {
          const uint32_t s2 = __byte_perm(kp[nt], 0, 0x1010), z2 = __byte_perm(kp[nt], 0, 0x3232);
          const uint32_t w4 = w == 0 ? kc[nt].x : (w == 1 ? kc[nt].y : (w == 2 ? kc[nt].z : kc[nt].w));
          mma16816(sc[nt], q[2 * w], qc_decode<0>(w4, s2, z2, p.sixteen), qc_decode<1>(w4, s2, z2, p.sixteen));
          mma16816(sd[nt], q[2 * w + 1], qc_decode<2>(w4, s2, z2, p.sixteen), qc_decode<3>(w4, s2, z2, p.sixteen));
        }
#pragma unroll
      for (int nt = 0; nt < 2; ++nt)
#pragma unroll
        for (int k = 0; k < 4; ++k) sc[nt][k] += sd[nt][k];
      load_k(next);
      if (left < QC_ROWS) {  // tokens behind the end: no score, and value 0 whatever the page holds there
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (t + 4 * i >= left) {
            sc[i >> 1][i & 1] = sc[i >> 1][2 + (i & 1)] = -INFINITY;
            vp[i] = 0;
          }
      }
      const float x0 = fmaxf(fmaxf(sc[0][0], sc[0][1]), fmaxf(sc[1][0], sc[1][1])) * p.scale_log2;
      const float x1 = fmaxf(fmaxf(sc[0][2], sc[0][3]), fmaxf(sc[1][2], sc[1][3])) * p.scale_log2;
      if (__any_sync(0xffffffffu, x0 > m0 + QT_THRESHOLD || x1 > m1 + QT_THRESHOLD)) {
        float n0 = fmaxf(x0, m0), n1 = fmaxf(x1, m1);
#pragma unroll
        for (int d = 1; d < 4; d <<= 1) {
          n0 = fmaxf(n0, __shfl_xor_sync(0xffffffffu, n0, d));
          n1 = fmaxf(n1, __shfl_xor_sync(0xffffffffu, n1, d));
        }
        const float a0 = m0 == -INFINITY ? 0.f : ex2(m0 - n0), a1 = m1 == -INFINITY ? 0.f : ex2(m1 - n1);
        le0 *= a0;
        le1 *= a1;
        sum[0] *= a0;
        sum[2] *= a1;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          o[i][0] *= a0;
          o[i][1] *= a0;
          o[i][2] *= a1;
          o[i][3] *= a1;
        }
        m0 = n0;
        m1 = n1;
        u0 = m0 == -INFINITY ? 0.f : m0;
        u1 = m1 == -INFINITY ? 0.f : m1;
      }
      uint32_t pr[4];
#pragma unroll
      for (int nt = 0; nt < 2; ++nt) {
#pragma unroll
        for (int k = 0; k < 4; ++k) sc[nt][k] = ex2(fmaf(sc[nt][k], p.scale_log2, k < 2 ? -u0 : -u1));
        pr[2 * nt] = pack_bf16x2(sc[nt][0], sc[nt][1]);
        pr[2 * nt + 1] = pack_bf16x2(sc[nt][2], sc[nt][3]);
      }
      if (p.lse) {
        le0 += (sc[0][0] + sc[0][1]) + (sc[1][0] + sc[1][1]);
        le1 += (sc[0][2] + sc[0][3]) + (sc[1][2] + sc[1][3]);
      }
      mma16816(sum, pr, 0x3F803F80u, 0x3F803F80u);
      // O += P V: column g of product n is element 16 g + n
      const uint32_t sa = __byte_perm(vp[0], vp[1], 0x5410), za = __byte_perm(vp[0], vp[1], 0x7632);
      const uint32_t sb = __byte_perm(vp[2], vp[3], 0x5410), zb = __byte_perm(vp[2], vp[3], 0x7632);
#pragma unroll
      for (int quad = 0; quad < 4; ++quad) {
        const uint32_t sel = (quad & 1) ? 0x7632u : 0x5410u;
        const uint32_t a = quad < 2 ? __byte_perm(vc[0].x, vc[1].x, sel) : __byte_perm(vc[0].y, vc[1].y, sel);
        const uint32_t b = quad < 2 ? __byte_perm(vc[2].x, vc[3].x, sel) : __byte_perm(vc[2].y, vc[3].y, sel);
        mma16816(o[4 * quad + 0], pr, qc_decode<0>(a, sa, za, p.sixteen), qc_decode<0>(b, sb, zb, p.sixteen));
        mma16816(o[4 * quad + 1], pr, qc_decode<1>(a, sa, za, p.sixteen), qc_decode<1>(b, sb, zb, p.sixteen));
        mma16816(o[4 * quad + 2], pr, qc_decode<2>(a, sa, za, p.sixteen), qc_decode<2>(b, sb, zb, p.sixteen));
        mma16816(o[4 * quad + 3], pr, qc_decode<3>(a, sa, za, p.sixteen), qc_decode<3>(b, sb, zb, p.sixteen));
      }
      load_v(next);
    }

    // ---- join the warps: rows' sums, references and O through shared memory
    le0 += __shfl_xor_sync(0xffffffffu, le0, 1);
    le1 += __shfl_xor_sync(0xffffffffu, le1, 1);
    le0 += __shfl_xor_sync(0xffffffffu, le0, 2);
    le1 += __shfl_xor_sync(0xffffffffu, le1, 2);
    if (t == 0) {
      s.m[warp][g] = m0;
      s.m[warp][g + 8] = m1;
      s.l[warp][g] = sum[0];
      s.l[warp][g + 8] = sum[2];
      s.le[warp][g] = le0;
      s.le[warp][g + 8] = le1;
    }
    float4* ow = reinterpret_cast<float4*>(qt_sm + warp * QT_WARP_BYTES);
#pragma unroll
    for (int half = 0; half < 2; ++half)
#pragma unroll
      for (int c = 0; c < 8; ++c) {  // elements 32 t + 4 c ..: products 4 (c % 4) .., column 2t (c < 4) or 2t + 1
        const int r = g + 8 * half, k = 2 * half + (c >> 2), i = 4 * (c & 3);
        ow[r * 32 + o_piece(r, t * 8 + c)] = make_float4(o[i][k], o[i + 1][k], o[i + 2][k], o[i + 3][k]);
      }
    __syncthreads();
    // a thread joins 4 x 4 elements of row tid / 8
    const int r = tid >> 3, cc = tid & 7;
    float mm = -INFINITY, ll = 0.f, ee = 0.f;
#pragma unroll
    for (int w = 0; w < QT_WARPS; ++w) mm = fmaxf(mm, s.m[w][r]);
    float4 acc[4] = {};
#pragma unroll
    for (int w = 0; w < QT_WARPS; ++w) {
      const float mw = s.m[w][r];
      const float f = mw == -INFINITY ? 0.f : ex2(mw - mm);
      ll += s.l[w][r] * f;
      ee += s.le[w][r] * f;
      const float4* src = reinterpret_cast<const float4*>(qt_sm + w * QT_WARP_BYTES);
#pragma unroll
      for (int k = 0; k < 4; ++k) add_scaled(acc[k], src[r * 32 + o_piece(r, 8 * k + cc)], f);
    }
    bool write = ns == 1;
    if (!write) {
      // partial rows [r][128], then reference and sums
      const int first = part.first;
      float* mine = p.part + static_cast<int64_t>(part.slot) * QT_PART;
#pragma unroll
      for (int k = 0; k < 4; ++k) __stcg(reinterpret_cast<float4*>(mine) + r * 32 + 8 * k + cc, acc[k]);
      if (cc == 0) {
        float* ex = mine + QT_ROWS * QC_D + r;
        __stcg(ex, mm);
        __stcg(ex + QT_ROWS, ll);
        __stcg(ex + 2 * QT_ROWS, ee);
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
        const auto rows = [&](int k) { return p.part + static_cast<int64_t>(qc_slot(first, k)) * QT_PART; };
        const auto ex = [&](int k) { return rows(k) + QT_ROWS * QC_D + r; };
        mm = -INFINITY;
#pragma unroll 4
        for (int k = 0; k < ns; ++k) mm = fmaxf(mm, __ldcg(ex(k)));
        ll = ee = 0.f;
#pragma unroll
        for (int k = 0; k < 4; ++k) acc[k] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
        for (int sp = 0; sp < ns; ++sp) {
          const float mw = __ldcg(ex(sp));
          const float f = mw == -INFINITY ? 0.f : ex2(mw - mm);
          ll += __ldcg(ex(sp) + QT_ROWS) * f;
          ee += __ldcg(ex(sp) + 2 * QT_ROWS) * f;
#pragma unroll
          for (int k = 0; k < 4; ++k)
            add_scaled(acc[k], __ldcg(reinterpret_cast<const float4*>(rows(sp)) + r * 32 + 8 * k + cc), f);
        }
      }
    }
    // the row, normalised, to O, and its log-sum-exp.  No tokens: 0 and -inf; NaN stays NaN
    const int rr = tile * QT_ROWS + r;
    if (write && rr < n_rows) {
      const int slot = rr / rows_per_cand;
      const int64_t at =
          (static_cast<int64_t>(__ldg(p.perm + seg + slot)) * p.H + hk * p.group) * p.Lq + (rr - slot * rows_per_cand);
      const float inv = ll > 0.f ? 1.0f / ll : (ll == 0.f ? 0.f : ll);
      uint2* dst = reinterpret_cast<uint2*>(p.O + at * QC_D);
#pragma unroll
      for (int k = 0; k < 4; ++k)
        dst[8 * k + cc] = make_uint2(pack_bf16x2(acc[k].x * inv, acc[k].y * inv), pack_bf16x2(acc[k].z * inv, acc[k].w * inv));
      if (p.lse && cc == 0) p.lse[at] = ee > 0.f ? (mm + __log2f(ee)) * 0.69314718055994531f : (ee == 0.f ? -INFINITY : ee);
    }
    __syncthreads();  // the next item writes the shared rows
  }
}

}  // namespace

int qattn_ctas(int num_sms) { return num_sms * QT_CTAS_PER_SM; }
size_t qattn_part_elems(int num_sms) { return static_cast<size_t>(QA_SLOTS) * qattn_ctas(num_sms) * QT_PART; }

cudaError_t launch_qattn(const QcAttnParams& p, cudaStream_t s) {
  constexpr size_t rows = QT_WARPS * QT_WARP_BYTES;
  const size_t smem = rows + sizeof(int64_t) * static_cast<size_t>(p.n_users);
  cudaError_t e = cudaFuncSetAttribute(qattn_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       static_cast<int>(rows + sizeof(int64_t) * SEG_MAX_USERS));
  if (e != cudaSuccess) return e;
  qattn_kernel<<<p.ctas, QT_THREADS, smem, s>>>(p);
  return cudaGetLastError();
}

}  // namespace ikbo
