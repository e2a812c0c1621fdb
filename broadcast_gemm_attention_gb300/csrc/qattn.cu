// qattn.cu -- broadcast attention straight from the 4-bit cache, for few
// query rows per user and K/V head.
//
//   O[i,h] = softmax(Q[i,h] K[map[i],g]^T * scale) V[map[i],g]
//
// The rows that read one history (user u, K/V head g) are its candidates'
// queries of the heads that share g: R = count[u] * (H / H_kv) * Lq.  With few
// of them the operator is bound by the cache's bytes (160 a token and head),
// and the work that counts besides is turning 4-bit codes into operands.
// Here that happens once per 16-row tile, in registers: the operand layout of
// the 16x8x16 warp-level matrix instruction lets a lane read its share of a
// block as whole 16- or 8-byte pieces of codes (the order of elements along a
// product's inner dimension is free, so Q is permuted to match), and one
// AND-OR and one FMA make two operands of four code bits each.  A tcgen05
// product would have to write them to shared memory first and would use 8 to
// 16 of its 128 rows.
//
// Work: a tile is 16 rows of one (u, g); its history is cut into splits of
// whole blocks (16 tokens, 2560 contiguous bytes), sized on the device so that
// the splits of all tiles fill the GPU.  A CTA takes one (tile, split); its
// four warps take every fourth block, each with a ring of its own filled by
// bulk copies (no CTA-wide barrier in the loop), and keep their own running
// maximum, sum and O in registers.  The warps are joined through shared
// memory; splits of a tile leave unnormalised partial rows, which the last
// split's CTA to finish adds in split order (so results repeat bit for bit).
//
// Softmax in fp32 in the log2 domain.  The reference maximum moves only when
// a score exceeds it by more than 2^8 (one vote per block instead of four
// shuffles); P is rounded to bf16 for P.V (at most 2^-8 relative, as in
// ikbo_attn_forward), the sum uses the unrounded values.
#include <cuda_bf16.h>

#include "ptx.cuh"
#include "qcache_internal.h"

namespace ikbo {
namespace {

constexpr int QT_WARPS = 4;
constexpr int QT_THREADS = 32 * QT_WARPS;
constexpr int QT_ROWS = 16;             // rows of a tile
constexpr int QT_STAGES = 4;            // blocks in flight per warp
constexpr int QT_CTAS_PER_SM = 4;
constexpr int QT_MIN_BLOCKS = 4 * QT_WARPS;  // blocks of a split, at least
constexpr float QT_THRESHOLD = 8.0f;    // log2 units
constexpr int QT_PART = QT_ROWS * (QC_D + 2);  // floats of a split's partial rows

constexpr uint32_t RING_BYTES = QT_STAGES * QC_BLOCK_BYTES;   // per warp; later 16 x 128 fp32 of its O
static_assert(RING_BYTES >= QT_ROWS * QC_D * 4, "a warp's O does not fit in its ring");

struct QtShared {
  uint64_t bars[QT_WARPS][QT_STAGES];
  int32_t left[QT_WARPS][QT_STAGES];  // tokens of the staged block that exist (0: page out of range)
  float m[QT_WARPS][QT_ROWS];
  float l[QT_WARPS][QT_ROWS];
  int64_t red[3][QT_WARPS];
  uint32_t abort;
  uint32_t last;
};

__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Sum over the CTA of three values at once.
__device__ __forceinline__ void block_sum(int64_t (&v)[3], QtShared& s) {
#pragma unroll
  for (int k = 0; k < 3; ++k) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
    if ((threadIdx.x & 31) == 0) s.red[k][threadIdx.x >> 5] = v[k];
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    v[k] = 0;
#pragma unroll
    for (int w = 0; w < QT_WARPS; ++w) v[k] += s.red[k][w];
  }
  __syncthreads();
}

// Exclusive scan over the CTA's threads of two values at once.
__device__ __forceinline__ void block_scan2(int64_t (&v)[2], int64_t (&total)[2], QtShared& s) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t incl[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    incl[k] = v[k];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, incl[k], o);
      if (lane >= o) incl[k] += y;
    }
    if (lane == 31) s.red[k][warp] = incl[k];
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    int64_t before = 0;
    total[k] = 0;
#pragma unroll
    for (int w = 0; w < QT_WARPS; ++w) {
      before += w < warp ? s.red[k][w] : 0;
      total[k] += s.red[k][w];
    }
    v[k] = before + incl[k] - v[k];
  }
  __syncthreads();
}

struct UserWork {
  int tiles;   // tiles of one K/V head
  int blocks;  // 16-token blocks of the history
};

__device__ __forceinline__ UserWork user_work(const QcAttnParams& p, int u, int64_t most, int64_t* len, bool& bad) {
  UserWork w;
  const int count = __ldg(p.offsets + u + 1) - __ldg(p.offsets + u);
  const int n = qc_length(p.lens, u, most, bad);
  *len = n;
  w.tiles = static_cast<int>((static_cast<int64_t>(count) * p.group * p.Lq + QT_ROWS - 1) / QT_ROWS);
  w.blocks = (n + QC_ROWS - 1) / QC_ROWS;
  return w;
}

__device__ __forceinline__ int splits_of(int blocks, int chunk) { return blocks <= chunk ? 1 : (blocks + chunk - 1) / chunk; }

// Place of 16-byte piece c (of 32) of a row of a warp's staged O: pieces are
// permuted so that the lanes' stores (rows g, quarters t) and the readers'
// loads spread over the banks.
__device__ __forceinline__ int o_piece(int row, int c) { return (c & ~7) | ((c & 7) ^ ((c >> 3) | ((row & 1) << 2))); }

__global__ void __launch_bounds__(QT_THREADS, QT_CTAS_PER_SM) qattn_kernel(const QcAttnParams p) {
  extern __shared__ __align__(128) uint8_t qt_sm[];
  __shared__ QtShared s;
  uint8_t* rings = qt_sm;
  int32_t* item0 = reinterpret_cast<int32_t*>(qt_sm + QT_WARPS * RING_BYTES);  // [n_users + 1] items before a user
  int32_t* part0 = item0 + p.n_users + 1;                                      // [n_users + 1] partial rows before
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, t = lane & 3;
  const int n = p.n_users;
  const int64_t most = (static_cast<int64_t>(p.max_blocks) << p.blocks_log2) * QC_ROWS;

  if (tid == 0) {
    for (int w = 0; w < QT_WARPS; ++w)
      for (int i = 0; i < QT_STAGES; ++i) mbar_init(&s.bars[w][i], 1);
    s.abort = 0;
    fence_barrier_init();
    fence_proxy_async_smem();
  }

  // ---- the list of items: (user, K/V head, split, tile), user-major
  const int per = (n + QT_THREADS - 1) / QT_THREADS;
  const int lo = min(tid * per, n), hi = min(lo + per, n);
  bool bad = false, ignored = false;
  int64_t sums[3] = {0, 0, 0};
  for (int u = lo; u < hi; ++u) {
    int64_t len;
    const UserWork w = user_work(p, u, most, &len, bad);
    sums[0] += static_cast<int64_t>(w.tiles) * w.blocks;
    sums[1] += len;
    sums[2] += w.tiles;
  }
  block_sum(sums, s);
  if (sums[1] > p.bound) bad = true;
  if (bad && blockIdx.x == 0) atomicOr(p.status, DEV_ERR_CACHE);
  const int64_t work = sums[0] * p.H_kv;
  int64_t chunk64 = (work + p.target - 1) / p.target;
  if (chunk64 < QT_MIN_BLOCKS) chunk64 = QT_MIN_BLOCKS;
  const int chunk = static_cast<int>(min(chunk64, static_cast<int64_t>(1 << 28)));
  int64_t v[2] = {0, 0}, total[2];
  for (int u = lo; u < hi; ++u) {
    int64_t len;
    const UserWork w = user_work(p, u, most, &len, ignored);
    const int ns = splits_of(w.blocks, chunk);
    const int64_t items = static_cast<int64_t>(w.tiles) * p.H_kv * ns;
    v[0] += items;
    v[1] += ns > 1 ? items : 0;
  }
  block_scan2(v, total, s);
  for (int u = lo; u < hi; ++u) {
    int64_t len;
    const UserWork w = user_work(p, u, most, &len, ignored);
    const int ns = splits_of(w.blocks, chunk);
    const int64_t items = static_cast<int64_t>(w.tiles) * p.H_kv * ns;
    item0[u] = static_cast<int32_t>(v[0]);
    part0[u] = static_cast<int32_t>(v[1]);
    v[0] += items;
    v[1] += ns > 1 ? items : 0;
  }
  __syncthreads();
  if (total[0] > 0x7fffffff || total[1] > 2 * static_cast<int64_t>(p.target)) {  // cannot be: see the host's checks
    if (tid == 0 && blockIdx.x == 0) atomicOr(p.status, DEV_ERR_BAD_WORK);
    return;
  }
  const int n_items = static_cast<int>(total[0]);

  uint8_t* ring = rings + warp * RING_BYTES;
  const int rows_per_cand = p.group * p.Lq;
  uint32_t done = 0;  // blocks this warp has staged so far (ring position and phase)

  for (int item = blockIdx.x; item < n_items; item += gridDim.x) {
    const int u = qc_find(item0, n, item);
    int64_t len64;
    const UserWork uw = user_work(p, u, most, &len64, ignored);
    const int len = static_cast<int>(len64);
    const int ns = splits_of(uw.blocks, chunk);
    int local = item - item0[u];
    const int tile = local % uw.tiles;
    local /= uw.tiles;
    const int split = local % ns, hk = local / ns;
    const int b0 = static_cast<int>(static_cast<int64_t>(uw.blocks) * split / ns);
    const int b1 = static_cast<int>(static_cast<int64_t>(uw.blocks) * (split + 1) / ns);
    const int nb = b1 - b0 > warp ? (b1 - b0 - warp + QT_WARPS - 1) / QT_WARPS : 0;  // this warp's blocks
    const int seg = __ldg(p.offsets + u), count = __ldg(p.offsets + u + 1) - seg;
    const int n_rows = count * rows_per_cand;

    // page numbers of this warp's next 32 blocks, one per lane
    const int32_t* table = p.table + static_cast<int64_t>(u) * p.max_blocks;
    const auto page_of = [&](int j) -> int {
      return j < nb ? __ldg(table + ((b0 + warp + j * QT_WARPS) >> p.blocks_log2)) : 0;
    };
    int pages = page_of(lane);
    const auto stage = [&](int j) {  // block j of this warp into its ring (whole warp)
      if (j > 0 && (j & 31) == 0) pages = page_of(j + lane);
      const int id = __shfl_sync(0xffffffffu, pages, j & 31);
      if (lane == 0) {
        const int b = b0 + warp + j * QT_WARPS;
        const uint32_t st = (done + j) % QT_STAGES;
        const bool legal = id >= 0 && id < p.n_pages;
        if (!legal) atomicOr(p.status, DEV_ERR_CACHE);
        s.left[warp][st] = legal ? min(QC_ROWS, len - b * QC_ROWS) : 0;
        const int64_t at = (((static_cast<int64_t>(legal ? id : 0) * p.H_kv + hk) << p.blocks_log2) +
                            (b & ((1 << p.blocks_log2) - 1))) * QC_BLOCK_BYTES;
        mbar_arrive_expect_tx(&s.bars[warp][st], QC_BLOCK_BYTES);
        bulk_load(ring + st * QC_BLOCK_BYTES, p.data + at, QC_BLOCK_BYTES, &s.bars[warp][st]);
      }
    };
    for (int j = 0; j < QT_STAGES && j < nb; ++j) stage(j);

    // Q: rows g and g + 8 of the tile; lane t holds elements 32t .. 32t+31,
    // in the order in which a block's codes unpack (element e of a word of
    // eight with e + 4)
    uint32_t q[8][4];
    int64_t row_at[2];
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int r = tile * QT_ROWS + g + 8 * half;
      row_at[half] = -1;
      uint4 x[4] = {};
      if (r < n_rows) {
        const int slot = r / rows_per_cand, rest = r - slot * rows_per_cand;
        const int cand = __ldg(p.perm + seg + slot);
        row_at[half] = (static_cast<int64_t>(cand) * p.H + hk * p.group) * p.Lq + rest;
        const uint4* src = reinterpret_cast<const uint4*>(p.Q + row_at[half] * QC_D + t * 32);
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

    float o[16][4];
#pragma unroll
    for (int i = 0; i < 16; ++i)
#pragma unroll
      for (int k = 0; k < 4; ++k) o[i][k] = 0.f;
    float m0 = -INFINITY, m1 = -INFINITY;  // reference of rows g, g + 8
    float u0 = 0.f, u1 = 0.f;              // the reference subtracted (0 while it is -inf)
    float l0 = 0.f, l1 = 0.f;              // this lane's part of the row sums

    bool alive = true;
    for (int j = 0; j < nb; ++j) {
      const uint32_t st = (done + j) % QT_STAGES, ph = ((done + j) / QT_STAGES) & 1u;
      alive = mbar_wait(&s.bars[warp][st], ph, &s.abort, p.timeout_ns, 1);
      alive = __all_sync(0xffffffffu, alive);
      if (!alive) break;  // the wait has set s.abort: the CTA leaves together below
      const uint8_t* blk = ring + st * QC_BLOCK_BYTES;
      const int left = s.left[warp][st];

      // scores of 16 tokens: lane (g, t) reads token (g >> 1) + 4 (g & 1) + 8 nt
      // for column g, so its own scores are of tokens t, t + 4, t + 8, t + 12
      float sc[2][4];
#pragma unroll
      for (int nt = 0; nt < 2; ++nt) {
        const int tok = nt * 8 + (g >> 1) + 4 * (g & 1);
        const uint4 c = *reinterpret_cast<const uint4*>(blk + tok * 64 + t * 16);
        const uint32_t sz = *reinterpret_cast<const uint32_t*>(blk + QC_CODE_BYTES + tok * 16 + t * 4);
        const uint32_t s2 = __byte_perm(sz, 0, 0x1010), z2 = __byte_perm(sz, 0, 0x3232);
        const uint32_t w4[4] = {c.x, c.y, c.z, c.w};
        sc[nt][0] = sc[nt][1] = sc[nt][2] = sc[nt][3] = 0.f;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          mma16816(sc[nt], q[2 * w], qc_decode<0>(w4[w], s2, z2), qc_decode<1>(w4[w], s2, z2));
          mma16816(sc[nt], q[2 * w + 1], qc_decode<2>(w4[w], s2, z2), qc_decode<3>(w4[w], s2, z2));
        }
      }
      // the values' codes and pairs of tokens t, t + 4, t + 8, t + 12
      uint2 vc[4];
      uint32_t vp[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int tok = t + 4 * i;
        vc[i] = *reinterpret_cast<const uint2*>(blk + QC_HALF_BYTES + tok * 64 + g * 8);
        vp[i] = *reinterpret_cast<const uint32_t*>(blk + QC_HALF_BYTES + QC_CODE_BYTES + tok * 16 + (g >> 1) * 4);
      }
      __syncwarp();  // the block is in registers
      if (j + QT_STAGES < nb) stage(j + QT_STAGES);
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
        l0 *= a0;
        l1 *= a1;
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
        const float p0 = ex2(fmaf(sc[nt][0], p.scale_log2, -u0)), p1 = ex2(fmaf(sc[nt][1], p.scale_log2, -u0));
        const float p2 = ex2(fmaf(sc[nt][2], p.scale_log2, -u1)), p3 = ex2(fmaf(sc[nt][3], p.scale_log2, -u1));
        l0 += p0 + p1;
        l1 += p2 + p3;
        pr[2 * nt] = pack_bf16x2(p0, p1);
        pr[2 * nt + 1] = pack_bf16x2(p2, p3);
      }
      // O += P V: column g of product n is element 16 g + n
      const uint32_t sa = __byte_perm(vp[0], vp[1], 0x5410), za = __byte_perm(vp[0], vp[1], 0x7632);
      const uint32_t sb = __byte_perm(vp[2], vp[3], 0x5410), zb = __byte_perm(vp[2], vp[3], 0x7632);
#pragma unroll
      for (int quad = 0; quad < 4; ++quad) {
        const uint32_t sel = (quad & 1) ? 0x7632u : 0x5410u;
        const uint32_t a = quad < 2 ? __byte_perm(vc[0].x, vc[1].x, sel) : __byte_perm(vc[0].y, vc[1].y, sel);
        const uint32_t b = quad < 2 ? __byte_perm(vc[2].x, vc[3].x, sel) : __byte_perm(vc[2].y, vc[3].y, sel);
        mma16816(o[4 * quad + 0], pr, qc_decode<0>(a, sa, za), qc_decode<0>(b, sb, zb));
        mma16816(o[4 * quad + 1], pr, qc_decode<1>(a, sa, za), qc_decode<1>(b, sb, zb));
        mma16816(o[4 * quad + 2], pr, qc_decode<2>(a, sa, za), qc_decode<2>(b, sb, zb));
        mma16816(o[4 * quad + 3], pr, qc_decode<3>(a, sa, za), qc_decode<3>(b, sb, zb));
      }
    }
    done += static_cast<uint32_t>(nb);

    // ---- join the warps: rows' sums, references and O through shared memory
#pragma unroll
    for (int d = 1; d < 4; d <<= 1) {
      l0 += __shfl_xor_sync(0xffffffffu, l0, d);
      l1 += __shfl_xor_sync(0xffffffffu, l1, d);
    }
    if (t == 0) {
      s.m[warp][g] = m0;
      s.m[warp][g + 8] = m1;
      s.l[warp][g] = l0;
      s.l[warp][g + 8] = l1;
    }
    float4* ow = reinterpret_cast<float4*>(ring);
#pragma unroll
    for (int half = 0; half < 2; ++half)
#pragma unroll
      for (int c = 0; c < 8; ++c) {  // elements 32 t + 4 c ..: products 4 (c % 4) .., column 2t (c < 4) or 2t + 1
        const int r = g + 8 * half, k = 2 * half + (c >> 2), i = 4 * (c & 3);
        ow[r * 32 + o_piece(r, t * 8 + c)] = make_float4(o[i][k], o[i + 1][k], o[i + 2][k], o[i + 3][k]);
      }
    __syncthreads();
    if (s.abort) break;
    // a thread joins 4 x 4 elements of row tid / 8
    const int r = tid >> 3, cc = tid & 7;
    float mm = -INFINITY;
#pragma unroll
    for (int w = 0; w < QT_WARPS; ++w) mm = fmaxf(mm, s.m[w][r]);
    float ll = 0.f;
    float4 acc[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) acc[k] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < QT_WARPS; ++w) {
      const float mw = s.m[w][r];
      const float f = mw == -INFINITY ? 0.f : ex2(mw - mm);
      ll += s.l[w][r] * f;
      const float4* src = reinterpret_cast<const float4*>(rings + w * RING_BYTES);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float4 x = src[r * 32 + o_piece(r, 8 * k + cc)];
        acc[k].x = fmaf(x.x, f, acc[k].x);
        acc[k].y = fmaf(x.y, f, acc[k].y);
        acc[k].z = fmaf(x.z, f, acc[k].z);
        acc[k].w = fmaf(x.w, f, acc[k].w);
      }
    }
    // every row's place, for the thread that writes it
    const int rr = tile * QT_ROWS + r;
    int64_t at = -1;
    if (rr < n_rows) {
      const int slot = rr / rows_per_cand;
      at = (static_cast<int64_t>(__ldg(p.perm + seg + slot)) * p.H + hk * p.group) * p.Lq + (rr - slot * rows_per_cand);
    }
    bool write = ns == 1;
    if (ns > 1) {
      // partial rows [r][128], then m, l; the tile's splits lie uw.tiles apart
      const int first = part0[u] + hk * ns * uw.tiles + tile;
      float* part = p.part + static_cast<int64_t>(first + split * uw.tiles) * QT_PART;
#pragma unroll
      for (int k = 0; k < 4; ++k) reinterpret_cast<float4*>(part)[r * 32 + 8 * k + cc] = acc[k];
      if (cc == 0) {
        part[QT_ROWS * QC_D + r] = mm;
        part[QT_ROWS * QC_D + QT_ROWS + r] = ll;
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
        mm = -INFINITY;
        const float* p0 = p.part + static_cast<int64_t>(first) * QT_PART;
        const int64_t step = static_cast<int64_t>(uw.tiles) * QT_PART;
        for (int k = 0; k < ns; ++k) mm = fmaxf(mm, __ldcg(p0 + k * step + QT_ROWS * QC_D + r));
        ll = 0.f;
#pragma unroll
        for (int k = 0; k < 4; ++k) acc[k] = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int sp = 0; sp < ns; ++sp) {
          const float* ps = p0 + sp * step;
          const float mw = __ldcg(ps + QT_ROWS * QC_D + r);
          const float f = mw == -INFINITY ? 0.f : ex2(mw - mm);
          ll += __ldcg(ps + QT_ROWS * QC_D + QT_ROWS + r) * f;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float4 x = __ldcg(reinterpret_cast<const float4*>(ps) + r * 32 + 8 * k + cc);
            acc[k].x = fmaf(x.x, f, acc[k].x);
            acc[k].y = fmaf(x.y, f, acc[k].y);
            acc[k].z = fmaf(x.z, f, acc[k].z);
            acc[k].w = fmaf(x.w, f, acc[k].w);
          }
        }
      }
    }
    if (write && at >= 0) {
      const float inv = ll > 0.f ? 1.0f / ll : (ll == 0.f ? 0.f : ll);  // no tokens: 0; NaN stays
      uint2* dst = reinterpret_cast<uint2*>(p.O + at * QC_D);
#pragma unroll
      for (int k = 0; k < 4; ++k)
        dst[8 * k + cc] = make_uint2(pack_bf16x2(acc[k].x * inv, acc[k].y * inv), pack_bf16x2(acc[k].z * inv, acc[k].w * inv));
      if (p.lse && cc == 0) p.lse[at] = ll > 0.f ? (mm + __log2f(ll)) * 0.69314718055994531f : (ll == 0.f ? -INFINITY : ll);
    }
    fence_proxy_async_smem();  // the rings were written by plain stores: order the next bulk copies after them
    __syncthreads();
  }
  if (s.abort && tid == 0) atomicOr(p.status, DEV_ERR_PIPE_TIMEOUT);
}

}  // namespace

int qattn_target(int num_sms) { return num_sms * QT_CTAS_PER_SM; }
size_t qattn_part_elems(int num_sms) { return static_cast<size_t>(2) * qattn_target(num_sms) * QT_PART; }

cudaError_t launch_qattn(const QcAttnParams& p, int num_sms, cudaStream_t s) {
  const size_t smem = QT_WARPS * RING_BYTES + 2 * sizeof(int32_t) * (static_cast<size_t>(p.n_users) + 1);
  cudaError_t e = cudaFuncSetAttribute(
      qattn_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
      static_cast<int>(QT_WARPS * RING_BYTES + 2 * sizeof(int32_t) * (SEG_MAX_USERS + 1)));
  if (e != cudaSuccess) return e;
  qattn_kernel<<<num_sms * QT_CTAS_PER_SM, QT_THREADS, smem, s>>>(p);
  return cudaGetLastError();
}

}  // namespace ikbo
