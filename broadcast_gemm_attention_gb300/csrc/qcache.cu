// qcache.cu -- the paged cache of 4-bit keys and values: lengths, pages and
// slots (resize), quantising new rows into their slots (append), and reading
// histories back as bf16 rows (load).  The layout is described in ikbo.h.
#include <cuda_bf16.h>

#include "ptx.cuh"
#include "qcache_internal.h"

namespace ikbo {
namespace {

// ------------------------------------------------------------------ resize
// One cluster; every CTA scans all users (pages taken, pages given back,
// tokens added) into its own shared memory, then the CTAs share the pages and
// tokens among them by flattened index, each finding its user by bisection.
// Pages released overwrite places of the free list that others still read,
// so the call has two phases with a cluster barrier between: first everything
// that reads the old state (pages taken, slots), then what replaces it.
// Bound: latency (a launch, one scan, two dependent loads): 15 users growing
// by 12 tokens each 5.8 us, one user 3.9; with many tokens the slots'
// bisections: 2048 users with 150 new tokens each, 30 us.
constexpr int QR_THREADS = 1024;

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Exclusive scans over the CTA's threads of three sums at once; v becomes the
// prefix, total the CTA's sums.
__device__ void scan3(int64_t (&v)[3], int64_t (&total)[3], int64_t (*warp_sums)[33]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t incl[3];
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    incl[k] = v[k];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, incl[k], o);
      if (lane >= o) incl[k] += y;
    }
    if (lane == 31) warp_sums[k][warp] = incl[k];
  }
  __syncthreads();
  if (warp < 3) {
    const int64_t s = warp_sums[warp][lane];
    int64_t si = s;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, si, o);
      if (lane >= o) si += y;
    }
    warp_sums[warp][lane] = si - s;
    if (lane == 31) warp_sums[warp][32] = si;
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    v[k] = incl[k] - v[k] + warp_sums[k][warp];
    total[k] = warp_sums[k][32];
  }
}

__global__ void __launch_bounds__(QR_THREADS) qc_resize_kernel(const QcResizeParams p) {
  extern __shared__ int32_t qr_sm[];
  int32_t* take0 = qr_sm;                      // [n_users] pages taken before this user
  int32_t* give0 = qr_sm + p.n_users;          // [n_users] pages given back before
  int32_t* token0 = qr_sm + 2 * p.n_users;     // [n_users] tokens added before
  int32_t* old = qr_sm + 3 * p.n_users;        // [n_users] lengths, as they were ..
  int32_t* fresh = qr_sm + 4 * p.n_users;      // .. and as they are to be
  __shared__ int64_t warp_sums[3][33];
  __shared__ int bad_users;
  const int tid = threadIdx.x, n = p.n_users;
  const int rank = static_cast<int>(blockIdx.x), ranks = static_cast<int>(gridDim.x);
  const int page = 1 << p.page_log2;
  const int64_t most = static_cast<int64_t>(p.max_blocks) << p.page_log2;
  if (tid == 0) bad_users = 0;
  bool bad = false;
  for (int u = tid; u < n; u += QR_THREADS) {
    old[u] = qc_length(p.lens, u, most, bad);
    fresh[u] = qc_length(p.new_lens, u, most, bad);
  }
  __syncthreads();

  const int per = (n + QR_THREADS - 1) / QR_THREADS;
  const int lo = min(tid * per, n), hi = min(lo + per, n);
  int64_t v[3] = {0, 0, 0}, total[3];
  for (int u = lo; u < hi; ++u) {
    const int before = old[u], after = fresh[u];
    const int have = (before + page - 1) >> p.page_log2, need = (after + page - 1) >> p.page_log2;
    v[0] += max(need - have, 0);
    v[1] += max(have - need, 0);
    v[2] += max(after - before, 0);
  }
  if (bad) bad_users = 1;
  scan3(v, total, warp_sums);
  for (int u = lo; u < hi; ++u) {
    const int before = old[u], after = fresh[u];
    const int have = (before + page - 1) >> p.page_log2, need = (after + page - 1) >> p.page_log2;
    take0[u] = static_cast<int32_t>(v[0]);
    give0[u] = static_cast<int32_t>(v[1]);
    token0[u] = static_cast<int32_t>(v[2]);
    v[0] += max(need - have, 0);
    v[1] += max(have - need, 0);
    v[2] += max(after - before, 0);
  }
  const int n_free = *p.n_free;
  __syncthreads();  // the prefixes and bad_users are complete
  const bool broken = bad_users != 0 || n_free < 0 || n_free > p.n_pages || total[2] > p.max_new ||
                      n_free - total[0] + total[1] > p.n_pages;
  const bool short_of = !broken && total[0] > n_free;
  const bool refused = broken || short_of;
  const int takes = refused ? 0 : static_cast<int>(total[0]), gives = refused ? 0 : static_cast<int>(total[1]);
  const int tokens = refused ? 0 : static_cast<int>(total[2]);
  if (refused && rank == 0 && tid == 0) atomicOr(p.status, broken ? DEV_ERR_CACHE : DEV_ERR_OUT_OF_PAGES);

  const int first = rank * QR_THREADS + tid, step = ranks * QR_THREADS;
  bool bad_page = false;
  for (int k = first; k < takes; k += step) {
    const int u = qc_find(take0, n, k);
    const int have = (old[u] + page - 1) >> p.page_log2;
    const int id = p.free_pages[n_free - 1 - k];
    if (id < 0 || id >= p.n_pages) bad_page = true;
    p.table[static_cast<int64_t>(u) * p.max_blocks + have + (k - take0[u])] = id;
  }
  // eight tokens in a row per thread: the first one's user is looked for, the
  // others follow; their page numbers are loaded together
  const bool wide = ((reinterpret_cast<uintptr_t>(p.slots) | reinterpret_cast<uintptr_t>(p.positions)) & 15) == 0;
  for (int64_t i0 = static_cast<int64_t>(first) * 8; i0 < p.max_new; i0 += static_cast<int64_t>(step) * 8) {
    int slot[8], pos[8];
    const int32_t* from[8];
    int u = i0 < tokens ? qc_find(token0, n, static_cast<int>(i0)) : 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      pos[j] = 0;
      from[j] = nullptr;
      const int i = static_cast<int>(i0) + j;
      if (i0 + j < tokens) {
        while (u + 1 < n && token0[u + 1] <= i) ++u;
        const int before = old[u], have = (before + page - 1) >> p.page_log2;
        pos[j] = before + (i - token0[u]);
        const int blk = pos[j] >> p.page_log2;
        from[j] = blk < have ? p.table + static_cast<int64_t>(u) * p.max_blocks + blk
                             : p.free_pages + (n_free - 1 - (take0[u] + blk - have));
      }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) slot[j] = from[j] ? *from[j] : -1;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (slot[j] >= 0 && slot[j] < p.n_pages) {
        slot[j] = (slot[j] << p.page_log2) + (pos[j] & (page - 1));
      } else {
        bad_page = bad_page || from[j] != nullptr;
        slot[j] = -1;
      }
    }
    if (wide && i0 + 8 <= p.max_new) {
#pragma unroll
      for (int j = 0; j < 8; j += 4) {
        *reinterpret_cast<int4*>(p.slots + i0 + j) = make_int4(slot[j], slot[j + 1], slot[j + 2], slot[j + 3]);
        if (p.positions) *reinterpret_cast<int4*>(p.positions + i0 + j) = make_int4(pos[j], pos[j + 1], pos[j + 2], pos[j + 3]);
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (i0 + j < p.max_new) {
          p.slots[i0 + j] = slot[j];
          if (p.positions) p.positions[i0 + j] = pos[j];
        }
    }
  }
  for (int u = first; u <= n; u += step) p.offsets[u] = refused ? 0 : (u == n ? tokens : token0[u]);

  cluster_sync();  // every read of the old lengths, table entries and free list is done

  for (int k = first; k < gives; k += step) {
    const int u = qc_find(give0, n, k);
    const int need = (fresh[u] + page - 1) >> p.page_log2;
    int32_t* entry = p.table + static_cast<int64_t>(u) * p.max_blocks + need + (k - give0[u]);
    const int id = *entry;
    if (id < 0 || id >= p.n_pages) bad_page = true;
    p.free_pages[n_free - takes + k] = id;
    *entry = -1;
  }
  if (!refused)
    for (int u = first; u < n; u += step) p.lens[u] = fresh[u];
  if (!refused && rank == 0 && tid == 0) *p.n_free = n_free - takes + gives;
  if (bad_page) atomicOr(p.status, DEV_ERR_CACHE);
}

// ------------------------------------------------------------------ append
// Eight lanes take a head of a row, sixteen elements of K and of V each, two
// lanes to a group of 32; a thread runs over its row's heads, so the slot and
// the address are worked out once.  Bound: issue, not memory (2 bytes read and
// 0.625 written an element): twelve instructions an element, although the
// arithmetic takes two elements in one; 77% of the issue slots and 71% of the
// integer pipe are busy, DRAM 63%.  So there is no
// division: q = (x - z) / s comes from an approximate reciprocal and one step of
// Markstein's correction ("Computation of elementary functions on the IBM RISC
// System/6000 processor", 1990), and so does the 7.5 below.  The codes are the
// division's: the corrected quotient is exact where the quotient is an fp32
// number, ties among them, and nowhere else does the quotient of these operands
// (a difference of bf16 values over a bf16 value) come close enough to a
// half-integer for its error of half an ulp to matter.
// Measured (caches cold and full of lines to write back): 15 histories of 2048
// tokens x 8 heads, 126 MB read and 39 MB written, 37.5 us, 4.4 TB/s; a row at a
// time without the packed arithmetic 40.9.
constexpr int QA_THREADS = 128;  // (256: 39.6 us for the histories below, against 37.5)
constexpr int QA_LANES = 8;  // of a head of a row

__device__ __forceinline__ uint32_t min2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ float low_half(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float high_half(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
__device__ __forceinline__ float rcp_approx(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

struct GroupCode {
  uint2 codes;    // of this lane's sixteen elements
  uint32_t pair;  // (s, z)
};

// The codes by division: groups of extreme scales, or without values (0, or NaN).
__device__ __noinline__ uint2 slow_codes(const uint4 x, const uint4 y, float s, float z) {
  const uint32_t w[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
  uint32_t c[2] = {0, 0};
  if (s > 0.f) {
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      const float t = ((j & 1) ? high_half(w[j >> 1]) : low_half(w[j >> 1])) - z;
      const float q = fminf(fmaxf(__fdiv_rn(t, s), 16.f), 31.f);
      c[j >> 3] |= (__float_as_uint(q + 8388608.f) & 15u) << (4 * (j & 7));
    }
  }
  return make_uint2(c[0], c[1]);
}

// Two fp32 numbers, in one instruction each operation.
struct F2 {
  uint64_t v;
  static __device__ __forceinline__ F2 of(float a, float b) {
    F2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(a), "f"(b));
    return r;
  }
  __device__ __forceinline__ void get(float& a, float& b) const { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v)); }
};
__device__ __forceinline__ F2 operator+(F2 x, F2 y) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(x.v), "l"(y.v));
  return r;
}
__device__ __forceinline__ F2 operator*(F2 x, F2 y) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(x.v), "l"(y.v));
  return r;
}
__device__ __forceinline__ F2 fma(F2 x, F2 y, F2 z) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(x.v), "l"(y.v), "l"(z.v));
  return r;
}

// Sixteen of a group's 32 elements; the other lane of the pair has the rest.
__device__ __forceinline__ GroupCode quantise16(const uint4 x, const uint4 y) {
  const uint32_t w[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
  uint32_t mn = min2(min2(min2(w[0], w[1]), min2(w[2], w[3])), min2(min2(w[4], w[5]), min2(w[6], w[7])));
  uint32_t mx = max2(max2(max2(w[0], w[1]), max2(w[2], w[3])), max2(max2(w[4], w[5]), max2(w[6], w[7])));
  mn = min2(mn, __shfl_xor_sync(0xffffffffu, mn, 1));
  mx = max2(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
  mn = min2(mn, mn >> 16);  // the low half holds the group's, also where it is NaN
  mx = max2(mx, mx >> 16);
  const float lo = low_half(mn), hi = low_half(mx);
  const float range = hi * 0.5f - lo * 0.5f;
  float step;
  if (range >= 1e-30f) {
    constexpr float inv = 1.0f / 7.5f;
    const float q0 = range * inv;
    step = fmaf(fmaf(-q0, 7.5f, range), inv, q0);
  } else {
    step = __fdiv_rn(range, 7.5f);  // remainders would not be normal numbers (or the range is NaN)
  }
  __nv_bfloat16 sb = __float2bfloat16_rn(step);
  __nv_bfloat16 zb = __float2bfloat16_rn(lo - 16.f * __bfloat162float(sb));
  float s = __bfloat162float(sb), z = __bfloat162float(zb);
  if (!(fabsf(s) <= 3.4e38f && fabsf(z) <= 3.4e38f)) {
    s = z = __uint_as_float(0x7fc00000u);
    sb = zb = __float2bfloat16_rn(s);
  }
  GroupCode g;
  g.pair = static_cast<uint32_t>(__bfloat16_as_ushort(sb)) | (static_cast<uint32_t>(__bfloat16_as_ushort(zb)) << 16);
  if (!(s >= 1e-30f && s <= 1e30f)) {  // the reciprocal or the remainders would not be normal numbers
    g.codes = slow_codes(x, y, s, z);
    return g;
  }
  // a quotient q in 16 .. 31 plus 2^23 is rounded to an integer in its low bits:
  // 0x4B000000 + q.  Sixteen-fold sums of those, less the constants', are the codes
  // (two elements at a time: the packed instructions round like the single ones)
  const float inv = rcp_approx(s);
  const F2 inv2 = F2::of(inv, inv), minus_s = F2::of(-s, -s), minus_z = F2::of(-z, -z);
  const F2 magic = F2::of(8388608.f, 8388608.f);
  uint32_t c[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    c[h] = 0;
#pragma unroll
    for (int j = 3; j >= 0; --j) {
      const uint32_t e = w[4 * h + j];
      const F2 t = F2::of(low_half(e), high_half(e)) + minus_z;
      const F2 q0 = t * inv2;
      float a, b;
      fma(fma(q0, minus_s, t), inv2, q0).get(a, b);
      (F2::of(fminf(fmaxf(a, 16.f), 31.f), fminf(fmaxf(b, 16.f), 31.f)) + magic).get(a, b);
      c[h] = (c[h] * 16u + __float_as_uint(b)) * 16u + __float_as_uint(a);
    }
    c[h] -= 0x4B000010u * 0x11111111u;
  }
  g.codes = make_uint2(c[0], c[1]);
  return g;
}

__global__ void __launch_bounds__(QA_THREADS) qc_append_kernel(const QcAppendParams p) {
  const int row = static_cast<int>(blockIdx.x) * (QA_THREADS / QA_LANES) + (static_cast<int>(threadIdx.x) / QA_LANES);
  const int lane8 = static_cast<int>(threadIdx.x) % QA_LANES;
  const int h0 = static_cast<int>(blockIdx.y) * p.heads_per_cta, h1 = min(p.H, h0 + p.heads_per_cta);
  const bool there = row < p.n_rows;
  const int slot = there ? __ldg(p.slots + row) : -1;
  const bool valid = slot >= 0 && slot < p.n_slots;
  if (there && slot != -1 && !valid && lane8 == 0 && h0 == 0) atomicOr(p.status, DEV_ERR_CACHE);
  const int64_t at = (valid ? row * p.row_stride : 0) + static_cast<int64_t>(h0) * QC_D + lane8 * 16;
  const uint4* k = reinterpret_cast<const uint4*>(p.K + at);
  const uint4* v = reinterpret_cast<const uint4*>(p.V + at);
  const int64_t block = slot >> 4;
  const int64_t page = block >> p.blocks_log2, sub = block & ((1 << p.blocks_log2) - 1);
  const int r = slot & 15;
  uint8_t* base = p.data + (((page * p.H + h0) << p.blocks_log2) + sub) * QC_BLOCK_BYTES + r * 64 + lane8 * 8;
  uint8_t* pairs = base - r * 64 - lane8 * 8 + QC_CODE_BYTES + r * 16 + (lane8 >> 1) * 4;
  const int64_t step = static_cast<int64_t>(QC_BLOCK_BYTES) << p.blocks_log2;  // from a head to the next
  const uint4 none = make_uint4(0, 0, 0, 0);
  // whole warps: lanes without a row code zeros; the next head's elements are on their way
  uint4 k0 = none, k1 = none, v0 = none, v1 = none;
  if (valid) {
    k0 = __ldg(k);
    k1 = __ldg(k + 1);
    v0 = __ldg(v);
    v1 = __ldg(v + 1);
  }
#pragma unroll 1
  for (int h = h0; h < h1; ++h) {
    const uint4 a0 = k0, a1 = k1, b0 = v0, b1 = v1;
    k += QC_D / 8;
    v += QC_D / 8;
    if (valid && h + 1 < h1) {
      k0 = __ldg(k);
      k1 = __ldg(k + 1);
      v0 = __ldg(v);
      v1 = __ldg(v + 1);
    }
    const GroupCode gk = quantise16(a0, a1), gv = quantise16(b0, b1);
    if (valid) {
      *reinterpret_cast<uint2*>(base) = gk.codes;
      *reinterpret_cast<uint2*>(base + QC_HALF_BYTES) = gv.codes;
      if ((lane8 & 1) == 0) {
        *reinterpret_cast<uint32_t*>(pairs) = gk.pair;
        *reinterpret_cast<uint32_t*>(pairs + QC_HALF_BYTES) = gv.pair;
      }
    }
    base += step;
    pairs += step;
  }
}

// -------------------------------------------------------------------- load
// A warp decodes one block (16 tokens) of one head: a lane turns four bytes
// of codes into eight bf16, a 16-byte store, so the warp writes two whole
// 256-byte rows at a time.  Blocks are numbered user-major over a prefix that
// every CTA scans for itself.  Bound: memory, mostly the bf16 rows written:
// 15 histories of 2048 tokens x 8 heads, 165 MB, 26.7 us alone (6.2 TB/s) and
// 34.5 where the caches are full of lines to write back.
// kPacked (for the attention's workspace): user u's rows start at a multiple
// of 128 of their own and are padded with zero rows to the next, so that no
// tile of one user meets another's rows.
constexpr int QL_THREADS = 256;

__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t* warp_sums, int64_t* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  constexpr int warps = QL_THREADS / 32;
  int64_t incl = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) warp_sums[warp] = incl;
  __syncthreads();
  int64_t before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < warps; ++w) {
    before += w < warp ? warp_sums[w] : 0;
    all += warp_sums[w];
  }
  __syncthreads();
  *total = all;
  return before + incl - v;
}

__device__ __forceinline__ void decode_rows(const uint8_t* half, uint16_t* out, int64_t row_elems, int rows, int zero_from) {
  const int lane = static_cast<int>(threadIdx.x & 31u);
  const uint32_t* codes = reinterpret_cast<const uint32_t*>(half);
  const uint32_t* pairs = reinterpret_cast<const uint32_t*>(half + QC_CODE_BYTES);
  const int piece = lane & 15;
  uint32_t w[8], sz[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const int r = 2 * k + (lane >> 4);
    const bool there = r < zero_from;
    w[k] = there ? __ldg(codes + r * 16 + piece) : 0u;
    sz[k] = there ? __ldg(pairs + r * 4 + (piece >> 2)) : 0u;
  }
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const int r = 2 * k + (lane >> 4);
    if (r >= rows) continue;
    const uint32_t s2 = __byte_perm(sz[k], 0, 0x1010), z2 = __byte_perm(sz[k], 0, 0x3232);
    // the decoded pairs are elements (0, 4), (1, 5), (2, 6), (3, 7)
    const uint32_t a = qc_decode<0>(w[k], s2, z2), b = qc_decode<1>(w[k], s2, z2);
    const uint32_t c = qc_decode<2>(w[k], s2, z2), d = qc_decode<3>(w[k], s2, z2);
    uint4 o;
    o.x = __byte_perm(a, b, 0x5410);
    o.y = __byte_perm(c, d, 0x5410);
    o.z = __byte_perm(a, b, 0x7632);
    o.w = __byte_perm(c, d, 0x7632);
    *reinterpret_cast<uint4*>(out + r * row_elems + piece * 8) = o;
  }
}

template <bool kPacked>
__global__ void __launch_bounds__(QL_THREADS) qc_load_kernel(const QcLoadParams p) {
  extern __shared__ int32_t ql_sm[];
  int32_t* block0 = ql_sm;  // [n_users + 1] blocks before each user
  __shared__ int64_t warp_sums[QL_THREADS / 32];
  const int tid = threadIdx.x, n = p.n_users;
  const int64_t most = (static_cast<int64_t>(p.max_blocks) << p.blocks_log2) * QC_ROWS;
  const int per = (n + QL_THREADS - 1) / QL_THREADS;
  const int lo = min(tid * per, n), hi = min(lo + per, n);
  // blocks of a user: its tokens' blocks, or when packed all of its padded rows'
  // (unsigned: a length may be 16 short of 2^31)
  const auto user_blocks = [](int len) {
    const uint32_t x = static_cast<uint32_t>(len);
    return static_cast<int>(kPacked ? (x + ATT_BN - 1) / ATT_BN * (ATT_BN / QC_ROWS) : (x + QC_ROWS - 1) / QC_ROWS);
  };
  int64_t mine = 0;
  bool bad = false;
  for (int u = lo; u < hi; ++u) {
    const int len = qc_length(p.lens, u, most, bad);
    mine += user_blocks(len);
  }
  int64_t total;
  int64_t before = block_scan(mine, warp_sums, &total);
  const bool too_many = total > 0x7fffffff;  // block numbers are 32 bits
  bool ignored = false;
  int64_t sum = 0;
  for (int u = lo; u < hi; ++u) {
    block0[u] = static_cast<int32_t>(before);
    const int len = qc_length(p.lens, u, most, ignored);
    const int b = user_blocks(len);
    if (kPacked && blockIdx.x == 0) {
      const int64_t first = before * QC_ROWS;
      const bool fits = !too_many && first + static_cast<int64_t>(b) * QC_ROWS <= p.n_rows;
      if (!fits) bad = true;
      p.ranges[u] = fits ? static_cast<int32_t>(first) : 0;
      p.ranges[n + u] = fits ? len : 0;
    }
    sum += len;
    before += b;
  }
  if (tid == 0) block0[n] = static_cast<int32_t>(total);
  if (blockIdx.x == 0) {
    bad = bad || too_many;
    if (kPacked) {
      __shared__ unsigned long long all;
      if (tid == 0) all = 0;
      __syncthreads();
      atomicAdd(&all, static_cast<unsigned long long>(sum));
      __syncthreads();
      if (all > static_cast<unsigned long long>(p.bound)) bad = true;
    }
    if (bad) atomicOr(p.status, DEV_ERR_CACHE);
  }
  if (too_many) return;
  __syncthreads();

  const int warps = QL_THREADS / 32;
  const int64_t items = total * p.H;
  const int64_t row_elems = static_cast<int64_t>(p.H) * QC_D;
  for (int64_t it = static_cast<int64_t>(blockIdx.x) * warps + (tid >> 5); it < items;
       it += static_cast<int64_t>(gridDim.x) * warps) {
    const int blk = static_cast<int>(it / p.H), h = static_cast<int>(it - static_cast<int64_t>(blk) * p.H);
    const int u = qc_find(block0, n, blk);
    const int b = blk - block0[u];  // the user's block
    const int len = qc_length(p.lens, u, most, ignored);
    const int left = len - b * QC_ROWS;  // tokens from this block on (<= 0: padding)
    int64_t row;
    int rows;
    if (kPacked) {
      row = static_cast<int64_t>(blk) * QC_ROWS;
      rows = row + QC_ROWS <= p.n_rows ? QC_ROWS : 0;
    } else {
      const int64_t r0 = __ldg(p.kv_offsets + u), r1 = __ldg(p.kv_offsets + u + 1);
      row = r0 + static_cast<int64_t>(b) * QC_ROWS;
      const bool legal = r0 >= 0 && r0 <= r1 && r1 <= p.n_rows;
      const int64_t room = legal ? r1 - row : 0;
      rows = static_cast<int>(max(static_cast<int64_t>(0), min(room, static_cast<int64_t>(min(left, QC_ROWS)))));
      if (rows < min(left, QC_ROWS) && (threadIdx.x & 31) == 0) atomicOr(p.status, DEV_ERR_CACHE);
    }
    if (rows == 0) continue;
    int zero_from = kPacked ? max(0, min(left, QC_ROWS)) : QC_ROWS;
    const uint8_t* src = p.data;
    if (left > 0) {
      const int id = __ldg(p.table + static_cast<int64_t>(u) * p.max_blocks + (b >> p.blocks_log2));
      if (id < 0 || id >= p.n_pages) {
        if ((threadIdx.x & 31) == 0) atomicOr(p.status, DEV_ERR_CACHE);
        if (!kPacked) continue;
        zero_from = 0;
      } else {
        src += (((static_cast<int64_t>(id) * p.H + h) << p.blocks_log2) + (b & ((1 << p.blocks_log2) - 1))) *
               QC_BLOCK_BYTES;
      }
    }
    const int64_t at = row * row_elems + h * QC_D;
    if (p.K) decode_rows(src, p.K + at, row_elems, rows, zero_from);
    if (p.V) decode_rows(src + QC_HALF_BYTES, p.V + at, row_elems, rows, zero_from);
  }
}

}  // namespace

cudaError_t launch_qc_resize(const QcResizeParams& p, cudaStream_t s) {
  const size_t smem = 5 * sizeof(int32_t) * static_cast<size_t>(p.n_users);
  cudaError_t e = cudaFuncSetAttribute(qc_resize_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       static_cast<int>(5 * sizeof(int32_t) * SEG_MAX_USERS));
  if (e != cudaSuccess) return e;
  // a CTA for each 8192 tokens, up to the portable cluster of 8
  int ctas = 1;
  while (ctas < 8 && static_cast<int64_t>(ctas) * 8192 < p.max_new) ctas *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas));
  cfg.blockDim = dim3(QR_THREADS);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = static_cast<unsigned>(ctas);
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, qc_resize_kernel, p);
}

cudaError_t launch_qc_append(QcAppendParams p, int num_sms, cudaStream_t s) {
  const int per = QA_THREADS / QA_LANES;
  const int ctas = (p.n_rows + per - 1) / per;
  // heads are spread over CTAs only while that gives work to more SMs
  int parts = 1;
  while (parts < p.H && static_cast<int64_t>(ctas) * parts < 16 * static_cast<int64_t>(num_sms)) parts *= 2;
  if (parts > p.H) parts = p.H;
  p.heads_per_cta = (p.H + parts - 1) / parts;
  const dim3 grid(static_cast<unsigned>(ctas), static_cast<unsigned>((p.H + p.heads_per_cta - 1) / p.heads_per_cta));
  if (grid.y > 65535) return cudaErrorInvalidValue;
  qc_append_kernel<<<grid, QA_THREADS, 0, s>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_qc_load(const QcLoadParams& p, int num_sms, cudaStream_t s) {
  const size_t smem = sizeof(int32_t) * (static_cast<size_t>(p.n_users) + 1);
  const int64_t blocks = (p.n_rows + QC_ROWS - 1) / QC_ROWS + (p.kv_offsets ? p.n_users : 0);
  const int64_t ctas_wanted = (blocks * p.H + QL_THREADS / 32 - 1) / (QL_THREADS / 32);
  const int64_t most = 8 * static_cast<int64_t>(num_sms);
  const unsigned ctas = static_cast<unsigned>(ctas_wanted < 1 ? 1 : (ctas_wanted < most ? ctas_wanted : most));
  if (p.kv_offsets) qc_load_kernel<false><<<ctas, QL_THREADS, smem, s>>>(p);
  else qc_load_kernel<true><<<ctas, QL_THREADS, smem, s>>>(p);
  return cudaGetLastError();
}

}  // namespace ikbo
