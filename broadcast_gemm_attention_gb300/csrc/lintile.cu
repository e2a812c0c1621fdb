// lintile.cu -- linear attention with a decay on the 5th-gen tensor cores, for
// histories of more than a few chunks (linattn.cu has the mathematics).
//
// In chunks of 128 rows, every product a 128 x 128 x 128 one with its result in
// tensor memory (x queries, y keys, z values, S the state before the chunk):
//   A  = x y^T            to registers, decayed and masked, back as bf16
//   O1 = x S              S's bf16 image in shared memory
//   O2 = A z
//   S  = decay^n S + (w y)^T z
//                         S stays in tensor memory in fp32; w y, each row with its
//                         decay to the chunk's end, as two bf16 parts in shared
//                         memory (2^-16), so two products
//   out = scale (O2 + decay^(i+1) O1)
// Of a scan whose state is a gradient the scale is in w, not in O1's factor.
//
// Per CTA (persistent, one per SM, 32 warps):
//   warp 0       loads x, y, z by TMA; warp 1 issues A, O1, O2; warp 2 issues S
//   warps 4-11   A's decays
//   warps 12-19  the outputs
//   warps 20-27  S: its image, and its decay before a chunk is added
//   warps 28-31  the two parts of w y
// The groups' work is bound by latencies (loads of tensor memory, barriers, a few
// dozen dependent instructions), so each has warps of its own.
// y and z have one buffer each, free once w y and A are formed, and after O2 and S's
// products, so that a chunk's loads lie beside the products of the one before.  x has two:
// the outputs leave by way of the one whose products have ended (54.2 us with a place of
// their own, 53.7 so; two buffers for z instead of x 55.0).
//
// Bound: a chunk of one scan takes 2.55 us, 5280 cycles, of which shared memory's 576 KB take 4608 (products 288,
// parts 96, image 32, outputs 64, loads 96).  120 scans at a time move 6.05 TB/s (2.60 us), and 152 6.8, memory's
// rate (2.92).  15 histories of 1200 to 2048 rows, 8 heads, bf16: 52.0 us, the longest's 16 chunks and 11 of start
// and end, 3.9 TB/s of the tensors' bytes, 0.34 of the tensor pipe's cycles; with 16x8x16 products in registers
// (linattn.cu) 142 us.  Their gradient at 524 to 1024 rows: 74 us (178).
//
// A reverse scan keeps the rows' order in its tiles and turns masks and decays around
// instead (row j reaches i <= j, and the chunk's first row is its end).
#include <cuda.h>
#include <cuda_bf16.h>

#include "launch.cuh"
#include "linattn_internal.h"
#include "mma_common.cuh"
#include "tile_common.cuh"

namespace ikbo {
namespace {

constexpr int LT_CHUNK = 128;
constexpr int LT_THREADS = 1024;
constexpr int DECAY_WARP0 = 4, OUT_WARP0 = 12, STATE_WARP0 = 20, PARTS_WARP0 = 28;
constexpr int GROUP_WARPS = 8, PARTS_WARPS = 4;
constexpr uint32_t TM_A = 0, TM_O1 = 128, TM_O2 = 256, TM_S = 384;

constexpr uint32_t TILE = 2 * HALF_TILE;  // 32 KB
constexpr uint32_t X_AT = 0, Y_AT = TILE, Z_AT = 2 * TILE, HI_AT = 3 * TILE, LO_AT = 4 * TILE, S_AT = 5 * TILE, X1_AT = 6 * TILE;
constexpr uint32_t OUT_BYTES = 32 * 128;  // of a tile, per warp of a group
static_assert(GROUP_WARPS * OUT_BYTES == TILE, "the outputs take x's place");
constexpr uint32_t AUX_AT = 7 * TILE;

struct Aux {
  uint64_t x_full[2], y_full, z_full, x_empty[2], y_empty, z_empty;
  uint64_t a_full, p_full, o_full, o_empty, s_full, s_empty, w_full[2], m_full, m_begun, w_empty[2], drain[2], group[2];
  float4 near[4];             // a 16-column block's decays to its nearest column
  float power[LT_CHUNK + 4];  // decay^n of the current item
  uint2 parts[LT_CHUNK];      // decay^n (and the scale, in a gradient's state) as a bf16 pair of the same, and what that lacks
  uint32_t tmem_slot, abort;
};
constexpr uint32_t LT_SMEM_USED = AUX_AT + sizeof(Aux);
constexpr uint32_t LT_SMEM = LT_SMEM_USED + 1024;
static_assert(LT_SMEM <= 227 * 1024, "tiles do not fit in shared memory");

struct LtMaps {
  CUtensorMap x[LIN_MAX_JOBS], y[LIN_MAX_JOBS], z[LIN_MAX_JOBS];
};

// One scan or segment of one.
struct Item {
  int job, u, h, seg, segs;
  int base, n;      // its rows: base .. base + n - 1 of the tensors
  bool reverse, whole_user_empty;
  int early;        // its first row takes the start as it is
  int chunks;
  // chunk c's rows, first and count
  __device__ __forceinline__ int rows(int c) const { return min(LT_CHUNK, n - c * LT_CHUNK); }
  __device__ __forceinline__ int first(int c) const { return base + (reverse ? n - c * LT_CHUNK - rows(c) : c * LT_CHUNK); }
};

// The rows of user u; none where the offsets are out of range.
__device__ __forceinline__ int user_rows(const LinParams& p, int u, int& first, bool report) {
  if (!p.offsets) {
    const int each = p.n_rows / p.n_users;
    first = u * each;
    return each;
  }
  const int a = __ldcg(p.offsets + u), b = __ldcg(p.offsets + u + 1);
  first = a;
  if (a >= 0 && b >= a && b <= p.n_rows && b - a <= p.max_len) return b - a;
  if (report) atomicOr(p.status, DEV_ERR_CACHE);
  first = 0;
  return 0;
}

// Of user u's scans, items a launch has of each: all segments, or (local) all but the last.
template <bool kLocal>
__device__ __forceinline__ int user_segs(const LinParams& p, int u) {
  if (u >= p.n_users) return 0;
  int first;
  const int len = user_rows(p, u, first, false);
  return max(1, (len + p.seg_len - 1) / p.seg_len) - (kLocal ? 1 : 0);
}

// A CTA's items, one after the other, by whole warps.
//
// Scans are dealt out longest first, back and forth over the CTAs (so that a CTA's long
// one meets a short one: the gradient of 15 users' 524 to 1024 rows 83 -> 76 us), where there
// are no segments, more than one a CTA, and a lane for each user; else in order.
template <bool kLocal>
struct Items {
  int per_job;    // items of one job
  int items, k;   // of the launch; turns taken
  bool sorted;
  int rank;       // of the lane's user, by rows

  __device__ __forceinline__ Items(const LinParams& p) : k(0) {
    const int lane = static_cast<int>(lane_id());
    sorted = p.segs == 1 && p.n_users <= 32 && p.n_users * p.H * p.n_jobs > static_cast<int>(gridDim.x);
    rank = lane;
    if (p.segs == 1) {
      per_job = p.n_users * p.H;
      if (sorted) {
        int first;
        const int len = lane < p.n_users ? user_rows(p, lane, first, false) : -1;
        rank = 0;
#pragma unroll 1
        for (int v = 0; v < 32; ++v) {
          const int other = __shfl_sync(0xffffffffu, len, v);
          rank += other > len || (other == len && v < lane);
        }
      }
    } else {
      int sum = 0;
#pragma unroll 1
      for (int u = 0; u < p.n_users; u += 32) sum += static_cast<int>(__reduce_add_sync(0xffffffffu, static_cast<uint32_t>(user_segs<kLocal>(p, u + lane))));
      per_job = sum * p.H;
    }
    items = per_job * p.n_jobs;
  }

  // The CTA's next item; false: none is left.
  __device__ __forceinline__ bool next(const LinParams& p, Item& x, bool report) {
    const int ctas = static_cast<int>(gridDim.x), cta = static_cast<int>(blockIdx.x);
#pragma unroll 1
    for (; k * ctas < items; ++k) {
      const int i = k & 1 ? (k + 1) * ctas - 1 - cta : k * ctas + cta;
      if (i >= items) continue;
      ++k;
      get(p, i, x, report);
      return true;
    }
    return false;
  }

  __device__ __forceinline__ void get(const LinParams& p, int i, Item& x, bool report) const {
    const int lane = static_cast<int>(lane_id());
    x.seg = 0;
    if (sorted) {
      const int each = p.n_jobs * p.H, which = i / each, r = i - which * each;
      x.u = __ffs(static_cast<int>(__ballot_sync(0xffffffffu, rank == which))) - 1;
      x.job = r / p.H;
      x.h = r - x.job * p.H;
    } else {
      x.job = i / per_job;
      const int r = i - x.job * per_job;
      if (p.segs == 1) {
        x.u = r / p.H;
        x.h = r - x.u * p.H;
      } else {  // users one after the other, each with its own number of segments for each head
        int before = 0, u0 = 0, mine, upto;
#pragma unroll 1
        for (;; u0 += 32) {
          mine = user_segs<kLocal>(p, u0 + lane);
          upto = mine;
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += y;
          }
          const int all = __shfl_sync(0xffffffffu, upto, 31);
          if (r < (before + all) * p.H || u0 + 32 >= p.n_users) break;
          before += all;
        }
        const int l = __ffs(static_cast<int>(__ballot_sync(0xffffffffu, r < (before + upto) * p.H))) - 1;
        mine = __shfl_sync(0xffffffffu, mine, l);
        const int in = r - (before + __shfl_sync(0xffffffffu, upto, l) - mine) * p.H;
        x.u = u0 + l;
        x.h = in / mine;
        x.seg = in - x.h * mine;
      }
    }
    int first;
    const int len = user_rows(p, x.u, first, report);
    x.reverse = p.job[x.job].reverse != 0;
    x.segs = p.segs > 1 ? max(1, (len + p.seg_len - 1) / p.seg_len) : 1;
    const int r0 = x.segs > 1 ? x.seg * p.seg_len : 0;
    x.n = x.segs > 1 ? min(p.seg_len, len - r0) : len;
    x.base = first + (x.reverse ? len - r0 - x.n : r0);
    x.whole_user_empty = len == 0;
    x.early = !kLocal && x.seg == 0 && x.reverse ? 1 : 0;
    x.chunks = (x.n + LT_CHUNK - 1) / LT_CHUNK;
  }
};

// Where an item's state comes from (null: zero), and whether rows there are z's elements.
template <bool kLocal>
__device__ __forceinline__ const float* state_from(const LinParams& p, const Item& it, bool& turned) {
  turned = false;
  if (kLocal) return nullptr;
  const int64_t uh = static_cast<int64_t>(it.u) * p.H + it.h;
  // of several segments the first one's start is in the workspace too, as s_out may be s_in
  if (it.segs > 1)
    return p.ws + ((static_cast<int64_t>(it.job) * p.n_users * p.H + uh) * p.segs + (it.seg > 0 ? it.seg - 1 : it.segs - 1)) * LIN_STATE;
  turned = p.job[it.job].s_in_turned != 0;
  return p.job[it.job].s_in ? p.job[it.job].s_in + uh * LIN_STATE : nullptr;
}

// A group's warps meet.  (Not a hardware barrier: a warp that gave up does not come.)
__device__ __forceinline__ bool group_sync(uint64_t* bar, uint32_t& phase, Aux& x, const LinParams& p) {
  warp_arrive(bar);
  return warp_wait(bar, phase++ & 1u, x, p);
}

// bf16 pairs: a b, and a b + c, in one rounding each.
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t fma_bf16x2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t r;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
  return r;
}
// v (w.x + w.y) in two parts: the first is v w.x, rounded; what it lacks of that
// product has few enough bits to be exact, and v w.y is added to it.
__device__ __forceinline__ void decayed(uint32_t v, uint2 w, uint32_t& hi, uint32_t& lo) {
  hi = mul_bf16x2(v, w.x);
  lo = fma_bf16x2(v, w.y, fma_bf16x2(v, w.x, hi ^ 0x80008000u));
}

// ------------------------------------------------------------------ loader
// Asks for a tile in L2.
__device__ __forceinline__ void prefetch_3d(const CUtensorMap* map, int x, int y, int z) {
  asm volatile("cp.async.bulk.prefetch.tensor.3d.L2.global [%0, {%1, %2, %3}];" ::"l"(map), "r"(x), "r"(y), "r"(z) : "memory");
}

template <bool kOutputs, bool kLocal>
__device__ void loader(const LinParams& p, const LtMaps& maps, uint8_t* sm, Aux& x) {
  uint32_t g = 0;  // chunks loaded
  const auto load = [&](uint32_t at, const CUtensorMap* map, uint64_t* full, int h, int row) {
    if (elect_one()) {
      mbar_arrive_expect_tx(full, TILE);
      tma_load_3d(sm + at, map, full, 0, h, row);
      tma_load_3d(sm + at + HALF_TILE, map, full, 64, h, row);
    }
    __syncwarp();
  };
  uint32_t ny = 0, nx = 0, nz = 0;
  bool ok = true;
  Items<kLocal> items(p);
  Item it;
  for (bool more = items.next(p, it, false); more && ok;) {
    for (int c = 0; c < it.chunks && ok; ++c, ++g) {
      const uint32_t free = (g & 1u) ^ 1u;
      const int row = it.first(c);
      ok = warp_wait(&x.y_empty, free, x, p);
      if (!ok) break;
      load(Y_AT, &maps.y[it.job], &x.y_full, it.h, row);
      ++ny;
      if (kOutputs) {
        ok = warp_wait(&x.x_empty[g & 1u], ((g >> 1) & 1u) ^ 1u, x, p);
        if (!ok) break;
        load(g & 1u ? X1_AT : X_AT, &maps.x[it.job], &x.x_full[g & 1u], it.h, row);
        ++nx;
      }
      ok = warp_wait(&x.z_empty, free, x, p);
      if (!ok) break;
      load(Z_AT, &maps.z[it.job], &x.z_full, it.h, row);
      ++nz;
      if (c + 1 < it.chunks && elect_one()) {  // the next chunk's tiles, ahead of their buffers
        const int next = it.first(c + 1);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          prefetch_3d(&maps.y[it.job], 64 * half, it.h, next);
          prefetch_3d(&maps.z[it.job], 64 * half, it.h, next);
          if (kOutputs) prefetch_3d(&maps.x[it.job], 64 * half, it.h, next);
        }
      }
      __syncwarp();
    }
    more = ok && items.next(p, it, false);
    bool turned;
    const float* state = more ? state_from<kLocal>(p, it, turned) : nullptr;
    if (state && elect_one()) asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(state), "n"(LIN_STATE * 4) : "memory");
    __syncwarp();
  }
  // the copies in flight end before the CTA does, whichever warp's wait ran out
  if (ny) wait_a_second(&x.y_full, (ny - 1) & 1u);
  for (uint32_t k = nx > 2 ? nx - 2 : 0; k < nx; ++k) wait_a_second(&x.x_full[k & 1u], (k >> 1) & 1u);
  if (nz) wait_a_second(&x.z_full, (nz - 1) & 1u);
  __syncwarp();
}

// ----------------------------------------------------------------- issuers
// O1 = x S: A K-major, B (rows of S's y elements) MN-major.
__device__ __forceinline__ void issue_xs(uint32_t o_tmem, uint32_t x_base, uint32_t s_base) {
  constexpr uint32_t idesc = idesc_bf16_f32(128, 128, false, true);
  const uint64_t xd = sdesc_sw128(x_base, 16, 1024), sd = sdesc_sw128(s_base, HALF_TILE, 1024);
#pragma unroll
  for (int ks = 0; ks < 8; ++ks)
    mma_bf16_ss(o_tmem, xd + (((ks >> 2) * HALF_TILE + (ks & 3) * 32) >> 4), sd + ((ks * 2048u) >> 4), idesc, ks > 0 ? 1u : 0u);
}

// O2 = A z over the chunk's first 16 `steps` rows.  A's columns 64 .. lie behind
// 32 unused ones (each half of the output warps writes where it has read).
__device__ __forceinline__ void issue_az(uint32_t o_tmem, uint32_t a_tmem, uint32_t z_base, int steps) {
  constexpr uint32_t idesc = idesc_bf16_f32(128, 128, false, true);
  const uint64_t zd = sdesc_sw128(z_base, HALF_TILE, 1024);
#pragma unroll
  for (int ks = 0; ks < 8; ++ks) {
    if (ks >= steps) break;
    mma_bf16_ts(o_tmem, a_tmem + ks * 8 + (ks & 4) * 8, zd + ((ks * 2048u) >> 4), idesc, ks > 0 ? 1u : 0u);
  }
}

// S += (w y)^T z: both MN-major.
__device__ __forceinline__ void issue_wyz(uint32_t m_tmem, uint32_t hi_base, uint32_t lo_base, uint32_t z_base, int steps) {
  constexpr uint32_t idesc = idesc_bf16_f32(128, 128, true, true);
  const uint64_t hd = sdesc_sw128(hi_base, HALF_TILE, 1024), ld = sdesc_sw128(lo_base, HALF_TILE, 1024),
                 zd = sdesc_sw128(z_base, HALF_TILE, 1024);
#pragma unroll
  for (int ks = 0; ks < 8; ++ks) {
    if (ks >= steps) break;
    const uint32_t off = (ks * 2048u) >> 4;
    mma_bf16_ss(m_tmem, hd + off, zd + off, idesc, 1u);
    mma_bf16_ss(m_tmem, ld + off, zd + off, idesc, 1u);
  }
}

template <bool kLocal>
__device__ void output_issuer(const LinParams& p, uint8_t* sm, Aux& x, uint32_t tmem) {
  uint32_t g = 0;
  const uint32_t xbs[2] = {smem_u32(sm + X_AT), smem_u32(sm + X1_AT)}, yb = smem_u32(sm + Y_AT), zb = smem_u32(sm + Z_AT), sb = smem_u32(sm + S_AT);
  Items<kLocal> items(p);
  for (Item it; items.next(p, it, false);) {
    for (int c = 0; c < it.chunks; ++c, ++g) {
      const uint32_t ph = g & 1u;
      const uint32_t xb = g & 1u ? xbs[1] : xbs[0];
      if (!warp_wait(&x.y_full, ph, x, p) || !warp_wait(&x.x_full[g & 1u], (g >> 1) & 1u, x, p)) return;
      // (A's place is free: O2 of the chunk before has ended)
      if (g > 0 && !warp_wait(&x.o_full, ph ^ 1u, x, p)) return;
      tc_fence_after();
      if (elect_one()) {
        issue_qk_ss(tmem + TM_A, xb, yb);
        mma_commit(&x.a_full);
        mma_commit(&x.y_empty);
      }
      __syncwarp();
      // (behind the state's products, which the next chunk's image waits for)
      if (!warp_wait(&x.m_begun, ph, x, p) || !warp_wait(&x.s_full, ph, x, p) || !warp_wait(&x.o_empty, ph ^ 1u, x, p)) return;
      tc_fence_after();
      if (elect_one()) {
        issue_xs(tmem + TM_O1, xb, sb);
        mma_commit(&x.s_empty);
      }
      __syncwarp();
      // (of a part of a chunk, z's rows behind it are zeros: w y was there before the state's products began.
      // No wait for it here, only sometimes: a waiter has to see every phase.)
      if (!warp_wait(&x.z_full, ph, x, p) || !warp_wait(&x.p_full, ph, x, p)) return;
      tc_fence_after();
      if (elect_one()) {
        issue_az(tmem + TM_O2, tmem + TM_A, zb, (it.rows(c) + 15) >> 4);
        mma_commit(&x.o_full);
        mma_commit(&x.z_empty);
      }
      __syncwarp();
    }
  }
}

// w y's parts have one place, or without outputs two by turns (x's tile and the image are
// not needed there); each place's barriers have a phase a turn.
template <bool kOutputs>
__device__ __forceinline__ uint32_t place(uint32_t g) {
  return kOutputs ? 0u : g & 1u;
}
template <bool kOutputs>
__device__ __forceinline__ uint32_t turn(uint32_t g) {
  return (kOutputs ? g : g >> 1) & 1u;
}

template <bool kOutputs, bool kLocal>
__device__ void state_issuer(const LinParams& p, uint8_t* sm, Aux& x, uint32_t tmem) {
  uint32_t g = 0;
  const uint32_t zb = smem_u32(sm + Z_AT);
  Items<kLocal> items(p);
  for (Item it; items.next(p, it, false);) {
    for (int c = 0; c < it.chunks; ++c, ++g) {
      const uint32_t ph = g & 1u;
      const uint32_t wb = place<kOutputs>(g);
      if (!warp_wait(&x.z_full, ph, x, p) || !warp_wait(&x.w_full[wb], turn<kOutputs>(g), x, p) || !warp_wait(&x.s_full, ph, x, p)) return;
      tc_fence_after();
      if (elect_one()) {
        issue_wyz(tmem + TM_S, smem_u32(sm + (wb ? X_AT : HI_AT)), smem_u32(sm + (wb ? S_AT : LO_AT)), zb, (it.rows(c) + 15) >> 4);
        mma_commit(&x.m_full);
        mma_commit(&x.w_empty[wb]);
        mma_commit(&x.z_empty);
      }
      warp_arrive(&x.m_begun);
    }
  }
}

__device__ __forceinline__ float decay_power(float log2_decay, int n) {
  return n == 0 ? 1.f : exp2f(static_cast<float>(n) * log2_decay);
}

// ---------------------------------------------------------------- A's decays
// Loops stay loops: code in straight lines is fetched at about 12 cycles an
// instruction (64 columns unrolled took 6200 cycles a chunk).
template <bool kLocal>
__device__ void decay_warps(const LinParams& p, Aux& x, uint32_t tmem) {
  const int tid = static_cast<int>(threadIdx.x) - 32 * DECAY_WARP0;
  const int warp = static_cast<int>(threadIdx.x >> 5), lane = static_cast<int>(lane_id());
  const int quarter = warp & 3, half = (warp - DECAY_WARP0) >> 2, i_row = quarter * 32 + lane;
  const uint32_t At = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + TM_A + half * 64;
  uint32_t g = 0, meet = 0;
  Items<kLocal> items(p);
  for (Item it; items.next(p, it, false);) {
    if (it.chunks == 0) continue;
    const float log2_decay = log2f(__ldcg(p.decay + it.h));
    if (!group_sync(&x.group[0], meet, x, p)) return;
    if (tid < LT_CHUNK) x.power[tid] = decay_power(log2_decay, tid) * p.scale;
    if (tid < 16) reinterpret_cast<float*>(x.near)[tid] = decay_power(log2_decay, it.reverse ? tid : 15 - tid);
    if (!group_sync(&x.group[0], meet, x, p)) return;
    for (int c = 0; c < it.chunks; ++c, ++g) {
      const int rows = it.rows(c);
      if (!warp_wait(&x.a_full, g & 1u, x, p)) return;
      tc_fence_after();
      // columns 64 half .. of row i_row, sixteen at a time, to where they came from
#pragma unroll 1
      for (int b = 0; b < 4; ++b) {
        uint32_t a[16];
        tmem_ld16(At + 16 * b, a);
        const int j0 = 64 * half + 16 * b;
        const int gap = it.reverse ? j0 - i_row : i_row - (j0 + 15);  // to the block's nearest column
        uint32_t pk[8] = {};
        if (__all_sync(0xffffffffu, gap >= 0) && (!it.reverse || j0 + 16 <= rows)) {  // every row reaches all columns
          const float w = x.power[gap];
          tmem_ld16_wait(a);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float4 n = x.near[k];
            float c0, c1, c2, c3;
            mul2(c0, c1, __uint_as_float(a[4 * k]), __uint_as_float(a[4 * k + 1]), n.x, n.y);
            mul2(c2, c3, __uint_as_float(a[4 * k + 2]), __uint_as_float(a[4 * k + 3]), n.z, n.w);
            mul2(c0, c1, c0, c1, w, w);
            mul2(c2, c3, c2, c3, w, w);
            pk[2 * k] = pack_bf16x2(c0, c1);
            pk[2 * k + 1] = pack_bf16x2(c2, c3);
          }
        } else {
          tmem_ld16_wait(a);
          if (__any_sync(0xffffffffu, gap >= -15)) {
            // row by column; columns from `rows` on are another user's, or none's
            const int most = it.reverse ? rows - 1 - i_row : LT_CHUNK;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              const int e = it.reverse ? j0 + 2 * k - i_row : i_row - j0 - 2 * k, d = it.reverse ? e + 1 : e - 1;
              const float w0 = e >= 0 && e <= most ? __uint_as_float(a[2 * k]) * x.power[max(e, 0)] : 0.f;
              const float w1 = d >= 0 && d <= most ? __uint_as_float(a[2 * k + 1]) * x.power[max(d, 0)] : 0.f;
              pk[k] = pack_bf16x2(w0, w1);
            }
          }
        }
        tmem_st8(At + 8 * b, pk);
      }
      tmem_st_wait();
      tc_fence_before();
      warp_arrive(&x.p_full);
    }
  }
}

// ----------------------------------------------------------------- outputs
// 8 columns of the lane's row from tensor memory.
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
      : "r"(taddr)
      : "memory");
}

// Outputs again, in plain arithmetic, where one is infinite or NaN whose part from the state is not: an infinity or NaN in
// z reaches rows of its chunk that do not read it, as 0 times infinity.  8 columns of the lane's row i of a chunk
// (`row0` its first row, `rows` of them) at a time, from the inputs; o1 is x S of them, `to` the row's place.
// (Behind that chunk the state has it, so that of a column one chunk is slow: 0.7 ms, 6 where all columns are.
// Looking for it in all chunks takes 1 to 1.5% of a call: 15 histories 51.6 -> 52.0 us, their gradient 73.2 -> 74.4.)
__device__ __forceinline__ void plain_outputs(const LinParams& p, const LinJob& job, int64_t row0, int rows, int at, int i, int column, float log2_decay,
                                              float w1, uint32_t o1, uint8_t* to) {
  uint32_t a[8];
  tmem_ld8(o1, a);
  uint4* piece = reinterpret_cast<uint4*>(to + ((((column & 63) >> 3) ^ (i & 7)) << 4));
  const uint4 now = *piece;
  bool any = false;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const uint32_t w = k < 4 ? (k < 2 ? now.x : now.y) : (k < 6 ? now.z : now.w);
    any |= is_finite(__uint_as_float(a[k])) && (not_finite(w) & (k & 1 ? 0x80000000u : 0x8000u));
  }
  if (!__any_sync(0xffffffffu, any && i < rows)) return;
  float acc[8] = {};
#pragma unroll 1
  for (int j = 0; j < rows; ++j) {
    const int gap = job.reverse ? j - i : i - j;
    if (gap < 0 || i >= rows) continue;
    const uint16_t *x = job.x + (row0 + i) * job.xs + at, *y = job.y + (row0 + j) * job.ys + at;
    float w = 0.f;
#pragma unroll 1
    for (int e = 0; e < LIN_D; e += 2) {
      const uint32_t f = *reinterpret_cast<const uint32_t*>(x + e), g = *reinterpret_cast<const uint32_t*>(y + e);
      w = fmaf(bf16_lo(f), bf16_lo(g), fmaf(bf16_hi(f), bf16_hi(g), w));
    }
    w = bf16_lo(pack_bf16x2(w * (decay_power(log2_decay, gap) * p.scale), 0.f));
    const uint16_t* z = job.z + (row0 + j) * job.zs + at + column;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t v = *reinterpret_cast<const uint32_t*>(z + 2 * k);
      acc[2 * k] = fmaf(w, bf16_lo(v), acc[2 * k]);
      acc[2 * k + 1] = fmaf(w, bf16_hi(v), acc[2 * k + 1]);
    }
  }
  __syncwarp();
  tmem_ld8(o1, a);
#pragma unroll
  for (int k = 0; k < 4; ++k)
    a[k] = pack_bf16x2(fmaf(__uint_as_float(a[2 * k]), w1, acc[2 * k]), fmaf(__uint_as_float(a[2 * k + 1]), w1, acc[2 * k + 1]));
  *piece = make_uint4(a[0], a[1], a[2], a[3]);
}

template <bool kLocal>
__device__ void output_warps(const LinParams& p, uint8_t* sm, Aux& x, uint32_t tmem) {
  const int warp = static_cast<int>(threadIdx.x >> 5), lane = static_cast<int>(lane_id());
  const int quarter = warp & 3, half = (warp - OUT_WARP0) >> 2, i_row = quarter * 32 + lane;
  const uint32_t lane_base = static_cast<uint32_t>(quarter * 32) << 16;
  const uint32_t O1 = tmem + lane_base + TM_O1 + half * 64, O2 = tmem + lane_base + TM_O2 + half * 64;
  uint32_t g = 0;
  Items<kLocal> items(p);
  for (Item it; items.next(p, it, false);) {
    const LinJob& job = p.job[it.job];
    const float log2_decay = log2f(__ldcg(p.decay + it.h));
    for (int c = 0; c < it.chunks; ++c, ++g) {
      const int rows = it.rows(c);
      const float w1 = decay_power(log2_decay, max(it.reverse ? rows - i_row - (c == 0 ? it.early : 0) : i_row + 1, 0)) * job.read;
      const bool stores = quarter * 32 < rows && job.out;
      uint8_t* stage = sm + (g & 1u ? X1_AT : X_AT) + (warp - OUT_WARP0) * OUT_BYTES;  // x's place: its products have ended
      if (!warp_wait(&x.o_full, g & 1u, x, p)) return;
      tc_fence_after();
      float odd0 = 0.f, odd1 = 0.f;  // NaN where an output is infinite or NaN
#pragma unroll 1
      for (int b = 0; b < 4 && stores; ++b) {
        uint32_t a[16], o[16], out[8];
        tmem_ld16(O1 + 16 * b, a);
        tmem_ld16(O2 + 16 * b, o);
        tmem_ld16_wait(a);
        tmem_ld16_wait(o);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          float u, v;
          fma2v(u, v, __uint_as_float(a[2 * j]), __uint_as_float(a[2 * j + 1]), w1, __uint_as_float(o[2 * j]), __uint_as_float(o[2 * j + 1]));
          out[j] = pack_bf16x2(u, v);
          fma2v(odd0, odd1, u, v, 0.f, odd0, odd1);
        }
#pragma unroll
        for (int q = 0; q < 2; ++q)
          *reinterpret_cast<uint4*>(stage + lane * 128 + (((2 * b + q) ^ (lane & 7)) << 4)) =
              make_uint4(out[4 * q], out[4 * q + 1], out[4 * q + 2], out[4 * q + 3]);
      }
      if (__builtin_expect(__any_sync(0xffffffffu, stores && i_row < rows && !(odd0 + odd1 == 0.f)), 0)) {
#pragma unroll 1
        for (int b = 0; b < 8; ++b)
          plain_outputs(p, job, it.first(c), rows, it.h * LIN_D, i_row, half * 64 + 8 * b, log2_decay, w1, O1 + 8 * b, stage + lane * 128);
      }
      tc_fence_before();
      warp_arrive(&x.o_empty);
      // through shared memory, so that a store fills whole lines: stores of a sector in each of 32 lines took the
      // unit that shared memory goes through for 57 cycles each
      if (stores) {
        uint16_t* dst = job.out + static_cast<int64_t>(it.first(c) + quarter * 32) * job.os + it.h * LIN_D + half * 64 + 8 * (lane & 7);
#pragma unroll 4
        for (int q = 0; q < 8; ++q) {
          const int r = 4 * q + (lane >> 3);
          const uint4 v = *reinterpret_cast<const uint4*>(stage + r * 128 + (((lane & 7) ^ (r & 7)) << 4));
          if (quarter * 32 + r < rows) *reinterpret_cast<uint4*>(dst + r * job.os) = v;
        }
        __syncwarp();
        fence_proxy_async_smem();  // (before x's next tile)
      }
      warp_arrive(&x.x_empty[g & 1u]);
    }
  }
}

// ------------------------------------------------------------------- state
template <bool kOutputs, bool kLocal>
__device__ void state_warps(const LinParams& p, uint8_t* sm, Aux& x, uint32_t tmem) {
  const int warp = static_cast<int>(threadIdx.x >> 5), lane = static_cast<int>(lane_id());
  const int quarter = warp & 3, half = (warp - STATE_WARP0) >> 2, e_row = quarter * 32 + lane;  // a row of the state, 64 half .. of its columns
  const uint32_t St = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + TM_S + half * 64;
  // the warp's rows of the image; without outputs a place of its own
  uint8_t* stage = sm + (kOutputs ? S_AT + half * HALF_TILE + quarter * 32 * 128 : X1_AT + (warp - STATE_WARP0) * OUT_BYTES);
  uint8_t* image = stage + lane * 128;
  uint32_t g = 0;
  Items<kLocal> items(p);
  for (Item it; items.next(p, it, threadIdx.x == 32 * STATE_WARP0);) {
    const LinJob& job = p.job[it.job];
    const float log2_decay = log2f(__ldcg(p.decay + it.h));
    const int64_t state = (static_cast<int64_t>(it.u) * p.H + it.h) * LIN_STATE;
    const int64_t ws = ((static_cast<int64_t>(it.job) * p.n_users + it.u) * p.H + it.h) * p.segs;
    bool turned;
    const float* from = state_from<kLocal>(p, it, turned);
    float* to = kLocal ? p.ws + (ws + it.seg) * LIN_STATE : (it.seg + 1 == it.segs && job.s_out ? job.s_out + state : nullptr);
    const float up = !kLocal && it.reverse && !it.whole_user_empty ? decay_power(log2_decay, 1) : 1.f;
    // The start to tensor memory.  Rows of a state are 512 bytes apart, a lane's place is a row: eight lanes load a row's
    // 128 bytes, by way of the warp's place in the image (a load of 16 bytes of each of 32 rows took 18000 cycles in all).
    if (kOutputs && !warp_wait(&x.s_empty, (g & 1u) ^ 1u, x, p)) return;
    const int sub = lane >> 3, piece = lane & 7;
#pragma unroll 1
    for (int b = 0; b < 2; ++b) {
      uint32_t v[32];
      if (from && !turned) {
        float4 f[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) f[q] = __ldcg(reinterpret_cast<const float4*>(from + (quarter * 32 + 4 * q + sub) * LIN_D + 64 * half + 32 * b) + piece);
#pragma unroll
        for (int q = 0; q < 8; ++q) *reinterpret_cast<float4*>(stage + (4 * q + sub) * 128 + ((piece ^ ((4 * q + sub) & 7)) << 4)) = f[q];
        __syncwarp();
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float4 r = *reinterpret_cast<const float4*>(stage + lane * 128 + ((k ^ (lane & 7)) << 4));
          v[4 * k] = __float_as_uint(r.x);
          v[4 * k + 1] = __float_as_uint(r.y);
          v[4 * k + 2] = __float_as_uint(r.z);
          v[4 * k + 3] = __float_as_uint(r.w);
        }
        __syncwarp();
      } else {
#pragma unroll
        for (int k = 0; k < 32; ++k) v[k] = __float_as_uint(from ? __ldcg(from + (64 * half + 32 * b + k) * LIN_D + e_row) : 0.f);
      }
      tmem_st32(St + 32 * b, v);
    }
    tmem_st_wait();
    // chunk by chunk: the image of the state before it, and the decay over it; then
    // the products add the chunk.  One turn more gives the end away.  (Without outputs
    // all decays reach to the end: the start's at once, a chunk's with w y.)
    for (int c = 0; c <= it.chunks; ++c) {
      const bool last = c == it.chunks;
      if (c > 0 && !warp_wait(&x.m_full, (g - 1) & 1u, x, p)) return;
      if (last && !to) break;
      if (kOutputs && !warp_wait(&x.s_empty, (g & 1u) ^ 1u, x, p)) return;
      tc_fence_after();
      if (!kOutputs && c > 0 && !last) {
        warp_arrive(&x.s_full);
        ++g;
        continue;
      }
      const float down = last ? up : decay_power(log2_decay, (kOutputs ? it.rows(c) : it.n) - (c == 0 ? it.early : 0));
#pragma unroll 1
      for (int b = 0; b < 2; ++b) {
        uint32_t v[32];
        tmem_ld32(St + 32 * b, v);
        tmem_ld_wait(v);
        if (kOutputs && !last) {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            uint32_t w[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) w[q] = pack_bf16x2(__uint_as_float(v[8 * k + 2 * q]), __uint_as_float(v[8 * k + 2 * q + 1]));
            *reinterpret_cast<uint4*>(image + (((4 * b + k) ^ (e_row & 7)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          float f0, f1;
          mul2(f0, f1, __uint_as_float(v[2 * k]), __uint_as_float(v[2 * k + 1]), down, down);
          v[2 * k] = __float_as_uint(f0);
          v[2 * k + 1] = __float_as_uint(f1);
        }
        if (!last) {
          tmem_st32(St + 32 * b, v);
          continue;
        }
#pragma unroll
        for (int k = 0; k < 8; ++k)
          *reinterpret_cast<uint4*>(stage + lane * 128 + ((k ^ (lane & 7)) << 4)) = make_uint4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
        __syncwarp();
#pragma unroll
        for (int q = 0; q < 8; ++q)
          reinterpret_cast<uint4*>(to + (quarter * 32 + 4 * q + sub) * LIN_D + 64 * half + 32 * b)[piece] =
              *reinterpret_cast<const uint4*>(stage + (4 * q + sub) * 128 + ((piece ^ ((4 * q + sub) & 7)) << 4));
        __syncwarp();
      }
      if (last) break;
      tmem_st_wait();
      tc_fence_before();
      fence_proxy_async_smem();
      warp_arrive(&x.s_full);
      ++g;
    }
  }
}

// -------------------------------------------------------------- w y's parts
template <bool kOutputs, bool kLocal>
__device__ void parts_warps(const LinParams& p, uint8_t* sm, Aux& x) {
  constexpr int kThreads = 32 * PARTS_WARPS;
  const int tid = static_cast<int>(threadIdx.x) - 32 * PARTS_WARP0;
  uint32_t g = 0, meet = 0;
  Items<kLocal> items(p);
  for (Item it; items.next(p, it, false);) {
    if (it.chunks == 0) continue;
    static_assert(kThreads == LT_CHUNK, "a decay a thread");
    const float log2_decay = log2f(__ldcg(p.decay + it.h));
    for (int c = 0; c < it.chunks; ++c, ++g) {
      const uint32_t ph = g & 1u;
      const int rows = it.rows(c);
      if (c == 0 || !kOutputs) {  // the decays: to the chunk's end, or to the scan's
        if (!group_sync(&x.group[1], meet, x, p)) return;
        const float w = decay_power(log2_decay, tid + (kOutputs ? 0 : it.n - c * LT_CHUNK - rows)) * p.job[it.job].add;
        const uint32_t hi = pack_bf16x2(w, w);
        const float rest = w - bf16_lo(hi);
        x.parts[tid] = make_uint2(hi, pack_bf16x2(rest, rest));
        if (!group_sync(&x.group[1], meet, x, p)) return;
      }
      // (element-wise: any order of the tile's 16-byte pieces)
      const uint32_t wb = place<kOutputs>(g);
      if (!warp_wait(&x.y_full, ph, x, p) || !warp_wait(&x.w_empty[wb], turn<kOutputs>(g) ^ 1u, x, p)) return;
      uint8_t *hi_to = sm + (wb ? X_AT : HI_AT), *lo_to = sm + (wb ? S_AT : LO_AT);
#pragma unroll 1
      for (int k0 = 0; k0 < 16; k0 += 4) {
        uint4 v[4];
        uint2 w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int e = (k0 + k) * kThreads + tid, j = (e >> 3) & (LT_CHUNK - 1);
          v[k] = *reinterpret_cast<const uint4*>(sm + Y_AT + e * 16);
          w[k] = x.parts[it.reverse ? j : max(rows - 1 - j, 0)];
          if (j >= rows) v[k] = uint4{};
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int e = (k0 + k) * kThreads + tid;
          uint4 hi, lo;
          decayed(v[k].x, w[k], hi.x, lo.x);
          decayed(v[k].y, w[k], hi.y, lo.y);
          decayed(v[k].z, w[k], hi.z, lo.z);
          decayed(v[k].w, w[k], hi.w, lo.w);
          *reinterpret_cast<uint4*>(hi_to + e * 16) = hi;
          *reinterpret_cast<uint4*>(lo_to + e * 16) = lo;
        }
      }
      if (rows < LT_CHUNK) {  // rows that are another user's, or none's: no value, whatever they hold
        // (after the products of the chunk before, so that z_full is not a phase behind)
        if (!kOutputs && g > 0 && !warp_wait(&x.w_empty[place<kOutputs>(g - 1)], turn<kOutputs>(g - 1), x, p)) return;
        if (!warp_wait(&x.z_full, ph, x, p)) return;
#pragma unroll 1
        for (int k = 0; k < 16; ++k) {
          const int e = k * kThreads + tid, j = (e >> 3) & (LT_CHUNK - 1);
          if (j >= rows) *reinterpret_cast<uint4*>(sm + Z_AT + e * 16) = uint4{};
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane_id() == 0) {
        mbar_arrive(&x.w_full[wb]);
        mbar_arrive(&x.y_empty);
      }
    }
  }
}

template <bool kOutputs, bool kLocal>
__global__ void __launch_bounds__(LT_THREADS, 1) lin_tile_kernel(const __grid_constant__ LinParams p, const __grid_constant__ LtMaps maps) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  uint8_t* sm = smem_raw + (((raw + 1023u) & ~1023u) - raw);
  Aux& x = *reinterpret_cast<Aux*>(sm + AUX_AT);
  const int warp = static_cast<int>(threadIdx.x >> 5);
  if (threadIdx.x == 0) {
    uint64_t* once[] = {&x.x_full[0], &x.x_full[1], &x.y_full, &x.z_full, &x.a_full, &x.o_full, &x.s_empty, &x.m_full, &x.m_begun, &x.w_empty[0], &x.w_empty[1], &x.drain[0], &x.drain[1]};
    for (uint64_t* b : once) mbar_init(b, 1);
    mbar_init(&x.y_empty, PARTS_WARPS + (kOutputs ? 1 : 0));
    mbar_init(&x.z_empty, kOutputs ? 2 : 1);
    uint64_t* warps[] = {&x.p_full, &x.o_empty, &x.s_full, &x.x_empty[0], &x.x_empty[1], &x.group[0]};
    for (uint64_t* b : warps) mbar_init(b, GROUP_WARPS);
    const int withheld = (p.debug & DEBUG_WITHHOLD_STATES) && (blockIdx.x & 3u) == 1u ? 1 : 0;
    mbar_init(&x.w_full[0], PARTS_WARPS + withheld);
    mbar_init(&x.w_full[1], PARTS_WARPS + withheld);
    mbar_init(&x.group[1], PARTS_WARPS);
    x.abort = 0;
    fence_barrier_init();
    fence_proxy_async_smem();
  }
  wait_for_launch_before();
  if (warp == 3) {
    tmem_alloc(&x.tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = x.tmem_slot;

  if (warp < DECAY_WARP0) {
    if (warp == 0) loader<kOutputs, kLocal>(p, maps, sm, x);
    if (warp == 1 && kOutputs) output_issuer<kLocal>(p, sm, x, tmem);
    if (warp == 2) state_issuer<kOutputs, kLocal>(p, sm, x, tmem);
    if (warp == 1 || warp == 2) drain(&x.drain[warp - 1]);
  } else if (warp < OUT_WARP0) {
    if (kOutputs) decay_warps<kLocal>(p, x, tmem);
  } else if (warp < STATE_WARP0) {
    if (kOutputs) output_warps<kLocal>(p, sm, x, tmem);
  } else if (warp < PARTS_WARP0) {
    state_warps<kOutputs, kLocal>(p, sm, x, tmem);
  } else {
    parts_warps<kOutputs, kLocal>(p, sm, x);
  }
  tc_fence_before();
  __syncthreads();
  if (x.abort && threadIdx.x == 0) atomicOr(p.status, DEV_ERR_PIPE_TIMEOUT);
  if (warp == 3) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <bool kOutputs, bool kLocal>
cudaError_t launch(const LinParams& p, const LtMaps& maps, int num_sms, cudaStream_t s) {
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = allow_smem(lin_tile_kernel<kOutputs, kLocal>, LT_SMEM, done);
  if (e != cudaSuccess) return e;
  // (segments of all users: no more than their rows hold, and one each)
  const int64_t segs = p.segs > 1 ? p.n_rows / p.seg_len + static_cast<int64_t>(p.n_users) : p.n_users;
  const int64_t items = segs * p.H * p.n_jobs;
  const unsigned grid = static_cast<unsigned>(items < num_sms ? items : num_sms);
  return launch_behind(lin_tile_kernel<kOutputs, kLocal>, dim3(grid), LT_THREADS, LT_SMEM, s, p, maps);
}

}  // namespace

bool encode_bf16(CUtensorMap* m, const void* base, int rank, const uint64_t* dims, const uint64_t* strides_bytes, const uint32_t* box);

size_t lin_tile_smem() { return LT_SMEM; }

// The scans, or (local) the segments' own parts.
cudaError_t launch_lin_tiles(const LinParams& p, bool local, int num_sms, cudaStream_t s) {
  LtMaps maps;
  const auto encode = [&](CUtensorMap* m, const uint16_t* t, int64_t stride) {
    const uint64_t dims[3] = {LIN_D, static_cast<uint64_t>(p.H), static_cast<uint64_t>(p.n_rows)};
    const uint64_t strides[2] = {LIN_D * 2, static_cast<uint64_t>(stride) * 2};
    const uint32_t box[3] = {64, 1, LT_CHUNK};
    return encode_bf16(m, t, 3, dims, strides, box);
  };
  const bool outputs = p.job[0].x != nullptr && !local;
  for (int k = 0; k < p.n_jobs; ++k) {
    const LinJob& j = p.job[k];
    if (!encode(&maps.y[k], j.y, j.ys) || !encode(&maps.z[k], j.z, j.zs) || (outputs && !encode(&maps.x[k], j.x, j.xs)))
      return cudaErrorInvalidValue;
  }
  for (int k = p.n_jobs; k < LIN_MAX_JOBS; ++k) maps.y[k] = maps.z[k] = maps.y[0];
  for (int k = outputs ? p.n_jobs : 0; k < LIN_MAX_JOBS; ++k) maps.x[k] = maps.y[0];
  if (local) return launch<false, true>(p, maps, num_sms, s);
  return outputs ? launch<true, false>(p, maps, num_sms, s) : launch<false, false>(p, maps, num_sms, s);
}

}  // namespace ikbo
