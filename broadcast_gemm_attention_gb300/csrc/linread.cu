// linread.cu -- candidates' queries of their users' states of linear attention,
// read through the map, and the gradient.
//
//   O[i,h] = scale Q[i,h] S[map[i],h]
//   dQ[i,h] = scale dO[i,h] S[map[i],h]^T,   dS[u,h] = scale sum_{map[i]=u} Q[i,h]^T dO[i,h]
//
// The broadcast's linear form: a user's 64 KB state serves all of its
// candidates, and the gradient of the state is the sum over them.
//
// A unit of the plan's work list is up to 128 rows (the queries of a few candidates)
// of one user and head.  Its tile is gathered by TMA, a box for each candidate, and
//   O = x S       with S's bf16 image as B (MN-major),
//   dQ = dO S^T   with the same image as a K-major B,
//   dS += Q^T dO  (backward) into tensor memory over all of a run of units of one
//                 (user, head), both operands MN-major: rows are the inner dimension.
// One pass over the rows serves both gradients.  Bound: memory, and each CTA's start.
// 1024 candidates of 15 users, 8 heads x 32 rows: 29.4 us among other calls, 4.8 TB/s
// (16x8x16 products in registers: 107); the gradient of 1024 candidates of 64 users
// unevenly, 8 heads x 16 rows: 45.8 us, 3.7 TB/s (138), 6 of it the parts' adding.
//
// Per CTA (persistent, one per SM, a share of the list, 20 warps):
//   warp 0       loads; warp 1 issues
//   warps 4-11   outputs, and at a run's end the state's gradient
//   warps 12-19  images of the states, one run ahead; zeros for users without candidates
// A run costs about as many bytes as a unit (its state, and that one's gradient), so
// shares are equal in units and runs together (in units alone the gradient of 1024
// candidates of 64 users, unevenly, had 63 tiles' bytes in its largest share, of 41 on
// average; so 45).
// Runs cut by a CTA's share leave their gradients as parts, which the last CTA to end
// adds in order (so results repeat bit for bit).
#include <cuda.h>
#include <cuda_bf16.h>

#include "launch.cuh"
#include "linattn_internal.h"
#include "mma_common.cuh"
#include "tile_common.cuh"

namespace ikbo {
int lin_read_ctas(int num_sms);
namespace {

constexpr int RT_THREADS = 640;
constexpr int OUT_WARP0 = 4, IMAGE_WARP0 = 12, GROUP_WARPS = 8;
constexpr uint32_t TILE = 2 * HALF_TILE;  // 32 KB
constexpr int RING_TILES = 4;             // a stage is a tile (forward) or two
constexpr uint32_t IMAGE_AT = RING_TILES * TILE, OUT_AT = IMAGE_AT + 2 * TILE;
constexpr uint32_t OUT_BYTES = 32 * 128;  // of the outputs, per warp
constexpr uint32_t AUX_AT = OUT_AT + GROUP_WARPS * OUT_BYTES;
constexpr uint32_t TM_O = 0, TM_DS = 256;

struct Aux {
  uint64_t full[RING_TILES], empty[RING_TILES];
  uint64_t o_full[2], o_empty[2], image_full[2], image_empty[2], ds_full[2], ds_empty[2], drain;
  uint32_t tmem_slot, abort;
  int begin, end;               // the CTA's share of the list
  uint32_t total;               // of all units' and runs' costs; 0: shares are equal in units
  uint2 sums[RT_THREADS / 32];  // units and runs of a warp's users
  int4 shared[2];               // runs shared with other CTAs: its user and head, its first and last CTA (-1: none)
  uint32_t parts[2], last[2];   // how many CTAs that are, whether this was the last of them
};
constexpr uint32_t RT_SMEM = AUX_AT + sizeof(Aux) + 1024;
static_assert(RT_SMEM <= 227 * 1024, "tiles do not fit in shared memory");

// This CTA's units a .. b - 1, and a walk over them with the runs of one (user, head).
// The unit after the current one is at hand already.
struct Walk {
  int a, b;
  uint32_t runs;   // begun so far
  int u, h;        // of the run
  bool begins, ends;
  int4 w, next;
  __device__ __forceinline__ Walk(const LinReadParams& p, const Aux& x) : runs(0), u(-1), h(-1) {
    a = x.begin;
    b = x.end;
    next = a < b ? unit(p, a) : make_int4(-1, -1, 0, 0);
  }
  __device__ __forceinline__ static int4 unit(const LinReadParams& p, int i) { return fresh(reinterpret_cast<const int4*>(p.work) + i); }
  // To unit i; false (to every role alike) where the list is not sound, which ends the share.
  __device__ __forceinline__ bool at(const LinReadParams& p, int i) {
    w = next;
    if (w.x < 0 || w.x >= p.n_users || w.y < 0 || w.y >= p.H || w.z < 0 || w.w <= 0 || w.z + w.w > p.n_cand || w.w * p.Lq > 128) {
      if (threadIdx.x == 0) atomicOr(p.status, DEV_ERR_BAD_WORK);
      return false;
    }
    next = i + 1 < b ? unit(p, i + 1) : make_int4(-1, -1, 0, 0);
    begins = w.x != u || w.y != h;
    runs += begins;
    u = w.x;
    h = w.y;
    ends = next.x != u || next.y != h;
    return true;
  }
  // The candidate of place k of unit w (0 for none).
  __device__ __forceinline__ static int cand(const LinReadParams& p, const int4& w, int k) {
    return k < w.w && w.z >= 0 && w.z + k < p.n_cand ? fresh(p.perm + w.z + k) : 0;
  }
};

// ------------------------------------------------------------------ shares
// Where a share of the list begins.  A unit costs 1 and its run's beginning 1 more; counted
// along the list (P before a run, that run's units at P, P + 2, P + 3, ..), unit i at cost(i)
// is CTA cost(i) * CTAs / total's.  Units alone count (total: how many) where there are fewer
// runs than CTAs (15 users' 8 heads: 1.6 us without finding the shares), and where shares
// are not two wide at least, so that what lies between a run's first CTA and its last has
// units of it.
__device__ __forceinline__ uint32_t share_begin(uint32_t c, uint32_t total) {
  if (total <= 0xffffffffu / 1024) return (c * total + gridDim.x - 1) / gridDim.x;
  return static_cast<uint32_t>((static_cast<uint64_t>(c) * total + gridDim.x - 1) / gridDim.x);
}
__device__ __forceinline__ int share_of(uint32_t cost, uint32_t total) {
  return static_cast<int>(static_cast<uint64_t>(cost) * gridDim.x / total);
}

__device__ __forceinline__ uint32_t listed_units(const LinReadParams& p) {
  return static_cast<uint32_t>(max(0, min(fresh(p.n_units), static_cast<int>(p.max_units))));
}

// Units of user u for each head.
__device__ __forceinline__ uint32_t units_of(const LinReadParams& p, int u, uint32_t cands) {
  const int count = fresh(p.offsets + u + 1) - fresh(p.offsets + u);
  return count > 0 ? (static_cast<uint32_t>(count) + cands - 1) / cands : 0u;
}

// By the whole CTA, each thread some users.
__device__ __forceinline__ void find_share(const LinReadParams& p, Aux& x) {
  const int tid = static_cast<int>(threadIdx.x), lane = tid & 31, warp = tid >> 5;
  const uint32_t c = blockIdx.x, n = listed_units(p);
  uint32_t units = 0, runs = 0, before = 0, cost = 0, all = 0, total = 0;
  const bool weigh = static_cast<int64_t>(p.n_users) * p.H > gridDim.x;
  const int per = (p.n_users + RT_THREADS - 1) / RT_THREADS, u0 = min(tid * per, p.n_users), u1 = min(u0 + per, p.n_users);
  const uint32_t cands = 128u / p.Lq;
  if (weigh) {
#pragma unroll 4
    for (int u = u0; u < u1; ++u) {
      const uint32_t k = units_of(p, u, cands);
      units += k * p.H;
      runs += k > 0 ? p.H : 0;
    }
    before = units;
    cost = runs;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t a = __shfl_up_sync(0xffffffffu, before, o), b = __shfl_up_sync(0xffffffffu, cost, o);
      if (lane >= o) {
        before += a;
        cost += b;
      }
    }
    if (lane == 31) x.sums[warp] = make_uint2(before, cost);
    __syncthreads();
    before -= units;
    cost += before - runs;  // of the thread's first user
#pragma unroll 4
    for (int w = 0; w < RT_THREADS / 32; ++w) {
      const uint2 v = x.sums[w];
      all += v.x;
      total += v.x + v.y;
      if (w >= warp) continue;
      before += v.x;
      cost += v.x + v.y;
    }
  }
  if (!weigh || all != n || total < 2 * gridDim.x) {
    if (tid == 0) {
      x.begin = static_cast<int>(share_begin(c, n));
      x.end = static_cast<int>(share_begin(c + 1, n));
      x.total = 0;
    }
    return;
  }
  if (tid == 0) x.total = total;
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const uint32_t ask = share_begin(c + e, total);
    int* to = e == 0 ? &x.begin : &x.end;
    if (tid == 0 && ask == total) *to = static_cast<int>(n);
    if (ask < cost || ask - cost >= units + runs) continue;
    uint32_t t = ask - cost, at = before;
    for (int u = u0; u < u1; ++u) {
      const uint32_t k = units_of(p, u, cands);
      if (k == 0) continue;
      if (t >= (k + 1) * p.H) {
        t -= (k + 1) * p.H;
        at += k * p.H;
        continue;
      }
      const uint32_t run = t / (k + 1), in = t - run * (k + 1);
      *to = static_cast<int>(at + run * k + (in == 0 ? 0u : max(in - 1, 1u)));
      break;
    }
  }
}

// ------------------------------------------------------------------ loader
template <bool kBack>
__device__ void loader(const LinReadParams& p, const CUtensorMap* mx, const CUtensorMap* mq, uint8_t* sm, Aux& x) {
  constexpr int kStages = kBack ? RING_TILES / 2 : RING_TILES;
  constexpr uint32_t kStage = (kBack ? 2 : 1) * TILE;
  const int lane = static_cast<int>(lane_id());
  Walk k(p, x);
  uint32_t g = 0;
  bool ok = true;
  int cand_next = Walk::cand(p, k.next, lane);
  for (int i = k.a; i < k.b && ok && k.at(p, i); ++i, ++g) {
    const uint32_t st = g % kStages;
    const int cand = cand_next;
    cand_next = Walk::cand(p, k.next, lane);
    ok = warp_wait(&x.empty[st], ((g / kStages) & 1u) ^ 1u, x, p);
    if (!ok) break;
    uint8_t* at = sm + st * kStage;
    const int rows = k.w.w * p.Lq;
    if (kBack && (rows & 15)) {  // eight rows more are multiplied: zeros
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        uint4* z = reinterpret_cast<uint4*>(at + q * HALF_TILE + rows * 128);
        z[lane] = uint4{};
        z[lane + 32] = uint4{};
      }
      fence_proxy_async_smem();
    }
    __syncwarp();
    if (lane == 0) mbar_arrive_expect_tx(&x.full[st], static_cast<uint32_t>(rows) * 256u * (kBack ? 2 : 1));
    __syncwarp();
    if (lane < k.w.w) {
      uint8_t* to = at + lane * p.Lq * 128;
      tma_load_4d(to, mx, &x.full[st], 0, 0, k.h, cand);
      tma_load_4d(to + HALF_TILE, mx, &x.full[st], 64, 0, k.h, cand);
      if (kBack) {
        tma_load_4d(to + TILE, mq, &x.full[st], 0, 0, k.h, cand);
        tma_load_4d(to + TILE + HALF_TILE, mq, &x.full[st], 64, 0, k.h, cand);
      }
    }
    __syncwarp();
  }
  // the copies in flight end before the CTA does, whichever warp's wait ran out
  for (uint32_t s = g > static_cast<uint32_t>(kStages) ? g - kStages : 0; s < g; ++s) wait_a_second(&x.full[s % kStages], (s / kStages) & 1u);
  __syncwarp();
}

// ------------------------------------------------------------------ issuer
// x S: A K-major, B the image, its rows the inner dimension; x S^T: its rows the columns.
__device__ __forceinline__ void issue_read(uint32_t o_tmem, uint32_t x_base, uint32_t image, bool turned) {
  const uint32_t idesc = turned ? idesc_bf16_f32(128, 128, false, false) : idesc_bf16_f32(128, 128, false, true);
  const uint64_t xd = sdesc_sw128(x_base, 16, 1024), sd = turned ? sdesc_sw128(image, 16, 1024) : sdesc_sw128(image, HALF_TILE, 1024);
#pragma unroll
  for (int ks = 0; ks < 8; ++ks) {
    const uint32_t a = ((ks >> 2) * HALF_TILE + (ks & 3) * 32) >> 4;
    mma_bf16_ss(o_tmem, xd + a, sd + (turned ? a : (ks * 2048u) >> 4), idesc, ks > 0 ? 1u : 0u);
  }
}

// Q^T dO: both MN-major.
__device__ __forceinline__ void issue_state(uint32_t s_tmem, uint32_t q_base, uint32_t o_base, int steps, bool more) {
  constexpr uint32_t idesc = idesc_bf16_f32(128, 128, true, true);
  const uint64_t qd = sdesc_sw128(q_base, HALF_TILE, 1024), od = sdesc_sw128(o_base, HALF_TILE, 1024);
#pragma unroll
  for (int ks = 0; ks < 8; ++ks) {
    if (ks >= steps) break;
    mma_bf16_ss(s_tmem, qd + ((ks * 2048u) >> 4), od + ((ks * 2048u) >> 4), idesc, more || ks > 0 ? 1u : 0u);
  }
}

template <bool kBack>
__device__ void issuer(const LinReadParams& p, uint8_t* sm, Aux& x, uint32_t tmem) {
  constexpr int kStages = kBack ? RING_TILES / 2 : RING_TILES;
  constexpr uint32_t kStage = (kBack ? 2 : 1) * TILE;
  const uint32_t ring = smem_u32(sm), images = smem_u32(sm + IMAGE_AT);
  const bool out = p.out != nullptr;
  Walk k(p, x);
  uint32_t g = 0;
  for (int i = k.a; i < k.b && k.at(p, i); ++i, ++g) {
    const uint32_t st = g % kStages, r = k.runs - 1, rb = r & 1u, rp = (r >> 1) & 1u, ob = g & 1u;
    if (!warp_wait(&x.full[st], (g / kStages) & 1u, x, p)) return;
    if (out && k.begins && !warp_wait(&x.image_full[rb], rp, x, p)) return;
    if (out && !warp_wait(&x.o_empty[ob], ((g >> 1) & 1u) ^ 1u, x, p)) return;
    if (kBack && k.begins && !warp_wait(&x.ds_empty[rb], rp ^ 1u, x, p)) return;
    tc_fence_after();
    if (elect_one()) {
      const uint32_t at = ring + st * kStage;
      if (out) {
        issue_read(tmem + TM_O + 128 * ob, at, images + rb * TILE, p.turned != 0);
        mma_commit(&x.o_full[ob]);
        if (k.ends) mma_commit(&x.image_empty[rb]);
      }
      if (kBack) {
        issue_state(tmem + TM_DS + 128 * rb, at + TILE, at, (k.w.w * p.Lq + 15) >> 4, !k.begins);
        if (k.ends) mma_commit(&x.ds_full[rb]);
      }
      mma_commit(&x.empty[st]);
    }
    __syncwarp();
  }
}

// ------------------------------------------------------------------ images
template <bool kBack>
__device__ void image_warps(const LinReadParams& p, uint8_t* sm, Aux& x) {
  const int tid = static_cast<int>(threadIdx.x) - 32 * IMAGE_WARP0, warp = tid >> 5, lane = tid & 31;
  if (kBack) {  // users without candidates
    for (int64_t uh = blockIdx.x; uh < static_cast<int64_t>(p.n_users) * p.H; uh += gridDim.x) {
      const int u = static_cast<int>(uh / p.H);
      if (fresh(p.offsets + u + 1) > fresh(p.offsets + u)) continue;
#pragma unroll 4
      for (int e = tid; e < LIN_STATE / 4; e += 32 * GROUP_WARPS) reinterpret_cast<float4*>(p.d_state + uh * LIN_STATE)[e] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
  }
  if (!p.out) return;
  Walk k(p, x), ahead(p, x);
  int j = ahead.a;
  for (int i = k.a; i < k.b && k.at(p, i); ++i) {
    if (!k.begins) continue;
    const uint32_t r = k.runs - 1, rb = r & 1u;
    const float4* s = reinterpret_cast<const float4*>(p.state + (static_cast<int64_t>(k.u) * p.H + k.h) * LIN_STATE) + lane;
    // row by row: four elements a lane (all on their way before the place is free)
    uint8_t* to = sm + IMAGE_AT + rb * TILE + (lane >> 4) * HALF_TILE + (lane & 1) * 8;
    float4 v[16];
#pragma unroll
    for (int c = 0; c < 16; ++c) v[c] = fresh(s + (8 * c + warp) * 32);
    if (warp == 0) {  // the next run's state is on its way to L2 meanwhile (47.1 -> 45.8 us)
      while (j < ahead.b && ahead.runs <= k.runs && ahead.at(p, j)) ++j;
      if (ahead.runs > k.runs && elect_one())
        asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p.state + (static_cast<int64_t>(ahead.u) * p.H + ahead.h) * LIN_STATE), "n"(LIN_STATE * 4) : "memory");
      __syncwarp();
    }
    if (!warp_wait(&x.image_empty[rb], ((r >> 1) & 1u) ^ 1u, x, p)) return;
#pragma unroll
    for (int c = 0; c < 16; ++c) {
      const int row = 8 * c + warp;
      *reinterpret_cast<uint2*>(to + row * 128 + ((((lane & 15) >> 1) ^ (row & 7)) << 4)) = make_uint2(pack_bf16x2(v[c].x, v[c].y), pack_bf16x2(v[c].z, v[c].w));
    }
    fence_proxy_async_smem();
    warp_arrive(&x.image_full[rb]);
  }
}

// ------------------------------------------------------------ shared runs
// Which runs this CTA shares, by one warp: its first and its last unit's.
__device__ void find_shared(const LinReadParams& p, Aux& x) {
  const int n = static_cast<int>(listed_units(p)), a = x.begin, b = x.end, cands = 128 / p.Lq;
  int done = -1;
#pragma unroll 1
  for (int k = 0; k < 2; ++k) {
    int4 run = make_int4(-1, -1, -1, -1);
    uint32_t parts = 0;
    const int i = k == 0 ? a : b - 1;
    const int4 w = a < b ? Walk::unit(p, i) : make_int4(-1, -1, 0, 0);
    if (w.x >= 0 && w.x < p.n_users) {
      const int first = fresh(p.offsets + w.x);
      const int lo = i - (w.z - first) / cands, hi = lo + (fresh(p.offsets + w.x + 1) - first + cands - 1) / cands;  // its units
      if ((lo < a || hi > b) && lo != done && lo >= 0 && hi <= n) {
        done = lo;
        uint32_t cost = static_cast<uint32_t>(lo), total = static_cast<uint32_t>(n);
        if (x.total > 0) {
          int users = 0;  // with candidates, before the run's
#pragma unroll 4
          for (int v = 0; v < w.x; v += 32) {
            const int u = min(v + static_cast<int>(lane_id()), w.x);
            users += __popc(__ballot_sync(0xffffffffu, u < w.x && fresh(p.offsets + u + 1) > fresh(p.offsets + u)));
          }
          cost += static_cast<uint32_t>(users * p.H + w.y);
          total = x.total;
        }
        const int c0 = share_of(cost, total);
        const int c1 = share_of(cost + static_cast<uint32_t>(hi - lo - 1) + (x.total > 0 && hi - lo > 1 ? 1u : 0u), total);
        const bool gaps = x.total == 0 && n < static_cast<int>(gridDim.x);  // fewer units than CTAs: each has one at most
        if (c0 <= c1 && c1 < static_cast<int>(gridDim.x)) {  // (always, in a sound list)
          run = make_int4(w.x, w.y, c0, c1);
          parts = static_cast<uint32_t>(gaps ? hi - lo : c1 - c0 + 1);
        }
      }
    }
    if (lane_id() == 0) {
      x.shared[k] = run;
      x.parts[k] = parts;
    }
  }
  __syncwarp();
}

// ----------------------------------------------------------------- outputs
template <bool kBack>
__device__ void output_warps(const LinReadParams& p, uint8_t* sm, Aux& x, uint32_t tmem) {
  const int warp = static_cast<int>(threadIdx.x >> 5), lane = static_cast<int>(lane_id());
  const int quarter = warp & 3, half = (warp - OUT_WARP0) >> 2, row = quarter * 32 + lane;
  const uint32_t lane_base = static_cast<uint32_t>(quarter * 32) << 16;
  uint8_t* stage = sm + OUT_AT + (warp - OUT_WARP0) * OUT_BYTES;
  const int piece = lane & 7, slot = row / p.Lq;
  Walk k(p, x);
  uint32_t g = 0;
  int cand_next = Walk::cand(p, k.next, slot);
  for (int i = k.a; i < k.b && k.at(p, i); ++i, ++g) {
    const uint32_t r = k.runs - 1, rb = r & 1u, rp = (r >> 1) & 1u, ob = g & 1u;
    const int cand = cand_next;
    cand_next = Walk::cand(p, k.next, slot);
    if (p.out) {
      const int64_t mine = row < k.w.w * p.Lq ? ((static_cast<int64_t>(cand) * p.H + k.h) * p.Lq + (row - slot * p.Lq)) * LIN_D : -1;
      if (!warp_wait(&x.o_full[ob], (g >> 1) & 1u, x, p)) return;
      tc_fence_after();
      const uint32_t Ot = tmem + lane_base + TM_O + 128 * ob + 64 * half;
      const bool any = quarter * 32 < k.w.w * p.Lq;
#pragma unroll 1
      for (int b = 0; b < 2 && any; ++b) {
        uint32_t v[32];
        tmem_ld32(Ot + 32 * b, v);
        tmem_ld_wait(v);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t o[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float f0, f1;
            mul2(f0, f1, __uint_as_float(v[8 * c + 2 * e]), __uint_as_float(v[8 * c + 2 * e + 1]), p.scale, p.scale);
            o[e] = pack_bf16x2(f0, f1);
          }
          *reinterpret_cast<uint4*>(stage + lane * 128 + (((4 * b + c) ^ piece) << 4)) = make_uint4(o[0], o[1], o[2], o[3]);
        }
      }
      tc_fence_before();
      warp_arrive(&x.o_empty[ob]);
      // whole lines: eight lanes to a row's half
      if (any) {
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          const int rr = 4 * q + (lane >> 3);
          const int64_t at = __shfl_sync(0xffffffffu, mine, rr);
          const uint4 v = *reinterpret_cast<const uint4*>(stage + rr * 128 + ((piece ^ (rr & 7)) << 4));
          if (at >= 0) *reinterpret_cast<uint4*>(p.out + at + 64 * half + 8 * piece) = v;
        }
        __syncwarp();
      }
    }
    if (kBack && k.ends) {  // the run's gradient: whole, or a part
      const auto same = [&](int j) {
        const int4 n = Walk::unit(p, j);
        return n.x == k.u && n.y == k.h;
      };
      const int64_t n = min(static_cast<int64_t>(fresh(p.n_units)), p.max_units);
      const bool begun = r > 0 || k.a == 0 || !same(k.a - 1), whole = begun && (i + 1 < k.b || i + 1 >= n || !same(i + 1));
      float* to = whole ? p.d_state + (static_cast<int64_t>(k.u) * p.H + k.h) * LIN_STATE
                        : p.part + (2 * static_cast<int64_t>(blockIdx.x) + (begun ? 1 : 0)) * LIN_STATE;
      const float f = whole ? p.scale : 1.f;
      if (!warp_wait(&x.ds_full[rb], rp, x, p)) return;
      tc_fence_after();
#pragma unroll 1
      for (int b = 0; b < 2; ++b) {
        uint32_t v[32];
        tmem_ld32(tmem + lane_base + TM_DS + 128 * rb + 64 * half + 32 * b, v);
        tmem_ld_wait(v);
#pragma unroll
        for (int c = 0; c < 8; ++c)
          *reinterpret_cast<float4*>(stage + lane * 128 + ((c ^ piece) << 4)) =
              make_float4(__uint_as_float(v[4 * c]) * f, __uint_as_float(v[4 * c + 1]) * f, __uint_as_float(v[4 * c + 2]) * f, __uint_as_float(v[4 * c + 3]) * f);
        __syncwarp();
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          const int rr = 4 * q + (lane >> 3);
          *reinterpret_cast<float4*>(to + (quarter * 32 + rr) * LIN_D + 64 * half + 32 * b + 4 * piece) =
              *reinterpret_cast<const float4*>(stage + rr * 128 + ((piece ^ (rr & 7)) << 4));
        }
        __syncwarp();
      }
      tc_fence_before();
      warp_arrive(&x.ds_empty[rb]);
    }
  }
}

// The parts of the runs that this CTA shares (its first and its last, at most), where it
// is the last of their CTAs.  Counted whatever happened before, so that counts are zero
// again for the next call.
__device__ void join_runs(const LinReadParams& p, Aux& x) {
  if (threadIdx.x == 0) {
    __threadfence();
    uint32_t had[2] = {};
#pragma unroll
    for (int k = 0; k < 2; ++k)
      if (x.parts[k]) had[k] = atomicAdd(p.tickets + x.shared[k].z, 1u);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      x.last[k] = x.parts[k] && had[k] + 1 == x.parts[k];
      if (x.last[k]) p.tickets[x.shared[k].z] = 0;
    }
  }
  __syncthreads();
#pragma unroll 1
  for (int k = 0; k < 2; ++k) {
    if (!x.last[k]) continue;
    __threadfence();
    const int4 run = x.shared[k];
    const uint32_t n = listed_units(p);
    const bool gaps = static_cast<int>(x.parts[k]) != run.w - run.z + 1;
    float4* to = reinterpret_cast<float4*>(p.d_state + (static_cast<int64_t>(run.x) * p.H + run.y) * LIN_STATE);
    constexpr int kMine = (LIN_STATE / 4 + RT_THREADS - 1) / RT_THREADS;
    float4 sum[kMine] = {};
#pragma unroll 2
    for (int c = run.z; c <= run.w; ++c) {
      if (gaps && share_begin(c, n) >= share_begin(c + 1, n)) continue;
      const float4* part = reinterpret_cast<const float4*>(p.part + (2 * static_cast<int64_t>(c) + (c == run.z ? 1 : 0)) * LIN_STATE);
#pragma unroll
      for (int q = 0; q < kMine; ++q) {
        const int e = q * RT_THREADS + static_cast<int>(threadIdx.x);
        const float4 v = e < LIN_STATE / 4 ? __ldcg(part + e) : make_float4(0.f, 0.f, 0.f, 0.f);
        sum[q].x += v.x;
        sum[q].y += v.y;
        sum[q].z += v.z;
        sum[q].w += v.w;
      }
    }
#pragma unroll
    for (int q = 0; q < kMine; ++q) {
      const int e = q * RT_THREADS + static_cast<int>(threadIdx.x);
      if (e < LIN_STATE / 4) to[e] = make_float4(sum[q].x * p.scale, sum[q].y * p.scale, sum[q].z * p.scale, sum[q].w * p.scale);
    }
  }
}

template <bool kBack>
__global__ void __launch_bounds__(RT_THREADS, 1)
    lin_read_kernel(const __grid_constant__ LinReadParams p, const __grid_constant__ CUtensorMap mx, const __grid_constant__ CUtensorMap mq) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  uint8_t* sm = smem_raw + (((raw + 1023u) & ~1023u) - raw);
  Aux& x = *reinterpret_cast<Aux*>(sm + AUX_AT);
  const int warp = static_cast<int>(threadIdx.x >> 5);
  if (threadIdx.x == 0) {
    for (int i = 0; i < RING_TILES; ++i) {
      mbar_init(&x.full[i], 1);
      mbar_init(&x.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&x.o_full[i], 1);
      mbar_init(&x.image_empty[i], 1);
      mbar_init(&x.ds_full[i], 1);
      mbar_init(&x.o_empty[i], GROUP_WARPS);
      mbar_init(&x.image_full[i], GROUP_WARPS + ((p.debug & DEBUG_WITHHOLD_STATES) && (blockIdx.x & 3u) == 1u ? 1 : 0));
      mbar_init(&x.ds_empty[i], GROUP_WARPS);
    }
    mbar_init(&x.drain, 1);
    x.abort = 0;
    fence_barrier_init();
    fence_proxy_async_smem();
  }
  wait_for_launch_before();
  if (warp == 3) {
    tmem_alloc(&x.tmem_slot, 512);
    tmem_relinquish();
  }
  find_share(p, x);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = x.tmem_slot;
  if (warp < OUT_WARP0) {
    if (warp == 0) loader<kBack>(p, &mx, &mq, sm, x);
    if (warp == 1) {
      issuer<kBack>(p, sm, x, tmem);
      drain(&x.drain);
    }
    if (warp == 2 && kBack) find_shared(p, x);
  } else if (warp < IMAGE_WARP0) {
    output_warps<kBack>(p, sm, x, tmem);
  } else {
    image_warps<kBack>(p, sm, x);
  }
  tc_fence_before();
  __syncthreads();
  if (x.abort && threadIdx.x == 0) atomicOr(p.status, DEV_ERR_PIPE_TIMEOUT);
  if (warp == 3) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  if (kBack) join_runs(p, x);
}

template <bool kBack>
cudaError_t launch(const LinReadParams& p, const CUtensorMap& mx, const CUtensorMap& mq, int num_sms, cudaStream_t s) {
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = allow_smem(lin_read_kernel<kBack>, RT_SMEM, done);
  if (e != cudaSuccess) return e;
  return launch_behind(lin_read_kernel<kBack>, dim3(static_cast<unsigned>(lin_read_ctas(num_sms))), RT_THREADS, RT_SMEM, s, p, mx, mq);
}

}  // namespace

bool encode_bf16(CUtensorMap* m, const void* base, int rank, const uint64_t* dims, const uint64_t* strides_bytes, const uint32_t* box);

size_t lin_read_smem() { return RT_SMEM; }
int lin_read_ctas(int num_sms) { return num_sms; }

cudaError_t launch_lin_read(const LinReadParams& p, int num_sms, cudaStream_t s) {
  CUtensorMap mx, mq;
  const uint64_t H = static_cast<uint64_t>(p.H), Lq = static_cast<uint64_t>(p.Lq);
  const uint64_t dims[4] = {LIN_D, Lq, H, static_cast<uint64_t>(p.n_cand)};
  const uint64_t strides[3] = {LIN_D * 2, Lq * LIN_D * 2, H * Lq * LIN_D * 2};
  const uint32_t box[4] = {64, static_cast<uint32_t>(p.Lq), 1, 1};
  if (!encode_bf16(&mx, p.x, 4, dims, strides, box)) return cudaErrorInvalidValue;
  mq = mx;
  if (p.d_state && !encode_bf16(&mq, p.q, 4, dims, strides, box)) return cudaErrorInvalidValue;
  return p.d_state ? launch<true>(p, mx, mq, num_sms, s) : launch<false>(p, mx, mq, num_sms, s);
}

}  // namespace ikbo
