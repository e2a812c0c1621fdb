// plan_internal.h -- the plan object behind ikbo_plan_t and the host helpers
// the ABI's source files share.  Not part of the public ABI.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstddef>
#include <cstdint>
#include <cstdlib>

#include "ikbo.h"
#include "ikbo_internal.h"

namespace ikbo {
// A workspace of the plan that captured graphs may hold (see grow_kept).
template <typename T>
struct KeptBuffer {
  T* ptr = nullptr;
  size_t elems = 0;
  bool captured = false;  // a call under stream capture has used it
};
}  // namespace ikbo

struct ikbo_plan_s {
  int device = 0;
  int num_sms = 0;
  size_t max_smem = 0;
  int max_cand = 0, max_users = 0, max_heads = 0;
  // the bound request
  bool planned = false;
  const int32_t* d_map = nullptr;
  int n_cand = 0, n_users = 0, H = 0, Lq = 0, cands_per_unit = 0;
  // plan-owned device memory
  int32_t* d_counts = nullptr;
  int32_t* d_offsets = nullptr;
  int32_t* d_runs = nullptr;
  int32_t* d_perm = nullptr;
  int32_t* d_work = nullptr;
  int32_t* d_n_units = nullptr;
  int64_t max_units = 0;
  uint32_t* d_status = nullptr;  // [0] status bits, [1] LCE flag-timeout word, [2] LCE finished-CTA count
  float* d_partial = nullptr;
  size_t partial_elems = 0;
  uint32_t* d_flags = nullptr;
  size_t flags_elems = 0;
  // LCE backward workspaces (grown on first use)
  float* d_bwd_S = nullptr;
  size_t bwd_S_elems = 0;
  uint16_t* d_bwd_Sb = nullptr;
  size_t bwd_Sb_elems = 0;
  float* d_bwd_seg = nullptr;
  size_t bwd_seg_elems = 0;
  float* d_bwd_wpart = nullptr;
  size_t bwd_wpart_elems = 0;
  float* d_bwd_spart = nullptr;  // candidate pass: S partials of each CTA's first and last run
  size_t bwd_spart_elems = 0;
  float* d_bwd_dbcta = nullptr;  // candidate pass: each CTA's share of db
  size_t bwd_dbcta_elems = 0;
  uint32_t* d_bwd_ctrl = nullptr;  // candidate pass: grid barrier counts
  size_t bwd_ctrl_elems = 0;
  // a second stream (created on first use) on which dW_u runs beside dU
  cudaStream_t side = nullptr;
  cudaEvent_t ev_fork = nullptr, ev_join = nullptr;
  // attention backward workspaces
  float* d_abwd_lse = nullptr;
  size_t abwd_lse_elems = 0;
  float* d_abwd_drow = nullptr;
  size_t abwd_drow_elems = 0;
  int32_t* d_abwd_blk = nullptr;
  size_t abwd_blk_elems = 0;
  // 4-bit cache attention (grown on first use)
  ikbo::KeptBuffer<float> qa_part;        // partial rows of histories split over several CTAs
  ikbo::KeptBuffer<uint32_t> qa_tickets;  // splits of a tile that have finished (zero between calls)
  ikbo::KeptBuffer<int4> qa_list;         // work items
  ikbo::KeptBuffer<uint16_t> qa_kv;       // decoded K rows, then V rows
  ikbo::KeptBuffer<int32_t> qa_ranges;    // each user's first decoded row, then each user's length
  void** retired = nullptr;               // replaced buffers that captured graphs may hold, freed with the plan
  int n_retired = 0;
  bool lce_flags_dirty = false;  // an LCE launch failed: its flags may still be set
  uint32_t debug = 0;
  uint64_t timeout_ns = 2000000000ull;
  int lce_schedule = ikbo::LCE_SCHEDULE_AUTO;
  std::atomic<uint64_t> launches{0};
};

namespace ikbo {

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// The device the plan was made on is the current one.
inline bool plan_device_current(const ikbo_plan_s* p) {
  int dev = -1;
  return cudaGetDevice(&dev) == cudaSuccess && dev == p->device;
}

inline cudaError_t is_capturing(cudaStream_t stream, bool* yes) {
  cudaStreamCaptureStatus st = cudaStreamCaptureStatusNone;
  const cudaError_t e = cudaStreamIsCapturing(stream, &st);
  *yes = st != cudaStreamCaptureStatusNone;
  return e;
}

// Makes a workspace hold `need` elements.  Sizes grow by a quarter at least (so
// that a plan meets few of them), up to `most` where that holds `need`, unless the
// memory for that is not there.  A buffer that a captured call has used is kept
// until the plan is destroyed, as its graph may be replayed at any time; others are
// freed before the new one is allocated.  A call under capture that would have to
// allocate is refused before anything is tried.  kZeroed: new memory is zeroed on
// `stream`.
template <bool kZeroed, typename T>
cudaError_t grow_kept(ikbo_plan_s* p, KeptBuffer<T>* b, size_t need, size_t most, bool capturing, cudaStream_t stream) {
  if (b->ptr && b->elems >= need) {
    b->captured = b->captured || capturing;
    return cudaSuccess;
  }
  // (asked again: for the default stream it is an error that another one is captured,
  // whose capture an allocation would end)
  cudaError_t e = is_capturing(stream, &capturing);
  if (e != cudaSuccess) return e;
  if (capturing) return cudaErrorStreamCaptureUnsupported;
  size_t size = b->elems + b->elems / 4;
  if (size > most) size = most;
  if (size < need) size = need;
  if (b->ptr && b->captured) {
    void** list = static_cast<void**>(std::realloc(p->retired, sizeof(void*) * (static_cast<size_t>(p->n_retired) + 1)));
    if (!list) return cudaErrorMemoryAllocation;
    p->retired = list;
    p->retired[p->n_retired++] = b->ptr;
  } else if (b->ptr) {  // (whichever stream the last call that used it ran on)
    e = cudaDeviceSynchronize();
    if (e != cudaSuccess) return e;
    cudaFree(b->ptr);
  }
  *b = KeptBuffer<T>();
  e = cudaMalloc(reinterpret_cast<void**>(&b->ptr), size * sizeof(T));
  if (e != cudaSuccess && size > need) {
    cudaGetLastError();
    size = need;
    e = cudaMalloc(reinterpret_cast<void**>(&b->ptr), size * sizeof(T));
  }
  if (e != cudaSuccess) {
    cudaGetLastError();
    b->ptr = nullptr;
    return e;
  }
  if (kZeroed) {
    e = cudaMemsetAsync(b->ptr, 0, size * sizeof(T), stream);
    if (e != cudaSuccess) {
      cudaFree(b->ptr);
      b->ptr = nullptr;
      return e;
    }
  }
  b->elems = size;
  return cudaSuccess;
}

// Broadcast attention over bf16 K/V (api.cu), every entry point's launch:
// target units of the plan's work list, plus self units when Q_user is given.
// kv_lens (with jagged kv_offsets): user u's keys are rows kv_offsets[u] ..
// kv_offsets[u] + kv_lens[u] - 1; null: they end where the next user's begin.
// H_kv heads of K/V serve the plan's H query heads (H % H_kv == 0).
struct AttnCall {
  const void *Q, *Q_user, *K, *V;
  const int32_t *kv_offsets, *kv_lens;
  void *O, *O_user;
  float* lse;
  int Lq_u, Lkv, d, H_kv;
  float scale;
};
ikbo_status_t attn_launch(ikbo_plan_s* p, const AttnCall& c, cudaStream_t stream);

}  // namespace ikbo
