// linattn_internal.h -- parameter blocks of linear attention with a decay
// (linattn.cu) and of the candidates' reads of its states (linread.cu).  Not
// part of the public ABI.
#pragma once
#include <cuda_runtime.h>

#include "ikbo_internal.h"

namespace ikbo {

// A debug switch (ikbo_plan_set_debug), beside those of ikbo_internal.h: some CTAs of the
// tile kernels never hand over what states are made of, or read by.
constexpr uint32_t DEBUG_WITHHOLD_STATES = 1u << 3;

constexpr int LIN_D = 128;                    // head dimension of queries, keys and values
constexpr int LIN_STATE = LIN_D * LIN_D;      // floats of a state
constexpr int LIN_MAX_JOBS = 3;
constexpr int LIN_STEP_MOST = 8;              // rows of a user up to which single steps are taken


// One scan: with queries x, keys y and values z,
//   S <- decay S + add y_t z_t^T,   out_t = read x_t S,   add read = scale
// from the first row of a user to the last, or (reverse) from the last to the
// first.  A reverse scan's start has been decayed already: its first step
// takes it as it is, and its end is decayed once more.  The scale is in what rows add where
// the state is a gradient, which the start and the end are too (a state without it
// would have to begin with the start divided by the scale, and may not hold that).
struct LinJob {
  const uint16_t *x, *y, *z;  // x null: no outputs
  uint16_t* out;
  int64_t xs, ys, zs, os;     // row strides in elements
  const float* s_in;          // [n_users][H][128][128], rows of y's elements; null: zero
  float* s_out;               // the same, or null; may be s_in
  float add, read;
  int s_in_turned;            // s_in has rows of z's elements
  int reverse;
};

struct LinParams {
  LinJob job[LIN_MAX_JOBS];
  const int32_t* offsets;  // [n_users + 1], or null: n_rows / n_users rows each
  const float* decay;      // [H]
  uint32_t* status;
  float* ws;               // states between segments [job][u][h][segs], at a segment's end
  int n_jobs, n_users, n_rows, H, max_len;
  int likely_len;          // what variants are chosen by: max_len, or without a bound four times the average
  int seg_len, segs;       // rows of a segment (a multiple of the chunk), segments of the longest user; 1: no segments
  int backward;            // the jobs are a gradient's (variants do not go by which of them are asked for)
  int steps;               // rows one by one (a forward scan alone)
  int tiles;               // the chunks' products on the 5th-gen tensor cores
  int ahead;               // in registers: the scan whose state is asked for in L2 meanwhile is this many later
  uint32_t debug;          // the plan's switches
  uint64_t timeout_ns;
  float scale;
};

// The gradient of a few rows a user, at once.
struct LinBackParams {
  const uint16_t *q, *k, *v, *d_o;
  int64_t qs, ks, vs, d_os;        // row strides in elements
  uint16_t *dq, *dk, *dv;          // null: not wanted
  int64_t dqs, dks, dvs;
  const float *s_in, *ds_out;      // null: zero
  float* ds_in;                    // null: not wanted
  const int32_t* offsets;
  const float* decay;
  uint32_t* status;
  int n_users, n_rows, H, max_len;
  int ahead;                       // CTAs that run at a time
  float scale;
};

struct LinReadParams {
  const uint16_t* x;        // rows [n_cand][H][Lq][128]
  const float* state;       // [n_users][H][128][128]
  uint16_t* out;            // like x
  const uint16_t* q;        // backward: the queries (x is dO), for d_state
  float* d_state;
  float* part;              // two states a CTA: of the first and the last run of units that it shares
  uint32_t* tickets;        // a count a CTA, zero between calls: parts of the run that begins there
  const int32_t* offsets;   // the plan's segments
  const int32_t* perm;
  const int32_t* work;      // units {u, h, first place, run}
  const int32_t* n_units;
  uint32_t* status;
  int64_t max_units;
  int n_cand, n_users, H, Lq;
  int turned;               // out = x S^T
  float scale;
  uint32_t debug;           // the plan's switches
  uint64_t timeout_ns;
};

}  // namespace ikbo
