// linattn_api.cu -- host side of linear attention with a decay and of the
// candidates' reads of its states (declared in ikbo.h): argument checks,
// workspaces and launches.
#include <algorithm>
#include <cmath>
#include <cstring>

#include "linattn_internal.h"
#include "plan_internal.h"

namespace ikbo {
cudaError_t launch_linattn(const LinParams& p, int num_sms, cudaStream_t s, int* launches);
cudaError_t launch_linattn_back(LinBackParams p, int num_sms, cudaStream_t s);
size_t lin_tile_smem();
cudaError_t launch_lin_read(const LinReadParams& p, int num_sms, cudaStream_t s);
size_t lin_read_smem();
int lin_read_ctas(int num_sms);
}  // namespace ikbo

using namespace ikbo;

namespace {

constexpr size_t ANY = ~size_t{0};

// A row stride of H heads of 128 elements, 16-byte pieces.
ikbo_status_t check_stride(int64_t stride, int H) {
  if (stride < static_cast<int64_t>(H) * LIN_D) return IKBO_ERR_INVALID_ARG;
  return stride % 8 != 0 ? IKBO_ERR_UNSUPPORTED : IKBO_OK;
}

// What forward and backward check alike, and the parameters that they share.
ikbo_status_t lin_params(ikbo_plan_t p, const int32_t* d_offsets, int n_users, int n_rows, int max_len, int H, int d,
                         const float* decay, float scale, LinParams* lp) {
  if (n_users < 1 || n_rows < 0 || max_len < 0 || H < 1 || !decay || !aligned4(decay) || !aligned4(d_offsets) || !(scale > 0.f) ||
      !std::isfinite(scale) || !std::isfinite(1.f / scale))
    return IKBO_ERR_INVALID_ARG;
  if (d != LIN_D || n_users > SEG_MAX_USERS || H > 1024) return IKBO_ERR_UNSUPPORTED;
  if (!d_offsets && n_rows % n_users != 0) return IKBO_ERR_INVALID_ARG;
  if (!p || !plan_device_current(p)) return IKBO_ERR_INVALID_ARG;
  std::memset(lp, 0, sizeof(*lp));
  lp->offsets = d_offsets;
  lp->decay = decay;
  lp->status = p->d_status;
  lp->n_users = n_users;
  lp->n_rows = n_rows;
  lp->H = H;
  lp->max_len = d_offsets ? (max_len > 0 ? std::min(max_len, n_rows) : n_rows) : n_rows / n_users;
  const int64_t each = (static_cast<int64_t>(n_rows) + n_users - 1) / n_users;
  lp->likely_len = !d_offsets || max_len > 0 ? lp->max_len : static_cast<int>(std::min<int64_t>(lp->max_len, 4 * each));
  lp->scale = scale;
  lp->segs = 1;
  lp->debug = p->debug;
  lp->timeout_ns = p->timeout_ns;
  return IKBO_OK;
}

// Whether, and into what, long histories are cut.  A scan is one CTA's, so a few
// long ones leave SMs idle; cut into segments each one's keys and values are read
// (and multiplied) once more, for the states between them.  With fewer scans than
// half the SMs, segments are as long as makes one for each SM; else only rows far
// above a CTA's share are cut, as where one user's history is much longer than the
// others'.  In us, of a scan of L rows 6 + 0.0195 L whole, 13 + 0.041 seg + 0.07 (states between
// segments) cut; the states alone 5 + 0.012 L and 10.8 + 0.0265 seg + 0.072 states (measured from 400 to
// 6000 rows and 4 to 76 scans: 16 scans of 1152 rows 29 and 29, of 4096 86 and 43; 40 of 2048 48 and 56, of
// 6000 126 and 104; 60 of 4096 89 and 122).  The gradient, which has three scans for one and begins at both ends, goes
// by the same: of 3 to 72 scans of 400 to 6000 rows it takes the faster way or one within 3% (12 scans of 1024 rows whole 26.7,
// cut 26.3; 24 of 1024 26.8 and 31.0, of 2048 47.7 and 39.4; 48 of 6000 127.8 and 124.1; 72 of 6000 128 and 212).  At most
// LIN_MOST_STATES states lie between segments, and with more than LIN_MOST_CUT users none is cut (each item looks for its place among all users').
constexpr int64_t LIN_MOST_STATES = 16384;  // 1 GiB
constexpr int LIN_LEAST_SEGMENT = 256;
constexpr int LIN_MOST_CUT = 256;

// The variant, from the bound on a user's rows (every variant takes any length).  Measured, 8 heads, with states, among other
// calls on the GPU (us):
//   forward, rows           15 users:  4     8    16    64    96   128   160   256   100 users: 8    16    64    96   128   256
//   row by row                       4.3   5.6   8.1  24.4        46.1  56.9  89.5           29.2  40.8             247   476
//   chunks, in registers             6.1   6.1   6.1   8.2  10.9  12.3  15.0  20.5           33.3  33.6  48.4  63.5  71.2 120
//   chunks, tensor memory           10.7  10.7  10.8  11.1  11.4  11.4  13.7  13.9           51.6  52.4  53.4  55.6  59.6  84.0
//     (1 user 80 rows 10.0 and 9.2, 96 10.6 and 9.3; 40 users 80 27.9 and 24.7; 400 users 64 166 and 173, 80 206 and 175, 128 248 and 194)
//   the states alone, rows  15 users:  8   128   192   224   256   320   100 users: 128   192   224   256   320
//   chunks, in registers             4.9   7.6   9.4  10.6  11.2  13.0             35.6  44.9  51.1  55.1  64.3
//   chunks, tensor memory            7.7   7.8   9.4   9.5   9.0  10.8             39.8  50.1  51.3  52.2  60.8
//     (row by row, 15 users: 4 rows 4.3, 16 5.6; 400 users in chunks: 192 149 and 164, 224 170 and 168, 256 184 and 163)
constexpr int LIN_TILES_FROM[2] = {96, 225};  // forward, states alone
//   gradient, rows             15 users: 1    16    32    48    64    96   400 users: 1    16    32    48    64    96
//   in one pass                        8.4   8.7  14.7  20.0  25.2  35.7            132   153   246   333   426   614
//   chunks, tensor memory             24.6  24.9  25.4  25.4  25.6  25.9            436   437   442   443   444   452
constexpr int LIN_BACK_MOST = 64;

void cut_segments(LinParams* lp, int num_sms) {
  const int64_t items = static_cast<int64_t>(lp->n_users) * lp->H * (lp->backward ? LIN_MAX_JOBS : 1);
  const int64_t rows = static_cast<int64_t>(lp->n_rows) * lp->H * (lp->backward ? LIN_MAX_JOBS : 1);
  // (each scan's last segment is a part of one: as many SMs are left out of the division)
  int64_t seg = std::max<int64_t>(items * 2 <= num_sms ? (rows + num_sms - items - 1) / (num_sms - items) : 4 * (rows / num_sms), LIN_LEAST_SEGMENT);
  const int64_t most = LIN_MOST_STATES / items;  // segments of a user
  if (most < 2 || lp->n_users > LIN_MOST_CUT) return;
  seg = std::max(seg, (lp->max_len + most - 1) / most);
  seg = (seg + 127) / 128 * 128;
  const int64_t states = std::min(items * ((lp->likely_len + seg - 1) / seg), rows / seg + items);
  if (lp->likely_len <= (lp->job[0].x ? 360 + 21 * seg / 10 + 36 * states / 10 : 480 + 22 * seg / 10 + 6 * states)) return;
  lp->seg_len = static_cast<int>(seg);
  lp->segs = static_cast<int>((lp->max_len + seg - 1) / seg);
}

ikbo_status_t lin_run(ikbo_plan_t p, LinParams* lp, cudaStream_t stream) {
  if (lin_tile_smem() > p->max_smem) return IKBO_ERR_UNSUPPORTED;
  if (!lp->steps) {
    lp->tiles = lp->backward || lp->likely_len >= LIN_TILES_FROM[lp->job[0].x ? 0 : 1];
    if (lp->tiles) cut_segments(lp, p->num_sms);
  }
  if (lp->segs > 1) {
    bool capturing = false;
    if (stream && is_capturing(stream, &capturing) != cudaSuccess) return IKBO_ERR_CUDA;
    const size_t need = static_cast<size_t>(lp->n_jobs) * lp->n_users * lp->H * lp->segs * LIN_STATE;
    if (grow_kept<false>(p, &p->lin_states, need, ANY, capturing, stream) != cudaSuccess) return IKBO_ERR_CUDA;
    lp->ws = p->lin_states.ptr;
  }
  lp->ahead = p->num_sms;
  int launches = 0;
  const cudaError_t e = launch_linattn(*lp, p->num_sms, stream, &launches);
  p->launches += launches;
  return e == cudaSuccess ? IKBO_OK : IKBO_ERR_CUDA;
}

ikbo_status_t read_call(ikbo_plan_t p, const void* x, const float* state, int d, float scale, LinReadParams* rp) {
  if (!x || !aligned16(x) || !aligned16(state) || !(scale > 0.f) || !std::isfinite(scale)) return IKBO_ERR_INVALID_ARG;
  if (d != LIN_D) return IKBO_ERR_UNSUPPORTED;
  if (!p) return IKBO_ERR_INVALID_ARG;
  if (!p->planned) return IKBO_ERR_NOT_PLANNED;
  if (!plan_device_current(p)) return IKBO_ERR_INVALID_ARG;
  if (lin_read_smem() > p->max_smem) return IKBO_ERR_UNSUPPORTED;
  std::memset(rp, 0, sizeof(*rp));
  rp->x = static_cast<const uint16_t*>(x);
  rp->state = state;
  rp->offsets = p->d_offsets;
  rp->perm = p->d_perm;
  rp->work = p->d_work;
  rp->n_units = p->d_n_units;
  rp->status = p->d_status;
  rp->max_units = p->max_units;
  rp->n_cand = p->n_cand;
  rp->n_users = p->n_users;
  rp->H = p->H;
  rp->Lq = p->Lq;
  rp->scale = scale;
  rp->debug = p->debug;
  rp->timeout_ns = p->timeout_ns;
  return IKBO_OK;
}

}  // namespace

extern "C" {

ikbo_status_t ikbo_linattn_forward(ikbo_plan_t p, const void* Q, const void* K, const void* V, const int64_t* row_strides,
                                   const int32_t* d_offsets, int n_users, int n_rows, int max_len, int H, int d,
                                   const float* decay, const float* state_in, float* state_out, void* O, float scale,
                                   cudaStream_t stream) {
  if ((Q == nullptr) != (O == nullptr) || (n_rows > 0 && (!K || !V)) || (!O && !state_out)) return IKBO_ERR_INVALID_ARG;
  const void* ptrs[] = {Q, K, V, O, state_in, state_out};
  for (const void* q : ptrs)
    if (!aligned16(q)) return IKBO_ERR_INVALID_ARG;
  if (O && (O == K || O == V || O == Q)) return IKBO_ERR_INVALID_ARG;
  int64_t strides[4] = {0, 0, 0, 0};
  for (int k = 0; k < 4; ++k) {
    strides[k] = row_strides ? row_strides[k] : static_cast<int64_t>(H) * LIN_D;
    if ((k == 0 || k == 3) && !Q) continue;
    const ikbo_status_t st = check_stride(strides[k], H);
    if (st != IKBO_OK) return st;
  }
  LinParams lp;
  ikbo_status_t st = lin_params(p, d_offsets, n_users, n_rows, max_len, H, d, decay, scale, &lp);
  if (st != IKBO_OK) return st;
  LinJob& j = lp.job[0];
  j.x = static_cast<const uint16_t*>(Q);
  j.y = static_cast<const uint16_t*>(K);
  j.z = static_cast<const uint16_t*>(V);
  j.out = static_cast<uint16_t*>(O);
  j.xs = strides[0];
  j.ys = strides[1];
  j.zs = strides[2];
  j.os = strides[3];
  j.s_in = state_in;
  j.s_out = state_out;
  j.add = 1.f;
  j.read = scale;
  lp.n_jobs = 1;
  lp.steps = lp.likely_len <= LIN_STEP_MOST;
  return lin_run(p, &lp, stream);
}

ikbo_status_t ikbo_linattn_backward(ikbo_plan_t p, const void* Q, const void* K, const void* V, const void* dO,
                                    const int64_t* row_strides, const int32_t* d_offsets, int n_users, int n_rows,
                                    int max_len, int H, int d, const float* decay, const float* state_in,
                                    const float* d_state_out, void* dQ, void* dK, void* dV, float* d_state_in, float scale,
                                    cudaStream_t stream) {
  const void* in[] = {Q, K, V, dO, state_in, d_state_out};
  const void* out[] = {dQ, dK, dV, d_state_in};
  for (int k = 0; k < 4; ++k)
    if (n_rows > 0 && !in[k]) return IKBO_ERR_INVALID_ARG;
  if (!dQ && !dK && !dV && !d_state_in) return IKBO_ERR_INVALID_ARG;
  for (const void* q : in)
    if (!aligned16(q)) return IKBO_ERR_INVALID_ARG;
  for (const void* q : out) {
    if (!aligned16(q)) return IKBO_ERR_INVALID_ARG;
    for (const void* r : in)
      if (q && q == r) return IKBO_ERR_INVALID_ARG;
  }
  int64_t strides[7];
  for (int k = 0; k < 7; ++k) {
    strides[k] = row_strides ? row_strides[k] : static_cast<int64_t>(H) * LIN_D;
    if (k >= 4 && !out[k - 4]) continue;
    const ikbo_status_t st = check_stride(strides[k], H);
    if (st != IKBO_OK) return st;
  }
  LinParams lp;
  ikbo_status_t st = lin_params(p, d_offsets, n_users, n_rows, max_len, H, d, decay, scale, &lp);
  if (st != IKBO_OK) return st;
  if (lp.likely_len <= LIN_BACK_MOST) {
    LinBackParams bp;
    std::memset(&bp, 0, sizeof(bp));
    bp.q = static_cast<const uint16_t*>(Q);
    bp.k = static_cast<const uint16_t*>(K);
    bp.v = static_cast<const uint16_t*>(V);
    bp.d_o = static_cast<const uint16_t*>(dO);
    bp.qs = strides[0];
    bp.ks = strides[1];
    bp.vs = strides[2];
    bp.d_os = strides[3];
    bp.dq = static_cast<uint16_t*>(dQ);
    bp.dk = static_cast<uint16_t*>(dK);
    bp.dv = static_cast<uint16_t*>(dV);
    bp.dqs = strides[4];
    bp.dks = strides[5];
    bp.dvs = strides[6];
    bp.s_in = state_in;
    bp.ds_out = d_state_out;
    bp.ds_in = d_state_in;
    bp.offsets = d_offsets;
    bp.decay = decay;
    bp.status = lp.status;
    bp.n_users = n_users;
    bp.n_rows = n_rows;
    bp.H = H;
    bp.max_len = lp.max_len;
    bp.scale = scale;
    if (launch_linattn_back(bp, p->num_sms, stream) != cudaSuccess) return IKBO_ERR_CUDA;
    p->launches++;
    return IKBO_OK;
  }
  lp.backward = 1;
  const auto add = [&](int x, int y, int z, void* o, int os, const float* s_in, bool turned, float* s_out, bool reverse) {
    LinJob& j = lp.job[lp.n_jobs++];
    j.x = static_cast<const uint16_t*>(in[x]);
    j.y = static_cast<const uint16_t*>(in[y]);
    j.z = static_cast<const uint16_t*>(in[z]);
    j.out = static_cast<uint16_t*>(o);
    j.xs = strides[x];
    j.ys = strides[y];
    j.zs = strides[z];
    j.os = strides[os];
    j.s_in = s_in;
    j.s_out = s_out;
    j.s_in_turned = turned;
    j.reverse = reverse;
    j.add = reverse ? scale : 1.f;
    j.read = reverse ? 1.f : scale;
  };
  if (dQ) add(3, 2, 1, dQ, 4, state_in, true, nullptr, false);
  if (dK) add(2, 3, 0, dK, 5, d_state_out, true, nullptr, true);
  if (dV || d_state_in) add(1, 0, 3, dV, 6, d_state_out, false, d_state_in, true);
  return lin_run(p, &lp, stream);
}

ikbo_status_t ikbo_linattn_read_forward(ikbo_plan_t p, const void* Q, const float* state, void* O, int d, float scale,
                                        cudaStream_t stream) {
  if (!O || !aligned16(O) || !state) return IKBO_ERR_INVALID_ARG;
  LinReadParams rp;
  const ikbo_status_t st = read_call(p, Q, state, d, scale, &rp);
  if (st != IKBO_OK) return st;
  rp.out = static_cast<uint16_t*>(O);
  if (launch_lin_read(rp, p->num_sms, stream) != cudaSuccess) return IKBO_ERR_CUDA;
  p->launches++;
  return IKBO_OK;
}

ikbo_status_t ikbo_linattn_read_backward(ikbo_plan_t p, const void* Q, const float* state, const void* dO, void* dQ,
                                         float* d_state, int d, float scale, cudaStream_t stream) {
  if ((!dQ && !d_state) || !aligned16(dQ) || !aligned16(d_state) || !aligned16(Q) || (dQ && !state) || (d_state && !Q) ||
      (dQ && d_state && (dQ == Q || dQ == dO)) || (d_state && d_state == state))
    return IKBO_ERR_INVALID_ARG;
  LinReadParams rp;
  const ikbo_status_t st = read_call(p, dO, state, d, scale, &rp);
  if (st != IKBO_OK) return st;
  rp.q = static_cast<const uint16_t*>(Q);
  if (d_state) {
    bool capturing = false;
    if (stream && is_capturing(stream, &capturing) != cudaSuccess) return IKBO_ERR_CUDA;
    const size_t need = 2 * static_cast<size_t>(lin_read_ctas(p->num_sms)) * LIN_STATE;
    if (grow_kept<false>(p, &p->lin_part, need, ANY, capturing, stream) != cudaSuccess ||
        grow_kept<true>(p, &p->lin_tickets, static_cast<size_t>(lin_read_ctas(p->num_sms)), ANY, capturing, stream) != cudaSuccess)
      return IKBO_ERR_CUDA;
    rp.part = p->lin_part.ptr;
    rp.tickets = p->lin_tickets.ptr;
    rp.d_state = d_state;
  }
  rp.out = static_cast<uint16_t*>(dQ);
  rp.turned = 1;
  if (launch_lin_read(rp, p->num_sms, stream) != cudaSuccess) return IKBO_ERR_CUDA;
  p->launches++;
  return IKBO_OK;
}

}  // extern "C"
