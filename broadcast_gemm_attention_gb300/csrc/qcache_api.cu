// qcache_api.cu -- host side of the rotary positions, the 4-bit cache and the
// attention that reads it (declared in ikbo.h): argument checks, workspaces
// and launches.  No computation of the method happens on the host but a
// rotation's table of frequencies, formed once.
#include <algorithm>
#include <cmath>
#include <cstring>
#include <new>

#include "plan_internal.h"
#include "qcache_internal.h"

namespace ikbo {
cudaError_t launch_rope(const RopeParams& p, int dtype, int num_sms, cudaStream_t s);
cudaError_t launch_qc_resize(const QcResizeParams& p, cudaStream_t s);
cudaError_t launch_qc_append(QcAppendParams p, int num_sms, cudaStream_t s);
cudaError_t launch_qc_load(const QcLoadParams& p, int num_sms, cudaStream_t s);
int qattn_ctas(int num_sms, bool eight);
size_t qattn_part_elems(int num_sms);
size_t qattn_tickets(int num_sms);
cudaError_t launch_qattn(const QcAttnParams& p, bool eight, bool solo, cudaStream_t s);
size_t qattn_tile_smem();
size_t qattn_tile_part_elems(int num_sms);
int64_t qattn_tile_items(int64_t rows, int n_users, int H_kv, int num_sms);
cudaError_t launch_qattn_tile(const QcAttnParams& p, cudaStream_t s);
cudaError_t launch_qtree(const QcTreeParams& p, int num_sms, cudaStream_t s);
}  // namespace ikbo

using namespace ikbo;

struct ikbo_rope_s {
  int rot, interleaved;
  float magnitude;
  int axes;  // 0: made for one axis
  uint64_t turn[ROPE_MAX_DIM / 2];
  uint8_t axis[ROPE_MAX_DIM / 2];
};

namespace {

constexpr double TWO_PI = 6.283185307179586476925286766559;
constexpr double TWO_PI_REST = 2.4492935982947064e-16;  // 2 pi - TWO_PI
constexpr int64_t INT32_LIMIT = 0x7fffffff;

// x modulo 1 in units of 2^-64, to the nearest.
uint64_t fixed_fraction(double x) {
  const double a = std::fabs(x), part = a - std::floor(a);  // both exact
  const uint64_t v = static_cast<uint64_t>(std::nearbyint(std::ldexp(part, 64)));  // below 2^64: part is at most 1 - 2^-53
  return x < 0 ? 0 - v : v;
}

// The turns of f radians, modulo 1, in units of 2^-64 turn: the quotient to 53 bits,
// and the same for what it leaves of f.  (The first alone is off by 2^-56 of a turn
// at f = 1, and in proportion to f; a position of 31 bits makes that 2^-25.)  Each
// is rounded to a unit, and the second's own rounding, 2^-106 f, is below one for f
// up to 2^40.
uint64_t fixed_turns(double f) {
  const double q = f / TWO_PI;
  const double left = std::fma(-q, TWO_PI, f) - q * TWO_PI_REST;
  return fixed_fraction(q) + fixed_fraction(left / TWO_PI);
}

// log2(page / 16), or -1 for a page that is not 16, 32, .., 1024
int blocks_log2_of(int page) {
  for (int k = 0; QC_ROWS << k <= QC_MAX_PAGE; ++k)
    if (page == QC_ROWS << k) return k;
  return -1;
}

// Sizes of a cache: IKBO_OK, or the refusal.
ikbo_status_t check_cache(int n_pages, int page, int H) {
  if (n_pages < 1 || H < 1) return IKBO_ERR_INVALID_ARG;
  if (blocks_log2_of(page) < 0) return IKBO_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(n_pages) * page > INT32_LIMIT) return IKBO_ERR_UNSUPPORTED;
  return IKBO_OK;
}

// A table of max_blocks pages per user: its lengths are 32 bits.
ikbo_status_t check_table(const int32_t* table, const int32_t* lens, int max_blocks, int n_users, int page) {
  if (!table || !lens || !aligned4(table) || !aligned4(lens) || max_blocks < 1 || n_users < 1)
    return IKBO_ERR_INVALID_ARG;
  if (n_users > SEG_MAX_USERS || static_cast<int64_t>(max_blocks) * page > INT32_LIMIT) return IKBO_ERR_UNSUPPORTED;
  return IKBO_OK;
}

// The attention's variant, from the average number of query rows that read a
// history's K/V head, R = rows / n_users, and the tokens there may be to read.
// Measured at 64 users x 8 heads x 4096 tokens, caches cold (us):
//   R                   8    16    32    64   128
//   in registers       85   105   190   358   695  (histories decoded once per 8 or 16 rows)
//   in tiles          126   126   126   130   135  (once per 128 rows)
// 1024 candidates of 32 queries x 8 heads over 2048 tokens each:
//   R                 546  1092  2184  4369 (2048 candidates)
//   in tiles          281   258   253   497
//   decoded first     338   248   208   375 (the first with an earlier attention forward, 3% slower)
// So up to 16 rows in registers, from 1024 on decoded first, between them in
// tiles, unless the tile kernel's longer start and end (about 12 us) are not
// made up for: the register kernel gets through 21000 (16-row tile, token,
// head)s in a microsecond, the tile kernel through 20500 of 128 rows (4
// candidates of one history of 32000 tokens, 32 rows: 40 and 49 us; 8 of the
// same with four heads sharing, 256 rows: 169 and 56).
// (And in tiles where the bound on the tokens is so large, or so loose, that
// decoded histories would take more than QA_MOST_DECODED bytes.)
enum QcAttnVariant { QATTN_REGISTERS = 1, QATTN_TILES = 2, QATTN_DECODED = 3 };

constexpr int64_t QA_MOST_DECODED = int64_t{8} << 30;

// Rows of decoded histories, each padded to the attention kernel's key tile.
int64_t decoded_rows(int n_users, int Lkv) {
  return (static_cast<int64_t>(Lkv) + static_cast<int64_t>(ATT_BN) * n_users + ATT_BN - 1) / ATT_BN * ATT_BN;
}
int64_t decoded_bytes(int n_users, int H_kv, int Lkv) { return decoded_rows(n_users, Lkv) * H_kv * QC_D * 4; }

QcAttnVariant qattn_variant(int64_t rows, int n_users, int H_kv, int Lkv) {
  if (rows <= 16 * static_cast<int64_t>(n_users)) return QATTN_REGISTERS;
  if (rows > 1024 * static_cast<int64_t>(n_users) && decoded_bytes(n_users, H_kv, Lkv) <= QA_MOST_DECODED) return QATTN_DECODED;
  const double tokens = static_cast<double>(Lkv) * H_kv;
  const double r = static_cast<double>(rows) / n_users;
  const double registers_us = std::ceil(r / 16) * tokens / 21000;
  const double tiles_us = 12 + std::ceil(r / 128) * tokens / 20500;
  return registers_us < tiles_us ? QATTN_REGISTERS : QATTN_TILES;
}

// What attention over the cache asks of its arguments (before anything is allocated or launched).
ikbo_status_t check_attn(ikbo_plan_t p, const void* Q, const void* data, int n_pages, int page, int H_kv, const int32_t* d_table,
                         int max_blocks, const int32_t* d_lens, const void* O, const float* lse, int Lkv, int d, float scale) {
  if (!Q || !O || !data || !aligned16(Q) || !aligned16(O) || !aligned16(data) || !aligned4(lse))
    return IKBO_ERR_INVALID_ARG;
  if (Lkv < 1 || !(scale > 0.f) || !std::isfinite(scale)) return IKBO_ERR_INVALID_ARG;
  if (d != QC_D) return IKBO_ERR_UNSUPPORTED;
  ikbo_status_t st = check_cache(n_pages, page, H_kv);
  if (st != IKBO_OK) return st;
  st = check_table(d_table, d_lens, max_blocks, p ? (p->planned ? p->n_users : 1) : 1, page);
  if (st != IKBO_OK) return st;
  if (!p) return IKBO_ERR_INVALID_ARG;
  if (!p->planned) return IKBO_ERR_NOT_PLANNED;
  if (p->H % H_kv != 0 || !plan_device_current(p)) return IKBO_ERR_INVALID_ARG;
  return static_cast<int64_t>(p->n_cand) * p->H * p->Lq > INT32_LIMIT ? IKBO_ERR_UNSUPPORTED : IKBO_OK;
}

// axes: a call with positions on the rotation's axes, d_pos and the stride from one
// item's to the next's among them.
ikbo_status_t rope_call(ikbo_plan_t p, ikbo_rope_t r, const void* X, const int64_t* xs, void* Y, const int64_t* ys,
                        const int32_t* d_start, int broadcast, int dtype, int n, int H, int L, int d, bool backward,
                        cudaStream_t stream, bool axes = false, const int32_t* d_pos = nullptr, int64_t pos_item = 0) {
  if (r && (axes ? r->axes < 1 || !aligned4(d_pos) || pos_item < 0 : r->axes > 0)) return IKBO_ERR_INVALID_ARG;
  if (!r || n < 0 || (n > 0 && (!X || !Y)) || H < 1 || L < 1 || d < 1) return IKBO_ERR_INVALID_ARG;
  if (dtype < IKBO_BF16 || dtype > IKBO_FP32) return IKBO_ERR_INVALID_ARG;
  const uintptr_t elt = dtype == IKBO_FP32 ? 4 : 2;
  if (reinterpret_cast<uintptr_t>(X) % elt || reinterpret_cast<uintptr_t>(Y) % elt || !aligned4(d_start))
    return IKBO_ERR_INVALID_ARG;
  if (r->rot > d) return IKBO_ERR_INVALID_ARG;
  if (d > ROPE_MAX_DIM || static_cast<int64_t>(n) * L > INT32_LIMIT) return IKBO_ERR_UNSUPPORTED;
  RopeParams rp;
  std::memset(&rp, 0, sizeof(rp));
  const int64_t plain[3] = {static_cast<int64_t>(H) * L * d, static_cast<int64_t>(L) * d, d};
  const int extent[3] = {n, H, L};
  bool same = X == Y;
  for (int k = 0; k < 3; ++k) {  // the stride of a dimension of extent 1 is never used
    rp.xs[k] = extent[k] <= 1 ? 0 : (xs ? xs[k] : plain[k]);
    rp.ys[k] = extent[k] <= 1 ? 0 : (ys ? ys[k] : plain[k]);
    same = same && rp.xs[k] == rp.ys[k];
  }
  if (X == Y && !same) return IKBO_ERR_INVALID_ARG;
  if (!p) return IKBO_ERR_INVALID_ARG;
  if (broadcast) {
    if (!p->planned) return IKBO_ERR_NOT_PLANNED;
    if (n != p->n_cand) return IKBO_ERR_INVALID_ARG;
    rp.map = p->d_map;
    rp.n_users = p->n_users;
  }
  if (!plan_device_current(p)) return IKBO_ERR_INVALID_ARG;
  if (n == 0) return IKBO_OK;
  rp.X = X;
  rp.Y = Y;
  rp.start = d_start;
  rp.status = p->d_status;
  rp.n = n;
  rp.H = H;
  rp.L = L;
  rp.d = d;
  rp.rot = r->rot;
  rp.interleaved = r->interleaved;
  rp.backward = backward ? 1 : 0;
  rp.copy_rest = (!same && r->rot < d) ? 1 : 0;
  rp.magnitude = r->magnitude;
  if (axes) {
    rp.axes = r->axes;
    rp.pos = d_pos;
    rp.pos_item = pos_item;
    std::memcpy(rp.axis, r->axis, sizeof(uint8_t) * (r->rot / 2));
  }
  std::memcpy(rp.turn, r->turn, sizeof(uint64_t) * (r->rot / 2));
  if (launch_rope(rp, dtype, p->num_sms, stream) != cudaSuccess) return IKBO_ERR_CUDA;
  p->launches++;
  return IKBO_OK;
}

}  // namespace

extern "C" {

// ---------------------------------------------------------------- rotation
ikbo_status_t ikbo_rope_frequencies(double* freqs, int rot_dim, double base, int scaling, double factor,
                                    double original_len, double low_turns, double high_turns) {
  if (!freqs || rot_dim < 2 || rot_dim % 2 != 0 || rot_dim > ROPE_MAX_DIM) return IKBO_ERR_INVALID_ARG;
  if (!(base > 0) || !std::isfinite(base) || !(factor > 0) || !std::isfinite(factor)) return IKBO_ERR_INVALID_ARG;
  if (scaling < IKBO_ROPE_PLAIN || scaling > IKBO_ROPE_TURNS) return IKBO_ERR_INVALID_ARG;
  if (scaling == IKBO_ROPE_TURNS &&
      (!(original_len > 0) || !std::isfinite(original_len) || !(low_turns >= 0) || !(high_turns > low_turns) ||
       !std::isfinite(high_turns)))
    return IKBO_ERR_INVALID_ARG;
  if (scaling == IKBO_ROPE_BASE && rot_dim > 2) base *= std::pow(factor, rot_dim / (rot_dim - 2.0));
  for (int j = 0; j < rot_dim / 2; ++j) {
    double f = std::pow(base, -2.0 * j / rot_dim);
    if (scaling == IKBO_ROPE_LINEAR) f /= factor;
    if (scaling == IKBO_ROPE_TURNS) {
      double keep = (original_len * f / TWO_PI - low_turns) / (high_turns - low_turns);
      keep = keep < 0 ? 0 : (keep > 1 ? 1 : keep);
      f = keep * f + (1 - keep) * f / factor;
    }
    freqs[j] = f;
  }
  return IKBO_OK;
}

ikbo_status_t ikbo_rope_create(ikbo_rope_t* out, int rot_dim, const double* freqs, int interleaved, float magnitude) {
  if (!out) return IKBO_ERR_INVALID_ARG;
  *out = nullptr;
  if (!freqs || rot_dim < 2 || rot_dim % 2 != 0 || rot_dim > ROPE_MAX_DIM || !std::isfinite(magnitude) ||
      magnitude == 0.f)
    return IKBO_ERR_INVALID_ARG;
  for (int j = 0; j < rot_dim / 2; ++j)
    if (!std::isfinite(freqs[j])) return IKBO_ERR_INVALID_ARG;
  ikbo_rope_t r = new (std::nothrow) ikbo_rope_s();
  if (!r) return IKBO_ERR_CUDA;
  r->rot = rot_dim;
  r->interleaved = interleaved ? 1 : 0;
  r->magnitude = magnitude;
  for (int j = 0; j < rot_dim / 2; ++j) r->turn[j] = fixed_turns(freqs[j]);
  *out = r;
  return IKBO_OK;
}

ikbo_status_t ikbo_rope_create_axes(ikbo_rope_t* out, int rot_dim, const double* freqs, int n_axes,
                                    const uint8_t* axis_of_pair, int interleaved, float magnitude) {
  if (!out) return IKBO_ERR_INVALID_ARG;
  *out = nullptr;
  if (n_axes < 1 || !axis_of_pair) return IKBO_ERR_INVALID_ARG;
  if (n_axes > ROPE_MAX_AXES) return IKBO_ERR_UNSUPPORTED;
  ikbo_rope_t r = nullptr;
  const ikbo_status_t st = ikbo_rope_create(&r, rot_dim, freqs, interleaved, magnitude);
  if (st != IKBO_OK) return st;
  for (int j = 0; j < rot_dim / 2; ++j) {
    if (axis_of_pair[j] >= n_axes) {
      delete r;
      return IKBO_ERR_INVALID_ARG;
    }
    r->axis[j] = axis_of_pair[j];
  }
  r->axes = n_axes;
  *out = r;
  return IKBO_OK;
}

void ikbo_rope_destroy(ikbo_rope_t r) { delete r; }

ikbo_status_t ikbo_rope_forward(ikbo_plan_t p, ikbo_rope_t r, const void* X, const int64_t* x_strides, void* Y,
                                const int64_t* y_strides, const int32_t* d_start, int broadcast, int dtype, int n,
                                int H, int L, int d, cudaStream_t stream) {
  return rope_call(p, r, X, x_strides, Y, y_strides, d_start, broadcast, dtype, n, H, L, d, false, stream);
}

ikbo_status_t ikbo_rope_backward(ikbo_plan_t p, ikbo_rope_t r, const void* dY, const int64_t* dy_strides, void* dX,
                                 const int64_t* dx_strides, const int32_t* d_start, int broadcast, int dtype, int n,
                                 int H, int L, int d, cudaStream_t stream) {
  return rope_call(p, r, dY, dy_strides, dX, dx_strides, d_start, broadcast, dtype, n, H, L, d, true, stream);
}

ikbo_status_t ikbo_rope_axes_forward(ikbo_plan_t p, ikbo_rope_t r, const void* X, const int64_t* x_strides, void* Y,
                                     const int64_t* y_strides, const int32_t* d_start, const int32_t* d_positions,
                                     int64_t positions_stride, int broadcast, int dtype, int n, int H, int L, int d,
                                     cudaStream_t stream) {
  return rope_call(p, r, X, x_strides, Y, y_strides, d_start, broadcast, dtype, n, H, L, d, false, stream, true, d_positions,
                   positions_stride);
}

ikbo_status_t ikbo_rope_axes_backward(ikbo_plan_t p, ikbo_rope_t r, const void* dY, const int64_t* dy_strides, void* dX,
                                      const int64_t* dx_strides, const int32_t* d_start, const int32_t* d_positions,
                                      int64_t positions_stride, int broadcast, int dtype, int n, int H, int L, int d,
                                      cudaStream_t stream) {
  return rope_call(p, r, dY, dy_strides, dX, dx_strides, d_start, broadcast, dtype, n, H, L, d, true, stream, true, d_positions,
                   positions_stride);
}

// ------------------------------------------------------------------- cache
uint64_t ikbo_qcache_bytes(int n_pages, int page, int H) {
  if (check_cache(n_pages, page, H) != IKBO_OK) return 0;
  return static_cast<uint64_t>(n_pages) * H * (page / QC_ROWS) * QC_BLOCK_BYTES;
}

ikbo_status_t ikbo_qcache_resize(ikbo_plan_t p, int32_t* d_lens, const int32_t* d_new_lens, int n_users,
                                 int32_t* d_table, int max_blocks, int page, int32_t* d_free, int32_t* d_n_free,
                                 int n_pages, int32_t* d_slots, int32_t* d_slot_offsets, int32_t* d_positions,
                                 int max_new, cudaStream_t stream) {
  ikbo_status_t st = check_cache(n_pages, page, 1);
  if (st != IKBO_OK) return st;
  st = check_table(d_table, d_lens, max_blocks, n_users, page);
  if (st != IKBO_OK) return st;
  if (!d_new_lens || !d_free || !d_n_free || !d_slot_offsets || max_new < 0 || (max_new > 0 && !d_slots))
    return IKBO_ERR_INVALID_ARG;
  const void* ptrs[] = {d_new_lens, d_free, d_n_free, d_slots, d_slot_offsets, d_positions};
  for (const void* q : ptrs)
    if (!aligned4(q)) return IKBO_ERR_INVALID_ARG;
  if (!p || !plan_device_current(p)) return IKBO_ERR_INVALID_ARG;
  QcResizeParams rp;
  rp.lens = d_lens;
  rp.new_lens = d_new_lens;
  rp.table = d_table;
  rp.free_pages = d_free;
  rp.n_free = d_n_free;
  rp.slots = d_slots;
  rp.offsets = d_slot_offsets;
  rp.positions = d_positions;
  rp.status = p->d_status;
  rp.n_users = n_users;
  rp.max_blocks = max_blocks;
  rp.page_log2 = blocks_log2_of(page) + 4;
  rp.n_pages = n_pages;
  rp.max_new = max_new;
  if (launch_qc_resize(rp, stream) != cudaSuccess) return IKBO_ERR_CUDA;
  p->launches++;
  return IKBO_OK;
}

ikbo_status_t ikbo_qcache_append(ikbo_plan_t p, const void* K, const void* V, int64_t row_stride,
                                 const int32_t* d_slots, int n_rows, int H, int d, void* data, int n_pages, int page,
                                 cudaStream_t stream) {
  if (n_rows < 0 || !data || !aligned16(data)) return IKBO_ERR_INVALID_ARG;
  if (d != QC_D) return IKBO_ERR_UNSUPPORTED;
  const ikbo_status_t st = check_cache(n_pages, page, H);
  if (st != IKBO_OK) return st;
  if (n_rows > 0 && (!K || !V || !d_slots)) return IKBO_ERR_INVALID_ARG;
  if (!aligned16(K) || !aligned16(V) || !aligned4(d_slots)) return IKBO_ERR_INVALID_ARG;
  if (row_stride < static_cast<int64_t>(H) * QC_D) return IKBO_ERR_INVALID_ARG;
  if (row_stride % 8 != 0) return IKBO_ERR_UNSUPPORTED;
  if (!p || !plan_device_current(p)) return IKBO_ERR_INVALID_ARG;
  if (n_rows == 0) return IKBO_OK;
  QcAppendParams ap;
  ap.K = static_cast<const uint16_t*>(K);
  ap.V = static_cast<const uint16_t*>(V);
  ap.slots = d_slots;
  ap.data = static_cast<uint8_t*>(data);
  ap.status = p->d_status;
  ap.row_stride = row_stride;
  ap.n_rows = n_rows;
  ap.H = H;
  ap.heads_per_cta = H;
  ap.blocks_log2 = blocks_log2_of(page);
  ap.n_slots = static_cast<int64_t>(n_pages) * page;
  if (launch_qc_append(ap, p->num_sms, stream) != cudaSuccess) return IKBO_ERR_CUDA;
  p->launches++;
  return IKBO_OK;
}

ikbo_status_t ikbo_qcache_load(ikbo_plan_t p, const void* data, int n_pages, int page, int H, int d,
                               const int32_t* d_table, int max_blocks, const int32_t* d_lens, int n_users,
                               const int32_t* d_kv_offsets, void* K, void* V, int n_rows, cudaStream_t stream) {
  if (!data || !aligned16(data) || !d_kv_offsets || !aligned4(d_kv_offsets) || n_rows < 0 || !aligned16(K) ||
      !aligned16(V))
    return IKBO_ERR_INVALID_ARG;
  if (d != QC_D) return IKBO_ERR_UNSUPPORTED;
  ikbo_status_t st = check_cache(n_pages, page, H);
  if (st != IKBO_OK) return st;
  st = check_table(d_table, d_lens, max_blocks, n_users, page);
  if (st != IKBO_OK) return st;
  if (!p || !plan_device_current(p)) return IKBO_ERR_INVALID_ARG;
  if (n_rows == 0 || (!K && !V)) return IKBO_OK;
  QcLoadParams lp;
  std::memset(&lp, 0, sizeof(lp));
  lp.data = static_cast<const uint8_t*>(data);
  lp.table = d_table;
  lp.lens = d_lens;
  lp.kv_offsets = d_kv_offsets;
  lp.K = static_cast<uint16_t*>(K);
  lp.V = static_cast<uint16_t*>(V);
  lp.status = p->d_status;
  lp.n_rows = n_rows;
  lp.n_users = n_users;
  lp.max_blocks = max_blocks;
  lp.n_pages = n_pages;
  lp.blocks_log2 = blocks_log2_of(page);
  lp.H = H;
  if (launch_qc_load(lp, p->num_sms, stream) != cudaSuccess) return IKBO_ERR_CUDA;
  p->launches++;
  return IKBO_OK;
}

// --------------------------------------------------------------- attention
ikbo_status_t ikbo_attn_qcache_forward(ikbo_plan_t p, const void* Q, const void* data, int n_pages, int page,
                                       int H_kv, const int32_t* d_table, int max_blocks, const int32_t* d_lens,
                                       void* O, float* lse, int Lkv, int d, float scale, cudaStream_t stream) {
  const ikbo_status_t st = check_attn(p, Q, data, n_pages, page, H_kv, d_table, max_blocks, d_lens, O, lse, Lkv, d, scale);
  if (st != IKBO_OK) return st;

  const int n_users = p->n_users, group = p->H / H_kv;
  const int64_t rows = static_cast<int64_t>(p->n_cand) * group * p->Lq;  // that read one K/V head, over all users
  const int blocks_log2 = blocks_log2_of(page);

  // (the default stream cannot be captured, and asking took half a microsecond)
  bool capturing = false;
  if (stream && is_capturing(stream, &capturing) != cudaSuccess) return IKBO_ERR_CUDA;
  constexpr size_t ANY = ~size_t{0};

  const QcAttnVariant variant = qattn_variant(rows, n_users, H_kv, Lkv);
  if (variant == QATTN_DECODED) {
    // decode each history once into padded bf16 rows, then the bf16 kernel
    const int64_t cap = decoded_rows(n_users, Lkv);  // (below 2^31: QA_MOST_DECODED)
    const size_t half = static_cast<size_t>(cap) * H_kv * QC_D;
    if (grow_kept<false>(p, &p->qa_kv, 2 * half, QA_MOST_DECODED / sizeof(uint16_t), capturing, stream) != cudaSuccess ||
        grow_kept<false>(p, &p->qa_ranges, 2 * static_cast<size_t>(n_users), ANY, capturing, stream) != cudaSuccess)
      return IKBO_ERR_CUDA;
    QcLoadParams lp;
    std::memset(&lp, 0, sizeof(lp));
    lp.data = static_cast<const uint8_t*>(data);
    lp.table = d_table;
    lp.lens = d_lens;
    lp.ranges = p->qa_ranges.ptr;
    lp.K = p->qa_kv.ptr;
    lp.V = p->qa_kv.ptr + half;
    lp.status = p->d_status;
    lp.n_rows = cap;
    lp.bound = Lkv;
    lp.n_users = n_users;
    lp.max_blocks = max_blocks;
    lp.n_pages = n_pages;
    lp.blocks_log2 = blocks_log2;
    lp.H = H_kv;
    if (launch_qc_load(lp, p->num_sms, stream) != cudaSuccess) return IKBO_ERR_CUDA;
    p->launches++;
    AttnCall c;
    std::memset(&c, 0, sizeof(c));
    c.Q = Q;
    c.K = lp.K;
    c.V = lp.V;
    c.kv_offsets = p->qa_ranges.ptr;
    c.kv_lens = p->qa_ranges.ptr + n_users;
    c.O = O;
    c.lse = lse;
    c.Lkv = static_cast<int>(cap);
    c.d = d;
    c.H_kv = H_kv;
    c.scale = scale;
    // (An ordinary launch, here and below, as launch_qtree needs: it begins when all before it has ended.)
    return attn_launch(p, c, stream);
  }

  const bool few = variant == QATTN_REGISTERS;
  if (!few && qattn_tile_smem() > p->max_smem) return IKBO_ERR_UNSUPPORTED;
  const bool eight = rows <= 8 * static_cast<int64_t>(n_users);  // rows of a register kernel's tile, or 16
  const int ctas = few ? qattn_ctas(p->num_sms, eight) : p->num_sms;
  const size_t part = few ? qattn_part_elems(p->num_sms) : qattn_tile_part_elems(p->num_sms);
  // In registers, warps work alone where there is an item for each; with fewer,
  // a CTA's four share one and join in shared memory.  Measured, four together
  // and alone: 1000 users of 30 to 100 tokens, 8 heads 91 and 52 us, 300 of 150 to
  // 500 56 and 52, 1024 of 600 to 2048 396 and 357; 64 of 1200 to 4096 62 and 64,
  // one of 1000 15 and 23.
  const bool solo = rows * H_kv >= static_cast<int64_t>(eight ? 8 : 16) * 4 * ctas;
  const size_t tickets = std::max(static_cast<size_t>(QA_SLOTS) * p->num_sms * 8, qattn_tickets(p->num_sms));
  const int64_t items = few ? 0 : qattn_tile_items(rows, n_users, H_kv, p->num_sms);
  if (grow_kept<false>(p, &p->qa_part, part, ANY, capturing, stream) != cudaSuccess ||
      grow_kept<true>(p, &p->qa_tickets, tickets, ANY, capturing, stream) != cudaSuccess ||
      (!few && grow_kept<false>(p, &p->qa_list, static_cast<size_t>(items) * 3, ANY, capturing, stream) != cudaSuccess))
    return IKBO_ERR_CUDA;
  QcAttnParams ap;
  std::memset(&ap, 0, sizeof(ap));
  ap.Q = static_cast<const uint16_t*>(Q);
  ap.O = static_cast<uint16_t*>(O);
  ap.lse = lse;
  ap.data = static_cast<const uint8_t*>(data);
  ap.table = d_table;
  ap.lens = d_lens;
  ap.offsets = p->d_offsets;
  ap.perm = p->d_perm;
  ap.part = p->qa_part.ptr;
  ap.tickets = p->qa_tickets.ptr;
  ap.status = p->d_status;
  ap.bound = Lkv;
  ap.n_cand = p->n_cand;
  ap.n_users = n_users;
  ap.H = p->H;
  ap.H_kv = H_kv;
  ap.group = group;
  ap.Lq = p->Lq;
  ap.n_pages = n_pages;
  ap.max_blocks = max_blocks;
  ap.blocks_log2 = blocks_log2;
  ap.ctas = ctas;
  ap.list = p->qa_list.ptr;
  ap.max_items = items;
  ap.scale_log2 = scale * 1.4426950408889634f;
  ap.sixteen = QC_SIXTEEN;
  ap.debug = p->debug;
  ap.timeout_ns = p->timeout_ns;
  // (Ordinary launches: the drafts' kernel behind them, launch_qtree, reads its inputs before they have ended.)
  if ((few ? launch_qattn(ap, eight, solo, stream) : launch_qattn_tile(ap, stream)) != cudaSuccess)
    return IKBO_ERR_CUDA;
  p->launches++;
  return IKBO_OK;
}

ikbo_status_t ikbo_attn_qcache_tree_forward(ikbo_plan_t p, const void* Q, const void* data, int n_pages, int page,
                                            int H_kv, const int32_t* d_table, int max_blocks, const int32_t* d_lens,
                                            const void* K_new, const void* V_new, int64_t row_stride,
                                            const int32_t* d_parents, void* O, float* lse, int Lkv, int d, float scale,
                                            cudaStream_t stream) {
  if (!K_new || !V_new || !aligned16(K_new) || !aligned16(V_new) || !aligned4(d_parents) || !Q || Q == O)
    return IKBO_ERR_INVALID_ARG;
  if (H_kv < 1 || row_stride < static_cast<int64_t>(H_kv) * QC_D) return IKBO_ERR_INVALID_ARG;
  if (row_stride % 8 != 0 || H_kv > TREE_MOST_HEADS) return IKBO_ERR_UNSUPPORTED;
  ikbo_status_t st = check_attn(p, Q, data, n_pages, page, H_kv, d_table, max_blocks, d_lens, O, lse, Lkv, d, scale);
  if (st != IKBO_OK) return st;
  float* hist = lse;
  if (!lse) {  // the history's log-sum-exp has to be somewhere
    bool capturing = false;
    if (stream && is_capturing(stream, &capturing) != cudaSuccess) return IKBO_ERR_CUDA;
    const size_t need = static_cast<size_t>(p->n_cand) * p->H * p->Lq;
    if (grow_kept<false>(p, &p->qa_lse, need, ~size_t{0}, capturing, stream) != cudaSuccess) return IKBO_ERR_CUDA;
    hist = p->qa_lse.ptr;
  }
  st = ikbo_attn_qcache_forward(p, Q, data, n_pages, page, H_kv, d_table, max_blocks, d_lens, O, hist, Lkv, d, scale, stream);
  if (st != IKBO_OK) return st;
  QcTreeParams tp;
  std::memset(&tp, 0, sizeof(tp));
  tp.Q = static_cast<const uint16_t*>(Q);
  tp.K = static_cast<const uint16_t*>(K_new);
  tp.V = static_cast<const uint16_t*>(V_new);
  tp.O = static_cast<uint16_t*>(O);
  tp.hist_lse = hist;
  tp.lse = lse;
  tp.parents = d_parents;
  tp.map = p->d_map;
  tp.status = p->d_status;
  tp.row_stride = row_stride;
  tp.cand_stride = row_stride * p->Lq;
  tp.n_cand = p->n_cand;
  tp.n_users = p->n_users;
  tp.H = p->H;
  tp.H_kv = H_kv;
  tp.group = p->H / H_kv;
  tp.Lq = p->Lq;
  tp.scale_log2 = scale * 1.4426950408889634f;
  if (launch_qtree(tp, p->num_sms, stream) != cudaSuccess) return IKBO_ERR_CUDA;
  p->launches++;
  return IKBO_OK;
}

}  // extern "C"
