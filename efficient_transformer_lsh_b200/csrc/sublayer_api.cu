// C ABI of the sublayer operators (norms, residual add, dropout, rotary
// positions): argument checks and dispatch.
#include <algorithm>
#include <cmath>
#include <initializer_list>

#include "internal.h"
#include "sublayer.h"

namespace lsh {
namespace {

// Rows (b, h, l) and tokens (b, l) are counted in 32 bits with room for one
// grid's stride beyond the last.
constexpr int64_t kMaxRows = 1 << 30;
constexpr int64_t kMaxStride = (int64_t)1 << 44;
constexpr int kMaxHead = 1 << 16;

bool is_aligned(const void* p, size_t a) { return (uintptr_t)p % a == 0; }
bool all_aligned(std::initializer_list<const void*> ps, size_t a) {
  for (const void* p : ps)
    if (!is_aligned(p, a)) return false;
  return true;
}
lsh_status from_cuda(cudaError_t e) { return e == cudaSuccess ? LSH_OK : LSH_ERR_CUDA; }

lsh_status check_sizes(int B, int H, int L, int d, int dtype) {
  if (B < 0 || H < 0 || L < 0 || d < 1) return LSH_ERR_INVALID_ARG;
  if (dtype != LSH_F32 && dtype != LSH_BF16) return LSH_ERR_INVALID_ARG;
  if (d > kMaxHead || (int64_t)H * d > (int64_t)INT32_MAX) return LSH_ERR_UNSUPPORTED;
  if ((int64_t)B * L > kMaxRows) return LSH_ERR_UNSUPPORTED;
  if ((int64_t)B * L > 0 && (int64_t)H > kMaxRows / ((int64_t)B * L)) return LSH_ERR_UNSUPPORTED;
  return LSH_OK;
}

// Resolves strides (all zero: contiguous); dimensions of one element get
// stride 0. False if two elements would share an address.
bool resolve(int B, int H, int L, int d, const lsh_strides& in, lsh_strides* out) {
  if (in.b == 0 && in.h == 0 && in.l == 0) {
    *out = {(int64_t)H * L * d, (int64_t)L * d, d};
  } else {
    *out = in;
  }
  struct Dim {
    int64_t n, s;
  } v[3] = {{B, out->b}, {H, out->h}, {L, out->l}};
  if (B <= 1) out->b = 0;
  if (H <= 1) out->h = 0;
  if (L <= 1) out->l = 0;
  if ((int64_t)B * H * L == 0) return true;
  std::sort(v, v + 3, [](const Dim& a, const Dim& b) { return a.s < b.s; });
  int64_t span = d;
  for (const Dim& m : v) {
    if (m.n <= 1) continue;
    if (m.s < span || m.s > kMaxStride) return false;
    span += m.s * (m.n - 1);
  }
  return true;
}

bool stride_multiple(const lsh_strides& s, int64_t n) {
  return s.b % n == 0 && s.h % n == 0 && s.l % n == 0;
}

// Whether every access of 8 features is aligned to 16 bytes.
bool wide_ok(int d, int dtype, std::initializer_list<const lsh_strides*> strides,
             std::initializer_list<const void*> ps) {
  const int64_t n = dtype == LSH_BF16 ? 8 : 4;
  if (d % 8 != 0) return false;
  for (const lsh_strides* s : strides)
    if (!stride_multiple(*s, n)) return false;
  return all_aligned(ps, 16);
}

bool drop_of(float p, uint32_t* t, float* scale) {
  if (!(p >= 0.f && p <= 1.f)) return false;
  *t = (uint32_t)std::nearbyint((double)p * 65536.0);
  *scale = *t < 65536u ? (float)(65536.0 / (65536.0 - *t)) : 0.f;
  return true;
}
bool slice_ok(int64_t s) { return s >= 0 && s <= (int64_t)INT32_MAX; }
bool kind_ok(int k) { return k == LSH_NORM_LAYER || k == LSH_NORM_RMS; }
bool eps_ok(float e) { return std::isfinite(e) && e > 0.f; }
size_t esize(int dtype) { return dtype == LSH_BF16 ? 2 : 4; }

lsh_status norm_call(const lsh_norm_problem* n, SubCall* c) {
  if (!n) return LSH_ERR_INVALID_ARG;
  lsh_status st = check_sizes(n->B, n->H, n->L, n->d, n->dtype);
  if (st != LSH_OK) return st;
  if (!kind_ok(n->kind) || !eps_ok(n->eps)) return LSH_ERR_INVALID_ARG;
  *c = SubCall{};
  if (!resolve(n->B, n->H, n->L, n->d, n->x, &c->sx) ||
      !resolve(n->B, n->H, n->L, n->d, n->h, &c->sh))
    return LSH_ERR_INVALID_ARG;
  if ((int64_t)n->H * n->d > kNormMaxD) return LSH_ERR_UNSUPPORTED;
  c->B = n->B, c->H = n->H, c->L = n->L, c->d = n->d, c->dtype = n->dtype;
  c->norm = n->kind, c->eps = n->eps, c->beta = 1.f;
  return LSH_OK;
}

lsh_status residual_call(const lsh_residual_problem* q, SubCall* c) {
  if (!q) return LSH_ERR_INVALID_ARG;
  lsh_status st = check_sizes(q->B, q->H, q->L, q->d, q->dtype);
  if (st != LSH_OK) return st;
  *c = SubCall{};
  if ((q->post != LSH_NORM_NONE && (!kind_ok(q->post) || !eps_ok(q->eps_post))) ||
      (q->norm != LSH_NORM_NONE && (!kind_ok(q->norm) || !eps_ok(q->eps))))
    return LSH_ERR_INVALID_ARG;
  if (q->gate < LSH_GATE_NONE || q->gate > LSH_GATE_SIGMOID) return LSH_ERR_INVALID_ARG;
  if (q->gate_batch != 0 && (q->gate_batch != 1 || q->gate != LSH_GATE_VECTOR))
    return LSH_ERR_INVALID_ARG;
  if (!std::isfinite(q->alpha) || !std::isfinite(q->beta) || !slice_ok(q->slice0) ||
      !drop_of(q->p, &c->drop_t, &c->drop_scale))
    return LSH_ERR_INVALID_ARG;
  if (!resolve(q->B, q->H, q->L, q->d, q->x, &c->sx) ||
      !resolve(q->B, q->H, q->L, q->d, q->f, &c->sf))
    return LSH_ERR_INVALID_ARG;
  if ((int64_t)q->H * q->d > kNormMaxD) return LSH_ERR_UNSUPPORTED;
  c->sh = c->sx;
  c->B = q->B, c->H = q->H, c->L = q->L, c->d = q->d, c->dtype = q->dtype;
  c->post = q->post, c->norm = q->norm, c->gate = q->gate, c->gate_batch = q->gate_batch;
  c->eps_post = q->eps_post, c->eps = q->eps, c->alpha = q->alpha, c->beta = q->beta;
  c->slice0 = q->slice0;
  c->branch = true;
  return LSH_OK;
}

}  // namespace
}  // namespace lsh

using namespace lsh;

extern "C" {

lsh_status lsh_norm_fwd(const lsh_norm_problem* n, const void* x, const float* w, const float* b,
                        void* h, lsh_stream_t stream) {
  SubCall c;
  lsh_status st = norm_call(n, &c);
  if (st != LSH_OK) return st;
  if ((int64_t)n->B * n->H * n->L == 0) return LSH_OK;
  if (!x || !h) return LSH_ERR_INVALID_ARG;
  if (!all_aligned({x, h}, esize(n->dtype)) || !all_aligned({w, b}, 4)) return LSH_ERR_INVALID_ARG;
  c.x = x, c.w = w, c.b = b, c.h = h;
  c.wide = wide_ok(n->d, n->dtype, {&c.sx, &c.sh}, {x, h, w, b});
  return from_cuda(launch_sub_fwd(c, (cudaStream_t)stream));
}

size_t lsh_norm_bwd_workspace_size(const lsh_norm_problem* n) {
  SubCall c;
  if (norm_call(n, &c) != LSH_OK) return 0;
  return sub_bwd_ws_bytes(n->B, n->H, n->L, n->d, false, false);
}

lsh_status lsh_norm_bwd(const lsh_norm_problem* n, const void* x, const float* w, const void* dh,
                        const void* dres, void* dx, float* dw, float* db, void* ws,
                        size_t ws_bytes, lsh_stream_t stream) {
  SubCall c;
  lsh_status st = norm_call(n, &c);
  if (st != LSH_OK) return st;
  if (n->H == 0) return LSH_OK;
  const bool empty = (int64_t)n->B * n->L == 0;
  if (!empty && (!x || !dh || !dx)) return LSH_ERR_INVALID_ARG;
  if (!all_aligned({x, dh, dres, dx}, esize(n->dtype)) || !all_aligned({w, dw, db}, 4))
    return LSH_ERR_INVALID_ARG;
  if (!empty && (dw || db) &&
      (!ws || ws_bytes < sub_bwd_ws_bytes(n->B, n->H, n->L, n->d, false, false) ||
       !is_aligned(ws, 256)))
    return LSH_ERR_WORKSPACE;
  c.x = x, c.w = w, c.dh = dh, c.dy = dres, c.dx = dx, c.dw = dw, c.db = db;
  c.wide = wide_ok(n->d, n->dtype, {&c.sx, &c.sh}, {x, dh, dres, dx, w});
  return from_cuda(launch_sub_bwd(c, ws, (cudaStream_t)stream));
}

lsh_status lsh_dropout_fwd(const lsh_dropout_problem* q, const void* x, uint64_t seed,
                           uint64_t offset, const uint64_t* counter, void* y,
                           lsh_stream_t stream) {
  if (!q) return LSH_ERR_INVALID_ARG;
  lsh_status st = check_sizes(q->B, q->H, q->L, q->d, q->dtype);
  if (st != LSH_OK) return st;
  uint32_t t;
  float scale;
  lsh_dropout_problem r = *q;
  if (!drop_of(q->p, &t, &scale) || !slice_ok(q->slice0) ||
      !resolve(q->B, q->H, q->L, q->d, q->x, &r.x) || !resolve(q->B, q->H, q->L, q->d, q->y, &r.y))
    return LSH_ERR_INVALID_ARG;
  if ((int64_t)q->B * q->H * q->L == 0) return LSH_OK;
  if (!x || !y || !all_aligned({x, y}, esize(q->dtype)) || !is_aligned(counter, 8))
    return LSH_ERR_INVALID_ARG;
  return from_cuda(launch_dropout(r, t, scale, x, seed, offset, counter, y,
                                  wide_ok(q->d, q->dtype, {&r.x, &r.y}, {x, y}),
                                  (cudaStream_t)stream));
}

lsh_status lsh_residual_fwd(const lsh_residual_problem* q, const void* x, const void* f,
                            const void* gate, const float* w_post, const float* b_post,
                            const float* w, const float* b, uint64_t seed, uint64_t offset,
                            const uint64_t* counter, void* y, void* h, lsh_stream_t stream) {
  SubCall c;
  lsh_status st = residual_call(q, &c);
  if (st != LSH_OK) return st;
  if ((int64_t)q->B * q->H * q->L == 0) return LSH_OK;
  if (!x || !f || !y || (q->gate != LSH_GATE_NONE && !gate) ||
      (q->norm != LSH_NORM_NONE && !h))
    return LSH_ERR_INVALID_ARG;
  const void* z = q->gate == LSH_GATE_SIGMOID ? gate : nullptr;
  const void* gv = q->gate == LSH_GATE_VECTOR ? gate : nullptr;
  if (q->post == LSH_NORM_NONE) w_post = b_post = nullptr;
  if (q->norm == LSH_NORM_NONE) w = b = nullptr, h = nullptr;
  if (!all_aligned({x, f, z, y, h}, esize(q->dtype)) ||
      !all_aligned({gv, w_post, b_post, w, b}, 4) || !is_aligned(counter, 8))
    return LSH_ERR_INVALID_ARG;
  c.x = x, c.f = f, c.gatep = q->gate == LSH_GATE_NONE ? nullptr : gate;
  c.wp = w_post, c.bp = b_post, c.w = w, c.b = b;
  c.seed = seed, c.offset = offset, c.counter = c.drop_t ? counter : nullptr;
  c.y = y, c.h = h;
  c.wide = wide_ok(q->d, q->dtype, {&c.sx, &c.sf}, {x, f, gate, w_post, b_post, w, b, y, h});
  return from_cuda(launch_sub_fwd(c, (cudaStream_t)stream));
}

size_t lsh_residual_bwd_workspace_size(const lsh_residual_problem* q) {
  SubCall c;
  if (residual_call(q, &c) != LSH_OK) return 0;
  return sub_bwd_ws_bytes(q->B, q->H, q->L, q->d, true, q->gate_batch != 0);
}

lsh_status lsh_residual_bwd(const lsh_residual_problem* q, const void* dy, const void* dh,
                            const void* y, const void* f, const void* gate, const float* w_post,
                            const float* b_post, const float* w, uint64_t seed, uint64_t offset,
                            const uint64_t* counter, void* dx, void* df, void* dgate,
                            float* dw_post, float* db_post, float* dw, float* db, void* ws,
                            size_t ws_bytes, lsh_stream_t stream) {
  SubCall c;
  lsh_status st = residual_call(q, &c);
  if (st != LSH_OK) return st;
  if (q->H == 0) return LSH_OK;
  const bool empty = (int64_t)q->B * q->L == 0;
  const bool norm = q->norm != LSH_NORM_NONE, post = q->post != LSH_NORM_NONE;
  if (!empty && (!f || !df || (q->gate != LSH_GATE_NONE && !gate) || (norm ? !y || !dh : !dy)))
    return LSH_ERR_INVALID_ARG;
  if (!norm) y = dh = nullptr, w = nullptr;
  if (!post) w_post = b_post = nullptr;
  // gradients of what is not there are refused, not left unwritten
  if ((!norm && (dw || db)) || (!post && (dw_post || db_post)) ||
      (q->gate == LSH_GATE_NONE && dgate))
    return LSH_ERR_INVALID_ARG;
  const bool sig = q->gate == LSH_GATE_SIGMOID, vec = q->gate == LSH_GATE_VECTOR;
  if (!all_aligned({dy, dh, y, f, sig ? gate : nullptr, dx, df, sig ? dgate : nullptr},
                   esize(q->dtype)) ||
      !all_aligned({vec ? gate : nullptr, vec ? dgate : nullptr, w_post, b_post, w, dw_post,
                    db_post, dw, db}, 4) ||
      !is_aligned(counter, 8))
    return LSH_ERR_INVALID_ARG;
  const bool sums = (vec && dgate) || dw_post || db_post || dw || db;
  if (!empty && sums &&
      (!ws || ws_bytes < sub_bwd_ws_bytes(q->B, q->H, q->L, q->d, true, q->gate_batch != 0) ||
       !is_aligned(ws, 256)))
    return LSH_ERR_WORKSPACE;
  c.dy = dy, c.dh = dh, c.x = y, c.f = f;
  c.gatep = q->gate == LSH_GATE_NONE ? nullptr : gate;
  c.wp = w_post, c.bp = b_post, c.w = w;
  c.seed = seed, c.offset = offset, c.counter = c.drop_t ? counter : nullptr;
  c.dx = dx, c.df = df;
  c.dz = sig ? dgate : nullptr, c.dgate = vec ? (float*)dgate : nullptr;
  c.dwp = dw_post, c.dbp = db_post, c.dw = dw, c.db = db;
  c.wide = wide_ok(q->d, q->dtype, {&c.sx, &c.sf},
                   {dy, dh, y, f, gate, w_post, b_post, w, dx, df, c.dz});
  return from_cuda(launch_sub_bwd(c, ws, (cudaStream_t)stream));
}

// Pairs of one access: the most that divides the pairs and the copied rest
// and that pointers and strides allow (at most `most` bytes at once).
static int rope_pairs(const lsh_rope_problem* q, const lsh_strides& x, const lsh_strides& y,
                      const void* in, const void* out, int most = 16) {
  const int64_t es = (int64_t)esize(q->dtype);
  const int per = q->interleaved ? 2 : 1;
  for (int vp = (int)(most / es) / per; vp > 1; vp /= 2) {
    const int64_t n = vp * per;
    if ((q->rot / 2) % vp == 0 && (q->d - q->rot) % (2 * vp) == 0 && stride_multiple(x, n) &&
        stride_multiple(y, n) && is_aligned(in, n * es) && is_aligned(out, n * es))
      return vp;
  }
  return 1;
}

static lsh_status check_rope(const lsh_rope_problem* q, int least) {
  if (!q) return LSH_ERR_INVALID_ARG;
  lsh_status st = check_sizes(q->B, q->H, q->L, q->d, q->dtype);
  if (st != LSH_OK) return st;
  if (q->rot < least || q->rot % 2 != 0 || q->rot > q->d || q->d % 2 != 0)
    return LSH_ERR_INVALID_ARG;
  if ((q->interleaved | 1) != 1 || (q->pos_batch | 1) != 1 || !std::isfinite(q->amp))
    return LSH_ERR_INVALID_ARG;
  return LSH_OK;
}

static lsh_status rope_run(const lsh_rope_problem* q, const void* in, const uint64_t* turns,
                           const int32_t* pos, int64_t pos0, void* out, bool inverse,
                           lsh_stream_t stream) {
  lsh_status st = check_rope(q, 2);
  if (st != LSH_OK) return st;
  lsh_strides x, y;
  if (!resolve(q->B, q->H, q->L, q->d, q->x, &x) || !resolve(q->B, q->H, q->L, q->d, q->y, &y))
    return LSH_ERR_INVALID_ARG;
  if (q->d > kRopeMaxHead) return LSH_ERR_UNSUPPORTED;
  if ((int64_t)q->B * q->H * q->L == 0) return LSH_OK;
  if (!in || !out || !turns || !all_aligned({in, out}, esize(q->dtype)) ||
      !is_aligned(turns, 8) || !is_aligned(pos, 4))
    return LSH_ERR_INVALID_ARG;
  if (inverse) std::swap(x, y);
  return from_cuda(launch_rope(*q, x, y, in, turns, pos, pos0, out, inverse,
                               rope_pairs(q, x, y, in, out), (cudaStream_t)stream));
}

lsh_status lsh_rope_fwd(const lsh_rope_problem* q, const void* x, const uint64_t* turns,
                        const int32_t* pos, int64_t pos0, void* y, lsh_stream_t stream) {
  return rope_run(q, x, turns, pos, pos0, y, false, stream);
}

lsh_status lsh_rope_bwd_sum(const lsh_rope_problem* q, const float* dqk, const float* dv,
                            const uint64_t* turns, const int32_t* pos, int64_t pos0, void* dx,
                            lsh_stream_t stream) {
  lsh_status st = check_rope(q, 0);
  if (st != LSH_OK) return st;
  lsh_strides x;
  if (!resolve(q->B, q->H, q->L, q->d, q->x, &x)) return LSH_ERR_INVALID_ARG;
  if (q->d > kRopeMaxHead) return LSH_ERR_UNSUPPORTED;
  if ((int64_t)q->B * q->H * q->L == 0) return LSH_OK;
  if (!dqk || !dv || !dx || (q->rot && !turns) || !is_aligned(dx, esize(q->dtype)) ||
      !all_aligned({dqk, dv, pos}, 4) || !is_aligned(turns, 8))
    return LSH_ERR_INVALID_ARG;
  // the float32 side's accesses decide the width: four features at once
  lsh_rope_problem f = *q;
  f.dtype = LSH_F32;
  lsh_strides c;
  resolve(q->B, q->H, q->L, q->d, {0, 0, 0}, &c);
  const int vp = std::min(rope_pairs(&f, c, c, dqk, dv), rope_pairs(q, x, x, dx, dx, 4 * (int)esize(q->dtype)));
  return from_cuda(launch_rope_sum(*q, x, dqk, dv, turns, pos, pos0, dx, vp, (cudaStream_t)stream));
}

lsh_status lsh_rope_bwd(const lsh_rope_problem* q, const void* dy, const uint64_t* turns,
                        const int32_t* pos, int64_t pos0, void* dx, lsh_stream_t stream) {
  return rope_run(q, dy, turns, pos, pos0, dx, true, stream);
}

}  // extern "C"
