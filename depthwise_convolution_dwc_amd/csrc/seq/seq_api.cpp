// seq_api.cpp -- entry points of the sequence-layer operators (extern "C"):
// every argument is checked on the host before anything is launched.
#include <hip/hip_runtime.h>

#include <cmath>

#include "seq_check.h"
#include "seq_chunk.h"
#include "seq_delta.h"
#include "seq_launch.h"

using namespace dwc;
using namespace dwc::seq;

namespace {

int check_norm(const dwc_norm_problem* p, bool bwd) {
  if (!p) return fail(DWC_ERR_BAD_PARAM, "problem pointer is NULL");
  if (p->rows < 0 || p->c < 1) return fail(DWC_ERR_BAD_PARAM, "need rows >= 0 and c >= 1");
  if (!is_type(p->x_dtype) || !is_type(p->y_dtype) || !is_type(p->w_dtype))
    return fail(DWC_ERR_BAD_PARAM, "layer norm types are DWC_F32, DWC_BF16 and DWC_F16");
  if (p->x_stride < p->c || (bwd && p->dy_stride < p->c))
    return fail(DWC_ERR_BAD_PARAM, "row strides must be at least c");
  if (!(p->eps >= 0.f) || std::isinf(p->eps))
    return fail(DWC_ERR_BAD_PARAM, "eps must be finite and >= 0");
  if (p->c > ((int64_t)1 << 31) || p->rows > ((int64_t)1 << 31) || p->x_stride > kMost >> 8 ||
      (bwd && p->dy_stride > kMost >> 8) || p->rows > kMost / p->x_stride ||
      (bwd && p->rows > kMost / p->dy_stride))
    return fail(DWC_ERR_UNSUPPORTED, "layer norm sizes past the index range");
  // a launch has fewer than 2^32 threads; the widest rows take 1024 each
  if (p->rows > (p->c > 512 ? (int64_t)1 << 22 : (int64_t)1 << 26) - 1)
    return fail(DWC_ERR_UNSUPPORTED, "layer norm rows past the launch range");
  // and the sums of dw and db take 64 a column
  if (bwd && p->c >= (int64_t)1 << 25)
    return fail(DWC_ERR_UNSUPPORTED, "layer norm columns past the launch range");
  return DWC_OK;
}

NormArgs norm_args(const dwc_norm_problem* p) {
  NormArgs a{};
  a.rows = p->rows;
  a.c = p->c;
  a.x_stride = p->x_stride;
  a.dy_stride = p->dy_stride;
  a.x_type = p->x_dtype;
  a.y_type = p->y_dtype;
  a.w_type = p->w_dtype;
  a.eps = p->eps;
  return a;
}

int64_t matrix_bytes(int64_t rows, int64_t c, int64_t stride, int type) {
  return rows > 0 ? ((rows - 1) * stride + c) * bytes_of(type) : 0;
}

int check_delta(const dwc_delta_problem* p, int max_dk) {
  if (!p) return fail(DWC_ERR_BAD_PARAM, "problem pointer is NULL");
  if (p->b < 0 || p->l < 0) return fail(DWC_ERR_BAD_PARAM, "need b >= 0 and l >= 0");
  if (p->hk < 1 || p->hv < 1 || p->hv % p->hk)
    return fail(DWC_ERR_BAD_PARAM, "need hk >= 1 and hv a multiple of hk");
  if (p->dk < 1 || p->dv < 1) return fail(DWC_ERR_BAD_PARAM, "need dk >= 1 and dv >= 1");
  if (!is_type(p->dtype))
    return fail(DWC_ERR_BAD_PARAM, "delta rule types are DWC_F32, DWC_BF16 and DWC_F16");
  if (!std::isfinite(p->scale)) return fail(DWC_ERR_BAD_PARAM, "scale must be finite");
  if (p->dk > max_dk || p->dv > 4096)
    return fail(DWC_ERR_UNSUPPORTED, max_dk == 128
                                         ? "the chunked delta rule needs dk <= 128 and dv <= 4096"
                                         : "the delta rule needs dk <= 256 and dv <= 4096");
  // b * l * heads * 4096 stays inside 63 bits; a launch has under 2^32 threads
  if (p->hv > 65536 || p->l > ((int64_t)1 << 30) || p->b > 65535 ||
      p->b * p->hv > ((int64_t)1 << 17) || p->b * p->hv * ((p->l + 63) / 64) > ((int64_t)1 << 24) - 1)
    return fail(DWC_ERR_UNSUPPORTED, "delta rule sizes past the launch range");
  // up to 512 threads for 64 tokens of a head, up to 256 for 16 of its columns
  if (max_dk == 128 && (p->b * p->hv * ((p->l + 63) / 64) >= ((int64_t)1 << 23) ||
                        p->b * p->hv * (((int64_t)p->dv + 15) / 16) >= ((int64_t)1 << 24)))
    return fail(DWC_ERR_UNSUPPORTED, "delta rule sizes past the launch range");
  return DWC_OK;
}

struct DeltaSpans {
  int64_t q, k, v, g, beta, dout, o, s, qk_dense, heads;
};

int delta_spans(const dwc_delta_problem* p, bool bwd, DeltaSpans* n) {
  const int64_t e = bytes_of(p->dtype);
  if (!strided_bytes(p->q_stride, p->b, p->l, p->hk, p->dk, e, &n->q) ||
      !strided_bytes(p->k_stride, p->b, p->l, p->hk, p->dk, e, &n->k) ||
      !strided_bytes(p->v_stride, p->b, p->l, p->hv, p->dv, e, &n->v) ||
      !strided_bytes(p->g_stride, p->b, p->l, p->hv, 1, 4, &n->g) ||
      !strided_bytes(p->beta_stride, p->b, p->l, p->hv, 1, 4, &n->beta) ||
      (bwd && !strided_bytes(p->do_stride, p->b, p->l, p->hv, p->dv, e, &n->dout)))
    return fail(DWC_ERR_BAD_PARAM, "strides must be >= 0 and inside the index range");
  n->o = p->b * p->l * p->hv * p->dv * e;
  n->s = p->b * p->hv * p->dk * p->dv * 4;
  n->qk_dense = p->b * p->l * p->hk * p->dk * e;
  n->heads = p->b * p->l * p->hv * 4;
  return DWC_OK;
}

DeltaArgs delta_args(const dwc_delta_problem* p, const void* q, const void* k, const void* v,
                     const float* g, const float* beta, const float* s0,
                     const int32_t* lengths) {
  DeltaArgs a{};
  a.q = q;
  a.k = k;
  a.v = v;
  a.g = g;
  a.beta = beta;
  a.s0 = s0;
  a.lengths = lengths;
  for (int i = 0; i < 3; ++i) {
    a.q_stride[i] = p->q_stride[i];
    a.k_stride[i] = p->k_stride[i];
    a.v_stride[i] = p->v_stride[i];
    a.g_stride[i] = p->g_stride[i];
    a.beta_stride[i] = p->beta_stride[i];
    a.do_stride[i] = p->do_stride[i];
  }
  a.b = p->b;
  a.l = p->l;
  a.hk = p->hk;
  a.hv = p->hv;
  a.dk = p->dk;
  a.dv = p->dv;
  a.type = p->dtype;
  a.scale = p->scale;
  return a;
}

// The chunked kernels' workspace, laid out from base (null: sizes only).
size_t delta_layout(const dwc_delta_problem* p, bool bwd, char* base, ChunkArgs* c) {
  const int64_t np = p->dtype == DWC_F32 ? 2 : 1;
  const int64_t dp = p->dk <= 64 ? 64 : 128;
  c->nc = (int)((p->l + kChunk - 1) / kChunk);
  c->dvp = (p->dv + 15) / 16 * 16;
  const int64_t nk = p->b * c->nc * p->hk, nv = p->b * c->nc * p->hv;
  const int64_t frags = nk * np * (dp / 8) * 64, tri = nv * kTri * 64;
  size_t at = 0;
  const auto take = [&](auto** field, int64_t bytes) {
    *field = reinterpret_cast<std::remove_reference_t<decltype(*field)>>(base + at);
    at += ((size_t)bytes + 255) & ~(size_t)255;
  };
  take(&c->ka, frags * 16);
  take(&c->kt, frags * 16);
  take(&c->xa, tri * 2 * 16);
  take(&c->gate, nv * (int64_t)sizeof(Gate));
  if (!bwd) {
    take(&c->qa, frags * 16);
    take(&c->pa, tri * 2 * 16);
  } else {
    take(&c->qt, frags * 16);
    take(&c->kk, nk * kLow * 64 * 16);
    take(&c->qk, nk * kLow * 64 * 16);
    take(&c->xt, tri * 2 * 16);
    take(&c->pt, tri * 2 * 16);
    take(&c->states, nv * dp * c->dvp * 4);
    take(&c->dstates, nv * dp * c->dvp * 4);
    take(&c->e, nv * kChunk * c->dvp * 4);
    take(&c->dw, nv * kChunk * c->dvp * 4);
  }
  return at;
}

int run_dropout(const dwc_dropout_problem* p, const void* x, const void* residual, void* y,
                const uint64_t* position, void* stream) {
  if (!p) return fail(DWC_ERR_BAD_PARAM, "problem pointer is NULL");
  if (p->n < 0) return fail(DWC_ERR_BAD_PARAM, "need n >= 0");
  if (!is_type(p->dtype))
    return fail(DWC_ERR_BAD_PARAM, "dropout types are DWC_F32, DWC_BF16 and DWC_F16");
  if (!(p->p >= 0.0 && p->p <= 1.0)) return fail(DWC_ERR_BAD_PARAM, "need 0 <= p <= 1");
  if (p->n > (int64_t)1 << 33)  // a launch has fewer than 2^32 threads
    return fail(DWC_ERR_UNSUPPORTED, "dropout sizes past the launch range");
  if (p->n == 0) return DWC_OK;
  if (!x || !y) return fail(DWC_ERR_BAD_PARAM, "x or y pointer is NULL");
  const int64_t e = bytes_of(p->dtype);
  const Span in[] = {{x, p->n * e, e}, {residual, residual ? p->n * e : 0, e},
                     {position, position ? 8 : 0, 8}};
  const Span out[] = {{y, p->n * e, e}};
  const int st = check_spans(in, out);
  if (st != DWC_OK) return st;
  DropArgs a{};
  a.x = x;
  a.res = residual;
  a.y = y;
  a.n = p->n;
  a.offset = p->offset;
  a.position = position;
  a.key0 = (uint32_t)p->seed;
  a.key1 = (uint32_t)(p->seed >> 32);
  const double t = std::nearbyint(p->p * 4294967296.0);  // ties to even
  a.drop_all = t >= 4294967296.0;
  a.threshold = a.drop_all ? 0xffffffffu : (uint32_t)t;
  a.scale = p->p < 1.0 ? (float)(1.0 / (1.0 - p->p)) : 0.f;
  a.type = p->dtype;
  return hip_result(launch_dropout(a, (hipStream_t)stream), "dropout launch");
}

}  // namespace

extern "C" {

int dwc_layer_norm(const dwc_norm_problem* p, const void* x, const void* w, const void* b,
                   void* y, float* mean, float* rstd, void* stream) {
  int st = check_norm(p, false);
  if (st != DWC_OK) return st;
  if (p->rows == 0) return DWC_OK;
  if (!x || !y) return fail(DWC_ERR_BAD_PARAM, "x or y pointer is NULL");
  if (!mean != !rstd) return fail(DWC_ERR_BAD_PARAM, "mean and rstd are given together or not");
  const int64_t xe = bytes_of(p->x_dtype), ye = bytes_of(p->y_dtype), we = bytes_of(p->w_dtype);
  const Span in[] = {{x, matrix_bytes(p->rows, p->c, p->x_stride, p->x_dtype), xe},
                     {w, w ? p->c * we : 0, we},
                     {b, b ? p->c * we : 0, we}};
  const Span out[] = {{y, p->rows * p->c * ye, ye},
                      {mean, mean ? p->rows * 4 : 0, 4},
                      {rstd, rstd ? p->rows * 4 : 0, 4}};
  st = check_spans(in, out);
  if (st != DWC_OK) return st;
  NormArgs a = norm_args(p);
  a.x = x;
  a.w = w;
  a.b = b;
  a.y = y;
  a.mean = mean;
  a.rstd = rstd;
  return hip_result(launch_norm_fwd(a, (hipStream_t)stream), "dwc_layer_norm launch");
}

int dwc_layer_norm_bwd_workspace_size(const dwc_norm_problem* p, size_t* bytes) {
  const int st = check_norm(p, true);
  if (st != DWC_OK) return st;
  if (!bytes) return fail(DWC_ERR_BAD_PARAM, "bytes pointer is NULL");
  // enough for either layout of the rows: the addresses are not known yet
  NormArgs a = norm_args(p);
  int groups = norm_groups(a, norm_shape(a, true));
  a.x_stride = a.c % 2 ? a.c : a.c + 1;  // no wide loads
  const int narrow = norm_groups(a, norm_shape(a, true));
  if (narrow > groups) groups = narrow;
  *bytes = p->rows > 0 ? (size_t)groups * 2 * (size_t)p->c * 4 : 0;
  return DWC_OK;
}

int dwc_layer_norm_bwd(const dwc_norm_problem* p, const void* dy, const void* x,
                       const float* mean, const float* rstd, const void* w, void* dx, float* dw,
                       float* db, void* workspace, size_t workspace_bytes, void* stream) {
  size_t need = 0;
  int st = dwc_layer_norm_bwd_workspace_size(p, &need);
  if (st != DWC_OK) return st;
  if (p->rows > 0 && (!dy || !x || !mean || !rstd || !dx))
    return fail(DWC_ERR_BAD_PARAM, "dy, x, mean, rstd or dx pointer is NULL");
  if (need > 0 && (!workspace || workspace_bytes < need))
    return fail(DWC_ERR_WORKSPACE, "workspace missing or smaller than required");
  const int64_t xe = bytes_of(p->x_dtype), ye = bytes_of(p->y_dtype), we = bytes_of(p->w_dtype);
  const Span in[] = {{x, matrix_bytes(p->rows, p->c, p->x_stride, p->x_dtype), xe},
                     {dy, matrix_bytes(p->rows, p->c, p->dy_stride, p->y_dtype), ye},
                     {w, w ? p->c * we : 0, we},
                     {mean, p->rows * 4, 4},
                     {rstd, p->rows * 4, 4}};
  const Span out[] = {{dx, p->rows * p->c * xe, xe},
                      {dw, dw ? p->c * 4 : 0, 4},
                      {db, db ? p->c * 4 : 0, 4},
                      {workspace, (int64_t)need, 4}};
  st = check_spans(in, out);
  if (st != DWC_OK) return st;
  NormArgs a = norm_args(p);
  a.x = x;
  a.dy = dy;
  a.w = w;
  a.y = dx;
  a.mean = const_cast<float*>(mean);
  a.rstd = const_cast<float*>(rstd);
  a.part = (float*)workspace;
  a.groups = norm_groups(a, norm_shape(a, true));
  return hip_result(launch_norm_bwd(a, dw, db, (hipStream_t)stream), "dwc_layer_norm_bwd launch");
}

int dwc_dropout(const dwc_dropout_problem* p, const void* x, const void* residual, void* y,
                void* stream) {
  return run_dropout(p, x, residual, y, nullptr, stream);
}

int dwc_dropout_at(const dwc_dropout_problem* p, const void* x, const void* residual, void* y,
                   const uint64_t* position, void* stream) {
  if (!position) return fail(DWC_ERR_BAD_PARAM, "position pointer is NULL");
  return run_dropout(p, x, residual, y, position, stream);
}

int dwc_delta_step(const dwc_delta_problem* p, const void* q, const void* k, const void* v,
                   const float* g, const float* beta, const float* s0, const int32_t* lengths,
                   void* o, float* s1, void* stream) {
  int st = check_delta(p, 256);
  if (st != DWC_OK) return st;
  DeltaSpans n{};
  st = delta_spans(p, false, &n);
  if (st != DWC_OK) return st;
  if (p->b == 0) return DWC_OK;
  if (!s1 || (p->l > 0 && (!q || !k || !v || !g || !beta || !o)))
    return fail(DWC_ERR_BAD_PARAM, "a tensor's pointer is NULL");
  const int64_t e = bytes_of(p->dtype);
  const Span in[] = {{q, n.q, e},       {k, n.k, e}, {v, n.v, e}, {g, n.g, 4},
                     {beta, n.beta, 4}, {s0 == s1 ? nullptr : s0, n.s, 4},
                     {lengths, lengths ? p->b * 4 : 0, 4}};
  const Span out[] = {{o, n.o, e}, {s1, n.s, 4}};
  st = check_spans(in, out);
  if (st != DWC_OK) return st;
  DeltaArgs a = delta_args(p, q, k, v, g, beta, s0, lengths);
  a.o = o;
  a.s1 = s1;
  return hip_result(launch_delta_token(a, (hipStream_t)stream), "dwc_delta_step launch");
}

int dwc_delta_workspace_size(const dwc_delta_problem* p, int op, size_t* bytes) {
  const int st = check_delta(p, 128);
  if (st != DWC_OK) return st;
  if (op != DWC_DELTA_FWD && op != DWC_DELTA_BWD)
    return fail(DWC_ERR_BAD_PARAM, "op must be DWC_DELTA_FWD or DWC_DELTA_BWD");
  if (!bytes) return fail(DWC_ERR_BAD_PARAM, "bytes pointer is NULL");
  ChunkArgs c{};
  *bytes = p->b > 0 && p->l > 0 ? delta_layout(p, op == DWC_DELTA_BWD, nullptr, &c) : 0;
  return DWC_OK;
}

int dwc_delta_fwd(const dwc_delta_problem* p, const void* q, const void* k, const void* v,
                  const float* g, const float* beta, const float* s0, const int32_t* lengths,
                  void* o, float* s1, void* workspace, size_t workspace_bytes, void* stream) {
  size_t need = 0;
  int st = dwc_delta_workspace_size(p, DWC_DELTA_FWD, &need);
  if (st != DWC_OK) return st;
  DeltaSpans n{};
  st = delta_spans(p, false, &n);
  if (st != DWC_OK) return st;
  if (p->b == 0) return DWC_OK;
  if (!s1 || (p->l > 0 && (!q || !k || !v || !g || !beta || !o)))
    return fail(DWC_ERR_BAD_PARAM, "a tensor's pointer is NULL");
  if (need > 0 && (!workspace || workspace_bytes < need))
    return fail(DWC_ERR_WORKSPACE, "workspace missing or smaller than required");
  const int64_t e = bytes_of(p->dtype);
  const Span in[] = {{q, n.q, e},       {k, n.k, e},  {v, n.v, e}, {g, n.g, 4},
                     {beta, n.beta, 4}, {s0, n.s, 4}, {lengths, lengths ? p->b * 4 : 0, 4}};
  const Span out[] = {{o, n.o, e}, {s1, n.s, 4}, {workspace, (int64_t)need, 256}};
  st = check_spans(in, out);
  if (st != DWC_OK) return st;
  ChunkArgs c{};
  c.a = delta_args(p, q, k, v, g, beta, s0, lengths);
  c.a.o = o;
  c.a.s1 = s1;
  const hipStream_t hs = (hipStream_t)stream;
  if (p->l == 0) return hip_result(launch_delta_token(c.a, hs), "dwc_delta_fwd launch");
  delta_layout(p, false, (char*)workspace, &c);
  hipError_t err = launch_delta_prep(c, false, hs);
  if (err == hipSuccess) err = launch_delta_scan(c, false, hs);
  return hip_result(err, "dwc_delta_fwd launch");
}

int dwc_delta_bwd(const dwc_delta_problem* p, const void* dout, const float* ds1, const void* q,
                  const void* k, const void* v, const float* g, const float* beta,
                  const float* s0, const int32_t* lengths, void* dq, void* dk_out, void* dv_out,
                  float* dg, float* dbeta, float* ds0, void* workspace, size_t workspace_bytes,
                  void* stream) {
  size_t need = 0;
  int st = dwc_delta_workspace_size(p, DWC_DELTA_BWD, &need);
  if (st != DWC_OK) return st;
  DeltaSpans n{};
  st = delta_spans(p, true, &n);
  if (st != DWC_OK) return st;
  if (p->b == 0) return DWC_OK;
  if (p->l > 0 && (!dout || !q || !k || !v || !g || !beta || !dq || !dk_out || !dv_out || !dg ||
                   !dbeta))
    return fail(DWC_ERR_BAD_PARAM, "a tensor's pointer is NULL");
  if (need > 0 && (!workspace || workspace_bytes < need))
    return fail(DWC_ERR_WORKSPACE, "workspace missing or smaller than required");
  const int64_t e = bytes_of(p->dtype);
  const Span in[] = {{q, n.q, e},       {k, n.k, e},
                     {v, n.v, e},       {g, n.g, 4},
                     {beta, n.beta, 4}, {s0, n.s, 4},
                     {dout, n.dout, e}, {ds1, n.s, 4},
                     {lengths, lengths ? p->b * 4 : 0, 4}};
  const Span out[] = {{dq, n.qk_dense, e}, {dk_out, n.qk_dense, e}, {dv_out, n.o, e},
                      {dg, n.heads, 4},    {dbeta, n.heads, 4},     {ds0, n.s, 4},
                      {workspace, (int64_t)need, 256}};
  st = check_spans(in, out);
  if (st != DWC_OK) return st;
  ChunkArgs c{};
  c.a = delta_args(p, q, k, v, g, beta, s0, lengths);
  c.a.dout = dout;
  c.a.ds1 = ds1;
  c.a.dq = dq;
  c.a.dk_out = dk_out;
  c.a.dv_out = dv_out;
  c.a.dg = dg;
  c.a.dbeta = dbeta;
  c.a.ds0 = ds0;
  const hipStream_t hs = (hipStream_t)stream;
  hipError_t err = hipSuccess;
  delta_layout(p, true, (char*)workspace, &c);
  if (p->l == 0) {  // the state passes through, and its gradient
    if (ds0) err = launch_delta_scan(c, true, hs);
    return hip_result(err, "dwc_delta_bwd launch");
  }
  err = launch_delta_prep(c, true, hs);
  if (err == hipSuccess) err = launch_delta_scan(c, true, hs);
  if (err == hipSuccess) err = launch_delta_grad(c, hs);
  return hip_result(err, "dwc_delta_bwd launch");
}

}  // extern "C"
