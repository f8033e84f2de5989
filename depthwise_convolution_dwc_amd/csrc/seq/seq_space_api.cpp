// seq_space_api.cpp -- entry points of the short causal convolution, the
// selective state space scan and the residual norm (extern "C"): every
// argument is checked on the host before anything is launched.
#include <hip/hip_runtime.h>

#include <cmath>

#include "seq_check.h"
#include "seq_space.h"

using namespace dwc;
using namespace dwc::seq;

namespace {

constexpr int64_t kLanes = (int64_t)1 << 32;  // a launch has fewer threads

bool token_bytes(const int64_t* stride, int64_t b, int64_t l, int64_t d, int64_t e,
                 int64_t* bytes) {
  const int64_t s[3] = {stride[0], stride[1], 0};
  return strided_bytes(s, b, l, 1, d, e, bytes);
}

// ---- short causal convolution -------------------------------------------

int check_conv(const dwc_causal_conv_problem* p, bool bwd) {
  if (!p) return fail(DWC_ERR_BAD_PARAM, "problem pointer is NULL");
  if (p->b < 0 || p->l < 0 || p->d < 1)
    return fail(DWC_ERR_BAD_PARAM, "need b >= 0, l >= 0 and d >= 1");
  if (!is_type(p->dtype) || !is_type(p->w_dtype))
    return fail(DWC_ERR_BAD_PARAM, "causal convolution types are DWC_F32, DWC_BF16 and DWC_F16");
  if (p->act != DWC_ACT_NONE && p->act != DWC_ACT_SILU)
    return fail(DWC_ERR_BAD_PARAM, "act must be DWC_ACT_NONE or DWC_ACT_SILU");
  if (p->taps < 1) return fail(DWC_ERR_BAD_PARAM, "need taps >= 1");
  if (p->taps > kMostTaps) return fail(DWC_ERR_UNSUPPORTED, "the causal convolution has up to 8 taps");
  // b l d stays inside 63 bits; a lane takes at least 8 tokens of a channel,
  // 64 channels a wave in the backward pass
  if (p->b > 65535 || p->l > (int64_t)1 << 30 || p->d > (int64_t)1 << 24 ||
      p->b * ((p->l + 31) / 32 + 1) * 4 >= kLanes / ((p->d + 63) / 64 * 64))
    return fail(DWC_ERR_UNSUPPORTED, "causal convolution sizes past the launch range");
  int64_t n = 0;
  if (!token_bytes(p->x_stride, p->b, p->l, p->d, 4, &n) ||
      (bwd && !token_bytes(p->dy_stride, p->b, p->l, p->d, 4, &n)))
    return fail(DWC_ERR_BAD_PARAM, "strides must be >= 0 and inside the index range");
  return DWC_OK;
}

ConvArgs conv_args(const dwc_causal_conv_problem* p, const void* x, const void* w,
                   const void* bias, const void* s0, const int32_t* lengths) {
  ConvArgs a{};
  a.x = x;
  a.w = w;
  a.bias = bias;
  a.s0 = p->taps > 1 ? s0 : nullptr;
  a.lengths = lengths;
  for (int i = 0; i < 2; ++i) {
    a.x_stride[i] = p->x_stride[i];
    a.dy_stride[i] = p->dy_stride[i];
  }
  a.b = p->b;
  a.l = p->l;
  a.d = p->d;
  a.taps = p->taps;
  a.type = p->dtype;
  a.w_type = p->w_dtype;
  a.silu = p->act == DWC_ACT_SILU;
  return a;
}

void conv_split(ConvArgs* a, bool bwd) {
  a->strip = conv_strip(*a, bwd);
  a->strips = (int)((a->l + a->strip - 1) / a->strip);
  if (a->strips < 1) a->strips = 1;
}

int run_conv(const dwc_causal_conv_problem* p, const void* x, const void* w, const void* bias,
             const void* s0, const int32_t* lengths, void* y, void* s1, bool step, void* stream) {
  int st = check_conv(p, false);
  if (st != DWC_OK) return st;
  if (p->b == 0) return DWC_OK;
  if (!w || (p->l > 0 && (!x || !y))) return fail(DWC_ERR_BAD_PARAM, "x, w or y pointer is NULL");
  const int64_t e = bytes_of(p->dtype), we = bytes_of(p->w_dtype);
  const int64_t state = p->b * (p->taps - 1) * p->d * e;
  int64_t xb = 0;
  token_bytes(p->x_stride, p->b, p->l, p->d, e, &xb);
  const Span in[] = {{x, xb, e},
                     {w, p->taps * p->d * we, we},
                     {bias, bias ? p->d * we : 0, we},
                     {step && s0 == s1 ? nullptr : s0, state, e},
                     {lengths, lengths ? p->b * 4 : 0, 4}};
  const Span out[] = {{y, p->b * p->l * p->d * e, e}, {s1, state, e}};
  st = check_spans(in, out);
  if (st != DWC_OK) return st;
  ConvArgs a = conv_args(p, x, w, bias, s0, lengths);
  a.y = y;
  a.s1 = s1;
  conv_split(&a, false);
  if (step) {  // one lane reads and writes a channel's state
    if (p->l > (int64_t)1 << 20)
      return fail(DWC_ERR_UNSUPPORTED, "the token form takes up to 2^20 tokens");
    a.strip = (int)(p->l > 0 ? p->l : 1);
    a.strips = 1;
  }
  return hip_result(launch_conv_fwd(a, (hipStream_t)stream), "dwc_causal_conv launch");
}

// ---- selective scan -----------------------------------------------------

int check_scan(const dwc_scan_problem* p) {
  if (!p) return fail(DWC_ERR_BAD_PARAM, "problem pointer is NULL");
  if (p->b < 0 || p->l < 0) return fail(DWC_ERR_BAD_PARAM, "need b >= 0 and l >= 0");
  if (p->d < 1 || p->n < 1 || p->g < 1 || p->d % p->g)
    return fail(DWC_ERR_BAD_PARAM, "need d >= 1, n >= 1, g >= 1 and d a multiple of g");
  if (!is_type(p->dtype))
    return fail(DWC_ERR_BAD_PARAM, "scan types are DWC_F32, DWC_BF16 and DWC_F16");
  if (p->softplus != 0 && p->softplus != 1) return fail(DWC_ERR_BAD_PARAM, "softplus must be 0 or 1");
  if (p->n > 256) return fail(DWC_ERR_UNSUPPORTED, "the scan has up to 256 states a channel");
  if (p->b > 65535 || p->l > (int64_t)1 << 30 || p->d > 1 << 22)
    return fail(DWC_ERR_UNSUPPORTED, "scan sizes past the index range");
  const int64_t e = 4;
  int64_t n = 0;
  if (!token_bytes(p->u_stride, p->b, p->l, p->d, e, &n) ||
      !token_bytes(p->delta_stride, p->b, p->l, p->d, e, &n) ||
      !token_bytes(p->z_stride, p->b, p->l, p->d, e, &n) ||
      !token_bytes(p->dy_stride, p->b, p->l, p->d, e, &n) ||
      !strided_bytes(p->b_stride, p->b, p->l, p->g, p->n, e, &n) ||
      !strided_bytes(p->c_stride, p->b, p->l, p->g, p->n, e, &n))
    return fail(DWC_ERR_BAD_PARAM, "strides must be >= 0 and inside the index range");
  // 64 lanes a token form's channel of 256 states
  const int64_t np = (p->n + 3) / 4;
  if (p->b * p->d >= kLanes / 2 / (np * 2))
    return fail(DWC_ERR_UNSUPPORTED, "scan sizes past the launch range");
  return DWC_OK;
}

ScanArgs scan_args(const dwc_scan_problem* p, const void* u, const void* delta, const float* A,
                   const void* B, const void* C, const float* D, const void* z, const float* bias,
                   const float* s0, const int32_t* lengths) {
  ScanArgs a{};
  a.u = u;
  a.delta = delta;
  a.z = z;
  a.bm = B;
  a.cm = C;
  a.a = A;
  a.skip = D;
  a.bias = bias;
  a.s0 = s0;
  a.lengths = lengths;
  for (int i = 0; i < 2; ++i) {
    a.u_stride[i] = p->u_stride[i];
    a.delta_stride[i] = p->delta_stride[i];
    a.z_stride[i] = p->z_stride[i];
    a.dy_stride[i] = p->dy_stride[i];
  }
  for (int i = 0; i < 3; ++i) {
    a.b_stride[i] = p->b_stride[i];
    a.c_stride[i] = p->c_stride[i];
  }
  a.b = p->b;
  a.l = p->l;
  a.d = p->d;
  a.n = p->n;
  a.g = p->g;
  a.dg = p->d / p->g;
  a.type = p->dtype;
  a.softplus = p->softplus;
  return a;
}

// The workspace, laid out from base (null: sizes only); 0 on sizes past the
// launch range.
int scan_layout(ScanArgs* a, bool bwd, char* base, size_t* bytes) {
  scan_split(a, bwd);
  const int64_t line = (int64_t)a->nblk * 2 * a->spl, np = (int64_t)a->nblk * a->spl;
  const int64_t tokens = a->b * a->lp, rows = a->b * a->nc;
  const int64_t pairs = (a->dg + kGradChannels - 1) / kGradChannels;
  // threads of the widest launches, and the index range
  if (tokens > kMost / (a->g * line) || tokens * a->g * line >= kLanes / 2 ||
      rows >= kLanes / 64 / ((int64_t)a->g * a->cblk * a->nblk) ||
      (a->nc > 1 && a->b * np * ((a->d + 63) / 64) >= kLanes / 128) ||
      (a->one && a->b * a->g * a->cblk >= kLanes / 1024) ||
      (bwd && (rows >= kLanes / 256 / ((int64_t)a->g * pairs * a->nblk) ||
               (int64_t)a->n * a->d * 64 >= kLanes / 2 || rows >= kLanes / a->d)))
    return fail(DWC_ERR_UNSUPPORTED, "scan sizes past the launch range");
  size_t at = 0;
  const auto take = [&](float** field, int64_t floats) {
    *field = reinterpret_cast<float*>(base + at);
    at += ((size_t)floats * 4 + 255) & ~(size_t)255;
  };
  take(&a->a2, np * a->d);
  take(&a->bc, tokens * a->g * line);
  if (a->nc > 1) {
    take(&a->states, rows * np * a->d);
    take(&a->dts, rows * a->d);
    if (bwd) take(&a->rstates, rows * np * a->d);
  }
  if (bwd) {
    take(&a->bcpart, pairs * tokens * a->g * line);
    take(&a->apart, rows * np * a->d);
    take(&a->dpart, rows * 2 * a->d);
    if (a->gblk > 1) take(&a->sums, 3 * a->gblk * tokens * a->d);
  }
  *bytes = at;
  return DWC_OK;
}

struct ScanSpans {
  int64_t u, delta, z, dy, b, c, dense, bc, state, vec;
};

ScanSpans scan_spans(const dwc_scan_problem* p) {
  ScanSpans n{};
  const int64_t e = bytes_of(p->dtype);
  token_bytes(p->u_stride, p->b, p->l, p->d, e, &n.u);
  token_bytes(p->delta_stride, p->b, p->l, p->d, e, &n.delta);
  token_bytes(p->z_stride, p->b, p->l, p->d, e, &n.z);
  token_bytes(p->dy_stride, p->b, p->l, p->d, e, &n.dy);
  strided_bytes(p->b_stride, p->b, p->l, p->g, p->n, e, &n.b);
  strided_bytes(p->c_stride, p->b, p->l, p->g, p->n, e, &n.c);
  n.dense = p->b * p->l * p->d * e;
  n.bc = p->b * p->l * p->g * p->n * e;
  n.state = p->b * p->d * p->n * 4;
  n.vec = (int64_t)p->d * 4;
  return n;
}

// ---- residual norm ------------------------------------------------------

int check_resnorm(const dwc_resnorm_problem* p, bool bwd) {
  if (!p) return fail(DWC_ERR_BAD_PARAM, "problem pointer is NULL");
  if (p->rows < 0 || p->c < 1) return fail(DWC_ERR_BAD_PARAM, "need rows >= 0 and c >= 1");
  if (!is_type(p->x_dtype) || !is_type(p->y_dtype) || !is_type(p->w_dtype))
    return fail(DWC_ERR_BAD_PARAM, "residual norm types are DWC_F32, DWC_BF16 and DWC_F16");
  if (p->x_dtype != DWC_F32 && p->x_dtype != p->y_dtype)
    return fail(DWC_ERR_BAD_PARAM, "x must be fp32 or of y's type");
  if (p->act < DWC_GATE_NONE || p->act > DWC_GATE_SIGMOID)
    return fail(DWC_ERR_BAD_PARAM, "act must be a DWC_GATE value");
  if ((p->post != 0 && p->post != 1) || (p->pre != 0 && p->pre != 1))
    return fail(DWC_ERR_BAD_PARAM, "post and pre must be 0 or 1");
  if (!(p->eps >= 0.f) || std::isinf(p->eps))
    return fail(DWC_ERR_BAD_PARAM, "eps must be finite and >= 0");
  const int64_t stride[] = {p->x_stride, p->y_stride, p->gate_stride, bwd ? p->dr_stride : p->c,
                            bwd ? p->dh_stride : p->c};
  for (const int64_t s : stride)
    if (s < p->c) return fail(DWC_ERR_BAD_PARAM, "row strides must be at least c");
  for (const int64_t s : stride)
    if (s > kMost >> 8 || p->rows > kMost / s)
      return fail(DWC_ERR_UNSUPPORTED, "residual norm sizes past the index range");
  // rows past 8192 values take 1024 threads each (the limit holds from 513 on),
  // the columns' sums 64 a column
  if (p->rows >= (p->c > 512 ? (int64_t)1 << 22 : (int64_t)1 << 26) ||
      p->c >= (bwd ? (int64_t)1 << 24 : (int64_t)1 << 31))
    return fail(DWC_ERR_UNSUPPORTED, "residual norm sizes past the launch range");
  return DWC_OK;
}

ResNormArgs resnorm_args(const dwc_resnorm_problem* p) {
  ResNormArgs a{};
  a.rows = p->rows;
  a.c = p->c;
  a.x_stride = p->x_stride;
  a.y_stride = p->y_stride;
  a.gate_stride = p->gate_stride;
  a.dr_stride = p->dr_stride;
  a.dh_stride = p->dh_stride;
  a.x_type = p->x_dtype;
  a.y_type = p->y_dtype;
  a.w_type = p->w_dtype;
  a.act = p->act;
  a.post = p->post;
  a.pre = p->pre;
  a.eps = p->eps;
  return a;
}

int64_t rows_bytes(int64_t rows, int64_t c, int64_t stride, int64_t e) {
  return rows > 0 ? ((rows - 1) * stride + c) * e : 0;
}

}  // namespace

extern "C" {

int dwc_causal_conv(const dwc_causal_conv_problem* p, const void* x, const void* w,
                    const void* bias, const void* s0, const int32_t* lengths, void* y, void* s1,
                    void* stream) {
  return run_conv(p, x, w, bias, s0, lengths, y, s1, false, stream);
}

int dwc_causal_conv_step(const dwc_causal_conv_problem* p, const void* x, const void* w,
                         const void* bias, const void* s0, const int32_t* lengths, void* y,
                         void* s1, void* stream) {
  if (p && p->b > 0 && p->taps > 1 && !s1) return fail(DWC_ERR_BAD_PARAM, "s1 pointer is NULL");
  return run_conv(p, x, w, bias, s0, lengths, y, s1, true, stream);
}

int dwc_causal_conv_bwd_workspace_size(const dwc_causal_conv_problem* p, size_t* bytes) {
  const int st = check_conv(p, true);
  if (st != DWC_OK) return st;
  if (!bytes) return fail(DWC_ERR_BAD_PARAM, "bytes pointer is NULL");
  ConvArgs a = conv_args(p, nullptr, nullptr, nullptr, nullptr, nullptr);
  conv_split(&a, true);
  *bytes = p->b > 0 ? (size_t)conv_rows(a) * (size_t)(p->taps + 1) * (size_t)p->d * 4 : 0;
  return DWC_OK;
}

int dwc_causal_conv_bwd(const dwc_causal_conv_problem* p, const void* dy, const void* ds1,
                        const void* x, const void* w, const void* bias, const void* s0,
                        const int32_t* lengths, void* dx, float* dw, float* dbias, void* ds0,
                        void* workspace, size_t workspace_bytes, void* stream) {
  size_t need = 0;
  int st = dwc_causal_conv_bwd_workspace_size(p, &need);
  if (st != DWC_OK) return st;
  if (!w || !dw || (p->b > 0 && p->l > 0 && (!dy || !x || !dx)))
    return fail(DWC_ERR_BAD_PARAM, "a tensor's pointer is NULL");
  if (need > 0 && (!workspace || workspace_bytes < need))
    return fail(DWC_ERR_WORKSPACE, "workspace missing or smaller than required");
  const int64_t e = bytes_of(p->dtype), we = bytes_of(p->w_dtype);
  const int64_t state = p->b * (p->taps - 1) * p->d * e;
  int64_t xb = 0, yb = 0;
  token_bytes(p->x_stride, p->b, p->l, p->d, e, &xb);
  token_bytes(p->dy_stride, p->b, p->l, p->d, e, &yb);
  const Span in[] = {{x, xb, e},       {dy, yb, e},
                     {ds1, state, e},  {w, p->taps * p->d * we, we},
                     {bias, bias ? p->d * we : 0, we}, {s0, state, e},
                     {lengths, lengths ? p->b * 4 : 0, 4}};
  const Span out[] = {{dx, p->b * p->l * p->d * e, e},
                      {dw, p->taps * p->d * 4, 4},
                      {dbias, dbias ? p->d * 4 : 0, 4},
                      {ds0, ds0 ? state : 0, e},
                      {workspace, (int64_t)need, 4}};
  st = check_spans(in, out);
  if (st != DWC_OK) return st;
  ConvArgs a = conv_args(p, x, w, bias, s0, lengths);
  a.y = dx;
  a.dy = dy;
  a.ds1 = p->taps > 1 ? ds1 : nullptr;
  a.ds0 = p->taps > 1 ? ds0 : nullptr;
  a.part = (float*)workspace;
  conv_split(&a, true);
  return hip_result(launch_conv_bwd(a, dw, dbias, (hipStream_t)stream),
                    "dwc_causal_conv_bwd launch");
}

int dwc_scan_step(const dwc_scan_problem* p, const void* u, const void* delta, const float* A,
                  const void* B, const void* C, const float* D, const void* z, const float* bias,
                  const float* s0, const int32_t* lengths, void* y, float* s1, void* stream) {
  int st = check_scan(p);
  if (st != DWC_OK) return st;
  if (p->b == 0) return DWC_OK;
  if (!A || !s1 || (p->l > 0 && (!u || !delta || !B || !C || !y)))
    return fail(DWC_ERR_BAD_PARAM, "a tensor's pointer is NULL");
  const int64_t e = bytes_of(p->dtype);
  const ScanSpans n = scan_spans(p);
  const Span in[] = {{u, n.u, e},    {delta, n.delta, e}, {A, n.vec * p->n, 4}, {B, n.b, e},
                     {C, n.c, e},    {D, D ? n.vec : 0, 4}, {z, z ? n.z : 0, e},
                     {bias, bias ? n.vec : 0, 4}, {s0 == s1 ? nullptr : s0, n.state, 4},
                     {lengths, lengths ? p->b * 4 : 0, 4}};
  const Span out[] = {{y, n.dense, e}, {s1, n.state, 4}};
  st = check_spans(in, out);
  if (st != DWC_OK) return st;
  ScanArgs a = scan_args(p, u, delta, A, B, C, D, z, bias, s0, lengths);
  a.y = y;
  a.s1 = s1;
  return hip_result(launch_scan_token(a, (hipStream_t)stream), "dwc_scan_step launch");
}

int dwc_scan_workspace_size(const dwc_scan_problem* p, int op, size_t* bytes) {
  const int st = check_scan(p);
  if (st != DWC_OK) return st;
  if (op != DWC_SCAN_FWD && op != DWC_SCAN_BWD)
    return fail(DWC_ERR_BAD_PARAM, "op must be DWC_SCAN_FWD or DWC_SCAN_BWD");
  if (!bytes) return fail(DWC_ERR_BAD_PARAM, "bytes pointer is NULL");
  ScanArgs a = scan_args(p, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr,
                         nullptr, nullptr);
  return scan_layout(&a, op == DWC_SCAN_BWD, nullptr, bytes);
}

int dwc_scan_fwd(const dwc_scan_problem* p, const void* u, const void* delta, const float* A,
                 const void* B, const void* C, const float* D, const void* z, const float* bias,
                 const float* s0, const int32_t* lengths, void* y, float* s1, void* workspace,
                 size_t workspace_bytes, void* stream) {
  size_t need = 0;
  int st = dwc_scan_workspace_size(p, DWC_SCAN_FWD, &need);
  if (st != DWC_OK) return st;
  if (p->b == 0) return DWC_OK;
  if (!A || !s1 || (p->l > 0 && (!u || !delta || !B || !C || !y)))
    return fail(DWC_ERR_BAD_PARAM, "a tensor's pointer is NULL");
  if (need > 0 && (!workspace || workspace_bytes < need))
    return fail(DWC_ERR_WORKSPACE, "workspace missing or smaller than required");
  const int64_t e = bytes_of(p->dtype);
  const ScanSpans n = scan_spans(p);
  const Span in[] = {{u, n.u, e},    {delta, n.delta, e}, {A, n.vec * p->n, 4}, {B, n.b, e},
                     {C, n.c, e},    {D, D ? n.vec : 0, 4}, {z, z ? n.z : 0, e},
                     {bias, bias ? n.vec : 0, 4}, {s0, n.state, 4},
                     {lengths, lengths ? p->b * 4 : 0, 4}};
  const Span out[] = {{y, n.dense, e}, {s1, n.state, 4}, {workspace, (int64_t)need, 256}};
  st = check_spans(in, out);
  if (st != DWC_OK) return st;
  ScanArgs a = scan_args(p, u, delta, A, B, C, D, z, bias, s0, lengths);
  a.y = y;
  a.s1 = s1;
  size_t bytes = 0;
  scan_layout(&a, false, (char*)workspace, &bytes);
  return hip_result(launch_scan_fwd(a, (hipStream_t)stream), "dwc_scan_fwd launch");
}

int dwc_scan_bwd(const dwc_scan_problem* p, const void* dy, const float* ds1, const void* u,
                 const void* delta, const float* A, const void* B, const void* C, const float* D,
                 const void* z, const float* bias, const float* s0, const int32_t* lengths,
                 void* du, void* ddelta, float* dA, void* dB, void* dC, float* dD, void* dz,
                 float* dbias, float* ds0, void* workspace, size_t workspace_bytes,
                 void* stream) {
  size_t need = 0;
  int st = dwc_scan_workspace_size(p, DWC_SCAN_BWD, &need);
  if (st != DWC_OK) return st;
  const bool some = p->b > 0 && p->l > 0;
  if (!A || !dA || (some && (!dy || !u || !delta || !B || !C || !du || !ddelta || !dB || !dC)))
    return fail(DWC_ERR_BAD_PARAM, "a tensor's pointer is NULL");
  if (some && !z != !dz) return fail(DWC_ERR_BAD_PARAM, "z and dz are given together or not");
  if (need > 0 && (!workspace || workspace_bytes < need))
    return fail(DWC_ERR_WORKSPACE, "workspace missing or smaller than required");
  const int64_t e = bytes_of(p->dtype);
  const ScanSpans n = scan_spans(p);
  const Span in[] = {{dy, n.dy, e},  {ds1, n.state, 4},   {u, n.u, e},   {delta, n.delta, e},
                     {A, n.vec * p->n, 4}, {B, n.b, e},   {C, n.c, e},   {D, D ? n.vec : 0, 4},
                     {z, z ? n.z : 0, e},  {bias, bias ? n.vec : 0, 4},  {s0, n.state, 4},
                     {lengths, lengths ? p->b * 4 : 0, 4}};
  const Span out[] = {{du, n.dense, e},  {ddelta, n.dense, e}, {dA, n.vec * p->n, 4},
                      {dB, n.bc, e},     {dC, n.bc, e},        {dD, dD ? n.vec : 0, 4},
                      {dz, dz ? n.dense : 0, e}, {dbias, dbias ? n.vec : 0, 4},
                      {ds0, ds0 ? n.state : 0, 4}, {workspace, (int64_t)need, 256}};
  st = check_spans(in, out);
  if (st != DWC_OK) return st;
  ScanArgs a = scan_args(p, u, delta, A, B, C, D, z, bias, s0, lengths);
  a.dy = dy;
  a.ds1 = ds1;
  a.du = du;
  a.ddelta = ddelta;
  a.da = dA;
  a.db = dB;
  a.dc = dC;
  a.dskip = dD;
  a.dz = dz;
  a.dbias = dbias;
  a.ds0 = ds0;
  size_t bytes = 0;
  scan_layout(&a, true, (char*)workspace, &bytes);
  return hip_result(launch_scan_bwd(a, (hipStream_t)stream), "dwc_scan_bwd launch");
}

int dwc_residual_norm(const dwc_resnorm_problem* p, const void* x, const void* y, const void* gate,
                      const void* scale, const void* w_post, const void* w_pre, void* r, void* h,
                      float* post_rstd, float* pre_rstd, void* stream) {
  int st = check_resnorm(p, false);
  if (st != DWC_OK) return st;
  if (p->rows == 0) return DWC_OK;
  if (!y || !r) return fail(DWC_ERR_BAD_PARAM, "y or r pointer is NULL");
  if (p->pre ? !h : (h || w_pre))
    return fail(DWC_ERR_BAD_PARAM, "h is given with pre, and w_pre not without it");
  if (!p->post && w_post) return fail(DWC_ERR_BAD_PARAM, "w_post is not given without post");
  const int64_t xe = bytes_of(p->x_dtype), ye = bytes_of(p->y_dtype), we = bytes_of(p->w_dtype);
  const int64_t n = p->rows * p->c, w = p->c * we;
  const Span in[] = {{x, rows_bytes(p->rows, p->c, p->x_stride, xe), xe},
                     {y, rows_bytes(p->rows, p->c, p->y_stride, ye), ye},
                     {gate, rows_bytes(p->rows, p->c, p->gate_stride, ye), ye},
                     {scale, w, we},
                     {w_post, w, we},
                     {w_pre, w, we}};
  const Span out[] = {{r, n * xe, xe}, {h, n * ye, ye}, {post_rstd, p->rows * 4, 4},
                      {pre_rstd, p->rows * 4, 4}};
  st = check_spans(in, out);
  if (st != DWC_OK) return st;
  ResNormArgs a = resnorm_args(p);
  a.x = x;
  a.y = y;
  a.gate = gate;
  a.scale = scale;
  a.w_post = w_post;
  a.w_pre = w_pre;
  a.r = r;
  a.h = h;
  a.post_rstd = post_rstd;
  a.pre_rstd = pre_rstd;
  return hip_result(launch_resnorm_fwd(a, (hipStream_t)stream), "dwc_residual_norm launch");
}

int dwc_residual_norm_bwd_workspace_size(const dwc_resnorm_problem* p, size_t* bytes) {
  const int st = check_resnorm(p, true);
  if (st != DWC_OK) return st;
  if (!bytes) return fail(DWC_ERR_BAD_PARAM, "bytes pointer is NULL");
  // enough for either layout of the rows: the addresses are not known yet
  ResNormArgs a = resnorm_args(p);
  size_t most = 0;
  for (int wide = 0; wide < 2; ++wide) {
    if (!wide) a.y = (const void*)1;  // no wide loads
    else a.y = nullptr;
    const ResNormShape s = resnorm_shape(a, true);
    const size_t need = (size_t)resnorm_groups(a, s, true) * 3 * (size_t)p->c * 4 +
                        (s.lpr == 0 ? (size_t)p->rows * 4 : 0);
    if (need > most) most = need;
  }
  *bytes = p->rows > 0 ? most : 0;
  return DWC_OK;
}

int dwc_residual_norm_bwd(const dwc_resnorm_problem* p, const void* dr, const void* dh,
                          const void* x, const void* y, const float* post_rstd,
                          const float* pre_rstd, const void* gate, const void* scale,
                          const void* w_post, const void* w_pre, void* dx, void* dy, void* dgate,
                          float* dscale, float* dw_post, float* dw_pre, void* workspace,
                          size_t workspace_bytes, void* stream) {
  size_t need = 0;
  int st = dwc_residual_norm_bwd_workspace_size(p, &need);
  if (st != DWC_OK) return st;
  if (p->rows > 0 && (!y || !dy || (!dr && !dh)))
    return fail(DWC_ERR_BAD_PARAM, "y, dy, or dr and dh pointers are NULL");
  if (p->rows > 0 && ((p->post && !post_rstd) || (p->pre && dh && !pre_rstd)))
    return fail(DWC_ERR_BAD_PARAM, "post_rstd or pre_rstd pointer is NULL");
  if (p->rows > 0 && !p->pre && dh) return fail(DWC_ERR_BAD_PARAM, "dh is not given without pre");
  if (!gate && dgate) return fail(DWC_ERR_BAD_PARAM, "dgate is not given without a gate");
  if ((!p->post && w_post) || (!p->pre && w_pre))
    return fail(DWC_ERR_BAD_PARAM, "weights are not given without their norm");
  if (need > 0 && (!workspace || workspace_bytes < need))
    return fail(DWC_ERR_WORKSPACE, "workspace missing or smaller than required");
  const int64_t xe = bytes_of(p->x_dtype), ye = bytes_of(p->y_dtype), we = bytes_of(p->w_dtype);
  const int64_t n = p->rows * p->c, w = p->c * we;
  const Span in[] = {{dr, rows_bytes(p->rows, p->c, p->dr_stride, xe), xe},
                     {dh, rows_bytes(p->rows, p->c, p->dh_stride, ye), ye},
                     {x, rows_bytes(p->rows, p->c, p->x_stride, xe), xe},
                     {y, rows_bytes(p->rows, p->c, p->y_stride, ye), ye},
                     {gate, rows_bytes(p->rows, p->c, p->gate_stride, ye), ye},
                     {post_rstd, p->rows * 4, 4},
                     {pre_rstd, p->rows * 4, 4},
                     {scale, w, we},
                     {w_post, w, we},
                     {w_pre, w, we}};
  const Span out[] = {{dx, n * xe, xe},      {dy, n * ye, ye},      {dgate, n * ye, ye},
                      {dscale, p->c * 4, 4}, {dw_post, p->c * 4, 4}, {dw_pre, p->c * 4, 4},
                      {workspace, (int64_t)need, 4}};
  st = check_spans(in, out);
  if (st != DWC_OK) return st;
  ResNormArgs a = resnorm_args(p);
  a.x = x;
  a.y = y;
  a.gate = gate;
  a.scale = scale;
  a.w_post = w_post;
  a.w_pre = w_pre;
  a.dr = dr;
  a.dh = dh;
  a.post_rstd = const_cast<float*>(post_rstd);
  a.pre_rstd = const_cast<float*>(pre_rstd);
  a.dx = dx;
  a.dy = dy;
  a.dgate = dgate;
  a.part = (float*)workspace;
  a.pre = p->pre && dh;  // (else nothing of that norm is read)
  a.groups = resnorm_groups(a, resnorm_shape(a, true), true);
  return hip_result(launch_resnorm_bwd(a, dscale, dw_post, dw_pre, (hipStream_t)stream),
                    "dwc_residual_norm_bwd launch");
}

}  // extern "C"
