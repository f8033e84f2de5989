// seq_space.h -- host-side launchers of the short causal convolution, the
// selective state space scan and the residual norm.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace dwc {
namespace seq {

// ---- sums of columns ----------------------------------------------------
// out[c] = sum over rows of part[row * stride + c], every sum in one order.
// With turn > 0 the columns are cols / turn x turn and out is the transpose.
struct ColumnSum {
  const float* part;
  float* out;  // null: skipped
  int64_t rows, stride, cols, turn;
};
constexpr int kColumnJobs = 3;
hipError_t launch_column_sums(const ColumnSum (&jobs)[kColumnJobs], hipStream_t st);

// ---- short causal convolution -------------------------------------------
struct ConvArgs {
  const void* x;
  const void* w;
  const void* bias;  // may be null
  const void* s0;    // may be null (zeros)
  const int32_t* lengths;
  void* y;  // dx in the backward pass
  void* s1;
  const void* dy;
  const void* ds1;  // may be null
  void* ds0;        // may be null
  float* part;      // [rows][taps + 1][d] partial sums of dw and dbias
  int64_t x_stride[2], dy_stride[2];
  int64_t b, l, d;
  int strip, strips;  // tokens a lane, lanes a sequence
  int taps, type, w_type, silu;
};
constexpr int kMostTaps = 8;
int conv_strip(const ConvArgs& a, bool bwd);
// rows of partial sums
int64_t conv_rows(const ConvArgs& a);
hipError_t launch_conv_fwd(const ConvArgs& a, hipStream_t st);
hipError_t launch_conv_bwd(const ConvArgs& a, float* dw, float* dbias, hipStream_t st);

// ---- selective state space scan -----------------------------------------
struct ScanArgs {
  const void *u, *delta, *z, *dy, *bm, *cm;  // z may be null
  const float *a, *skip, *bias, *s0, *ds1;   // all but a may be null
  const int32_t* lengths;
  void* y;
  float* s1;
  void *du, *ddelta, *dz, *db, *dc;
  float *da, *dskip, *dbias, *ds0;
  int64_t u_stride[2], delta_stride[2], z_stride[2], dy_stride[2], b_stride[3], c_stride[3];
  int64_t b, l;
  int d, n, g, type, softplus;
  // how the work is split: dg channels a group; spl states a lane in blocks of
  // that many, cblk blocks of 64 channels a group, nc chunks of tc tokens
  int dg, spl, nblk, cblk, tc, nc;
  int one;   // one pass over all tokens, no chunks
  int gblk;  // blocks of states of the gradients' workgroups
  // workspace
  float* a2;       // [nblk spl][d]: A log2 e, zeros past n
  int64_t lp;      // l up to whole chunks of the gradients
  float* bc;       // [b][g][nblk][lp][2 spl]: B and C in fp32, zeros past n and past a length
  float* states;   // [b][nc][nblk spl][d]
  float* rstates;  // the same, of the gradients
  float* dts;      // [b][nc][d]: sum of the steps
  float* bcpart;   // [channel blocks a group][b][g][nblk][lp][2 spl]
  float* apart;    // [b nc][nblk spl][d]
  float* dpart;    // [b nc][2][d]
  float* sums;     // [gblk][3][b l d]
};
constexpr int kGradChannels = 64, kGradChunk = 32;  // of a workgroup of the gradients
// Fills the split of the work.
void scan_split(ScanArgs* a, bool bwd);
hipError_t launch_scan_token(const ScanArgs& a, hipStream_t st);
hipError_t launch_scan_fwd(const ScanArgs& a, hipStream_t st);
hipError_t launch_scan_bwd(const ScanArgs& a, hipStream_t st);

// ---- residual norm ------------------------------------------------------
struct ResNormArgs {
  const void* x;     // may be null (zeros)
  const void* y;
  const void* gate;  // may be null (1)
  const void* scale; // may be null (1)
  const void* w_post;
  const void* w_pre;
  void* r;
  void* h;  // may be null (pre == 0)
  float* post_rstd;
  float* pre_rstd;
  // backward
  const void* dr;  // may be null
  const void* dh;  // may be null
  void* dx;        // may be null
  void* dy;
  void* dgate;  // may be null
  float* part;  // [groups][3][c] partial sums of dscale, dw_post and dw_pre
  int64_t rows, c, x_stride, y_stride, gate_stride, dr_stride, dh_stride;
  int x_type, y_type, w_type, act, post, pre;
  float eps;
  int groups;
};
struct ResNormShape {
  int vec, lpr, nv;
};
ResNormShape resnorm_shape(const ResNormArgs& a, bool bwd);
int resnorm_groups(const ResNormArgs& a, const ResNormShape& s, bool bwd);
hipError_t launch_resnorm_fwd(ResNormArgs a, hipStream_t st);
hipError_t launch_resnorm_bwd(const ResNormArgs& a, float* dscale, float* dw_post, float* dw_pre,
                              hipStream_t st);

}  // namespace seq
}  // namespace dwc
