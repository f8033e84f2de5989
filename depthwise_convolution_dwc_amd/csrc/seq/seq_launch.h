// seq_launch.h -- host-side launchers of the sequence-layer kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace dwc {
namespace seq {

// ---- layer norm ---------------------------------------------------------
struct NormArgs {
  const void* x;
  const void* dy;
  const void* w;  // may be null (w = 1)
  const void* b;  // may be null (b = 0)
  void* y;        // dx in the backward pass
  float* mean;    // may be null in the forward pass
  float* rstd;
  float* part;    // [groups][2][c] column partials of the backward pass
  int64_t rows, c, x_stride, dy_stride;
  int x_type, y_type, w_type;
  float eps;
  int groups;
};

// How the rows are laid on lanes: vec elements per load, lpr lanes a row,
// nv loads a lane; lpr == 0 means the looping kernels (rows longer than the
// register forms).
struct NormShape {
  int vec, lpr, nv;
};
NormShape norm_shape(const NormArgs& a, bool bwd);
int norm_groups(const NormArgs& a, const NormShape& s);
hipError_t launch_norm_fwd(const NormArgs& a, hipStream_t st);
hipError_t launch_norm_bwd(const NormArgs& a, float* dw, float* db, hipStream_t st);

// ---- dropout ------------------------------------------------------------
struct DropArgs {
  const void* x;
  const void* res;  // may be null
  void* y;
  int64_t n;
  uint64_t offset;
  const uint64_t* position;  // added to offset where the kernel runs; may be null
  uint32_t key0, key1;
  uint32_t threshold;
  int drop_all;
  float scale;
  int type;
};
hipError_t launch_dropout(const DropArgs& a, hipStream_t st);

}  // namespace seq
}  // namespace dwc
