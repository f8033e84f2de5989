// seq_delta.h -- arguments and launchers of the gated delta rule's kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace dwc {
namespace seq {

struct DeltaArgs {
  const void *q, *k, *v, *dout;
  const float *g, *beta, *s0, *ds1;
  const int32_t* lengths;  // may be null: every sequence has l tokens
  void *o, *dq, *dk_out, *dv_out;
  float *s1, *dg, *dbeta, *ds0;
  // strides in elements: batch, token, head
  int64_t q_stride[3], k_stride[3], v_stride[3], g_stride[3], beta_stride[3], do_stride[3];
  int64_t b, l;
  int hk, hv, dk, dv, type;
  float scale;
};

hipError_t launch_delta_token(const DeltaArgs& a, hipStream_t st);

}  // namespace seq
}  // namespace dwc
