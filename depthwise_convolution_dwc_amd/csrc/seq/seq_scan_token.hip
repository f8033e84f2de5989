// seq_scan_token.hip -- the selective scan token by token, for one or a few
// new tokens of each sequence.
//
// A lane owns four states of a channel, LPC lanes a channel, for all tokens:
// a wave reads and writes 1 KB of states in one instruction each.  Bound for
// many sequences: memory, the states read and written once; for one sequence
// the latency of its loads.
#include "seq_scan.h"

namespace dwc {
namespace seq {
namespace scan {

template <int T, int LPC, bool WIDE>
__global__ void __launch_bounds__(256) scan_token(ScanArgs a) {
  const int64_t i = (int64_t)blockIdx.x * (256 / LPC) + threadIdx.x / LPC;  // of b d
  const int s0 = 4 * (threadIdx.x % LPC);
  const bool on = i < a.b * a.d;  // (lanes past the end stay for the sums)
  const int64_t b = on ? i / a.d : 0;
  const int c = on ? (int)(i - b * a.d) : 0, g = c / a.dg;
  const int64_t len = length_of(a, b);
  const int64_t at = (b * a.d + c) * a.n + s0;
  float h[4], a2[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) h[j] = a2[j] = 0.f;
  if constexpr (WIDE) {
    if (s0 < a.n) {
      if (a.s0) load_vec<T_F32, 4>(a.s0, at, h);
      load_vec<T_F32, 4>(a.a, (int64_t)c * a.n + s0, a2);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (s0 + j < a.n) {
        if (a.s0) h[j] = a.s0[at + j];
        a2[j] = a.a[(int64_t)c * a.n + s0 + j];
      }
  }
  const float bias = a.bias ? a.bias[c] : 0.f, skip = a.skip ? a.skip[c] : 0.f;
#pragma unroll
  for (int j = 0; j < 4; ++j) a2[j] *= kLog2e;
  for (int64_t t = 0; t < a.l; ++t) {
    float y = 0.f;
    if (t < len) {
      const int64_t bb = b * a.b_stride[0] + t * a.b_stride[1] + g * a.b_stride[2] + s0;
      const int64_t cb = b * a.c_stride[0] + t * a.c_stride[1] + g * a.c_stride[2] + s0;
      float bv[4], cv[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        bv[j] = s0 + j < a.n ? load1<T>(a.bm, bb + j) : 0.f;
        cv[j] = s0 + j < a.n ? load1<T>(a.cm, cb + j) : 0.f;
      }
      const float u = load1<T>(a.u, b * a.u_stride[0] + t * a.u_stride[1] + c);
      float dt = load1<T>(a.delta, b * a.delta_stride[0] + t * a.delta_stride[1] + c) + bias;
      float z = 0.f;
      if (a.z) z = load1<T>(a.z, b * a.z_stride[0] + t * a.z_stride[1] + c);
      if (a.softplus) dt = softplus(dt);
      const float du = dt * u;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        h[j] = fmaf(exp2_of(dt * a2[j]), h[j], du * bv[j]);
        y = fmaf(cv[j], h[j], y);
      }
      y = fmaf(skip, u, lane_sum<LPC>(y));
      if (a.z) y *= z * sigmoid(z);
    }
    if (on && s0 == 0) store1<T>(a.y, (b * a.l + t) * a.d + c, y);
  }
  if (!on) return;
  if constexpr (WIDE) {
    if (s0 < a.n) store_vec<T_F32, 4>(a.s1, at, h);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (s0 + j < a.n) a.s1[at + j] = h[j];
  }
}

template <int T, int LPC>
void go_token(const ScanArgs& a, hipStream_t st) {
  const bool wide = a.n % 4 == 0 && ((uintptr_t)a.s0 | (uintptr_t)a.s1 | (uintptr_t)a.a) % 16 == 0;
  const dim3 grid((uint32_t)((a.b * a.d + 256 / LPC - 1) / (256 / LPC)));
  if (wide) hipLaunchKernelGGL((scan_token<T, LPC, true>), grid, dim3(256), 0, st, a);
  else hipLaunchKernelGGL((scan_token<T, LPC, false>), grid, dim3(256), 0, st, a);
}

template <int T>
void go_lanes(const ScanArgs& a, hipStream_t st) {
  if (a.n <= 4) go_token<T, 1>(a, st);
  else if (a.n <= 8) go_token<T, 2>(a, st);
  else if (a.n <= 16) go_token<T, 4>(a, st);
  else if (a.n <= 32) go_token<T, 8>(a, st);
  else if (a.n <= 64) go_token<T, 16>(a, st);
  else if (a.n <= 128) go_token<T, 32>(a, st);
  else go_token<T, 64>(a, st);
}

}  // namespace scan

hipError_t launch_scan_token(const ScanArgs& a, hipStream_t st) {
  if (a.type == T_F32) scan::go_lanes<T_F32>(a, st);
  else if (a.type == T_BF16) scan::go_lanes<T_BF16>(a, st);
  else scan::go_lanes<T_F16>(a, st);
  return hipGetLastError();
}

}  // namespace seq
}  // namespace dwc
