// seq_scan_token.hip -- the selective scan token by token, for one or a few
// new tokens of each sequence.
//
// A lane owns four states of a channel, LPC lanes a channel, for all tokens:
// a wave reads and writes 1 KB of states in one instruction each.  Bound for
// many sequences: memory, the states read and written once (128 sequences of
// 4096 channels, 16 states: 17.5 us, 4.1 TB/s; two or four channels a lane took
// 21 and 23 where one took 19); for one sequence the latency of its loads.
#include "seq_scan.h"

namespace dwc {
namespace seq {
namespace scan {

// Four elements, those past n zero; one load where WIDE.
template <int T, bool WIDE>
__device__ __forceinline__ void load_four(const void* p, int64_t i, int left, float (&v)[4]) {
  if constexpr (WIDE) {
    if (left > 0) {
      load_vec<T, 4>(p, i, v);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = 0.f;
    }
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = j < left ? load1<T>(p, i + j) : 0.f;
  }
}

template <int T, int LPC, bool WIDE>
__global__ void __launch_bounds__(256) scan_token(ScanArgs a) {
  constexpr int CH = 256 / LPC;  // channels a workgroup
  const uint32_t blocks = (uint32_t)((a.d + CH - 1) / CH);
  const int64_t b = blockIdx.x / blocks;
  const int c0 = (int)(blockIdx.x - (uint32_t)b * blocks) * CH + (int)threadIdx.x / LPC;
  const bool on = c0 < a.d;  // (lanes past the end repeat the last channel, for the sums)
  const int c = on ? c0 : a.d - 1, g = c / a.dg;
  const int s0 = 4 * (threadIdx.x % LPC), left = a.n - s0;
  const int64_t len = length_of(a, b), at = (b * a.d + c) * a.n + s0;
  float h[4] = {0.f, 0.f, 0.f, 0.f}, a2[4];
  if (a.s0) load_four<T_F32, WIDE>(a.s0, at, left, h);
  load_four<T_F32, WIDE>(a.a, (int64_t)c * a.n + s0, left, a2);
  const float bias = a.bias ? a.bias[c] : 0.f, skip = a.skip ? a.skip[c] : 0.f;
#pragma unroll
  for (int j = 0; j < 4; ++j) a2[j] = rate_of(a2[j]);
  for (int64_t t = 0; t < a.l; ++t) {
    float y = 0.f;
    if (t < len) {
      float bv[4], cv[4];
      load_four<T, WIDE>(a.bm, b * a.b_stride[0] + t * a.b_stride[1] + g * a.b_stride[2] + s0, left, bv);
      load_four<T, WIDE>(a.cm, b * a.c_stride[0] + t * a.c_stride[1] + g * a.c_stride[2] + s0, left, cv);
      const float u = load1<T>(a.u, b * a.u_stride[0] + t * a.u_stride[1] + c);
      const float x = load1<T>(a.delta, b * a.delta_stride[0] + t * a.delta_stride[1] + c);
      const float z = a.z ? load1<T>(a.z, b * a.z_stride[0] + t * a.z_stride[1] + c) : 0.f;
      const float dt = step_of(a.softplus, x + bias), du = dt * u;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        h[j] = fmaf(exp2_of(dt * a2[j]), h[j], du * bv[j]);
        y = fmaf(cv[j], h[j], y);
      }
      y = fmaf(skip, u, lane_sum<LPC>(y));
      const float gate = z * sigmoid(z);
      y *= a.z ? gate : 1.f;
    }
    if (on && s0 == 0) store1<T>(a.y, (b * a.l + t) * a.d + c, y);
  }
  if (!on || left <= 0) return;
  if constexpr (WIDE) {
    store_vec<T_F32, 4>(a.s1, at, h);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (j < left) a.s1[at + j] = h[j];
  }
}

template <int T, int LPC>
void go_token(const ScanArgs& a, hipStream_t st) {
  const size_t e = T == T_F32 ? 16 : 8;
  bool wide = a.n % 4 == 0 && ((uintptr_t)a.s0 | (uintptr_t)a.s1 | (uintptr_t)a.a) % 16 == 0 &&
              ((uintptr_t)a.bm | (uintptr_t)a.cm) % e == 0;
  for (int i = 0; i < 3; ++i) wide = wide && a.b_stride[i] % 4 == 0 && a.c_stride[i] % 4 == 0;
  constexpr int per = 256 / LPC;
  const dim3 grid((uint32_t)(a.b * ((a.d + per - 1) / per)));
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
