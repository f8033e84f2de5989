// seq_scan_wide.hip -- the selective scan in one pass over the tokens, for
// many sequences or channels and for short sequences.
//
// A workgroup takes 64 channels of a sequence, wave w states 4 w to 4 w + 3
// with a channel a lane.  Stages of 16 tokens: the waves share out the tokens'
// steps, inputs and gates (tokens w, w + NW, ...), all run the stage on their
// own states, and join the parts of C . h in LDS, where each finishes its own
// tokens.  B and C go through LDS too, a stage ahead: there are few waves to
// wait for the scalar cache.  A state takes its exp and four
// other instructions once, not twice as in chunks; bound: the vector units.
#include "seq_scan.h"

namespace dwc {
namespace seq {
namespace scan {

constexpr int kStage = 16;

template <int T, int NW, bool GATE>
__global__ void __launch_bounds__(64 * NW) scan_wide(ScanArgs a) {
  constexpr int NT = kStage / NW, SPL = 16;  // tokens a wave shares; states a line of bc
  __shared__ float of[2][kStage][64];        // dt, u
  __shared__ float parts[kStage][NW][64];    // of C . h
  __shared__ __align__(16) float rows[2][kStage][8 * NW];  // B and C, four and four of a wave in turn
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  uint32_t i = blockIdx.x;
  const int block = (int)(i % (uint32_t)a.cblk);
  i /= (uint32_t)a.cblk;
  const int g = (int)(i % (uint32_t)a.g);
  const int64_t b = i / (uint32_t)a.g;
  const int len = (int)length_of(a, b);
  const int64_t g0 = (int64_t)g * a.dg;
  const uint32_t c0 = (uint32_t)(block * 64 + lane);
  const bool on = (int)c0 < a.dg;
  const uint32_t in = on ? c0 : 0;  // (lanes past the end repeat the first channel)
  const int n0 = 4 * wave;
  float a2[4], h[4];
  const auto states = [&](const float* p, float(&v)[4]) {  // of d x n
#pragma unroll
    for (int s = 0; s < 4; ++s) v[s] = (p + (n0 + s < a.n ? n0 + s : 0))[in * (uint32_t)a.n];
#pragma unroll
    for (int s = 0; s < 4; ++s) v[s] = n0 + s < a.n ? v[s] : 0.f;
  };
  states(a.a + g0 * a.n, a2);
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    a2[s] *= kLog2e;
    h[s] = 0.f;
  }
  if (a.s0) states(a.s0 + (b * a.d + g0) * a.n, h);
  const float bias = a.bias ? (a.bias + g0)[in] : 0.f, skip = a.skip ? (a.skip + g0)[in] : 0.f;
  // B and C of a stage: two values a thread; rows up to a multiple of the stage
  // are there, but for blocks of 16 states past the last
  const int row = threadIdx.x / (4 * NW), at_row = 2 * (threadIdx.x % (4 * NW)), of16 = at_row / 32;
  const bool some = of16 < a.nblk;
  const float* bc = a.bc + (((b * a.g + g) * a.nblk + (some ? of16 : 0)) * a.lp + row) * (2 * SPL) +
                    at_row % 32;
  f32x2 bc_next;
  // the wave's tokens of the next stage: next[] is the address of the first
  constexpr int N = GATE ? 3 : 2;
  const char* next[N];
  int64_t step[N];  // NW tokens
  const auto set = [&](int k, const void* p, const int64_t(&stride)[2]) {
    next[k] = (const char*)((const Raw<T>*)p + (b * stride[0] + wave * stride[1] + g0));
    step[k] = NW * stride[1] * (int64_t)sizeof(Raw<T>);
  };
  set(0, a.u, a.u_stride);
  set(1, a.delta, a.delta_stride);
  if constexpr (GATE) set(2, a.z, a.z_stride);
  Raw<T> raw[N][NT];
  const auto fetch = [&](int t0) {
    if (t0 + kStage <= len) {
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int k = 0; k < N; ++k) {
          raw[k][j] = ((const Raw<T>*)next[k])[in];
          next[k] += step[k];
        }
    } else {  // a token past the last one is read as the last
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        const int t = t0 + j * NW + wave, back = t < len ? 0 : t - (len - 1);
#pragma unroll
        for (int k = 0; k < N; ++k)
          raw[k][j] = ((const Raw<T>*)(next[k] + j * step[k] - back * (step[k] / NW)))[in];
      }
    }
    bc_next = *(const f32x2*)(bc + (int64_t)t0 * (2 * SPL));
  };
  const auto keep = [&](int side) {
    *(f32x2*)&rows[side][row][at_row] = some ? bc_next : f32x2{0.f, 0.f};
  };
  Raw<T>* const out = (Raw<T>*)a.y + (b * a.l * a.d + g0);
  if (len > 0) {
    fetch(0);
    keep(0);
  }
  int side = 0;
  for (int t0 = 0; t0 < len; t0 += kStage, side ^= 1) {
    // (the stage before has been read: its readers passed the barrier below)
    Raw<T> gate[NT];
    float u[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const int at = j * NW + wave;
      const bool live = t0 + at < len;
      u[j] = value<T>(raw[0][j]);
      const float dt = step_of(a.softplus, value<T>(raw[1][j]) + bias);
      if constexpr (GATE) gate[j] = raw[GATE ? 2 : 0][j];
      of[0][at][lane] = live ? dt : 0.f;
      of[1][at][lane] = live ? u[j] : 0.f;
    }
    __syncthreads();
    if (t0 + kStage < len) fetch(t0 + kStage);
    // LDS is read two tokens ahead and the decays are made one ahead: a SIMD
    // may have no other wave to fill the wait
    f32x4 bb[3], cc[3];
    float dt[3], du[3], k[2][4];
    const auto read = [&](int j) {
      bb[j % 3] = *(const f32x4*)&rows[side][j][8 * wave];
      cc[j % 3] = *(const f32x4*)&rows[side][j][8 * wave + 4];
      dt[j % 3] = of[0][j][lane];
      du[j % 3] = of[1][j][lane];
    };
    const auto decays = [&](int j) {
      du[j % 3] *= dt[j % 3];
#pragma unroll
      for (int s = 0; s < 4; ++s) k[j % 2][s] = exp2_of(dt[j % 3] * a2[s]);
    };
    read(0);
    read(1);
    decays(0);
#pragma unroll
    for (int j = 0; j < kStage; ++j) {
      __builtin_amdgcn_sched_barrier(0);
      if (j + 2 < kStage) read(j + 2);
      if (j + 1 < kStage) decays(j + 1);
      float y = 0.f;
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        h[s] = fmaf(k[j % 2][s], h[s], du[j % 3] * bb[j % 3][s]);
        y = fmaf(cc[j % 3][s], h[s], y);
      }
      parts[j][wave][lane] = y;
    }
    if (t0 + kStage < len) keep(side ^ 1);
    __syncthreads();
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const int at = j * NW + wave;
      float y = 0.f;
#pragma unroll
      for (int k = 0; k < NW; ++k) y += parts[at][k][lane];
      y = fmaf(skip, u[j], y);
      if constexpr (GATE) {
        const float z = value<T>(gate[j]);
        y *= z * sigmoid(z);
      }
      if (on && t0 + at < len) store1<T>(out + (int64_t)(t0 + at) * a.d, in, y);
    }
  }
  for (int64_t t = len + wave; t < a.l; t += NW)
    if (on) store1<T>(out + t * a.d, in, 0.f);
  float* const s1 = a.s1 + (b * a.d + g0) * a.n;
#pragma unroll
  for (int s = 0; s < 4; ++s)
    if (on && n0 + s < a.n) (s1 + n0 + s)[in * (uint32_t)a.n] = h[s];
}

template <int T, bool GATE>
void go_wide(const ScanArgs& a, hipStream_t st) {
  const dim3 grid((uint32_t)(a.b * a.g * a.cblk));
  if (a.waves == 4) hipLaunchKernelGGL((scan_wide<T, 4, GATE>), grid, dim3(256), 0, st, a);
  else if (a.waves == 8) hipLaunchKernelGGL((scan_wide<T, 8, GATE>), grid, dim3(512), 0, st, a);
  else hipLaunchKernelGGL((scan_wide<T, 16, GATE>), grid, dim3(1024), 0, st, a);
}

template <int T>
void go_wide_gate(const ScanArgs& a, hipStream_t st) {
  if (a.z) go_wide<T, true>(a, st);
  else go_wide<T, false>(a, st);
}

}  // namespace scan

void launch_scan_wide(const ScanArgs& a, hipStream_t st) {
  if (a.type == T_F32) scan::go_wide_gate<T_F32>(a, st);
  else if (a.type == T_BF16) scan::go_wide_gate<T_BF16>(a, st);
  else scan::go_wide_gate<T_F16>(a, st);
}

}  // namespace seq
}  // namespace dwc
