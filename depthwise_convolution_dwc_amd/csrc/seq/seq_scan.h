// seq_scan.h -- device helpers of the selective state space scan.
//
// Per sequence and channel, with a state h of n values:
//   dt_t = softplus(delta_t + bias), a_t = exp(dt_t A)
//   h_t = a_t h_(t-1) + dt_t u_t B_t,  o_t = C_t . h_t + D u_t,  y_t = o_t silu(z_t)
#pragma once

#include "seq_device.h"
#include "seq_space.h"

namespace dwc {
namespace seq {
namespace scan {

constexpr float kLog2e = 1.44269504088896341f, kLn2 = 0.693147180559945309f;

typedef float f32x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
template <int N> struct VecOf;
template <> struct VecOf<4> { typedef f32x4 type; };
template <> struct VecOf<8> { typedef f32x8 type; };
template <> struct VecOf<16> { typedef f32x16 type; };

// N floats from an address that is the same in all lanes, through the scalar
// cache into scalar registers (read-only memory of an earlier kernel).
template <int N>
__device__ __forceinline__ typename VecOf<N>::type load_scalar(const float* p) {
  typedef const __attribute__((address_space(4))) typename VecOf<N>::type cvec;
  return *(cvec*)(uintptr_t)p;
}

// An element as it stands in memory (Elem) and in a register (Raw: a whole one,
// or the compiler packs elements in pairs, which waits for their loads).
template <int T> struct RawOf {
  typedef uint16_t elem;
  typedef uint32_t reg;
};
template <> struct RawOf<T_F32> {
  typedef float elem;
  typedef float reg;
};
template <int T>
using Elem = typename RawOf<T>::elem;
template <int T>
using Raw = typename RawOf<T>::reg;

template <int T>
__device__ __forceinline__ float value(Raw<T> v) {
  if constexpr (T == T_F32) return v;
  else return from16<T>(v);
}

// Where a line of bc holds B and C of state s.  The gradients' waves have four
// states each and take both with one load.
template <int SPL, bool BWD>
constexpr int b_at(int s) { return BWD ? s / 4 * 8 + s % 4 : s; }
template <int SPL, bool BWD>
constexpr int c_at(int s) { return BWD ? s / 4 * 8 + 4 + s % 4 : SPL + s; }

// A in units of the decays' exp2.  Infinities become the largest values: a
// token that is not there has a step of 0, and 0 times infinity would be NaN.
__device__ __forceinline__ float rate_of(float a) {
  const float v = kLog2e * a;
  return fabsf(v) == __builtin_inff() ? copysignf(__FLT_MAX__, v) : v;
}

__device__ __forceinline__ float exp2_of(float x) { return __builtin_amdgcn_exp2f(x); }

// The decay 2^x of many tokens, m 2^e with m in (1/2, 1].  As one number it is
// past fp32's range where decays grow long enough, and infinity times a state
// of 0, or one that is small enough, is not what the tokens make of it one by
// one.
struct Decay {
  float m, e;
  __device__ __forceinline__ float of(float v) const {
    return __builtin_ldexpf(m * v, (int)e);
  }
};
__device__ __forceinline__ Decay decay_of(float x) {
  // (e is held where sums of it stay exact; m takes the rest, and a NaN)
  const float e = __builtin_ceilf(fminf(fmaxf(x, -1e6f), 1e6f));
  return {exp2_of(x - e), e};
}

__device__ __forceinline__ float sigmoid(float x) {
  return __builtin_amdgcn_rcpf(1.f + exp2_of(-kLog2e * x));
}

// max(x, 0) + log(1 + e), e = exp(-|x|).  1 + e drops low bits of a small e:
// log(w) e / (w - 1) with w = 1 + e as it was rounded gives them back (Higham,
// Accuracy and Stability of Numerical Algorithms, chapter 1).
__device__ __forceinline__ float softplus(float x) {
  const float e = exp2_of(-kLog2e * fabsf(x));
  const float w = 1.f + e, d = w - 1.f;
  const float l = kLn2 * __builtin_amdgcn_logf(w) * (e * __builtin_amdgcn_rcpf(d));
  return fmaxf(x, 0.f) + (d == 0.f ? e : l);
}

// (A select: a branch would split the code of several tokens.)
__device__ __forceinline__ float step_of(int soft, float x) {
  const float s = softplus(x);
  return soft ? s : x;
}

__device__ __forceinline__ int64_t length_of(const ScanArgs& a, int64_t b) {
  if (!a.lengths) return a.l;
  const int64_t n = a.lengths[b];
  return n < 0 ? 0 : (n < a.l ? n : a.l);
}

// The kernel's arguments, read again from their segment: held in registers
// over the whole kernel they push others out to memory.
typedef const __attribute__((address_space(4))) ScanArgs FreshArgs;
__device__ __forceinline__ FreshArgs& fresh_args() {
  FreshArgs* p = (FreshArgs*)__builtin_amdgcn_kernarg_segment_ptr();
  asm volatile("" : "+s"(p));
  return *p;
}

}  // namespace scan
}  // namespace seq
}  // namespace dwc
