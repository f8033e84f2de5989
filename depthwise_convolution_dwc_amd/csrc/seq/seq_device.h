// seq_device.h -- device helpers of the sequence-layer kernels (layer norm,
// dropout, gated delta rule) on gfx950.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace dwc {
namespace seq {

enum { T_F32 = 0, T_BF16 = 1, T_F16 = 2 };  // = DWC_F32, DWC_BF16, DWC_F16

template <int T> struct ElemBytes { static constexpr int value = T == T_F32 ? 4 : 2; };

__device__ __forceinline__ float bf16_to_f32(uint32_t bits) {
  return __builtin_bit_cast(float, bits << 16);
}

__device__ __forceinline__ float f16_to_f32(uint32_t bits) {
  return (float)__builtin_bit_cast(_Float16, (uint16_t)bits);
}

// Round to nearest even, NaN kept: the hardware conversion.
__device__ __forceinline__ uint32_t f32_to_bf16(float x) {
  return (uint32_t)__builtin_bit_cast(uint16_t, (__bf16)x);
}

__device__ __forceinline__ uint32_t f32_to_f16(float x) {
  return (uint32_t)__builtin_bit_cast(uint16_t, (_Float16)x);
}

template <int T>
__device__ __forceinline__ float from16(uint32_t bits) {
  if constexpr (T == T_BF16) return bf16_to_f32(bits);
  else return f16_to_f32(bits);
}

template <int T>
__device__ __forceinline__ uint32_t to16(float x) {
  if constexpr (T == T_BF16) return f32_to_bf16(x);
  else return f32_to_f16(x);
}

// One element, any of the three types.
template <int T>
__device__ __forceinline__ float load1(const void* p, int64_t i) {
  if constexpr (T == T_F32) return ((const float*)p)[i];
  else return from16<T>(((const uint16_t*)p)[i]);
}

template <int T>
__device__ __forceinline__ void store1(void* p, int64_t i, float v) {
  if constexpr (T == T_F32) ((float*)p)[i] = v;
  else ((uint16_t*)p)[i] = (uint16_t)to16<T>(v);
}

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

// N consecutive elements from an address aligned to min(16, N * size).
template <int T, int N>
__device__ __forceinline__ void load_vec(const void* p, int64_t i, float* v) {
  if constexpr (N == 1) {
    v[0] = load1<T>(p, i);
  } else if constexpr (T == T_F32) {
    static_assert(N % 4 == 0, "");
#pragma unroll
    for (int k = 0; k < N / 4; ++k) {
      const f32x4 t = *(const f32x4*)((const float*)p + i + 4 * k);
#pragma unroll
      for (int j = 0; j < 4; ++j) v[4 * k + j] = t[j];
    }
  } else {
    static_assert(N == 4 || N == 8, "");
    uint32_t w[N / 2];
    if constexpr (N == 8) {
      const u32x4 t = *(const u32x4*)((const uint16_t*)p + i);
#pragma unroll
      for (int j = 0; j < 4; ++j) w[j] = t[j];
    } else {
      const u32x2 t = *(const u32x2*)((const uint16_t*)p + i);
      w[0] = t[0];
      w[1] = t[1];
    }
#pragma unroll
    for (int j = 0; j < N / 2; ++j) {
      v[2 * j] = from16<T>(w[j] & 0xffffu);
      v[2 * j + 1] = from16<T>(w[j] >> 16);
    }
  }
}

template <int T, int N>
__device__ __forceinline__ void store_vec(void* p, int64_t i, const float* v) {
  if constexpr (N == 1) {
    store1<T>(p, i, v[0]);
  } else if constexpr (T == T_F32) {
#pragma unroll
    for (int k = 0; k < N / 4; ++k) {
      f32x4 t;
#pragma unroll
      for (int j = 0; j < 4; ++j) t[j] = v[4 * k + j];
      *(f32x4*)((float*)p + i + 4 * k) = t;
    }
  } else {
    uint32_t w[N / 2];
#pragma unroll
    for (int j = 0; j < N / 2; ++j) w[j] = to16<T>(v[2 * j]) | (to16<T>(v[2 * j + 1]) << 16);
    if constexpr (N == 8) *(u32x4*)((uint16_t*)p + i) = u32x4{w[0], w[1], w[2], w[3]};
    else *(u32x2*)((uint16_t*)p + i) = u32x2{w[0], w[1]};
  }
}

// The same with the type a launch argument (a scalar branch).
template <int N>
__device__ __forceinline__ void load_any(int t, const void* p, int64_t i, float* v) {
  if (t == T_F32) load_vec<T_F32, N>(p, i, v);
  else if (t == T_BF16) load_vec<T_BF16, N>(p, i, v);
  else load_vec<T_F16, N>(p, i, v);
}

template <int N>
__device__ __forceinline__ void store_any(int t, void* p, int64_t i, const float* v) {
  if (t == T_F32) store_vec<T_F32, N>(p, i, v);
  else if (t == T_BF16) store_vec<T_BF16, N>(p, i, v);
  else store_vec<T_F16, N>(p, i, v);
}

// v of another lane of the same row of 16, by a move inside the row (CTRL: a
// permutation of each four, a mirror of 8 or 16, a rotation).
template <int CTRL>
__device__ __forceinline__ float row_move(float v) {
  return __builtin_bit_cast(
      float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xf, 0xf, false));
}

// a = v of the even of two halves of a wave (of each two rows of 16), o = v
// of the odd one, both in all lanes.  The swap exchanges the odd halves
// (rows) of its first register with the even ones of its second.  (The
// compiler's builtin returns its first result twice.)
__device__ __forceinline__ void halves(float& a, float& o) {
  o = a;
  asm("s_nop 1\n\tv_permlane32_swap_b32 %0, %1" : "+v"(a), "+v"(o));
}
__device__ __forceinline__ void rows16(float& a, float& o) {
  o = a;
  asm("s_nop 1\n\tv_permlane16_swap_b32 %0, %1" : "+v"(a), "+v"(o));
}

// Sum over groups of W adjacent lanes (W a power of two up to 64); every
// lane of a group gets the same bits.  Moves inside the registers: an
// exchange through LDS costs each of the steps ten times as long.
template <int W>
__device__ __forceinline__ float lane_sum(float v) {
  if constexpr (W >= 2) v += row_move<0xB1>(v);    // 1 0 3 2
  if constexpr (W >= 4) v += row_move<0x4E>(v);    // 2 3 0 1
  if constexpr (W >= 8) v += row_move<0x141>(v);   // mirror of 8
  if constexpr (W >= 16) v += row_move<0x140>(v);  // mirror of 16
  float o;
  if constexpr (W >= 32) {
    rows16(v, o);
    v += o;
  }
  if constexpr (W >= 64) {
    halves(v, o);
    v += o;
  }
  return v;
}

// Sum over the lanes before this one in its row of 16: shifted by one lane,
// then summed up to this lane.
__device__ __forceinline__ float sum_before16(float v) {
  v = row_move<0x111>(v);
  v += row_move<0x111>(v);
  v += row_move<0x112>(v);
  v += row_move<0x114>(v);
  return v + row_move<0x118>(v);
}

}  // namespace seq
}  // namespace dwc
