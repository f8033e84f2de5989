// seq_dropout.hip -- dropout from a counter-based generator.
//
// Element i is kept where word i % 4 of Philox4x32 with 7 rounds (Salmon,
// Moraes, Dror and Shaw, "Parallel random numbers: as easy as 1, 2, 3",
// SC 2011; 7 rounds is the count the paper reports as passing all its
// statistical tests) is at least round(p 2^32); the counter is
// offset + i / 4, the key is the seed.  The mask is a function of (seed,
// offset, i), so the backward pass computes it again and nothing is stored.
//
// Bound: memory.  A thread makes the words of 8 elements of 16 bits (4 of
// 32), which is one 16-byte load and store a stream; the 7 rounds cost 14
// wide integer products per 4 elements, which the loads hide.  MI355X, 51.4M
// bf16: with a residual 57 us (5.4 TB/s), without 34 us (6.0 TB/s).
#include "seq_device.h"
#include "seq_launch.h"

namespace dwc {
namespace seq {
namespace drop {

__device__ __forceinline__ void philox7(uint64_t counter, uint32_t k0, uint32_t k1,
                                        uint32_t out[4]) {
  uint32_t c0 = (uint32_t)counter, c1 = (uint32_t)(counter >> 32), c2 = 0, c3 = 0;
#pragma unroll
  for (int r = 0; r < 7; ++r) {
    const uint64_t p0 = (uint64_t)c0 * 0xD2511F53u, p1 = (uint64_t)c2 * 0xCD9E8D57u;
    c0 = (uint32_t)(p1 >> 32) ^ c1 ^ k0;
    c1 = (uint32_t)p1;
    c2 = (uint32_t)(p0 >> 32) ^ c3 ^ k1;
    c3 = (uint32_t)p0;
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  out[0] = c0;
  out[1] = c1;
  out[2] = c2;
  out[3] = c3;
}

// VEC elements a thread (4 or 8, one or two counters).  WIDE: 16-byte
// vectors of aligned tensors; otherwise element by element.  AT: the position
// in device memory counts too (a form of its own: a branch on it costs the
// others 1.3 us of 32 at 51.4M bf16).
template <int T, int VEC, bool WIDE, bool RES, bool AT>
__global__ void __launch_bounds__(256) dropout(DropArgs a) {
  const int64_t i0 = ((int64_t)blockIdx.x * 256 + threadIdx.x) * VEC;
  if (i0 >= a.n) return;
  const uint64_t first = AT ? a.offset + *a.position : a.offset;
  float x[VEC], r[VEC];
  const bool whole = WIDE && i0 + VEC <= a.n;
  if (whole) {
    load_vec<T, VEC>(a.x, i0, x);
    if constexpr (RES) load_vec<T, VEC>(a.res, i0, r);
  } else {
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      x[j] = i0 + j < a.n ? load1<T>(a.x, i0 + j) : 0.f;
      if constexpr (RES) r[j] = i0 + j < a.n ? load1<T>(a.res, i0 + j) : 0.f;
    }
  }
#pragma unroll
  for (int q = 0; q < VEC / 4; ++q) {
    uint32_t w[4];
    philox7(first + (uint64_t)(i0 / 4 + q), a.key0, a.key1, w);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      // a select, so that a dropped infinity or NaN leaves zero
      const bool kept = w[j] >= a.threshold && !a.drop_all;
      float v = kept ? x[4 * q + j] * a.scale : 0.f;
      if constexpr (RES) v += r[4 * q + j];
      x[4 * q + j] = v;
    }
  }
  if (whole) {
    store_vec<T, VEC>(a.y, i0, x);
  } else {
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      if (i0 + j < a.n) store1<T>(a.y, i0 + j, x[j]);
    }
  }
}

template <int T, bool WIDE, bool RES, bool AT>
void go_one(const DropArgs& a, hipStream_t st) {
  constexpr int VEC = T == T_F32 ? 4 : 8;
  const dim3 grid((uint32_t)((a.n + 256 * VEC - 1) / (256 * VEC)));
  hipLaunchKernelGGL((dropout<T, VEC, WIDE, RES, AT>), grid, dim3(256), 0, st, a);
}

template <int T, bool WIDE>
void go_wide(const DropArgs& a, hipStream_t st) {
  if (a.res) a.position ? go_one<T, WIDE, true, true>(a, st) : go_one<T, WIDE, true, false>(a, st);
  else a.position ? go_one<T, WIDE, false, true>(a, st) : go_one<T, WIDE, false, false>(a, st);
}

template <int T>
void go(const DropArgs& a, hipStream_t st) {
  const bool wide = ((uintptr_t)a.x | (uintptr_t)a.y | (uintptr_t)a.res) % 16 == 0;
  if (wide) go_wide<T, true>(a, st);
  else go_wide<T, false>(a, st);
}

}  // namespace drop

hipError_t launch_dropout(const DropArgs& a, hipStream_t st) {
  if (a.type == T_F32) drop::go<T_F32>(a, st);
  else if (a.type == T_BF16) drop::go<T_BF16>(a, st);
  else drop::go<T_F16>(a, st);
  return hipGetLastError();
}

}  // namespace seq
}  // namespace dwc
