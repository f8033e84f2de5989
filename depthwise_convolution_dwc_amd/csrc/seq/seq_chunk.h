// seq_chunk.h -- what the chunked kernels of the gated delta rule share: the
// workspace, the matrix-core fragments and how fp32 values are multiplied.
//
// In a chunk of 64 tokens (G the running sum of g inside it, S the state
// before it, D_tj = exp(G_t - G_j) for j <= t):
//   N = strictly lower part of D o (K K^T),   X = (1 + N beta)^-1 N,
//   e = V - exp(G) o (K S),                   E = e - X (beta o e),
//   U = beta o E,   P = scale D o (Q K^T) (lower part),
//   O = scale exp(G) o (Q S) + P U,
//   S <- exp(G_64) S + K^T (exp(G_64 - G) o U).
// X needs no division by beta and gives both inverses that the rule and its
// gradient want: (1 + N beta)^-1 = 1 - X beta, (1 + beta N)^-1 = 1 - beta X.
//
// Arithmetic.  The matrix cores multiply fp16.  A value v is kept as one or
// two fp16 numbers hi + lo with v 2^s = hi + lo, hi the nearest fp16 and lo
// the nearest of the rest: together 22 bits and a sign, so a product of
// pairs (hi hi + hi lo + lo hi, summed in fp32 by the instruction) is off by
// about 2^-23 of its size, as an fp32 product is.  The scale 2^s brings the
// largest magnitude of the operand (a column of a state, a whole tile of the
// others) to 2^14..2^15.  hi then keeps 11 bits down to 2^-28 of the largest,
// and lo, a multiple of 2^-24, the other 11 down to about 2^-17 of it: below
// that a pair is off by at most 2^-39 of the largest.  fp16 inputs, and bf16
// ones down to 2^-31 of the largest, are exact in one fp16 number.  States,
// sums and statistics stay fp32.
#pragma once

#include "seq_delta.h"
#include "seq_device.h"

namespace dwc {
namespace seq {

constexpr int kChunk = 64;
constexpr double kLog2e = 1.4426950408889634074;  // sums of g are kept for exp2

typedef _Float16 half8 __attribute__((ext_vector_type(8)));
typedef _Float16 half4 __attribute__((ext_vector_type(4)));

// Per chunk and value head.
struct Gate {
  float into[kChunk];  // exp(G_t)
  float out[kChunk];   // exp(G_64 - G_t)
  float beta[kChunk];
  float total;         // exp(G_64)
  // the packed values of X, P, K and Q times these are the true ones
  float xinv, pinv, kinv, qinv;
  // (backward) the larger of the last two, and what each of them is of it
  float top, kpart, qpart;
  double g[kChunk];    // G_t log2(e)
};

// Fragment blocks of 64 lanes x 16 bytes.  Inside a block of 32 along the
// summed axis, lane group q = lane / 16 holds elements 4q..4q+3 and
// 16+4q..16+4q+3: the order in which two 16x16 results of an earlier
// product lie in the lanes, so a result becomes the next product's operand
// without leaving its lane.
typedef half8 Frag;  // one lane's part

// Blocks of the strictly or weakly lower triangular 64x64 operands: rows
// 0..31 need the first 32 columns only; and of their transposes.
__device__ __forceinline__ constexpr int tri_block(int m, int ks) {
  return m < 2 ? m : 2 + 2 * (m - 2) + ks;
}
__device__ __forceinline__ constexpr int tri_block_t(int m, int ks) {
  return m < 2 ? 2 * m + ks : 4 + (m - 2);
}
constexpr int kTri = 6;

// 16x16 blocks of the weakly lower triangle of a 64x64 matrix, as results of
// the matrix cores: lane l of block (i, j) has rows 16 i + 4 (l / 16) .. + 3
// of column 16 j + l % 16.
__device__ __forceinline__ constexpr int low_block(int i, int j) { return i * (i + 1) / 2 + j; }
constexpr int kLow = 10;

struct ChunkArgs {
  DeltaArgs a;
  int nc;        // chunks of the longest sequence
  int dvp;       // dv rounded up to 16
  Frag *ka, *qa, *kt, *qt;   // per (b, chunk, hk): [piece][block][64]
  Frag *xa, *pa, *xt, *pt;   // per (b, chunk, hv): [piece][kTri][64]
  f32x4 *kk, *qk;            // K K^T and Q K^T per (b, chunk, hk): [kLow][64]
  Gate* gate;                // per (b, chunk, hv)
  float *states, *dstates;   // per (b, chunk, hv): dp x dvp, before the chunk / after it
  float *e, *dw;             // per (b, chunk, hv): 64 x dvp
  bool wide;  // dout can be read 16 bytes at a time, dv is a multiple of 8
};

__device__ __forceinline__ int64_t live_tokens(const DeltaArgs& a, int64_t b) {
  if (!a.lengths) return a.l;
  const int64_t n = a.lengths[b];
  return n < 0 ? 0 : (n < a.l ? n : a.l);
}

__device__ __forceinline__ f32x4 mfma(half8 a, half8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}

// The power of two that brings a largest magnitude m to 2^14..2^15, and its
// inverse.  m below 2^-101 (and zero) is treated as 2^-101: both stay normal
// numbers, also times a decay, and an inverse times another one is exact
// down to 2^-149.  Factors of an operand go to the product's result and not
// into the operand, whose scale would then meet the limit earlier.
struct Scale {
  float mul, inv;
};
__device__ __forceinline__ Scale scale_of(float m) {
  int e = (int)((__builtin_bit_cast(uint32_t, m) >> 23) & 255) - 126;  // m < 2^e
  e = e < -100 ? -100 : (e > 125 ? 125 : e);
  return Scale{__builtin_bit_cast(float, (uint32_t)(127 + 15 - e) << 23),
               __builtin_bit_cast(float, (uint32_t)(127 + e - 15) << 23)};
}

// hi and lo of scaled values.
__device__ __forceinline__ void split(float v, _Float16* hi, _Float16* lo) {
  *hi = (_Float16)v;
  *lo = (_Float16)(v - (float)*hi);
}

// Largest magnitude over the lanes that share a column (lane % 16).
__device__ __forceinline__ float column_max(float m) {
  float o;
  halves(m, o);
  m = fmaxf(m, o);
  rows16(m, o);
  return fmaxf(m, o);
}

// Largest magnitude over a wave: over each 16 lanes by rotations of a row,
// then over the rows.
__device__ __forceinline__ float wave_max(float m) {
  m = fmaxf(m, row_move<0x128>(m));
  m = fmaxf(m, row_move<0x124>(m));
  m = fmaxf(m, row_move<0x122>(m));
  m = fmaxf(m, row_move<0x121>(m));
  return column_max(m);
}

// Element lane of a block at a uniform address: the address stays in scalar
// registers, the lane's part is one 32-bit offset.
template <typename V>
__device__ __forceinline__ V at_lane(const V* block, uint32_t offset) {
  return *(const V*)((const char*)block + offset);
}

// acc += A B from pieces: PA of A, PB of B, the products that matter.
template <int PA, int PB>
__device__ __forceinline__ f32x4 mfma_pieces(const half8* a, const half8* b, f32x4 c) {
  if constexpr (PA == 2) c = mfma(a[1], b[0], c);
  if constexpr (PB == 2) c = mfma(a[0], b[1], c);
  return mfma(a[0], b[0], c);
}

// Two 16-row results (rows 4q + r of each) as the operand fragments of 32
// rows, scaled by s.
template <int P>
__device__ __forceinline__ void to_frag(const f32x4& t0, const f32x4& t1, float s, half8* f) {
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    _Float16 h, l;
    split(t0[r] * s, &h, &l);
    f[0][r] = h;
    if constexpr (P == 2) f[1][r] = l;
    split(t1[r] * s, &h, &l);
    f[0][4 + r] = h;
    if constexpr (P == 2) f[1][4 + r] = l;
  }
}

template <int N>
__device__ __forceinline__ float abs_max(const f32x4 (&v)[N]) {
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < N; ++i)
#pragma unroll
    for (int r = 0; r < 4; ++r) m = fmaxf(m, fabsf(v[i][r]));
  return m;
}

hipError_t launch_delta_prep(const ChunkArgs& c, bool bwd, hipStream_t st);
// Chunk by chunk: o and s1, or (bwd) the state before each chunk and E, and
// back from the last chunk dv, the state's gradient after each chunk and dw.
hipError_t launch_delta_scan(const ChunkArgs& c, bool bwd, hipStream_t st);
// dq, dk, dg, dbeta of each chunk.
hipError_t launch_delta_grad(ChunkArgs c, hipStream_t st);

}  // namespace seq
}  // namespace dwc
