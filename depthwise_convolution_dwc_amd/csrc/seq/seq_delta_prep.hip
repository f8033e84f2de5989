// seq_delta_prep.hip -- what each chunk of the gated delta rule needs and no
// state enters: fragments of K, Q and their transposes, the gates, and the
// triangular X and P (see seq_chunk.h).  All chunks run at once.
//
// One workgroup of 4 waves a (sequence, chunk, key head); the value heads
// that share the key head reuse K K^T and Q K^T from registers.
//
// Bound: memory where chunks are many (8x2048 tokens of 16 heads, 128
// dimensions, bf16: 134 MB in, 308 MB out in 105 us, for the backward pass
// 442 MB out in 130 us), else one workgroup's chain of phases, 15 us.  The
// triangular solve by 16x16 blocks took it there from 202 us with a solve row
// by row.
#include "../dwc_device.h"
#include "seq_chunk.h"

namespace dwc {
namespace seq {
namespace prep {

// Of the 64x64 fp32 tiles in LDS: rows stay 16-byte aligned, and 16 rows read
// 16 bytes each at one column cover all 64 banks.
constexpr int kPitch = 68;

// The largest of each of two values over the workgroup.
__device__ __forceinline__ f32x2 block_max2(float u, float v, float (*red)[4]) {
  u = wave_max(u);
  v = wave_max(v);
  if ((threadIdx.x & 63) == 0) {
    red[0][threadIdx.x >> 6] = u;
    red[1][threadIdx.x >> 6] = v;
  }
  __syncthreads();
  return f32x2{fmaxf(fmaxf(red[0][0], red[0][1]), fmaxf(red[0][2], red[0][3])),
               fmaxf(fmaxf(red[1][0], red[1][1]), fmaxf(red[1][2], red[1][3]))};
}

// acc += A B for 16x16 fp32 blocks: a holds A's row lane % 16, columns
// 4 q .. 4 q + 3 (q = lane / 16); b is a result of an earlier product.  Step
// r sums the columns 4 q + r, which is where register r of a result lies.
__device__ __forceinline__ f32x4 mul16(const f32x4& a, const f32x4& b, f32x4 acc) {
#pragma unroll
  for (int r = 0; r < 4; ++r) acc = __builtin_amdgcn_mfma_f32_16x16x4f32(a[r], b[r], acc, 0, 0, 0);
  return acc;
}

template <int P>
constexpr int lds_bytes(int dp) {
  const int rows = 2 * P * kChunk * (dp + 8) * 2, tiles = 2 * kChunk * kPitch * 4;
  return rows > tiles ? rows : tiles;
}

// A row block's 8 halves of the summed axis, in fragment order.
__device__ __forceinline__ half8 row_frag(const _Float16* row, int ks, int q) {
  const half4 u = *(const half4*)(row + 32 * ks + 4 * q);
  const half4 v = *(const half4*)(row + 32 * ks + 16 + 4 * q);
  return half8{u[0], u[1], u[2], u[3], v[0], v[1], v[2], v[3]};
}

// Both pieces of the lower triangular tile in LDS (or of its transpose) to their
// blocks.  Wave w takes every fourth block.
template <bool TRANSPOSED>
__device__ __forceinline__ void write_tri(const float* tile, float s, Frag* dst) {
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, m = lane & 15, q = lane >> 4;
  for (int blk = w; blk < kTri; blk += 4) {
    int mt, ks;
    if (!TRANSPOSED) {
      mt = blk < 2 ? blk : 2 + (blk - 2) / 2;
      ks = blk < 2 ? 0 : (blk - 2) % 2;
    } else {
      mt = blk < 4 ? blk / 2 : blk - 2;
      ks = blk < 4 ? blk % 2 : 1;
    }
    half8 hi, lo;
    f32x4 rows[2] = {};
    if constexpr (!TRANSPOSED) {
      rows[0] = *(const f32x4*)(tile + (16 * mt + m) * kPitch + 32 * ks + 4 * q);
      rows[1] = *(const f32x4*)(tile + (16 * mt + m) * kPitch + 32 * ks + 16 + 4 * q);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int r = 16 * mt + m, c = 32 * ks + (j < 4 ? 4 * q + j : 12 + 4 * q + j);
      _Float16 h, l;
      split((TRANSPOSED ? tile[c * kPitch + r] : rows[j / 4][j % 4]) * s, &h, &l);
      hi[j] = h;
      lo[j] = l;
    }
    dst[blk * 64 + lane] = hi;
    dst[(kTri + blk) * 64 + lane] = lo;
  }
}

// T: type of q and k.  DP: head size padded.  NP: pieces of an input.  BWD:
// also the transposes.
template <int T, int DP, bool WIDE, bool BWD>
__global__ void __launch_bounds__(256, BWD ? 3 : 4) delta_prep(ChunkArgs c) {
  constexpr int NP = T == T_F32 ? 2 : 1;
  constexpr int KS = DP / 32, PITCH = DP + 8, PER = DP / 4;
  extern __shared__ __align__(16) char lds[];
  __shared__ float red[4][4];
  __shared__ __align__(16) double sg[4][kChunk];
  __shared__ __align__(16) float sbeta[4][kChunk];
  _Float16* rows = (_Float16*)lds;  // [k, q][piece][64][PITCH]
  float* tn = (float*)lds;          // N, then P
  float* tx = tn + kChunk * kPitch;
  const DeltaArgs& a = c.a;
  const int tid = threadIdx.x, lane = tid & 63, m = lane & 15, q = lane >> 4;
  const int w = uniform(tid >> 6);
  const int64_t id = blockIdx.x;
  const int hk = (int)(id % a.hk);
  const int64_t bc = id / a.hk;
  const int chunk = (int)(bc % c.nc);
  const int64_t b = bc / c.nc;
  const int64_t len = live_tokens(a, b), t0 = (int64_t)chunk * kChunk;
  if (t0 >= len) return;
  const int n = (int)(len - t0 < kChunk ? len - t0 : kChunk);

  const int per = a.hv / a.hk;
  // Wave w makes the gates of the w-th of the next four heads.
  const auto gates = [&](int first) {
    if (first + w >= per) return;
    const int h = hk * per + first + w;
    Gate* gate = c.gate + bc * a.hv + h;
    double g = 0.0;
    float beta = 0.f;
    if (lane < n) {
      // below -1e5 the decay is 0 anyway, and sums of it stay finite
      const float x = a.g[b * a.g_stride[0] + (t0 + lane) * a.g_stride[1] + h * a.g_stride[2]];
      g = (x < -1e5f ? -1e5 : (double)x) * kLog2e;
      beta = a.beta[b * a.beta_stride[0] + (t0 + lane) * a.beta_stride[1] + h * a.beta_stride[2]];
    }
    // sums in 64 bits: differences of far sums are what decays are made of
#pragma unroll
    for (int i = 1; i < 64; i <<= 1) {
      const double o = __shfl_up(g, i, 64);
      if (lane >= i) g += o;
    }
    const double all = __shfl(g, 63, 64);
    sg[w][lane] = g;
    sbeta[w][lane] = beta;
    gate->into[lane] = __builtin_amdgcn_exp2f((float)g);
    gate->out[lane] = __builtin_amdgcn_exp2f((float)(all - g));
    gate->beta[lane] = beta;
    gate->g[lane] = g;
    if (lane == 0) gate->total = __builtin_amdgcn_exp2f((float)all);
  };

  // K and Q to LDS as scaled pieces; places past the sequence or the head
  // size are zero whatever memory holds there
  float kinv = 0.f, qinv = 0.f;
  {
    // a thread takes every fourth 8 values of a row
    const int row = tid >> 2, part = tid & 3;
    float v[2][PER], mx[2] = {0.f, 0.f};
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const void* p = x ? a.q : a.k;
      const int64_t* st = x ? a.q_stride : a.k_stride;
      const int64_t base = b * st[0] + (t0 + row) * st[1] + hk * st[2];
#pragma unroll
      for (int i = 0; i < PER; i += 8) {
        const int col = 4 * i + 8 * part;
        if constexpr (WIDE) {
          if (row < n && col < a.dk) {
            load_vec<T, 8>(p, base + col, &v[x][i]);
          } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) v[x][i + j] = 0.f;
          }
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j)
            v[x][i + j] = row < n && col + j < a.dk ? load1<T>(p, base + col + j) : 0.f;
        }
      }
    }
    gates(0);
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
      for (int i = 0; i < PER; ++i) mx[x] = fmaxf(mx[x], fabsf(v[x][i]));
    const f32x2 top = block_max2(mx[0], mx[1], red);
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const Scale s = scale_of(top[x]);
      (x ? qinv : kinv) = s.inv;
#pragma unroll
      for (int i = 0; i < PER; i += 8) {
        half8 hi, lo;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          _Float16 h, l;
          split(v[x][i + j] * s.mul, &h, &l);
          hi[j] = h;
          lo[j] = l;
        }
        _Float16* dst = rows + ((x * NP) * kChunk + row) * PITCH + 4 * i + 8 * part;
        *(half8*)dst = hi;
        if constexpr (NP == 2) *(half8*)(dst + kChunk * PITCH) = lo;
      }
    }
    __syncthreads();
  }
  // fragments of K and Q (rows are tokens), and this wave's rows of K K^T
  // and Q K^T
  f32x4 kk[4], qk[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) kk[j] = qk[j] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int ks = 0; ks < KS; ++ks) {
    half8 fk[NP], fq[NP];
#pragma unroll
    for (int p = 0; p < NP; ++p) {
      fk[p] = row_frag(rows + (p * kChunk + 16 * w + m) * PITCH, ks, q);
      fq[p] = row_frag(rows + ((NP + p) * kChunk + 16 * w + m) * PITCH, ks, q);
      const int64_t at = ((id * NP + p) * 4 * KS + w * KS + ks) * 64 + lane;
      c.ka[at] = fk[p];
      if (!BWD) c.qa[at] = fq[p];
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (j > w) continue;
      half8 fb[NP];
#pragma unroll
      for (int p = 0; p < NP; ++p)
        fb[p] = row_frag(rows + (p * kChunk + 16 * j + m) * PITCH, ks, q);
      kk[j] = mfma_pieces<NP, NP>(fk, fb, kk[j]);
      qk[j] = mfma_pieces<NP, NP>(fq, fb, qk[j]);
    }
  }
  if constexpr (BWD) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (j > w) continue;
      const int64_t at = (id * kLow + low_block(w, j)) * 64 + lane;
      c.kk[at] = kk[j] * kinv * kinv;
      c.qk[at] = qk[j] * kinv * qinv;
    }
  }
  // fragments of the transposes (rows are key dimensions)
#pragma unroll
  for (int p = 0; p < NP; ++p) {
    for (int blk = w; blk < DP / 16 * 2; blk += 4) {
      const int mt = blk >> 1, ks = blk & 1;
      half8 fk, fq;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int t = 32 * ks + (j < 4 ? 4 * q + j : 12 + 4 * q + j);
        fk[j] = rows[(p * kChunk + t) * PITCH + 16 * mt + m];
        if (BWD) fq[j] = rows[((NP + p) * kChunk + t) * PITCH + 16 * mt + m];
      }
      const int64_t at = ((id * NP + p) * (DP / 16 * 2) + blk) * 64 + lane;
      c.kt[at] = fk;
      if (BWD) c.qt[at] = fq;
    }
  }

  for (int r = 0; r < per; ++r) {
    const int h = hk * per + r;
    const int64_t hid = bc * a.hv + h;
    Gate* gate = c.gate + hid;
    __syncthreads();  // the rows, or the last head's tiles, are read
    if (r && r % 4 == 0) {
      gates(r);
      __syncthreads();
    }
    const double* g = sg[r % 4];
    const float* beta = sbeta[r % 4];
    f32x4 pv[4];
    float pmax = 0.f;
    double grow[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) grow[i] = g[16 * w + 4 * q + i];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      pv[j] = f32x4{0.f, 0.f, 0.f, 0.f};
      f32x4 nv = pv[j];
      if (j <= w) {
        const double gcol = g[16 * j + m];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int row = 16 * w + 4 * q + i, col = 16 * j + m;
          const float d =
              col <= row ? __builtin_amdgcn_exp2f((float)(grow[i] - gcol)) : 0.f;
          nv[i] = col < row ? d * (kk[j][i] * kinv * kinv) : 0.f;
          pv[j][i] = a.scale * d * (qk[j][i] * kinv * qinv);
          pmax = fmaxf(pmax, fabsf(pv[j][i]));
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) tn[(16 * w + 4 * q + i) * kPitch + 16 * j + m] = nv[i];
    }
    __syncthreads();
    // X = N - N beta X in 16x16 blocks, wave w the block column w.  On the
    // diagonal by substitution (a lane a column, four lanes the same one) ...
    f32x4 x[4];
    {
      float y[16];
#pragma unroll
      for (int t = 0; t < 16; ++t) {
        const float* row = tn + (16 * w + t) * kPitch + 16 * w;
        y[t] = row[m];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          if (4 * k >= t) continue;
          const f32x4 nb = *(const f32x4*)(row + 4 * k) * *(const f32x4*)(beta + 16 * w + 4 * k);
#pragma unroll
          for (int z = 0; z < 4; ++z)
            if (4 * k + z < t) y[t] = fmaf(-nb[z], y[4 * k + z], y[t]);
        }
      }
      f32x4 d;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        d[i] = q < 2 ? (q == 0 ? y[i] : y[4 + i]) : (q == 2 ? y[8 + i] : y[12 + i]);
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = i == w ? d : f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (i > w) break;
#pragma unroll
        for (int z = 0; z < 4; ++z) tx[(16 * i + 4 * q + z) * kPitch + 16 * w + m] = x[i][z];
      }
    }
    __syncthreads();
    // ... and below it, with (1 + N_ii beta)^-1 = 1 - X_ii beta:
    // X_iw = R - X_ii beta R,  R = N_iw - sum over k of N_ik beta X_kw
#pragma unroll
    for (int i = 1; i < 4; ++i) {
      if (i <= w) continue;
      f32x4 acc = {0.f, 0.f, 0.f, 0.f}, nw;
#pragma unroll
      for (int k = 0; k < 3; ++k) {
        if (k >= i || k < w) continue;
        const f32x4 nb = *(const f32x4*)(tn + (16 * i + m) * kPitch + 16 * k + 4 * q) *
                         *(const f32x4*)(beta + 16 * k + 4 * q);
        acc = mul16(nb, x[k], acc);
      }
#pragma unroll
      for (int z = 0; z < 4; ++z)
        nw[z] = tn[(16 * i + 4 * q + z) * kPitch + 16 * w + m] - acc[z];
      const f32x4 xb = *(const f32x4*)(tx + (16 * i + m) * kPitch + 16 * i + 4 * q) *
                       *(const f32x4*)(beta + 16 * i + 4 * q);
      x[i] = nw - mul16(xb, nw, f32x4{0.f, 0.f, 0.f, 0.f});
#pragma unroll
      for (int z = 0; z < 4; ++z) tx[(16 * i + 4 * q + z) * kPitch + 16 * w + m] = x[i][z];
    }
    const f32x2 top = block_max2(abs_max(x), pmax, red + 2);
    const Scale xs = scale_of(top[0]), ps = scale_of(top[1]);
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) tn[(16 * w + 4 * q + i) * kPitch + 16 * j + m] = pv[j][i];
    __syncthreads();
    if (tid == 0) {
      gate->xinv = xs.inv;
      gate->pinv = ps.inv;
      gate->kinv = kinv;
      gate->qinv = qinv;
      if constexpr (BWD) {
        const float most = fmaxf(kinv, qinv);
        gate->top = most;
        gate->kpart = kinv / most;  // powers of two: exact
        gate->qpart = qinv / most;
      }
    }
    write_tri<false>(tx, xs.mul, c.xa + hid * 2 * kTri * 64);
    if constexpr (BWD) {
      write_tri<true>(tx, xs.mul, c.xt + hid * 2 * kTri * 64);
      write_tri<true>(tn, ps.mul, c.pt + hid * 2 * kTri * 64);
    } else {
      write_tri<false>(tn, ps.mul, c.pa + hid * 2 * kTri * 64);
    }
  }
}

template <int T, int DP, bool BWD>
hipError_t go(const ChunkArgs& c, hipStream_t st) {
  const DeltaArgs& a = c.a;
  const int64_t e = ElemBytes<T>::value, unit = 16 / e;
  bool wide = a.dk % 8 == 0;
  for (int i = 0; i < 3; ++i) wide = wide && a.q_stride[i] % unit == 0 && a.k_stride[i] % unit == 0;
  wide = wide && (((uintptr_t)a.q | (uintptr_t)a.k) % 16) == 0;
  constexpr int bytes = lds_bytes<T == T_F32 ? 2 : 1>(DP);
  const dim3 grid((uint32_t)(a.b * c.nc * a.hk));
  auto* f = wide ? &delta_prep<T, DP, true, BWD> : &delta_prep<T, DP, false, BWD>;
  if (bytes > 64 * 1024) {  // more than a launch may ask for unasked
    const hipError_t err = hipFuncSetAttribute(reinterpret_cast<const void*>(f),
                                               hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (err != hipSuccess) return err;
  }
  hipLaunchKernelGGL(f, grid, dim3(256), bytes, st, c);
  return hipGetLastError();
}

template <int T>
hipError_t go_dp(const ChunkArgs& c, bool bwd, hipStream_t st) {
  if (c.a.dk <= 64) return bwd ? go<T, 64, true>(c, st) : go<T, 64, false>(c, st);
  return bwd ? go<T, 128, true>(c, st) : go<T, 128, false>(c, st);
}

}  // namespace prep

hipError_t launch_delta_prep(const ChunkArgs& c, bool bwd, hipStream_t st) {
  if (c.a.type == T_F32) return prep::go_dp<T_F32>(c, bwd, st);
  if (c.a.type == T_BF16) return prep::go_dp<T_BF16>(c, bwd, st);
  return prep::go_dp<T_F16>(c, bwd, st);
}

}  // namespace seq
}  // namespace dwc
