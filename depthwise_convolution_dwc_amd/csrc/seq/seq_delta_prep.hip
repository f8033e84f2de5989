// seq_delta_prep.hip -- what each chunk of the gated delta rule needs and no
// state enters: fragments of K, Q and their transposes, the gates, and the
// triangular X and P (see seq_chunk.h).  All chunks run at once.
//
// One workgroup of 4 waves a (sequence, chunk, key head); the value heads
// that share the key head reuse K K^T and Q K^T from registers.
#include "seq_chunk.h"

namespace dwc {
namespace seq {
namespace prep {

constexpr int kPitch = 65;  // of the 64x64 fp32 tiles in LDS: no two rows on one bank

__device__ __forceinline__ float block_max(float m, float* red) {
#pragma unroll
  for (int i = 1; i < 64; i <<= 1) m = fmaxf(m, __shfl_xor(m, i, 64));
  __syncthreads();
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = m;
  __syncthreads();
  return fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
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

// Pieces of the lower triangular tile in LDS (or of its transpose) to their
// blocks.  Wave w takes every fourth block.
template <int P, bool TRANSPOSED>
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
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int r = 16 * mt + m, c = 32 * ks + (j < 4 ? 4 * q + j : 12 + 4 * q + j);
      const float v = (TRANSPOSED ? tile[c * kPitch + r] : tile[r * kPitch + c]) * s;
      _Float16 h, l;
      split(v, &h, &l);
      hi[j] = h;
      lo[j] = l;
    }
    dst[blk * 64 + lane] = hi;
    if constexpr (P == 2) dst[(kTri + blk) * 64 + lane] = lo;
  }
}

// T: type of q and k.  DP: head size padded.  NP: pieces of an input.  OP:
// pieces of P in the forward pass.  BWD: also the transposes.
template <int T, int DP, bool WIDE, bool BWD>
__global__ void __launch_bounds__(256) delta_prep(ChunkArgs c) {
  constexpr int NP = T == T_F32 ? 2 : 1, OP = T == T_BF16 ? 1 : 2;
  constexpr int KS = DP / 32, PITCH = DP + 8, PER = DP / 4;
  extern __shared__ __align__(16) char lds[];
  __shared__ float red[4];
  __shared__ double sg[kChunk];
  __shared__ float sbeta[kChunk];
  _Float16* rows = (_Float16*)lds;  // [k, q][piece][64][PITCH]
  float* tn = (float*)lds;          // N, then P
  float* tx = tn + kChunk * kPitch;
  const DeltaArgs& a = c.a;
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6, m = lane & 15, q = lane >> 4;
  const int64_t id = blockIdx.x;
  const int hk = (int)(id % a.hk);
  const int64_t bc = id / a.hk;
  const int chunk = (int)(bc % c.nc);
  const int64_t b = bc / c.nc;
  const int64_t len = live_tokens(a, b), t0 = (int64_t)chunk * kChunk;
  if (t0 >= len) return;
  const int n = (int)(len - t0 < kChunk ? len - t0 : kChunk);

  // K and Q to LDS as scaled pieces; places past the sequence or the head
  // size are zero whatever memory holds there
  float kinv, qinv;
  {
    const int row = tid >> 2, part = tid & 3;
    float v[2][PER];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const void* p = x ? a.q : a.k;
      const int64_t* st = x ? a.q_stride : a.k_stride;
      const int64_t base = b * st[0] + (t0 + row) * st[1] + hk * st[2] + part * PER;
      float mx = 0.f;
      if constexpr (WIDE) {
#pragma unroll
        for (int i = 0; i < PER; i += 8) {
          if (row < n && part * PER + i < a.dk) {
            load_vec<T, 8>(p, base + i, &v[x][i]);
          } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) v[x][i + j] = 0.f;
          }
        }
      } else {
#pragma unroll
        for (int i = 0; i < PER; ++i)
          v[x][i] = row < n && part * PER + i < a.dk ? load1<T>(p, base + i) : 0.f;
      }
#pragma unroll
      for (int i = 0; i < PER; ++i) mx = fmaxf(mx, fabsf(v[x][i]));
      const Scale s = scale_of(block_max(mx, red));
      (x ? qinv : kinv) = s.inv;
#pragma unroll
      for (int i = 0; i < PER; i += 4) {
        half4 hi, lo;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          _Float16 h, l;
          split(v[x][i + j] * s.mul, &h, &l);
          hi[j] = h;
          lo[j] = l;
        }
        _Float16* dst = rows + ((x * NP) * kChunk + row) * PITCH + part * PER + i;
        *(half4*)dst = hi;
        if constexpr (NP == 2) *(half4*)(dst + kChunk * PITCH) = lo;
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

  const int per = a.hv / a.hk;
  for (int r = 0; r < per; ++r) {
    const int h = hk * per + r;
    const int64_t hid = bc * a.hv + h;
    Gate* gate = c.gate + hid;
    __syncthreads();  // the rows, or the last head's tiles, are read
    if (w == 0) {
      double g = 0.0;
      float beta = 0.f;
      if (lane < n) {
        // below -1e5 the decay is 0 anyway, and sums of it stay finite
        const float x =
            a.g[b * a.g_stride[0] + (t0 + lane) * a.g_stride[1] + h * a.g_stride[2]];
        g = x < -1e5f ? -1e5 : (double)x;
        beta = a.beta[b * a.beta_stride[0] + (t0 + lane) * a.beta_stride[1] +
                      h * a.beta_stride[2]];
      }
      // sums in 64 bits: differences of far sums are what decays are made of
#pragma unroll
      for (int i = 1; i < 64; i <<= 1) {
        const double o = __shfl_up(g, i, 64);
        if (lane >= i) g += o;
      }
      const double all = __shfl(g, 63, 64);
      sg[lane] = g;
      sbeta[lane] = beta;
      gate->into[lane] = expf((float)g);
      gate->out[lane] = expf((float)(all - g));
      gate->beta[lane] = beta;
      gate->g[lane] = g;
      if (lane == 0) gate->total = expf((float)all);
    }
    __syncthreads();
    f32x4 pv[4];
    float pmax = 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int row = 16 * w + 4 * q + i, col = 16 * j + m;
        float nv = 0.f;
        pv[j][i] = 0.f;
        if (col <= row) {
          const float d = expf((float)(sg[row] - sg[col]));
          if (col < row) nv = d * (kk[j][i] * kinv * kinv);
          pv[j][i] = a.scale * d * (qk[j][i] * kinv * qinv);
        }
        pmax = fmaxf(pmax, fabsf(pv[j][i]));
        tn[row * kPitch + col] = nv;
      }
    }
    __syncthreads();
    // X = N - N beta X, 16 rows at a time: what the rows above give, by all
    // waves (a lane a column), then the 16 rows among themselves
    for (int i = 0; i < 4; ++i) {
      float acc[4];
#pragma unroll
      for (int x = 0; x < 4; ++x) acc[x] = tn[(16 * i + 4 * w + x) * kPitch + lane];
      for (int j = 0; j < 16 * i; ++j) {
        const float y = sbeta[j] * tx[j * kPitch + lane];
#pragma unroll
        for (int x = 0; x < 4; ++x)
          acc[x] = fmaf(-tn[(16 * i + 4 * w + x) * kPitch + j], y, acc[x]);
      }
#pragma unroll
      for (int x = 0; x < 4; ++x) tx[(16 * i + 4 * w + x) * kPitch + lane] = acc[x];
      __syncthreads();
      if (w == 0) {
        float x[16];
#pragma unroll
        for (int t = 0; t < 16; ++t) {
          x[t] = tx[(16 * i + t) * kPitch + lane];
#pragma unroll
          for (int s = 0; s < t; ++s)
            x[t] = fmaf(-tn[(16 * i + t) * kPitch + 16 * i + s] * sbeta[16 * i + s], x[s], x[t]);
          tx[(16 * i + t) * kPitch + lane] = x[t];
        }
      }
      __syncthreads();
    }
    float xmax = 0.f;
#pragma unroll
    for (int t = 0; t < 16; ++t) xmax = fmaxf(xmax, fabsf(tx[(16 * w + t) * kPitch + lane]));
    const Scale xs = scale_of(block_max(xmax, red)), ps = scale_of(block_max(pmax, red));
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
    }
    write_tri<2, false>(tx, xs.mul, c.xa + hid * 2 * kTri * 64);
    if constexpr (BWD) {
      write_tri<2, true>(tx, xs.mul, c.xt + hid * 2 * kTri * 64);
      write_tri<2, true>(tn, ps.mul, c.pt + hid * 2 * kTri * 64);
    } else {
      write_tri<OP, false>(tn, ps.mul, c.pa + hid * OP * kTri * 64);
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
