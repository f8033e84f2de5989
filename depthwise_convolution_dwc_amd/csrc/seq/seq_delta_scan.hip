// seq_delta_scan.hip -- the serial part of the chunked gated delta rule, and
// of its gradient (formulas in seq_chunk.h).
//
// A column of the state depends on no other, so a wave owns 16 columns for
// the whole sequence and holds them in fp32 as 16x16 results of the matrix
// cores (MT tiles of 4 registers).  Every product of the recurrence has the
// state or something made of it on the right and a shared fragment on the
// left, and each result is the next operand without leaving its lane: waves
// share nothing and never wait for each other.
#include "seq_chunk.h"

namespace dwc {
namespace seq {
namespace scan {

// The 4 fp32 values of rows 16 i + 4 q .. + 3.
__device__ __forceinline__ f32x4 row4(const float* p, int i, int q) {
  return *(const f32x4*)(p + 16 * i + 4 * q);
}

// The wave's part in one (sequence, value head) and its 16 columns.
struct Place {
  int64_t b, head;
  int h, hk, col, groups;
  bool ok, any;
};

__device__ __forceinline__ Place place_of(const ChunkArgs& c) {
  Place p;
  const DeltaArgs& a = c.a;
  const int groups = c.dvp / 16;
  const int64_t wave = (int64_t)blockIdx.x * (blockDim.x >> 6) + (threadIdx.x >> 6);
  p.any = wave < a.b * a.hv * groups;
  p.head = wave / groups;
  p.col = (int)(wave - p.head * groups) * 16 + (threadIdx.x & 15);
  p.b = p.head / a.hv;
  p.h = (int)(p.head - p.b * a.hv);
  p.hk = p.h / (a.hv / a.hk);
  p.ok = p.col < a.dv;
  p.groups = groups;
  return p;
}

template <int T, int DP, bool BWD>
__global__ void __launch_bounds__(256) delta_scan(ChunkArgs c) {
  constexpr int NP = T == T_F32 ? 2 : 1, OP = T == T_BF16 ? 1 : 2;
  constexpr int KS = DP / 32, MT = DP / 16;
  const DeltaArgs& a = c.a;
  const Place p = place_of(c);
  if (!p.any) return;
  const int lane = threadIdx.x & 63, m = lane & 15, q = lane >> 4;
  const int64_t len = live_tokens(a, p.b);
  const int chunks = (int)((len + kChunk - 1) / kChunk);
  f32x4 s[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int row = 16 * i + 4 * q + r;
      s[i][r] = a.s0 && p.ok && row < a.dk
                    ? a.s0[(p.head * a.dk + row) * a.dv + p.col] : 0.f;
    }
  for (int chunk = 0; chunk < chunks; ++chunk) {
    const int64_t bc = p.b * c.nc + chunk, kid = bc * a.hk + p.hk, hid = bc * a.hv + p.h;
    const int64_t t0 = (int64_t)chunk * kChunk;
    const int n = (int)(len - t0 < kChunk ? len - t0 : kChunk);
    const Gate* gate = c.gate + hid;
    const float kinv = c.kq_inv[2 * kid], qinv = c.kq_inv[2 * kid + 1];
    const Frag* ka = c.ka + kid * NP * 4 * KS * 64 + lane;
    const Frag* kt = c.kt + kid * NP * MT * 2 * 64 + lane;
    const Frag* xa = c.xa + hid * 2 * kTri * 64 + lane;
    if constexpr (BWD) {
      float* st = c.states + hid * DP * c.dvp + p.col;
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) st[(int64_t)(16 * i + 4 * q + r) * c.dvp] = s[i][r];
    }
    f32x4 e[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int t = 16 * i + 4 * q + r;
        e[i][r] = p.ok && t < n ? load1<T>(a.v, p.b * a.v_stride[0] + (t0 + t) * a.v_stride[1] +
                                                    p.h * a.v_stride[2] + p.col)
                                : 0.f;
      }
    half8 fs[KS][2];
    const Scale ss = scale_of(column_max(abs_max(s)));
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) to_frag<2>(s[2 * ks], s[2 * ks + 1], ss.mul, fs[ks]);
    // e = V - exp(G) o (K S)
    const float cks = kinv * ss.inv;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        half8 f[NP];
#pragma unroll
        for (int x = 0; x < NP; ++x) f[x] = ka[((x * 4 + i) * KS + ks) * 64];
        acc = mfma_pieces<NP, 2>(f, fs[ks], acc);
      }
      const f32x4 into = row4(gate->into, i, q);
#pragma unroll
      for (int r = 0; r < 4; ++r) e[i][r] -= into[r] * (cks * acc[r]);
    }
    // E = e - X (beta o e)
    f32x4 u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const f32x4 beta = row4(gate->beta, i, q);
#pragma unroll
      for (int r = 0; r < 4; ++r) u[i][r] = beta[r] * e[i][r];
    }
    half8 fu[2][2];
    Scale us = scale_of(column_max(abs_max(u)));
    to_frag<2>(u[0], u[1], us.mul, fu[0]);
    to_frag<2>(u[2], u[3], us.mul, fu[1]);
    const float cx = gate->xinv * us.inv;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int ks = 0; ks < (i < 2 ? 1 : 2); ++ks) {
        const half8 f[2] = {xa[tri_block(i, ks) * 64], xa[(kTri + tri_block(i, ks)) * 64]};
        acc = mfma_pieces<2, 2>(f, fu[ks], acc);
      }
#pragma unroll
      for (int r = 0; r < 4; ++r) e[i][r] -= cx * acc[r];
    }
    if constexpr (BWD) {
      float* ep = c.e + hid * kChunk * c.dvp + p.col;
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) ep[(int64_t)(16 * i + 4 * q + r) * c.dvp] = e[i][r];
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const f32x4 beta = row4(gate->beta, i, q);
#pragma unroll
      for (int r = 0; r < 4; ++r) u[i][r] = beta[r] * e[i][r];
    }
    if constexpr (!BWD) {
      // O = scale exp(G) o (Q S) + P U; an output of 16 bits takes fewer
      // pieces: bf16 one of each (2^-12 against its 2^-9), fp16 two
      const Frag* qa = c.qa + kid * NP * 4 * KS * 64 + lane;
      const Frag* pa = c.pa + hid * OP * kTri * 64 + lane;
      us = scale_of(column_max(abs_max(u)));
      to_frag<OP>(u[0], u[1], us.mul, fu[0]);
      to_frag<OP>(u[2], u[3], us.mul, fu[1]);
      const float cq = a.scale * qinv * ss.inv, cp = gate->pinv * us.inv;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        f32x4 acc = {0.f, 0.f, 0.f, 0.f}, acc2 = acc;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
          half8 f[NP];
#pragma unroll
          for (int x = 0; x < NP; ++x) f[x] = qa[((x * 4 + i) * KS + ks) * 64];
          acc = mfma_pieces<NP, OP>(f, fs[ks], acc);
        }
#pragma unroll
        for (int ks = 0; ks < (i < 2 ? 1 : 2); ++ks) {
          half8 f[OP];
#pragma unroll
          for (int x = 0; x < OP; ++x) f[x] = pa[(x * kTri + tri_block(i, ks)) * 64];
          acc2 = mfma_pieces<OP, OP>(f, fu[ks], acc2);
        }
        const f32x4 into = row4(gate->into, i, q);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int64_t t = t0 + 16 * i + 4 * q + r;
          if (p.ok && t < a.l)
            store1<T>(a.o, ((p.b * a.l + t) * a.hv + p.h) * a.dv + p.col,
                      t < len ? fmaf(cq * into[r], acc[r], cp * acc2[r]) : 0.f);
        }
      }
    }
    // S <- exp(G_64) S + K^T (exp(G_64 - G) o U)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const f32x4 out = row4(gate->out, i, q);
#pragma unroll
      for (int r = 0; r < 4; ++r) u[i][r] *= out[r];
    }
    us = scale_of(column_max(abs_max(u)));
    to_frag<2>(u[0], u[1], us.mul, fu[0]);
    to_frag<2>(u[2], u[3], us.mul, fu[1]);
    const float ck = kinv * us.inv, total = gate->total;
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) {
        half8 f[NP];
#pragma unroll
        for (int x = 0; x < NP; ++x) f[x] = kt[((x * MT + i) * 2 + ks) * 64];
        acc = mfma_pieces<NP, 2>(f, fu[ks], acc);
      }
#pragma unroll
      for (int r = 0; r < 4; ++r) s[i][r] = fmaf(ck, acc[r], total * s[i][r]);
    }
  }
  if constexpr (!BWD) {
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int row = 16 * i + 4 * q + r;
        if (p.ok && row < a.dk) a.s1[(p.head * a.dk + row) * a.dv + p.col] = s[i][r];
      }
    // outputs past the last live chunk
    if (p.ok)
      for (int64_t t = (int64_t)chunks * kChunk + q; t < a.l; t += 4)
        store1<T>(a.o, ((p.b * a.l + t) * a.hv + p.h) * a.dv + p.col, 0.f);
  }
}

// With W = dL/dU in full, dS the gradient of the state after the chunk:
//   dU = P^T dO + exp(G_64 - G) o (K dS),   W = dU - X^T (beta o dU),
//   dV = beta o W,
//   dS <- exp(G_64) dS + Q^T (scale exp(G) o dO) - K^T (exp(G) o dV).
template <int T, int DP>
__global__ void __launch_bounds__(256) delta_scan_bwd(ChunkArgs c) {
  constexpr int NP = T == T_F32 ? 2 : 1;
  constexpr int KS = DP / 32, MT = DP / 16;
  const DeltaArgs& a = c.a;
  const Place p = place_of(c);
  if (!p.any) return;
  const int lane = threadIdx.x & 63, q = lane >> 4;
  const int64_t len = live_tokens(a, p.b);
  const int chunks = (int)((len + kChunk - 1) / kChunk);
  f32x4 s[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int row = 16 * i + 4 * q + r;
      s[i][r] = a.ds1 && p.ok && row < a.dk
                    ? a.ds1[(p.head * a.dk + row) * a.dv + p.col] : 0.f;
    }
  for (int chunk = chunks - 1; chunk >= 0; --chunk) {
    const int64_t bc = p.b * c.nc + chunk, kid = bc * a.hk + p.hk, hid = bc * a.hv + p.h;
    const int64_t t0 = (int64_t)chunk * kChunk;
    const int n = (int)(len - t0 < kChunk ? len - t0 : kChunk);
    const Gate* gate = c.gate + hid;
    const float kinv = c.kq_inv[2 * kid], qinv = c.kq_inv[2 * kid + 1];
    const Frag* ka = c.ka + kid * NP * 4 * KS * 64 + lane;
    const Frag* kt = c.kt + kid * NP * MT * 2 * 64 + lane;
    const Frag* qt = c.qt + kid * NP * MT * 2 * 64 + lane;
    const Frag* xt = c.xt + hid * 2 * kTri * 64 + lane;
    const Frag* pt = c.pt + hid * 2 * kTri * 64 + lane;
    float* st = c.dstates + hid * DP * c.dvp + p.col;
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r) st[(int64_t)(16 * i + 4 * q + r) * c.dvp] = s[i][r];
    f32x4 d[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int t = 16 * i + 4 * q + r;
        d[i][r] = p.ok && t < n
                      ? load1<T>(a.dout, p.b * a.do_stride[0] + (t0 + t) * a.do_stride[1] +
                                             p.h * a.do_stride[2] + p.col)
                      : 0.f;
      }
    half8 fd[2][NP];
    const Scale ds = scale_of(column_max(abs_max(d)));
    to_frag<NP>(d[0], d[1], ds.mul, fd[0]);
    to_frag<NP>(d[2], d[3], ds.mul, fd[1]);
    half8 fs[KS][2];
    const Scale ss = scale_of(column_max(abs_max(s)));
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) to_frag<2>(s[2 * ks], s[2 * ks + 1], ss.mul, fs[ks]);
    const float cks = kinv * ss.inv, cp = gate->pinv * ds.inv;
    f32x4 w[4], y[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f32x4 acc = {0.f, 0.f, 0.f, 0.f}, acc2 = acc;
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        half8 f[NP];
#pragma unroll
        for (int x = 0; x < NP; ++x) f[x] = ka[((x * 4 + i) * KS + ks) * 64];
        acc = mfma_pieces<NP, 2>(f, fs[ks], acc);
      }
#pragma unroll
      for (int ks = (i < 2 ? 0 : 1); ks < 2; ++ks) {
        const half8 f[2] = {pt[tri_block_t(i, ks) * 64], pt[(kTri + tri_block_t(i, ks)) * 64]};
        acc2 = mfma_pieces<2, NP>(f, fd[ks], acc2);
      }
      const f32x4 out = row4(gate->out, i, q), beta = row4(gate->beta, i, q);
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        w[i][r] = fmaf(cks * out[r], acc[r], cp * acc2[r]);
        y[i][r] = beta[r] * w[i][r];
      }
    }
    half8 fy[2][2];
    Scale ys = scale_of(column_max(abs_max(y)));
    to_frag<2>(y[0], y[1], ys.mul, fy[0]);
    to_frag<2>(y[2], y[3], ys.mul, fy[1]);
    const float cx = gate->xinv * ys.inv;
    float* wp = c.dw + hid * kChunk * c.dvp + p.col;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int ks = (i < 2 ? 0 : 1); ks < 2; ++ks) {
        const half8 f[2] = {xt[tri_block_t(i, ks) * 64], xt[(kTri + tri_block_t(i, ks)) * 64]};
        acc = mfma_pieces<2, 2>(f, fy[ks], acc);
      }
      const f32x4 beta = row4(gate->beta, i, q), into = row4(gate->into, i, q);
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int64_t t = t0 + 16 * i + 4 * q + r;
        w[i][r] -= cx * acc[r];
        wp[(int64_t)(16 * i + 4 * q + r) * c.dvp] = w[i][r];
        const float dv = beta[r] * w[i][r];
        if (p.ok && t < a.l)
          store1<T>(a.dv_out, ((p.b * a.l + t) * a.hv + p.h) * a.dv + p.col, t < len ? dv : 0.f);
        y[i][r] = -into[r] * dv * kinv;
        d[i][r] *= a.scale * into[r] * qinv;
      }
    }
    // one scale for both operands, so that one sum takes both products
    half8 fq[2][2];
    ys = scale_of(column_max(fmaxf(abs_max(y), abs_max(d))));
    to_frag<2>(y[0], y[1], ys.mul, fy[0]);
    to_frag<2>(y[2], y[3], ys.mul, fy[1]);
    to_frag<2>(d[0], d[1], ys.mul, fq[0]);
    to_frag<2>(d[2], d[3], ys.mul, fq[1]);
    const float total = gate->total;
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) {
        half8 f[NP], g[NP];
#pragma unroll
        for (int x = 0; x < NP; ++x) {
          f[x] = kt[((x * MT + i) * 2 + ks) * 64];
          g[x] = qt[((x * MT + i) * 2 + ks) * 64];
        }
        acc = mfma_pieces<NP, 2>(f, fy[ks], acc);
        acc = mfma_pieces<NP, 2>(g, fq[ks], acc);
      }
#pragma unroll
      for (int r = 0; r < 4; ++r) s[i][r] = fmaf(ys.inv, acc[r], total * s[i][r]);
    }
  }
  if (a.ds0) {
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int row = 16 * i + 4 * q + r;
        if (p.ok && row < a.dk) a.ds0[(p.head * a.dk + row) * a.dv + p.col] = s[i][r];
      }
  }
  if (p.ok)
    for (int64_t t = (int64_t)chunks * kChunk + q; t < a.l; t += 4)
      store1<T>(a.dv_out, ((p.b * a.l + t) * a.hv + p.h) * a.dv + p.col, 0.f);
}

inline dim3 grid_of(const ChunkArgs& c, int waves) {
  const int64_t n = c.a.b * c.a.hv * (c.dvp / 16);
  return dim3((uint32_t)((n + waves - 1) / waves));
}

// Waves of a workgroup share fragments through the L1; with few columns one
// wave a workgroup spreads them over more compute units.
inline int waves_of(const ChunkArgs& c) {
  return c.a.b * c.a.hv * (c.dvp / 16) >= 1024 ? 4 : 1;
}

template <int T, int DP>
void go(const ChunkArgs& c, int what, hipStream_t st) {
  const int waves = waves_of(c);
  if (what == 0)
    hipLaunchKernelGGL((delta_scan<T, DP, false>), grid_of(c, waves), dim3(64 * waves), 0, st, c);
  else if (what == 1)
    hipLaunchKernelGGL((delta_scan<T, DP, true>), grid_of(c, waves), dim3(64 * waves), 0, st, c);
  else
    hipLaunchKernelGGL((delta_scan_bwd<T, DP>), grid_of(c, waves), dim3(64 * waves), 0, st, c);
}

template <int T>
void go_dp(const ChunkArgs& c, int what, hipStream_t st) {
  if (c.a.dk <= 64) go<T, 64>(c, what, st);
  else go<T, 128>(c, what, st);
}

inline hipError_t go_type(const ChunkArgs& c, int what, hipStream_t st) {
  if (c.a.type == T_F32) go_dp<T_F32>(c, what, st);
  else if (c.a.type == T_BF16) go_dp<T_BF16>(c, what, st);
  else go_dp<T_F16>(c, what, st);
  return hipGetLastError();
}

}  // namespace scan

hipError_t launch_delta_scan(const ChunkArgs& c, bool bwd, hipStream_t st) {
  return scan::go_type(c, bwd ? 1 : 0, st);
}

hipError_t launch_delta_scan_bwd(const ChunkArgs& c, hipStream_t st) {
  return scan::go_type(c, 2, st);
}

}  // namespace seq
}  // namespace dwc
