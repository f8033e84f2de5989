// seq_delta_token.hip -- the gated delta rule token by token:
//   u = beta (v - (a S)^T k),  S <- a S + k u^T,  o = scale S^T q,  a = exp(g)
// and so o = scale (a S^T q + (q.k) u): both products of the state that a
// token needs are of the state before it, which is read once.
//
// A wave owns 4 CL columns of one head's state for all tokens and keeps them
// in registers, CL lanes across (16 bytes each) and 64 / CL groups of RPL
// rows down, so tokens need no barrier and waves nothing of each other, and a
// lane's part of q and k is contiguous.  Bound for one
// token of many sequences: memory, the state read and written once (128
// sequences of 32 heads, 128x128: 94 us, 5.7 TB/s); for one sequence the
// latency of its loads (8 heads: 5 us).
#include "seq_delta.h"
#include "seq_device.h"

namespace dwc {
namespace seq {
namespace token {

// Sum over the lanes of a column: lanes that agree modulo CL.  Every one gets
// the same bits.
template <int CL>
__device__ __forceinline__ float group_sum(float v) {
  if constexpr (CL <= 8) v += row_move<0x128>(v);
  if constexpr (CL <= 4) v += row_move<0x124>(v);
  if constexpr (CL <= 2) v += row_move<0x122>(v);
  float o;
  rows16(v, o);
  v += o;
  halves(v, o);
  return v + o;
}

// RPL elements from element i of a row of dk; 8 (or 4) at a time where KWIDE.
template <int T, int RPL, bool KWIDE>
__device__ __forceinline__ void load_part(const void* p, int64_t base, int i, int dk, float* v) {
  constexpr int N = RPL < 8 ? RPL : 8;
#pragma unroll
  for (int r = 0; r < RPL; r += N) {
    if constexpr (KWIDE) {
      if (i + r < dk) {
        load_vec<T, N>(p, base + i + r, v + r);
      } else {
#pragma unroll
        for (int j = 0; j < N; ++j) v[r + j] = 0.f;
      }
    } else {
#pragma unroll
      for (int j = 0; j < N; ++j) v[r + j] = i + r + j < dk ? load1<T>(p, base + i + r + j) : 0.f;
    }
  }
}

template <int T, int CL, int RPL, bool WIDE, bool KWIDE>
__global__ void __launch_bounds__(256) delta_token(DeltaArgs a) {
  const int lane = threadIdx.x & 63, cl = lane % CL, i0 = lane / CL * RPL;
  const int tiles = (a.dv + 4 * CL - 1) / (4 * CL);
  const int64_t wave = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (wave >= (int64_t)a.b * a.hv * tiles) return;
  const int64_t head = wave / tiles;  // b * hv + h
  const int c0 = (int)(wave - head * tiles) * 4 * CL + 4 * cl;
  const int64_t b = head / a.hv;
  const int h = (int)(head - b * a.hv), hk = h / (a.hv / a.hk);
  int64_t len = a.l;
  if (a.lengths) {
    const int64_t n = a.lengths[b];
    len = n < 0 ? 0 : (n < a.l ? n : a.l);
  }
  bool col[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) col[j] = c0 + j < a.dv;
  const int64_t sbase = head * a.dk * a.dv + c0;
  float s[RPL][4];
#pragma unroll
  for (int r = 0; r < RPL; ++r) {
    const int i = i0 + r;
#pragma unroll
    for (int j = 0; j < 4; ++j) s[r][j] = 0.f;
    if (a.s0 && i < a.dk) {
      if constexpr (WIDE) {
        if (col[0]) {
          const f32x4 v = __builtin_nontemporal_load((const f32x4*)(a.s0 + sbase + (int64_t)i * a.dv));
#pragma unroll
          for (int j = 0; j < 4; ++j) s[r][j] = v[j];
        }
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (col[j]) s[r][j] = a.s0[sbase + (int64_t)i * a.dv + j];
      }
    }
  }
  for (int64_t t = 0; t < a.l; ++t) {
    const int64_t obase = ((b * a.l + t) * a.hv + h) * a.dv + c0;
    float o[4] = {0.f, 0.f, 0.f, 0.f};
    if (t < len) {
      const int64_t kb = b * a.k_stride[0] + t * a.k_stride[1] + hk * a.k_stride[2];
      const int64_t qb = b * a.q_stride[0] + t * a.q_stride[1] + hk * a.q_stride[2];
      const int64_t vb = b * a.v_stride[0] + t * a.v_stride[1] + h * a.v_stride[2] + c0;
      const float decay = expf(a.g[b * a.g_stride[0] + t * a.g_stride[1] + h * a.g_stride[2]]);
      const float beta =
          a.beta[b * a.beta_stride[0] + t * a.beta_stride[1] + h * a.beta_stride[2]];
      float k[RPL], q[RPL], qk = 0.f, ks[4] = {0.f, 0.f, 0.f, 0.f}, qs[4] = {0.f, 0.f, 0.f, 0.f}, v[4];
      load_part<T, RPL, KWIDE>(a.k, kb, i0, a.dk, k);
      load_part<T, RPL, KWIDE>(a.q, qb, i0, a.dk, q);
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = col[j] ? load1<T>(a.v, vb + j) : 0.f;
#pragma unroll
      for (int r = 0; r < RPL; ++r) {
        qk = fmaf(q[r], k[r], qk);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          ks[j] = fmaf(k[r], s[r][j], ks[j]);
          qs[j] = fmaf(q[r], s[r][j], qs[j]);
        }
      }
      qk = group_sum<CL>(qk);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        ks[j] = group_sum<CL>(ks[j]);
        qs[j] = group_sum<CL>(qs[j]);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float u = beta * (v[j] - decay * ks[j]);
        o[j] = a.scale * fmaf(qk, u, decay * qs[j]);
#pragma unroll
        for (int r = 0; r < RPL; ++r) s[r][j] = fmaf(k[r], u, decay * s[r][j]);
      }
    }
    if (i0 == 0) {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (col[j]) store1<T>(a.o, obase + j, o[j]);
    }
  }
#pragma unroll
  for (int r = 0; r < RPL; ++r) {
    const int i = i0 + r;
    if (i >= a.dk) continue;
    if constexpr (WIDE) {
      if (col[0])
        *(f32x4*)(a.s1 + sbase + (int64_t)i * a.dv) = f32x4{s[r][0], s[r][1], s[r][2], s[r][3]};
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (col[j]) a.s1[sbase + (int64_t)i * a.dv + j] = s[r][j];
    }
  }
}

template <int T, int CL, int RPL>
void go_wide(const DeltaArgs& a, hipStream_t st) {
  const int64_t waves = (int64_t)a.b * a.hv * ((a.dv + 4 * CL - 1) / (4 * CL));
  const dim3 grid((uint32_t)((waves + 3) / 4));
  const bool wide = a.dv % 4 == 0 && ((uintptr_t)a.s0 | (uintptr_t)a.s1) % 16 == 0;
  bool kwide = a.dk % 8 == 0 && ((uintptr_t)a.q | (uintptr_t)a.k) % 16 == 0;
  for (int i = 0; i < 3; ++i) kwide = kwide && a.q_stride[i] % 8 == 0 && a.k_stride[i] % 8 == 0;
  auto* f = wide ? (kwide ? &delta_token<T, CL, RPL, true, true>
                          : &delta_token<T, CL, RPL, true, false>)
                 : (kwide ? &delta_token<T, CL, RPL, false, true>
                          : &delta_token<T, CL, RPL, false, false>);
  hipLaunchKernelGGL(f, grid, dim3(256), 0, st, a);
}

template <int T>
void go(const DeltaArgs& a, hipStream_t st) {
  // 8 lanes across make a wave's row one 128-byte line.  Two lanes across
  // make four times the waves, each with a quarter of the loads before its
  // answer; taken while the device has room for them all at once (states of
  // 128x128: 8 heads 5.1 us against 9.3, 128 heads 6.8 us against 8.3 for 136
  // heads eight across).
  if (a.b * a.hv * a.dv <= 16384) {
    if (a.dk <= 128) return go_wide<T, 2, 4>(a, st);
    return go_wide<T, 2, 8>(a, st);
  }
  if (a.dk <= 32) go_wide<T, 8, 4>(a, st);
  else if (a.dk <= 64) go_wide<T, 8, 8>(a, st);
  else if (a.dk <= 128) go_wide<T, 8, 16>(a, st);
  else go_wide<T, 8, 32>(a, st);
}

}  // namespace token

hipError_t launch_delta_token(const DeltaArgs& a, hipStream_t st) {
  if (a.type == T_F32) token::go<T_F32>(a, st);
  else if (a.type == T_BF16) token::go<T_BF16>(a, st);
  else token::go<T_F16>(a, st);
  return hipGetLastError();
}

}  // namespace seq
}  // namespace dwc
