// seq_scan_grad.hip -- gradients of the selective scan.
//
//   do_t = dy_t silu(z_t),  dz_t = dy_t o_t silu'(z_t)
//   G_t = C_t do_t + a_(t+1) G_(t+1)  (behind the last token: ds1)
//   dC_t = sum_c do_t h_t,  dB_t = sum_c G_t dt_t u_t,  q_t = G_t a_t h_(t-1)
//   du_t = dt_t sum_n G_t B_t + D do_t,  ddt_t = sum_n A q_t + u_t sum_n G_t B_t
//   dA = sum_t dt_t q_t,  dD = sum_t do_t u_t,  ddelta = ddt softplus',
//   dbias = sum_t ddelta,  ds0 = a_1 G_1
//
// Chunks of 32 tokens side by side: scan_chunk and scan_combine give each its
// first state and the gradient that reaches its last one.  A workgroup takes a
// chunk of 128 channels, wave w states 4 w to 4 w + 3 of two channels a lane.
// It first runs forward and leaves the state before every 8 tokens in LDS,
// then takes the eights from the last to the first: forward with the states
// and decays in registers, and back.  The sums over the channels (dB, dC) are
// made by exchanges that halve the values a lane holds at each step, so that
// all 64 lanes add; the sums over the states go through LDS, where wave w
// finishes token w of each four.
#include "seq_scan.h"

namespace dwc {
namespace seq {
hipError_t launch_scan_prepare_bwd(const ScanArgs& a, hipStream_t st);

namespace scan {

constexpr int kEight = 8, kSubs = 4, kGradChunk = kEight * kSubs, kPair = 128;

// a = sums of the halves of a (lanes 0 to 31) and of b (32 to 63), the same
// by rows of 16, by halves of a row and by its fours.
__device__ __forceinline__ void swap32(float& a, float& b, float& c, float& d, float& e, float& f,
                                       float& g, float& h) {
  asm("s_nop 1\n\tv_permlane32_swap_b32 %0, %1\n\tv_permlane32_swap_b32 %2, %3\n\t"
      "v_permlane32_swap_b32 %4, %5\n\tv_permlane32_swap_b32 %6, %7"
      : "+v"(a), "+v"(b), "+v"(c), "+v"(d), "+v"(e), "+v"(f), "+v"(g), "+v"(h));
}
__device__ __forceinline__ void swap16(float& a, float& b, float& c, float& d) {
  asm("s_nop 1\n\tv_permlane16_swap_b32 %0, %1\n\tv_permlane16_swap_b32 %2, %3"
      : "+v"(a), "+v"(b), "+v"(c), "+v"(d));
}

// Sums over the lanes that agree in lane % 8 of eight values; lane has value
// (lane >> 5) + 2 (lane >> 4 & 1) + 4 (lane >> 3 & 1).
__device__ __forceinline__ float fold8(float (&v)[8], int lane) {
  swap32(v[0], v[1], v[2], v[3], v[4], v[5], v[6], v[7]);
  float a = v[0] + v[1], b = v[2] + v[3], c = v[4] + v[5], d = v[6] + v[7];
  swap16(a, b, c, d);
  const float e = a + b, f = c + d;
  const float x = e + row_move<0x128>(e), y = f + row_move<0x128>(f);  // rotated by 8
  return lane & 8 ? y : x;
}
// Of two such, the sums over the last eight lanes too; lanes with 4 set have
// the second one's.
__device__ __forceinline__ float fold2(float a, float b, int lane) {
  const float x = a + row_move<0x141>(a), y = b + row_move<0x141>(b);  // mirror of 8
  float v = lane & 4 ? y : x;
  v += row_move<0xB1>(v);
  return v + row_move<0x4E>(v);
}

// One token of two neighbouring channels.  base: the index of the first
// channel of the group at batch b and token t (the same in all lanes of
// scan_grad, so that lanes add a 32-bit offset to a scalar address).
template <int T>
struct Token {
  float u[2], dt[2], slope[2], go[2], dz[2];  // slope of dt in delta; dy silu'(z)
  __device__ __forceinline__ void load(const ScanArgs& a, int64_t b, int64_t t, int64_t first,
                                       uint32_t in, bool live, const bool (&on)[2],
                                       const float (&bias)[2]) {
    typedef const Raw<T>* ptr;
    const ptr pu = (ptr)a.u + (b * a.u_stride[0] + t * a.u_stride[1] + first);
    const ptr pd = (ptr)a.delta + (b * a.delta_stride[0] + t * a.delta_stride[1] + first);
    const ptr py = (ptr)a.dy + (b * a.dy_stride[0] + t * a.dy_stride[1] + first);
    const ptr pz = (ptr)a.z + (b * a.z_stride[0] + t * a.z_stride[1] + first);
    Raw<T> ru[2], rd[2], ry[2], rz[2];
#pragma unroll
    for (int k = 0; k < 2; ++k)
      if (live && on[k]) {
        ru[k] = pu[in + k];
        rd[k] = pd[in + k];
        ry[k] = py[in + k];
        if (a.z) rz[k] = pz[in + k];
      }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      u[k] = dt[k] = slope[k] = go[k] = dz[k] = 0.f;
      if (live && on[k]) {
        u[k] = value<T>(ru[k]);
        dt[k] = value<T>(rd[k]) + bias[k];
        slope[k] = 1.f;
        if (a.softplus) {
          slope[k] = sigmoid(dt[k]);
          dt[k] = softplus(dt[k]);
        }
        go[k] = value<T>(ry[k]);
        if (a.z) {
          const float z = value<T>(rz[k]), s = sigmoid(z);
          dz[k] = go[k] * fmaf(z * s, 1.f - s, s);
          go[k] *= z * s;
        }
      }
    }
  }
};

// Outputs of one token of one channel from its sums over the states: of
// G B, of A q (in units of 1 / log2 e) and of C h.
template <int T>
__device__ __forceinline__ void finish(const ScanArgs& a, int64_t at, uint32_t in, float gb, float aq,
                                       float ch, float u, float dt, float slope, float go,
                                       float dz, float skip, float& dskip, float& dbias) {
  const float dd = fmaf(u, gb, kLn2 * aq) * slope;
  store1<T>((Raw<T>*)a.du + at, in, fmaf(dt, gb, skip * go));
  store1<T>((Raw<T>*)a.ddelta + at, in, dd);
  if (a.z) store1<T>((Raw<T>*)a.dz + at, in, dz * fmaf(skip, u, ch));
  dskip = fmaf(go, u, dskip);
  dbias += dd;
}

enum { DT = 0, U, GO, SLOPE, DZ, kOf };  // of a token and channel, in LDS

// Zeros behind a sequence's last token.
template <int T>
__device__ __forceinline__ void finish_none(const ScanArgs& a, int64_t at, uint32_t in) {
  store1<T>((Raw<T>*)a.du + at, in, 0.f);
  store1<T>((Raw<T>*)a.ddelta + at, in, 0.f);
  if (a.z) store1<T>((Raw<T>*)a.dz + at, in, 0.f);
}

template <int T, bool MULTI>
__global__ void __launch_bounds__(256, 2) scan_grad(ScanArgs a) {
  constexpr int NW = 4, SPL = 4 * NW;
  __shared__ float of[kOf][kEight][kPair];
  __shared__ float sums[3][4][NW][kPair];     // over a wave's states
  __shared__ float first[kSubs][2 * 4][256];  // states before the eights
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int pairs = (a.dg + kPair - 1) / kPair;
  uint32_t i = blockIdx.x;
  const int blk = MULTI ? (int)(i % (uint32_t)a.nblk) : 0;
  if (MULTI) i /= (uint32_t)a.nblk;
  const int block = (int)(i % (uint32_t)pairs);
  i /= (uint32_t)pairs;
  const int g = (int)(i % (uint32_t)a.g);
  i /= (uint32_t)a.g;
  const int chunk = (int)(i % (uint32_t)a.nc);
  const int64_t b = i / (uint32_t)a.nc;
  const int64_t len = length_of(a, b), t0 = (int64_t)chunk * kGradChunk;
  const int64_t t1 = t0 + kGradChunk < a.l ? t0 + kGradChunk : a.l;
  const int64_t end = t1 < len ? t1 : len;
  const uint32_t in = (uint32_t)(block * kPair + 2 * lane);  // of the group's channels
  const int64_t g0 = (int64_t)g * a.dg;
  bool on[2];
  float dskip[2], dbias[2], a2[2][4], da[2][4], carry[2][4], h[2][4];
  const int64_t row = b * a.nc + chunk;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    on[k] = (int)in + k < a.dg;
    dskip[k] = dbias[k] = 0.f;
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const int n = blk * SPL + 4 * wave + s;
      a2[k][s] = da[k][s] = carry[k][s] = h[k][s] = 0.f;
      if (on[k] && n < a.n) {
        const int64_t own = (b * a.d + g0) * a.n + n, at = (row * a.nblk * SPL + n) * a.d + g0;
        const uint32_t lanes = (in + k) * (uint32_t)a.n;  // d n is below 2^32
        a2[k][s] = kLog2e * (a.a + (g0 * a.n + n))[lanes];
        if (a.nc > 1) {
          h[k][s] = (a.states + at)[in + k];
          carry[k][s] = (a.rstates + at)[in + k];
        } else {
          if (a.s0) h[k][s] = (a.s0 + own)[lanes];
          if (a.ds1) carry[k][s] = (a.ds1 + own)[lanes];
        }
      }
    }
  }
  const int64_t line = (int64_t)a.g * a.nblk * 2 * SPL;
  const int64_t lines = (int64_t)(g * a.nblk + blk) * 2 * SPL;
  const float* bc = a.bc + b * a.l * line + lines + 4 * wave;
  // rows of B and C past the last token are not there
  const auto bc_at = [&](int64_t t) { return bc + (t < a.l ? t : a.l - 1) * line; };

  // a wave's own tokens of an eight: wave and 4 + wave
  const auto share = [&](int64_t ts, int j, bool all) {
    // (read again for each eight: registers are short)
    const float bias[2] = {a.bias && on[0] ? (a.bias + g0)[in] : 0.f,
                           a.bias && on[1] ? (a.bias + g0)[in + 1] : 0.f};
    Token<T> x;
    x.load(a, b, ts + j, g0, in, ts + j < end, on, bias);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      of[DT][j][2 * lane + k] = x.dt[k];
      of[U][j][2 * lane + k] = x.u[k];
      if (all) {
        of[GO][j][2 * lane + k] = x.go[k];
        of[SLOPE][j][2 * lane + k] = x.slope[k];
        of[DZ][j][2 * lane + k] = x.dz[k];
      }
    }
  };

  // the states before the eights
#pragma unroll 1
  for (int sub = 0; sub < kSubs; ++sub) {
    const int64_t ts = t0 + sub * kEight;
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int s = 0; s < 4; ++s) first[sub][4 * k + s][threadIdx.x] = h[k][s];
    if (sub + 1 == kSubs || ts >= end) continue;  // (the same in all waves)
    __syncthreads();
    share(ts, wave, false);
    share(ts, 4 + wave, false);
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kEight; ++j) {
      const f32x4 bb = load_scalar<4>(bc_at(ts + j));
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const float dt = of[DT][j][2 * lane + k], du = dt * of[U][j][2 * lane + k];
#pragma unroll
        for (int s = 0; s < 4; ++s) h[k][s] = fmaf(exp2_of(dt * a2[k][s]), h[k][s], du * bb[s]);
      }
    }
  }

#pragma unroll 1
  for (int sub = kSubs - 1; sub >= 0; --sub) {
    const int64_t ts = t0 + sub * kEight;
    if (ts >= t1) continue;  // (the same in all waves)
    __syncthreads();
    share(ts, wave, true);
    share(ts, 4 + wave, true);
    __syncthreads();
    float h[kEight + 1][2][4], decay[kEight][2][4];
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int s = 0; s < 4; ++s) h[0][k][s] = first[sub][4 * k + s][threadIdx.x];
#pragma unroll
    for (int j = 0; j < kEight; ++j) {
      const f32x4 bb = load_scalar<4>(bc_at(ts + j));
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const float dt = of[DT][j][2 * lane + k], du = dt * of[U][j][2 * lane + k];
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          decay[j][k][s] = exp2_of(dt * a2[k][s]);
          h[j + 1][k][s] = fmaf(decay[j][k][s], h[j][k][s], du * bb[s]);
        }
      }
    }
#pragma unroll
    for (int half = 1; half >= 0; --half) {
      __builtin_amdgcn_sched_barrier(0);
      float folded = 0.f;
#pragma unroll
      for (int q = 3; q >= 0; --q) {
        const int j = 4 * half + q;
        const f32x4 bb = load_scalar<4>(bc_at(ts + j)), cc = load_scalar<4>(bc_at(ts + j) + SPL);
        float v[8], gb[2], aq[2], ch[2];
#pragma unroll
        for (int s = 0; s < 8; ++s) v[s] = 0.f;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const float dt = of[DT][j][2 * lane + k], du = dt * of[U][j][2 * lane + k];
          const float go = of[GO][j][2 * lane + k];
          gb[k] = aq[k] = ch[k] = 0.f;
#pragma unroll
          for (int s = 0; s < 4; ++s) {
            const float G = fmaf(cc[s], go, carry[k][s]);
            v[s] = fmaf(G, du, v[s]);
            v[4 + s] = fmaf(go, h[j + 1][k][s], v[4 + s]);
            gb[k] = fmaf(G, bb[s], gb[k]);
            ch[k] = fmaf(cc[s], h[j + 1][k][s], ch[k]);
            carry[k][s] = G * decay[j][k][s];
            const float w = carry[k][s] * h[j][k][s];
            aq[k] = fmaf(a2[k][s], w, aq[k]);
            da[k][s] = fmaf(dt, w, da[k][s]);
          }
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          sums[0][q][wave][2 * lane + k] = gb[k];
          sums[1][q][wave][2 * lane + k] = aq[k];
          sums[2][q][wave][2 * lane + k] = ch[k];
        }
        const float f = fold8(v, lane);
        if (q & 1) {
          folded = f;
        } else {
          // tokens j (lanes without 4) and j + 1
          const float x = fold2(f, folded, lane);
          const int64_t t = ts + j + (lane >> 2 & 1);
          const int s = (lane >> 5) + 2 * (lane >> 4 & 1);
          if ((lane & 3) == 0 && t < t1)
            a.bcpart[((int64_t)block * a.b + b) * a.l * line + t * line + lines + 4 * wave + s +
                     (lane & 8 ? SPL : 0)] = x;
        }
      }
      __syncthreads();
      const int j = 4 * half + wave;
      const int64_t t = ts + j;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        float gb = 0.f, aq = 0.f, ch = 0.f;
#pragma unroll
        for (int m = 0; m < NW; ++m) {
          gb += sums[0][wave][m][2 * lane + k];
          aq += sums[1][wave][m][2 * lane + k];
          ch += sums[2][wave][m][2 * lane + k];
        }
        if (!on[k] || t >= t1) continue;
        const int64_t at = (b * a.l + t) * a.d + g0, all = a.b * a.l * a.d;
        if constexpr (MULTI) {
          float* out = a.sums + blk * 3 * all + at;
          out[in + k] = gb;
          (out + all)[in + k] = aq;
          (out + 2 * all)[in + k] = ch;
        } else if (t < end) {
          finish<T>(a, at, in + k, gb, aq, ch, of[U][j][2 * lane + k], of[DT][j][2 * lane + k],
                    of[SLOPE][j][2 * lane + k], of[GO][j][2 * lane + k], of[DZ][j][2 * lane + k],
                    a.skip ? (a.skip + g0)[in + k] : 0.f, dskip[k], dbias[k]);
        } else {
          finish_none<T>(a, at, in + k);
        }
      }
      __syncthreads();
    }
  }
#pragma unroll
  for (int k = 0; k < 2; ++k)
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const int n = blk * SPL + 4 * wave + s;
      if (on[k]) (a.apart + ((row * a.nblk * SPL + n) * a.d + g0))[in + k] = da[k][s];
      if (on[k] && n < a.n && chunk == 0 && a.ds0)
        (a.ds0 + ((b * a.d + g0) * a.n + n))[(in + k) * (uint32_t)a.n] = carry[k][s];
    }
  if constexpr (!MULTI) {
    // dD and dbias over the waves' tokens
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      sums[0][0][wave][2 * lane + k] = dskip[k];
      sums[1][0][wave][2 * lane + k] = dbias[k];
    }
    __syncthreads();
    if (wave == 0) {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        float x = 0.f, y = 0.f;
#pragma unroll
        for (int m = 0; m < NW; ++m) {
          x += sums[0][0][m][2 * lane + k];
          y += sums[1][0][m][2 * lane + k];
        }
        if (on[k]) {
          (a.dpart + (row * 2 * a.d + g0))[in + k] = x;
          (a.dpart + ((row * 2 + 1) * a.d + g0))[in + k] = y;
        }
      }
    }
  }
}

// States in more than one block: the blocks' sums joined, one lane a channel
// of a chunk.
template <int T>
__global__ void __launch_bounds__(256) scan_finish(ScanArgs a) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t row = i / a.d;
  if (row >= a.b * a.nc) return;
  const uint32_t c = (uint32_t)(i - row * a.d);
  const bool on[2] = {true, false};
  const int64_t b = row / a.nc, len = length_of(a, b), t0 = (row - b * a.nc) * kGradChunk;
  const int64_t t1 = t0 + kGradChunk < a.l ? t0 + kGradChunk : a.l;
  const float bias[2] = {a.bias ? a.bias[c] : 0.f, 0.f};
  const float skip = a.skip ? a.skip[c] : 0.f;
  const int64_t all = a.b * a.l * a.d;
  float dskip = 0.f, dbias = 0.f;
  for (int64_t t = t0; t < t1; ++t) {
    const int64_t at = (b * a.l + t) * a.d;
    if (t < len) {
      Token<T> x;
      x.load(a, b, t, 0, c, true, on, bias);
      float gb = 0.f, aq = 0.f, ch = 0.f;
      for (int k = 0; k < a.nblk; ++k) {
        gb += a.sums[3 * k * all + at + c];
        aq += a.sums[(3 * k + 1) * all + at + c];
        ch += a.sums[(3 * k + 2) * all + at + c];
      }
      finish<T>(a, at, c, gb, aq, ch, x.u[0], x.dt[0], x.slope[0], x.go[0], x.dz[0], skip, dskip,
                dbias);
    } else {
      finish_none<T>(a, at, c);
    }
  }
  a.dpart[row * 2 * a.d + c] = dskip;
  a.dpart[(row * 2 + 1) * a.d + c] = dbias;
}

// dB and dC from the channel blocks' parts, in order.
template <int T>
__global__ void __launch_bounds__(256) scan_bc_sum(ScanArgs a) {
  const int64_t vals = a.b * a.l * a.g * a.n;
  int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= 2 * vals) return;
  const bool second = i >= vals;
  if (second) i -= vals;
  const int64_t row = i / a.n, token = row / a.g;
  const int s = (int)(i - row * a.n), blk = s / a.spl;
  const int64_t b = token / a.l, t = token - b * a.l;
  const int pairs = (a.dg + kPair - 1) / kPair;
  float v = 0.f;
  if (t < length_of(a, b)) {
    const int64_t size = a.b * a.l * a.g * a.nblk * 2 * a.spl;
    const float* p = a.bcpart + (row * a.nblk + blk) * 2 * a.spl + s - blk * a.spl +
                     (second ? a.spl : 0);
    for (int k = 0; k < pairs; ++k) v += p[k * size];
  }
  store1<T>(second ? a.dc : a.db, i, v);
}

template <int T>
void go_grad(const ScanArgs& a, hipStream_t st) {
  const int pairs = (a.dg + kPair - 1) / kPair;
  const dim3 grid((uint32_t)(a.b * a.nc * a.g * pairs * a.nblk));
  if (a.nblk > 1) {
    hipLaunchKernelGGL((scan_grad<T, true>), grid, dim3(256), 0, st, a);
    hipLaunchKernelGGL((scan_finish<T>), dim3((uint32_t)((a.b * a.nc * a.d + 255) / 256)),
                       dim3(256), 0, st, a);
  } else {
    hipLaunchKernelGGL((scan_grad<T, false>), grid, dim3(256), 0, st, a);
  }
  const int64_t vals = 2 * a.b * a.l * a.g * a.n;
  if (vals > 0)
    hipLaunchKernelGGL((scan_bc_sum<T>), dim3((uint32_t)((vals + 255) / 256)), dim3(256), 0, st, a);
}

}  // namespace scan

hipError_t launch_scan_bwd(const ScanArgs& a, hipStream_t st) {
  if (a.b > 0) {  // (else the sums of no rows: zeros)
    hipError_t e = launch_scan_prepare_bwd(a, st);
    if (e != hipSuccess) return e;
    if (a.type == T_F32) scan::go_grad<T_F32>(a, st);
    else if (a.type == T_BF16) scan::go_grad<T_BF16>(a, st);
    else scan::go_grad<T_F16>(a, st);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  const int64_t rows = a.b * a.nc, np = (int64_t)a.nblk * a.spl;
  const ColumnSum jobs[kColumnJobs] = {
      {a.apart, a.da, rows, np * a.d, (int64_t)a.n * a.d, a.d},
      {a.dpart, a.dskip, rows, 2 * (int64_t)a.d, a.d, 0},
      {a.dpart + a.d, a.dbias, rows, 2 * (int64_t)a.d, a.d, 0}};
  return launch_column_sums(jobs, st);
}

}  // namespace seq
}  // namespace dwc
