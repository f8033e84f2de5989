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
// chunk of 64 channels, wave w states 4 w to 4 w + 3 with a channel a lane.
// It first runs forward and leaves the state before every 8 tokens in LDS,
// then takes the eights from the last to the first: forward with the states
// and decays in registers, and back.  The sums over the channels (dB, dC) are
// made by exchanges that halve the values a lane holds at each step, so that
// all 64 lanes add; the sums over the states go through LDS, where wave w
// finishes token w of each four.
//
// Bound: the vector units, 88% busy at the four waves a SIMD that the registers
// leave (28 instructions a state and token, two of them exps).  8 sequences of
// 2048 tokens of 2048 channels and 16 states: 473 us of 724 for the whole
// gradient; the chunks' states before it 158, between the chunks 58.  (Two
// channels a lane: half the waves, 711 and 560 us when both were tried.)
#include "seq_scan.h"

namespace dwc {
namespace seq {
hipError_t launch_scan_prepare_bwd(const ScanArgs& a, hipStream_t st);

namespace scan {

constexpr int kEight = 8, kSubs = kGradChunk / kEight;
constexpr int NC = kGradChannels / 64, kPair = kGradChannels;  // channels a lane, a workgroup

// Sums of eight values over the lanes that agree in lane % 4 and lane / 32:
// first over lanes 8 apart in a row of 16, where the upper half takes the odd
// value of each pair (an addition that writes two of a row's four banks), then
// over lanes mirrored in a half row, where every other bank takes the next
// pair's, then over rows 16 apart.  A lane has value
//   (lane >> 3 & 1) + 2 (lane >> 2 & 1) + 4 (lane >> 4 & 1).
// The first wait is for the values, written just before.
__device__ __forceinline__ float fold8(const float (&v)[8]) {
  float a, b, c, d;
  asm("s_nop 1\n\t"
      "v_add_f32_dpp %0, %4, %4 row_ror:8 row_mask:0xf bank_mask:0xf\n\t"
      "v_add_f32_dpp %0, %5, %5 row_ror:8 row_mask:0xf bank_mask:0xc\n\t"
      "v_add_f32_dpp %1, %6, %6 row_ror:8 row_mask:0xf bank_mask:0xf\n\t"
      "v_add_f32_dpp %1, %7, %7 row_ror:8 row_mask:0xf bank_mask:0xc\n\t"
      "v_add_f32_dpp %2, %8, %8 row_ror:8 row_mask:0xf bank_mask:0xf\n\t"
      "v_add_f32_dpp %2, %9, %9 row_ror:8 row_mask:0xf bank_mask:0xc\n\t"
      "v_add_f32_dpp %3, %10, %10 row_ror:8 row_mask:0xf bank_mask:0xf\n\t"
      "v_add_f32_dpp %3, %11, %11 row_ror:8 row_mask:0xf bank_mask:0xc\n\t"
      "v_add_f32_dpp %0, %0, %0 row_half_mirror row_mask:0xf bank_mask:0xf\n\t"
      "v_add_f32_dpp %2, %2, %2 row_half_mirror row_mask:0xf bank_mask:0xf\n\t"
      "v_add_f32_dpp %0, %1, %1 row_half_mirror row_mask:0xf bank_mask:0xa\n\t"
      "v_add_f32_dpp %2, %3, %3 row_half_mirror row_mask:0xf bank_mask:0xa\n\t"
      "s_nop 1\n\t"
      "v_permlane16_swap_b32 %0, %2"
      : "=&v"(a), "=&v"(b), "=&v"(c), "=&v"(d)
      : "v"(v[0]), "v"(v[1]), "v"(v[2]), "v"(v[3]), "v"(v[4]), "v"(v[5]), "v"(v[6]), "v"(v[7]));
  return a + c;
}
// Of two such, the sums over all lanes of a value; lanes from 32 on have the
// second one's.
__device__ __forceinline__ float fold2(float a, float b) {
  asm("s_nop 1\n\tv_permlane32_swap_b32 %0, %1" : "+v"(a), "+v"(b));
  a += b;
  a += row_move<0xB1>(a);
  return a + row_move<0x4E>(a);
}

// Raw operands of one token of NC channels: u, delta, dy and, with a gate, z.
template <int T, int NC, bool GATE>
struct RawToken {
  static constexpr int N = GATE ? 4 : 3;
  Raw<T> v[N][NC];
  // p: addresses that are the same in all lanes
  __device__ __forceinline__ void load(const char* const (&p)[N], const uint32_t (&in)[NC]) {
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
      for (int k = 0; k < NC; ++k) v[i][k] = ((const Elem<T>*)p[i])[in[k]];
  }
};

// Addresses of token t, channel `first`, and the bytes between tokens.
template <int T, int N>
__device__ __forceinline__ void addresses(const ScanArgs& a, int64_t b, int64_t t, int64_t first,
                                          const char* (&p)[N], int64_t (&step)[N]) {
  const auto set = [&](int i, const void* q, const int64_t (&stride)[2]) {
    p[i] = (const char*)((const Elem<T>*)q + (b * stride[0] + t * stride[1] + first));
    step[i] = stride[1] * (int64_t)sizeof(Elem<T>);
  };
  set(0, a.u, a.u_stride);
  set(1, a.delta, a.delta_stride);
  set(2, a.dy, a.dy_stride);
  if constexpr (N > 3) set(3, a.z, a.z_stride);
}

// What they say: the step, its slope in delta, do and dy silu'(z).  Zeros
// where the token or the channel is not there.
struct Token {
  float u, dt, slope, go, dz;
};
template <int T, int NC, bool GATE>
__device__ __forceinline__ Token token_of(int soft, const RawToken<T, NC, GATE>& r, int k,
                                          float bias, bool live) {
  Token v;
  v.u = value<T>(r.v[0][k]);
  const float x = value<T>(r.v[1][k]) + bias, s = softplus(x);
  v.dt = soft ? s : x;  // (selects: branches would split the code)
  v.slope = soft ? sigmoid(x) : 1.f;
  v.go = value<T>(r.v[2][k]);
  v.dz = 0.f;
  if constexpr (GATE) {
    const float z = value<T>(r.v[GATE ? 3 : 0][k]), g = sigmoid(z);
    v.dz = v.go * fmaf(z * g, 1.f - g, g);
    v.go *= z * g;
  }
  v.u = live ? v.u : 0.f;
  v.dt = live ? v.dt : 0.f;
  v.slope = live ? v.slope : 0.f;
  v.go = live ? v.go : 0.f;
  v.dz = live ? v.dz : 0.f;
  return v;
}

// Outputs of one token of one channel from its sums over the states: of
// G B, of A q (in units of 1 / log2 e) and of C h.
template <int T, bool GATE, class Args>
__device__ __forceinline__ void finish(const Args& a, int64_t at, uint32_t in, float gb,
                                       float aq, float ch, const Token& v, float skip,
                                       float& dskip, float& dbias) {
  const float dd = fmaf(v.u, gb, kLn2 * aq) * v.slope;
  store1<T>((Elem<T>*)a.du + at, in, fmaf(v.dt, gb, skip * v.go));
  store1<T>((Elem<T>*)a.ddelta + at, in, dd);
  if constexpr (GATE) store1<T>((Elem<T>*)a.dz + at, in, v.dz * fmaf(skip, v.u, ch));
  dskip = fmaf(v.go, v.u, dskip);
  dbias += dd;
}

// Zeros behind a sequence's last token.
template <int T, bool GATE, class Args>
__device__ __forceinline__ void finish_none(const Args& a, int64_t at, uint32_t in) {
  store1<T>((Elem<T>*)a.du + at, in, 0.f);
  store1<T>((Elem<T>*)a.ddelta + at, in, 0.f);
  if constexpr (GATE) store1<T>((Elem<T>*)a.dz + at, in, 0.f);
}

enum { DT = 0, U, GO, SLOPE, DZ, kOf };  // of a token and channel, in LDS

// What the way back needs of one token.
struct OneToken {
  f32x8 bc;
  float dt[NC], u[NC], go[NC];
  __device__ __forceinline__ void load(const float* p, const float (&of)[kOf][kEight][kPair], int j,
                                       int lane) {
    bc = load_scalar<8>(p);
#pragma unroll
    for (int k = 0; k < NC; ++k) {
      dt[k] = of[DT][j][NC * lane + k];
      u[k] = of[U][j][NC * lane + k];
      go[k] = of[GO][j][NC * lane + k];
    }
  }
};

template <int T, int NW, bool GATE, bool MULTI>
__global__ void __launch_bounds__(64 * NW, 4) scan_grad(ScanArgs a) {
  constexpr int SPL = 16;                       // states of a line of bc
  constexpr int NT = NW < kEight ? kEight / NW : 1;  // tokens of an eight that a wave shares
  __shared__ float of[kOf][kEight][kPair];
  __shared__ float sums[3][4][NW][kPair];     // over a wave's states
  __shared__ float first[kSubs][NC * 4][64 * NW];  // states before the eights
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int pairs = (a.dg + kPair - 1) / kPair;
  uint32_t i = blockIdx.x;
  const int blk = MULTI ? (int)(i % (uint32_t)a.gblk) : 0;
  if (MULTI) i /= (uint32_t)a.gblk;
  const int block = (int)(i % (uint32_t)pairs);
  i /= (uint32_t)pairs;
  const int g = (int)(i % (uint32_t)a.g);
  i /= (uint32_t)a.g;
  const int chunk = (int)(i % (uint32_t)a.nc);
  const int64_t b = i / (uint32_t)a.nc;
  const int64_t len = length_of(a, b), t0 = (int64_t)chunk * kGradChunk;
  // tokens of the chunk, and of those inside the sequence's length
  const int tokens = a.l - t0 < kGradChunk ? (int)(a.l - t0) : kGradChunk;
  const int live = len <= t0 ? 0 : (len - t0 < tokens ? (int)(len - t0) : tokens);
  const int64_t g0 = (int64_t)g * a.dg, row = b * a.nc + chunk;
  // channels of the group; lanes past its end read its first one again
  const uint32_t c0 = (uint32_t)(block * kPair + NC * lane);
  bool on[NC];
  uint32_t in[NC];
  float dskip[NC], dbias[NC];
#pragma unroll
  for (int k = 0; k < NC; ++k) {
    on[k] = (int)c0 + k < a.dg;
    in[k] = on[k] ? c0 + k : 0;
    dskip[k] = dbias[k] = 0.f;
  }
  float a2[NC][4], da[NC][4], carry[NC][4], h[NC][4];
  const int n0 = 4 * (blk * NW + wave);
  // (all loads under way together, then what is not there made zero)
  {
#pragma unroll
    for (int k = 0; k < NC; ++k)
#pragma unroll
      for (int s = 0; s < 4; ++s) a2[k][s] = (a.a2 + ((int64_t)(n0 + s) * a.d + g0))[in[k]];
    if (a.nc > 1) {
      const int64_t at = (row * a.nblk * SPL + n0) * a.d + g0;
#pragma unroll
      for (int k = 0; k < NC; ++k)
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          h[k][s] = (a.states + at + (int64_t)s * a.d)[in[k]];
          carry[k][s] = (a.rstates + at + (int64_t)s * a.d)[in[k]];
        }
    } else {
      const int64_t at = (b * a.d + g0) * a.n;
#pragma unroll
      for (int k = 0; k < NC; ++k)
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          const bool is = n0 + s < a.n;
          const int64_t i = at + (int64_t)in[k] * a.n + (is ? n0 + s : 0);
          h[k][s] = a.s0 && is ? a.s0[i] : 0.f;
          carry[k][s] = a.ds1 && is ? a.ds1[i] : 0.f;
        }
    }
#pragma unroll
    for (int k = 0; k < NC; ++k)
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        h[k][s] = on[k] ? h[k][s] : 0.f;
        carry[k][s] = on[k] ? carry[k][s] : 0.f;
        da[k][s] = 0.f;
      }
  }
  // B and C of the wave's states, tokens 2 SPL apart; rows up to whole chunks
  // are there
  const int64_t lines = (((b * a.g + g) * a.nblk + n0 / 16) * a.lp + t0) * (2 * SPL) + 8 * (wave % 4);
  const float* const bc = a.bc + lines;

  // a wave's own tokens of an eight, wave and NW + wave; next[] is the address
  // of the first of them in the eight to be read.  Chunks cut short read a
  // token past the last one as the chunk's first.
  constexpr int N = GATE ? 4 : 3;
  RawToken<T, NC, GATE> raw[NT];
  const bool whole = live == kGradChunk, mine = wave < kEight;
  const char* next[N];
  int64_t eight[N];  // bytes of eight tokens
  addresses<T, N>(a, b, t0 + (whole && mine ? wave : 0), g0, next, eight);
#pragma unroll
  for (int i = 0; i < N; ++i) eight[i] *= kEight;
  const auto fetch = [&](int sub, int turn) {
    const char* p[N];
    if (whole) {
#pragma unroll
      for (int j = 0; j < NT; ++j) {
#pragma unroll
        for (int i = 0; i < N; ++i) p[i] = next[i] + j * (eight[i] / NT);
        raw[j].load(p, in);
      }
#pragma unroll
      for (int i = 0; i < N; ++i) next[i] += turn * eight[i];
    } else {
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        const int t = sub * kEight + NW * j + wave;
#pragma unroll
        for (int i = 0; i < N; ++i) p[i] = next[i] + (t < live ? t : 0) * (eight[i] / kEight);
        raw[j].load(p, in);
      }
    }
  };
  const auto share = [&](int sub, bool all) {
    if (!mine) return;
    // (the bias is read again for each eight: registers are short)
    FreshArgs& f = fresh_args();
    const float* pb = f.bias ? f.bias + g0 : nullptr;
    float bias[NC];
#pragma unroll
    for (int k = 0; k < NC; ++k) bias[k] = pb ? pb[in[k]] : 0.f;
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const int at = NW * j + wave;
#pragma unroll
      for (int k = 0; k < NC; ++k) {
        const Token v = token_of(f.softplus, raw[j], k, bias[k], on[k] && sub * kEight + at < live);
        of[DT][at][NC * lane + k] = v.dt;
        of[U][at][NC * lane + k] = v.u;
        if (all) {
          of[GO][at][NC * lane + k] = v.go;
          of[SLOPE][at][NC * lane + k] = v.slope;
          of[DZ][at][NC * lane + k] = v.dz;
        }
      }
    }
  };

  const int64_t row_out = (b * a.l + t0) * a.d + g0;  // of du, ddelta and dz

  // where fold2 leaves this lane's value: B of state s, C of it four further,
  // the second token's a line further
  const uint32_t out_at = (uint32_t)((lane >> 3 & 1) + 2 * (lane >> 2 & 1) + 4 * (lane >> 4 & 1) +
                                     (lane & 32 ? 2 * SPL : 0));

  // the states before the eights
  const int last = (tokens + kEight - 1) / kEight - 1;  // of the eights; -1 without tokens
  if (last >= 0) fetch(0, 1);
#pragma unroll 1
  for (int sub = 0; sub < kSubs; ++sub) {
#pragma unroll
    for (int k = 0; k < NC; ++k)
#pragma unroll
      for (int s = 0; s < 4; ++s) first[sub][4 * k + s][threadIdx.x] = h[k][s];
    if (sub >= last) break;  // (the same in all waves)
    __syncthreads();
    share(sub, false);
    fetch(sub + 1, sub + 1 < last ? 1 : -1);
    __syncthreads();
    const float* const rows = bc + sub * (kEight * 2 * SPL);
#pragma unroll
    for (int j = 0; j < kEight; ++j) {
      const f32x4 bb = load_scalar<4>(rows + j * (2 * SPL));
#pragma unroll
      for (int k = 0; k < NC; ++k) {
        const float dt = of[DT][j][NC * lane + k], du = dt * of[U][j][NC * lane + k];
#pragma unroll
        for (int s = 0; s < 4; ++s) h[k][s] = fmaf(exp2_of(dt * a2[k][s]), h[k][s], du * bb[s]);
      }
    }
  }

#pragma unroll 1
  for (int sub = last; sub >= 0; --sub) {
    __syncthreads();
    share(sub, true);
    __syncthreads();
    const float* const rows = bc + sub * (kEight * 2 * SPL);
    FreshArgs& o = fresh_args();
    float* const rows_out = o.bcpart + block * (o.b * o.g * o.nblk * o.lp * 2 * SPL) + lines +
                            sub * (kEight * 2 * SPL);
    float h[kEight + 1][NC][4], decay[kEight][NC][4];
#pragma unroll
    for (int k = 0; k < NC; ++k)
#pragma unroll
      for (int s = 0; s < 4; ++s) h[0][k][s] = first[sub][4 * k + s][threadIdx.x];
#pragma unroll
    for (int j = 0; j < kEight; ++j) {
      const f32x4 bb = load_scalar<4>(rows + j * (2 * SPL));
#pragma unroll
      for (int k = 0; k < NC; ++k) {
        const float dt = of[DT][j][NC * lane + k], du = dt * of[U][j][NC * lane + k];
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          decay[j][k][s] = exp2_of(dt * a2[k][s]);
          h[j + 1][k][s] = fmaf(decay[j][k][s], h[j][k][s], du * bb[s]);
        }
      }
      if (j % 2) __builtin_amdgcn_sched_barrier(0);
    }
    OneToken ahead;
    ahead.load(rows + (kEight - 1) * (2 * SPL), of, kEight - 1, lane);
#pragma unroll
    for (int half = 1; half >= 0; --half) {
      __builtin_amdgcn_sched_barrier(0);
      // (half of the eight's registers are free again)
      if (half == 0 && sub > 0) fetch(sub - 1, -1);
      float folded = 0.f;
#pragma unroll
      for (int q = 3; q >= 0; --q) {
        __builtin_amdgcn_sched_barrier(0);
        const int j = 4 * half + q;
        const OneToken now = ahead;  // (read while the token before it was computed)
        if (j > 0) ahead.load(rows + (j - 1) * (2 * SPL), of, j - 1, lane);
        const float bb[4] = {now.bc[0], now.bc[1], now.bc[2], now.bc[3]};
        const float cc[4] = {now.bc[4], now.bc[5], now.bc[6], now.bc[7]};
        float v[8], gb[NC], aq[NC], ch[NC];
#pragma unroll
        for (int s = 0; s < 8; ++s) v[s] = 0.f;
#pragma unroll
        for (int k = 0; k < NC; ++k) {
          const float dt = now.dt[k], du = dt * now.u[k], go = now.go[k];
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
        for (int k = 0; k < NC; ++k) {
          sums[0][q][wave][NC * lane + k] = gb[k];
          sums[1][q][wave][NC * lane + k] = aq[k];
          sums[2][q][wave][NC * lane + k] = ch[k];
        }
        const float f = fold8(v);
        if (q & 1) {
          folded = f;
        } else {
          // tokens j (lanes below 32) and j + 1
          const float x = fold2(f, folded);
          if ((lane & 3) == 0) rows_out[out_at + j * (2 * SPL)] = x;
        }
      }
      __syncthreads();
      FreshArgs& f = fresh_args();
      const int j = 4 * half + (NW > 4 ? wave % 4 : wave);
      const int t = sub * kEight + j;
      const int64_t at = row_out + (int64_t)t * f.d;
#pragma unroll
      for (int k = 0; k < NC; ++k) {
        float gb = 0.f, aq = 0.f, ch = 0.f;
#pragma unroll 4
        for (int m = 0; m < NW; ++m) {
          gb += sums[0][j % 4][m][NC * lane + k];
          aq += sums[1][j % 4][m][NC * lane + k];
          ch += sums[2][j % 4][m][NC * lane + k];
        }
        if (!on[k] || t >= tokens || wave >= 4) continue;
        if constexpr (MULTI) {
          const int64_t all = f.b * f.l * f.d;
          float* out = f.sums + blk * 3 * all + at;
          out[in[k]] = gb;
          (out + all)[in[k]] = aq;
          (out + 2 * all)[in[k]] = ch;
        } else if (t < live) {
          const int i = NC * lane + k;
          const Token v = {of[U][j][i], of[DT][j][i], of[SLOPE][j][i], of[GO][j][i], of[DZ][j][i]};
          finish<T, GATE>(f, at, in[k], gb, aq, ch, v, f.skip ? (f.skip + g0)[in[k]] : 0.f,
                          dskip[k], dbias[k]);
        } else {
          finish_none<T, GATE>(f, at, in[k]);
        }
      }
      __syncthreads();
    }
  }
  FreshArgs& e = fresh_args();
#pragma unroll
  for (int k = 0; k < NC; ++k)
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const int n = n0 + s;
      if (on[k]) (e.apart + ((row * e.nblk * SPL + n) * e.d + g0))[in[k]] = da[k][s];
      if (on[k] && n < e.n && chunk == 0 && e.ds0)
        (e.ds0 + ((b * e.d + g0) * e.n + n))[in[k] * (uint32_t)e.n] = carry[k][s];
    }
  if constexpr (!MULTI) {
    // dD and dbias over the waves' tokens
#pragma unroll
    for (int k = 0; k < NC; ++k) {
      sums[0][0][wave][NC * lane + k] = dskip[k];
      sums[1][0][wave][NC * lane + k] = dbias[k];
    }
    __syncthreads();
    if (wave == 0) {
#pragma unroll
      for (int k = 0; k < NC; ++k) {
        float x = 0.f, y = 0.f;
#pragma unroll 4
        for (int m = 0; m < NW; ++m) {
          x += sums[0][0][m][NC * lane + k];
          y += sums[1][0][m][NC * lane + k];
        }
        if (on[k]) {
          (e.dpart + (row * 2 * e.d + g0))[in[k]] = x;
          (e.dpart + ((row * 2 + 1) * e.d + g0))[in[k]] = y;
        }
      }
    }
  }
}

// States in more than one block: the blocks' sums joined, one lane a channel
// of a chunk.
template <int T, bool GATE>
__global__ void __launch_bounds__(256) scan_finish(ScanArgs a) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t row = i / a.d;
  if (row >= a.b * a.nc) return;
  const uint32_t c[1] = {(uint32_t)(i - row * a.d)};
  const int64_t b = row / a.nc, len = length_of(a, b), t0 = (row - b * a.nc) * kGradChunk;
  const int64_t t1 = t0 + kGradChunk < a.l ? t0 + kGradChunk : a.l;
  const float bias = a.bias ? a.bias[c[0]] : 0.f, skip = a.skip ? a.skip[c[0]] : 0.f;
  const int64_t all = a.b * a.l * a.d;
  float dskip = 0.f, dbias = 0.f;
  for (int64_t t = t0; t < t1; ++t) {
    const int64_t at = (b * a.l + t) * a.d;
    if (t < len) {
      constexpr int N = GATE ? 4 : 3;
      RawToken<T, 1, GATE> r;
      const char* p[N];
      int64_t step[N];
      addresses<T, N>(a, b, t, 0, p, step);
      r.load(p, c);
      float gb = 0.f, aq = 0.f, ch = 0.f;
      for (int k = 0; k < a.gblk; ++k) {
        gb += a.sums[3 * k * all + at + c[0]];
        aq += a.sums[(3 * k + 1) * all + at + c[0]];
        ch += a.sums[(3 * k + 2) * all + at + c[0]];
      }
      finish<T, GATE>(a, at, c[0], gb, aq, ch, token_of(a.softplus, r, 0, bias, true), skip, dskip, dbias);
    } else {
      finish_none<T, GATE>(a, at, c[0]);
    }
  }
  a.dpart[row * 2 * a.d + c[0]] = dskip;
  a.dpart[(row * 2 + 1) * a.d + c[0]] = dbias;
}

// dB and dC from the channel blocks' parts, in order: four states' dB or dC a
// lane.
template <int T>
__global__ void __launch_bounds__(256) scan_bc_sum(ScanArgs a) {
  const int w = a.nblk * 8;  // fours of a token and group
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t row = i / w, gr = row / a.l, t = row - gr * a.l, b = gr / a.g;
  if (b >= a.b) return;
  const int k = (int)(i - row * w), g = (int)(gr - b * a.g), blk = k / 8, four = k % 8;
  const int s0 = blk * 16 + four / 2 * 4;
  const int pairs = (a.dg + kPair - 1) / kPair;
  const int64_t size = a.b * a.lp * a.g * a.nblk * 32;
  f32x4 v = {0.f, 0.f, 0.f, 0.f};
  if (t < length_of(a, b)) {
    const float* p = a.bcpart + ((gr * a.nblk + blk) * a.lp + t) * 32 + four * 4;
#pragma unroll 8
    for (int j = 0; j < pairs; ++j) v += *(const f32x4*)(p + j * size);
  }
  void* const out = four % 2 ? a.dc : a.db;
  const int64_t at = ((b * a.l + t) * a.g + g) * a.n + s0;
#pragma unroll
  for (int s = 0; s < 4; ++s)
    if (s0 + s < a.n) store1<T>(out, at + s, v[s]);
}

template <int T, bool GATE>
void go_gate(const ScanArgs& a, hipStream_t st) {
  const int pairs = (a.dg + kPair - 1) / kPair;
  const dim3 grid((uint32_t)(a.b * a.nc * a.g * pairs * a.gblk));
  if (a.gblk > 1) {
    hipLaunchKernelGGL((scan_grad<T, 16, GATE, true>), grid, dim3(1024), 0, st, a);
    hipLaunchKernelGGL((scan_finish<T, GATE>), dim3((uint32_t)((a.b * a.nc * a.d + 255) / 256)),
                       dim3(256), 0, st, a);
  } else if (a.nblk == 1) {
    hipLaunchKernelGGL((scan_grad<T, 4, GATE, false>), grid, dim3(256), 0, st, a);
  } else if (a.nblk == 2) {
    hipLaunchKernelGGL((scan_grad<T, 8, GATE, false>), grid, dim3(512), 0, st, a);
  } else {
    hipLaunchKernelGGL((scan_grad<T, 16, GATE, false>), grid, dim3(1024), 0, st, a);
  }
}

template <int T>
void go_grad(const ScanArgs& a, hipStream_t st) {
  if (a.z) go_gate<T, true>(a, st);
  else go_gate<T, false>(a, st);
  const int64_t vals = a.b * a.l * a.g * a.nblk * 8;
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
