// seq_scan_wide.hip -- the selective scan in one pass over the tokens, for
// many sequences or channels and for short sequences.
//
// A workgroup takes 64 / Q channels of a sequence, a wave Q times two or four of
// the states with a channel a lane.  Stages of 16 tokens: the waves share out the
// tokens' steps, inputs and gates (tokens w, w + NW, ...), all run the stage on
// their own states, and join the parts of C . h in LDS, where each finishes its
// own tokens.  B and C go through LDS too, a stage ahead: there are few waves to
// wait for the scalar cache.
//
// A decay near 1 loses what is below 2^-24, and a product of many loses that
// much each time (16 states, 491 tokens: the last state off by 8e-7 of its
// norm).  So a second state starts from zero every 64 tokens and the first one
// is made again from it there, with one decay for the sum of their steps: 1.4e-7,
// for 5 to 10% of the time.
//
// Bound: the vector units, of which a state of a token takes an exp and five
// other instructions once, not twice as in chunks.  8 sequences of 2048 tokens
// of 2048 channels and 16 states: 219 us, the vector units 65% busy at the two
// waves a SIMD that there are.  (One barrier a stage, with the outputs of the
// stage before and the steps of the next one among the tokens: 1% less there,
// 2 to 7% more for 32 sequences and up, where its LDS leaves fewer waves.)
#include "seq_scan.h"

namespace dwc {
namespace seq {
namespace scan {

constexpr int kStage = 16, kAgain = 4;  // tokens; stages until the states are made again

template <int T, int NW, int S, bool GATE, int Q>
__global__ void __launch_bounds__(64 * NW) scan_wide(ScanArgs a) {
  constexpr int CH = 64 / Q, SPL = 16;  // channels; states a line of bc
  constexpr int NT = kStage / (NW * Q);  // tokens a lane shares
  constexpr int ROW = 2 * S * NW * Q;    // B and C of all states
  __shared__ f32x2 of[kStage][CH];       // dt, dt u
  __shared__ float parts[kStage][NW][64];  // of C . h
  __shared__ __align__(16) float rows[2][kStage][ROW];  // a wave's B and its C in turn
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  uint32_t i = blockIdx.x;
  const uint32_t blocks = Q == 1 ? (uint32_t)a.cblk : (uint32_t)((a.dg + CH - 1) / CH);
  const int block = (int)(i % blocks);
  i /= blocks;
  const int g = (int)(i % (uint32_t)a.g);
  const int64_t b = i / (uint32_t)a.g;
  const int len = (int)length_of(a, b);
  const int64_t g0 = (int64_t)g * a.dg;
  const int ch = lane % CH, q = Q == 1 ? 0 : lane / CH;
  const uint32_t c0 = (uint32_t)(block * CH + ch);
  const bool on = (int)c0 < a.dg;
  const uint32_t in = on ? c0 : 0;  // (lanes past the end repeat the first channel)
  const int n0 = S * (Q * wave + q);
  const bool mine = S * Q * wave < a.n;  // (the same in a wave; the others leave zeros)
  float a2[S], h[S], start[S], from[S], sum = 0.f;  // from: from zero, start: at that time
  const auto states = [&](const float* p, float(&v)[S]) {  // of d x n
#pragma unroll
    for (int s = 0; s < S; ++s) v[s] = (p + (n0 + s < a.n ? n0 + s : 0))[in * (uint32_t)a.n];
#pragma unroll
    for (int s = 0; s < S; ++s) v[s] = n0 + s < a.n ? v[s] : 0.f;
  };
#pragma unroll
  for (int s = 0; s < S; ++s) {
    // (waves past the last block of states have none)
    a2[s] = n0 + s < a.nblk * SPL ? (a.a2 + ((int64_t)(n0 + s) * a.d + g0))[in] : 0.f;
    h[s] = 0.f;
  }
  if (a.s0) states(a.s0 + (b * a.d + g0) * a.n, h);
#pragma unroll
  for (int s = 0; s < S; ++s) {
    start[s] = h[s];
    from[s] = 0.f;
  }
  const float bias = a.bias ? (a.bias + g0)[in] : 0.f, skip = a.skip ? (a.skip + g0)[in] : 0.f;
  // B and C of a stage: S Q / 2 values a thread; rows up to a multiple of the
  // stage are there, but for blocks of 16 states past the last
  constexpr int PER = S * Q / 2, ACROSS = ROW / PER;
  const int row = threadIdx.x / ACROSS, at_row = PER * (threadIdx.x % ACROSS), of16 = at_row / 32;
  const bool some = of16 < a.nblk;
  const float* bc = a.bc + (((b * a.g + g) * a.nblk + (some ? of16 : 0)) * a.lp + row) * (2 * SPL) +
                    at_row % 32;
  // in LDS a wave's B and C stand together
  const auto to_row = [](int i) {
    return S == 4 ? i : i / 8 * 8 + i % 4 / 2 * 4 + i % 8 / 4 * 2 + i % 2;
  };
  float bc_next[PER];
  // the lane's tokens of a stage, and the address of the first of the next
  // stage's, but for q tokens
  const auto token = [&](int j) { return (j * NW + wave) * Q + q; };
  constexpr int N = GATE ? 3 : 2;
  const char* next[N];
  int64_t one[N];  // bytes between tokens
  const auto set = [&](int k, const void* p, const int64_t(&stride)[2]) {
    next[k] = (const char*)((const Elem<T>*)p + (b * stride[0] + wave * Q * stride[1] + g0));
    one[k] = stride[1] * (int64_t)sizeof(Elem<T>);
  };
  set(0, a.u, a.u_stride);
  set(1, a.delta, a.delta_stride);
  if constexpr (GATE) set(2, a.z, a.z_stride);
  Raw<T> even[N][NT], odd[N][NT];  // of the next two stages
  const auto fetch = [&](int t0, Raw<T>(&raw)[N][NT]) {
    if (t0 >= len) return;
    if (t0 + kStage <= len) {
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int k = 0; k < N; ++k) {
          raw[k][j] = ((const Elem<T>*)(next[k] + q * one[k]))[in];
          next[k] += NW * Q * one[k];
        }
    } else {  // a token past the last one is read as the last
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        const int t = t0 + token(j), back = t < len ? 0 : t - (len - 1);
#pragma unroll
        for (int k = 0; k < N; ++k)
          raw[k][j] = ((const Elem<T>*)(next[k] + (j * NW * Q + q - back) * one[k]))[in];
      }
    }
  };
  const auto fetch_rows = [&](int t0) {
#pragma unroll
    for (int i = 0; i < PER; ++i) bc_next[i] = bc[(int64_t)t0 * (2 * SPL) + i];
  };
  const auto keep = [&](int side) {
#pragma unroll
    for (int i = 0; i < PER; ++i) rows[side][row][to_row(at_row + i)] = some ? bc_next[i] : 0.f;
  };
  Elem<T>* const out = (Elem<T>*)a.y + (b * a.l * a.d + g0);
  if (!mine) {
#pragma unroll
    for (int j = 0; j < kStage; ++j) parts[j][wave][lane] = 0.f;
  }
  if (len > 0) {
    fetch_rows(0);
    fetch(0, even);
    fetch(kStage, odd);
    keep(0);
  }
  const auto stage = [&](int t0, int side, Raw<T>(&raw)[N][NT]) {
    // (the stage before has been read: its readers passed the barrier below)
    Raw<T> gate[NT];
    float u[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const int at = token(j);
      const bool live = t0 + at < len;
      u[j] = value<T>(raw[0][j]);
      const float dt = step_of(a.softplus, value<T>(raw[1][j]) + bias);
      if constexpr (GATE) gate[j] = raw[GATE ? 2 : 0][j];
      of[at][ch] = live ? f32x2{dt, dt * u[j]} : f32x2{0.f, 0.f};
    }
    __syncthreads();
    // (the rows first: they are waited for first, a stage before the rest)
    if (t0 + kStage < len) fetch_rows(t0 + kStage);
    fetch(t0 + 2 * kStage, raw);
    if (mine) {
      // LDS is read two tokens ahead and the decays are made one ahead: a SIMD
      // may have no other wave to fill the wait
      float bb[3][S], cc[3][S], dt[3], du[3], k[2][S];
      const int b_at = 2 * n0, c_at = b_at + S;
      const auto read = [&](int j) {
#pragma unroll
        for (int s = 0; s < S; ++s) {
          bb[j % 3][s] = rows[side][j][b_at + s];
          cc[j % 3][s] = rows[side][j][c_at + s];
        }
        const f32x2 x = of[j][ch];
        dt[j % 3] = x[0];
        du[j % 3] = x[1];
      };
      const auto decays = [&](int j) {
#pragma unroll
        for (int s = 0; s < S; ++s) k[j % 2][s] = exp2_of(dt[j % 3] * a2[s]);
      };
      read(0);
      read(1);
      decays(0);
      float steps = 0.f;
#pragma unroll
      for (int j = 0; j < kStage; ++j) {
        __builtin_amdgcn_sched_barrier(0);
        if (j + 2 < kStage) read(j + 2);
        if (j + 1 < kStage) decays(j + 1);
        float y = 0.f;
#pragma unroll
        for (int s = 0; s < S; ++s) {
          const float x = du[j % 3] * bb[j % 3][s];
          h[s] = fmaf(k[j % 2][s], h[s], x);
          from[s] = fmaf(k[j % 2][s], from[s], x);
          y = fmaf(cc[j % 3][s], h[s], y);
        }
        steps += dt[j % 3];
        // (nothing reads these before the end: without this all 16 steps of them
        // are put off to there, their operands held in registers)
#pragma unroll
        for (int s = 0; s < S; ++s) asm volatile("" : "+v"(from[s]));
        asm volatile("" : "+v"(steps));
        parts[j][wave][lane] = y;
      }
      sum += steps;
      if (t0 / kStage % kAgain == kAgain - 1) {
#pragma unroll
        for (int s = 0; s < S; ++s) {
          h[s] = start[s] = decay_of(a2[s] * sum).of(start[s]) + from[s];
          from[s] = 0.f;
        }
        sum = 0.f;
      }
    }
    if (t0 + kStage < len) keep(side ^ 1);
    __syncthreads();
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const int at = token(j);
      float y = 0.f;
#pragma unroll
      for (int k = 0; k < NW; ++k)
#pragma unroll
        for (int e = 0; e < Q; ++e) y += parts[at][k][e * CH + ch];
      y = fmaf(skip, u[j], y);
      if constexpr (GATE) {
        const float z = value<T>(gate[j]);
        y *= z * sigmoid(z);
      }
      if (on && t0 + at < len) store1<T>(out + (int64_t)(t0 + at) * a.d, in, y);
    }
  };
  for (int t0 = 0; t0 < len; t0 += 2 * kStage) {
    stage(t0, 0, even);
    if (t0 + kStage < len) stage(t0 + kStage, 1, odd);
  }
  for (int64_t t = len + token(0); t < a.l; t += NW * Q)
    if (on) store1<T>(out + t * a.d, in, 0.f);
  float* const s1 = a.s1 + (b * a.d + g0) * a.n;
#pragma unroll
  for (int s = 0; s < S; ++s)
    if (on && n0 + s < a.n)
      (s1 + n0 + s)[in * (uint32_t)a.n] = decay_of(a2[s] * sum).of(start[s]) + from[s];
}

template <int T, int NW, int S, bool GATE, int Q = 1>
void go_shape(const ScanArgs& a, hipStream_t st) {
  const int64_t blocks = (a.dg + 64 / Q - 1) / (64 / Q);
  hipLaunchKernelGGL((scan_wide<T, NW, S, GATE, Q>), dim3((uint32_t)(a.b * a.g * blocks)),
                     dim3(64 * NW), 0, st, a);
}

template <int T, bool GATE>
void go_wide(const ScanArgs& a, hipStream_t st) {
  const int64_t groups = a.b * a.g * a.cblk;
  // Few channels are spread over as many SIMDs as there are by taking 32 or 16 of
  // them a workgroup.  us, with 64 first: 256 tokens of 2048 channels, 16 states:
  // 33 and 28; 5 sequences of 333 tokens of 600 channels, 32 states: 57, 40 and
  // 33; 16 of 700 tokens of 512: 115 and 78, 64 states 176 and 114.
  if (a.n <= 8) return go_shape<T, 4, 2, GATE>(a, st);
  if (a.n <= 16 && groups <= 128) return go_shape<T, 4, 2, GATE, 2>(a, st);
  if (a.n <= 32 && groups <= 64) return go_shape<T, 4, 2, GATE, 4>(a, st);
  if (a.n <= 32 && groups <= 128) return go_shape<T, 8, 2, GATE, 2>(a, st);
  // two states a wave while that leaves no SIMD more than two waves (8 and 16
  // sequences of 2048 tokens of 2048 channels: 224 and 350 us, with four 280
  // and 357; 32 of 1024 tokens, 128 of 256: 328 and 321, with four 306 and 290)
  if (a.n <= 16)
    return groups <= 256 ? go_shape<T, 8, 2, GATE>(a, st) : go_shape<T, 4, 4, GATE>(a, st);
  // (up to 24 states twos load the SIMDs more evenly: 32 sequences of 700 tokens
  // of 512 channels, 24 states: 99 and 116 us, 28 states 113 and 118; 48
  // sequences, 24 states: 185 and 177)
  if (a.n <= 32)
    return a.n <= 24 && groups <= 256 ? go_shape<T, 16, 2, GATE>(a, st)
                                      : go_shape<T, 8, 4, GATE>(a, st);
  if (groups <= 64) return go_shape<T, 4, 4, GATE, 4>(a, st);
  if (groups <= 128) return go_shape<T, 8, 4, GATE, 2>(a, st);
  go_shape<T, 16, 4, GATE>(a, st);
}

template <int T>
void go_wide_gate(const ScanArgs& a, hipStream_t st) {
  if (a.z) go_wide<T, true>(a, st);
  else go_wide<T, false>(a, st);
}

}  // namespace scan

void launch_scan_wide(const ScanArgs& a, hipStream_t st) {
  if (a.type == T_F32) scan::go_wide_gate<T_F32>(a, st);
  else if (a.type == T_BF16) scan::go_wide_gate<T_BF16>(a, st);
  else scan::go_wide_gate<T_F16>(a, st);
}

}  // namespace seq
}  // namespace dwc
