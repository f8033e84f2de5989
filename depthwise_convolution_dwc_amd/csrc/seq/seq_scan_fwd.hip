// seq_scan_fwd.hip -- the selective scan over whole sequences.
//
// A lane owns one channel and up to 16 of its states in registers and walks
// tokens; B and C of a token are the same for a wave's 64 channels, so they
// come through the scalar cache as scalar operands (scan_prep lays them out in
// fp32, padded to the block of states).  Where there are too few channels to
// fill the device, the tokens are split in chunks: scan_chunk finds each
// chunk's state from zero, scan_combine carries the states over the chunks and
// scan_out runs again from the right ones.
//
// Bound: the vector units.  A state of a token takes an exp (two instructions'
// time) and four other instructions: 4096 tokens of 2048 channels and 16 states
// take 33 us for the chunks' states (three of the four), 10 between the chunks
// and 40 for the outputs; 5 for the layout before them.
#include "seq_scan.h"

namespace dwc {
namespace seq {
void launch_scan_wide(const ScanArgs& a, hipStream_t st);

namespace scan {

// B and C four values a thread, then A with its states' rows across: waves
// read 64 channels of a state from one place.
template <int T, bool FOURS>
__global__ void __launch_bounds__(256) scan_prep(ScanArgs a) {
  const uint32_t w = (uint32_t)a.spl / 2;  // threads a line
  const uint32_t rows = (uint32_t)(a.b * a.g * a.nblk), lp = (uint32_t)a.lp;
  uint32_t i = blockIdx.x * 256 + threadIdx.x;
  if (i < rows * lp * w) {
    const uint32_t line = i / w, j = (i - line * w) * 4, row = line / lp;
    const int64_t t = line - row * lp;
    const uint32_t gr = row / (uint32_t)a.nblk, blk = row - gr * (uint32_t)a.nblk;
    const int64_t b = gr / (uint32_t)a.g, g = gr - (uint32_t)b * (uint32_t)a.g;
    // states in order, or by fours with B and C in turn
    const bool second = FOURS ? j & 4 : j >= (uint32_t)a.spl;
    const int s0 = (int)(blk * a.spl + (FOURS ? j / 8 * 4 : (second ? j - a.spl : j)));
    f32x4 v = {0.f, 0.f, 0.f, 0.f};
    if (t < length_of(a, b)) {
      const int64_t at =
          second ? b * a.c_stride[0] + t * a.c_stride[1] + g * a.c_stride[2] + s0
                 : b * a.b_stride[0] + t * a.b_stride[1] + g * a.b_stride[2] + s0;
      const void* p = second ? a.cm : a.bm;
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (s0 + k < a.n) v[k] = load1<T>(p, at + k);
    }
    ((f32x4*)a.bc)[i] = v;
    return;
  }
  i -= rows * lp * w;
  const uint32_t s = i / (uint32_t)a.d, c = i - s * (uint32_t)a.d;
  if (s < (uint32_t)(a.nblk * a.spl))
    a.a2[i] = s < (uint32_t)a.n ? rate_of(a.a[(int64_t)c * a.n + s]) : 0.f;
}

// What a workgroup works on.
struct Where {
  int g, blk, c;  // group, block of states, channel of d
  uint32_t in;    // channel of the group
  int64_t g0;     // the group's first channel
  bool on;
  int chunk;
  int64_t b, len, t0, t1;  // tokens of the chunk
};

__device__ __forceinline__ Where where(const ScanArgs& a, int blk, uint32_t i, int nblk) {
  Where w;
  const uint32_t per = (uint32_t)(a.g * a.cblk * nblk);
  const uint32_t row = i / per;
  uint32_t k = i - row * per;
  if (nblk > 1) {
    blk = (int)(k % (uint32_t)nblk);
    k /= (uint32_t)nblk;
  }
  w.blk = blk;
  w.g = (int)(k / (uint32_t)a.cblk);
  const uint32_t in = (k - (uint32_t)w.g * a.cblk) * 64 + (threadIdx.x & 63);
  w.on = (int)in < a.dg;
  w.in = w.on ? in : 0;
  w.g0 = (int64_t)w.g * a.dg;
  w.c = (int)w.g0 + (int)w.in;
  w.chunk = (int)(row % (uint32_t)a.nc);
  w.b = row / (uint32_t)a.nc;
  w.len = length_of(a, w.b);
  w.t0 = (int64_t)w.chunk * a.tc;
  w.t1 = w.t0 + a.tc < a.l ? w.t0 + a.tc : a.l;
  return w;
}

template <int SPL>
__device__ __forceinline__ void load_a(const ScanArgs& a, const Where& w, float (&v)[SPL]) {
  const float* p = a.a2 + ((int64_t)w.blk * SPL * a.d + w.g0);
#pragma unroll
  for (int s = 0; s < SPL; ++s) v[s] = (p + (int64_t)s * a.d)[w.in];
}

// B and C of the chunk's first token.
template <int SPL>
__device__ __forceinline__ const float* lines(const ScanArgs& a, const Where& w) {
  return a.bc + (((w.b * a.g + w.g) * a.nblk + w.blk) * a.lp + w.t0) * (2 * SPL);
}

constexpr int kAhead = 4;  // tokens whose loads are under way together

// Raw operands of N tensors, U tokens of them.  p: addresses of the next
// token that are the same in all lanes, of the group's first channel; step:
// bytes between tokens.
template <int T, int N, int U>
struct Ahead {
  Raw<T> v[N][U];
  __device__ __forceinline__ void load(const char* (&p)[N], const int64_t (&step)[N],
                                       uint32_t in) {
#pragma unroll
    for (int i = 0; i < U; ++i)
#pragma unroll
      for (int k = 0; k < N; ++k) {
        v[k][i] = ((const Elem<T>*)p[k])[in];
        p[k] += step[k];
      }
  }
};

// Address of token t0 of a tensor.
template <int T>
__device__ __forceinline__ const char* from(const void* p, const int64_t (&stride)[2],
                                            const Where& w, int64_t& step) {
  step = stride[1] * (int64_t)sizeof(Elem<T>);
  return (const char*)((const Elem<T>*)p + (w.b * stride[0] + w.t0 * stride[1] + w.g0));
}

// The gradient that a chunk hands to the state before it, from zero at its
// end: r_t = a_t (r_(t+1) + C_t do_t).
template <int T, int SPL, bool GATE>
__device__ __forceinline__ void from_the_end(const Where& w, int64_t end, const float (&a2)[SPL],
                                             float (&r)[SPL]) {
  FreshArgs& a = fresh_args();
  const float bias = a.bias ? a.bias[w.c] : 0.f;
  const float* bc = a.bc + ((w.b * a.g + w.g) * a.nblk + w.blk) * a.lp * (2 * SPL);
  asm volatile("" : "+v"(bc));  // (vector loads: scalar registers are short)
#pragma unroll
  for (int s = 0; s < SPL; ++s) r[s] = 0.f;
#pragma unroll 1
  for (int64_t t = end - 1; t >= w.t0; --t) {
    const float x = load1<T>(a.delta, w.b * a.delta_stride[0] + t * a.delta_stride[1] + w.c);
    const float dt = step_of(a.softplus, x + bias);
    float go = load1<T>(a.dy, w.b * a.dy_stride[0] + t * a.dy_stride[1] + w.c);
    if constexpr (GATE) {
      const float z = load1<T>(a.z, w.b * a.z_stride[0] + t * a.z_stride[1] + w.c);
      go *= z * sigmoid(z);
    }
#pragma unroll
    for (int s = 0; s < SPL; ++s)
      r[s] = exp2_of(dt * a2[s]) * fmaf(bc[t * (2 * SPL) + c_at<SPL, true>(s)], go, r[s]);
  }
}

// Each chunk's state from zero and the sum of its steps.  With BWD also, from
// zero at its end, the gradient that it hands to the state before it:
//   sum_t (a_t0 ... a_t) C_t do_t,  do = dy silu(z).
template <int T, int SPL, bool BWD, bool GATE>
__global__ void __launch_bounds__(64) scan_chunk(ScanArgs a) {
  const Where w = where(a, 0, blockIdx.x, a.nblk);
  if (!w.on) return;
  const int64_t end = w.t1 < w.len ? w.t1 : w.len;
  float a2[SPL], h[SPL], p[SPL], r[SPL];
  load_a<SPL>(a, w, a2);
#pragma unroll
  for (int s = 0; s < SPL; ++s) {
    h[s] = r[s] = 0.f;
    p[s] = 1.f;
  }
  double sum = 0.0;
  if (w.t0 < end) {
    const float bias = a.bias ? a.bias[w.c] : 0.f;
    constexpr int N = BWD ? (GATE ? 4 : 3) : 2;
    const char* ptr[N];
    int64_t step[N];
    ptr[0] = from<T>(a.u, a.u_stride, w, step[0]);
    ptr[1] = from<T>(a.delta, a.delta_stride, w, step[1]);
    if constexpr (BWD) {
      ptr[2] = from<T>(a.dy, a.dy_stride, w, step[2]);
      if constexpr (GATE) ptr[3] = from<T>(a.z, a.z_stride, w, step[3]);
    }
    const float* bc = lines<SPL>(a, w);
    const auto token = [&](const auto& x, int i) {
      // (forward only B is read)
      const auto lo = load_scalar<SPL>(bc), hi = load_scalar<SPL>(bc + (BWD ? SPL : 0));
      const auto at = [&](int k) { return k < SPL ? lo[k < SPL ? k : 0] : hi[k < SPL ? 0 : k - SPL]; };
      const float dt = step_of(a.softplus, value<T>(x.v[1][i]) + bias), du = dt * value<T>(x.v[0][i]);
      sum += dt;
      float k[SPL];
#pragma unroll
      for (int s = 0; s < SPL; ++s) {
        k[s] = exp2_of(dt * a2[s]);
        h[s] = fmaf(k[s], h[s], du * at(b_at<SPL, BWD>(s)));
      }
      if constexpr (BWD) {
        float go = value<T>(x.v[2][i]);
        if constexpr (GATE) {
          const float z = value<T>(x.v[3][i]);
          go *= z * sigmoid(z);
        }
#pragma unroll
        for (int s = 0; s < SPL; ++s) {
          p[s] *= k[s];
          r[s] = fmaf(p[s], at(c_at<SPL, BWD>(s)) * go, r[s]);
        }
      }
      bc += 2 * SPL;
    };
    Ahead<T, N, kAhead> now, next;
    int64_t t = w.t0;
    if (t + kAhead <= end) now.load(ptr, step, w.in);
    for (; t + kAhead <= end; t += kAhead) {
      if (t + 2 * kAhead <= end) next.load(ptr, step, w.in);
#pragma unroll
      for (int i = 0; i < kAhead; ++i) token(now, i);
      now = next;
    }
    for (; t < end; ++t) {
      Ahead<T, N, 1> one;
      one.load(ptr, step, w.in);
      token(one, 0);
    }
  }
  const int64_t at = ((w.b * a.nc + w.chunk) * a.nblk + w.blk) * SPL * a.d + w.g0;
#pragma unroll
  for (int s = 0; s < SPL; ++s) (a.states + at + (int64_t)s * a.d)[w.in] = h[s];
  if constexpr (BWD) {
    // a product of decays past fp32's range: token by token from the end
    bool past = false;
#pragma unroll
    for (int s = 0; s < SPL; ++s) past = past || !(p[s] <= __FLT_MAX__);
    if (past) from_the_end<T, SPL, GATE>(w, end, a2, r);
#pragma unroll
    for (int s = 0; s < SPL; ++s) (a.rstates + at + (int64_t)s * a.d)[w.in] = r[s];
  }
  if (w.blk == 0) (a.dts + (w.b * a.nc + w.chunk) * a.d + w.g0)[w.in] = (float)sum;
}

// From each chunk's own part to the state that it starts from; blockIdx.y = 1:
// to the gradient that reaches its last state.  RUNS waves take as many runs
// of up to kRun chunks of the same 64 channels: each sums its run from zero,
// all find their first value from the runs before, and each goes over its run
// again, which is still in its registers.
constexpr int kRun = 16;
template <int RUNS>
__global__ void __launch_bounds__(64 * RUNS) scan_combine(ScanArgs a) {
  __shared__ float part[2][RUNS][3][64];
  const int np = a.nblk * a.spl, blocks = (a.d + 63) / 64;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t row = blockIdx.x / (uint32_t)blocks;  // of b np
  const int c0 = (int)(blockIdx.x - row * (uint32_t)blocks) * 64 + lane;
  const int c = c0 < a.d ? c0 : a.d - 1;  // (lanes past the end repeat the last channel)
  const int64_t b = row / (uint32_t)np;
  const int s = (int)(row - (uint32_t)b * np);
  const bool back = blockIdx.y == 1, in = s < a.n;
  const int64_t own = (b * a.d + c) * a.n + (in ? s : 0), step = (int64_t)np * a.d;
  const float a2 = a.a2[(int64_t)s * a.d + c];
  const float* from = back ? a.ds1 : a.s0;
  float carry = from && in ? from[own] : 0.f;
  float* x = (back ? a.rstates : a.states) + (b * a.nc * np + s) * a.d + c;
  const float* dts = a.dts + b * a.nc * a.d + c;
  const int run = a.nc >= kRun * RUNS ? kRun : (a.nc + RUNS - 1) / RUNS;
  int side = 0;
  for (int k0 = 0; k0 < a.nc; k0 += run * RUNS, side ^= 1) {
    const int first = k0 + wave * run;
    float v[kRun], dt[kRun];
#pragma unroll
    for (int j = 0; j < kRun; ++j) {
      const int k = first + j, q = back ? a.nc - 1 - k : k;
      v[j] = dt[j] = 0.f;  // (a chunk that is not there changes nothing)
      if (j < run && k < a.nc) {
        v[j] = x[q * step];
        dt[j] = dts[(int64_t)q * a.d];
      }
    }
    Decay p[kRun], keep = {1.f, 0.f};
    float sum = 0.f;
#pragma unroll
    for (int j = 0; j < kRun; ++j) {
      p[j] = decay_of(a2 * dt[j]);
      sum = p[j].of(sum) + v[j];
      keep.m *= p[j].m;
      keep.e += p[j].e;
    }
    part[side][wave][0][lane] = sum;
    // (16 factors above 1/2: the product is brought back there)
    part[side][wave][1][lane] = __builtin_amdgcn_frexp_mantf(keep.m);
    part[side][wave][2][lane] = keep.e + (float)__builtin_amdgcn_frexp_expf(keep.m);
    __syncthreads();  // (two sides: one barrier keeps readers and writers apart)
    float mine = carry;
#pragma unroll
    for (int i = 0; i < RUNS; ++i) {
      if (i == wave) mine = carry;
      const Decay all = {part[side][i][1][lane], part[side][i][2][lane]};
      carry = all.of(carry) + part[side][i][0][lane];
    }
#pragma unroll
    for (int j = 0; j < kRun; ++j) {
      const int k = first + j, q = back ? a.nc - 1 - k : k;
      if (j < run && k < a.nc) {
        if (c0 < a.d) x[q * step] = mine;
        mine = p[j].of(mine) + v[j];
      }
    }
  }
}

// Outputs, a chunk from its first state on.  With MULTI a workgroup's waves
// hold the blocks of one channel block's states and their parts of C . h are
// joined in LDS, token i of each four by wave i.
template <int T, int SPL, bool GATE, bool MULTI>
__global__ void __launch_bounds__(MULTI ? 1024 : 64) scan_out(ScanArgs a) {
  __shared__ float lds[MULTI ? 2 : 1][MULTI ? 16 : 1][kAhead][64];
  const int wave = MULTI ? __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) : 0;
  const int lane = threadIdx.x & 63;
  const Where w = where(a, wave, blockIdx.x, 1);
  if (!w.on) return;  // (no whole wave: barriers still count all)
  const int64_t end = w.t1 < w.len ? w.t1 : w.len;
  float a2[SPL], h[SPL];
  load_a<SPL>(a, w, a2);
  if (a.nc > 1) {
    const float* p = a.states + ((w.b * a.nc + w.chunk) * a.nblk + w.blk) * SPL * a.d + w.g0;
#pragma unroll
    for (int s = 0; s < SPL; ++s) h[s] = (p + (int64_t)s * a.d)[w.in];
  } else if (a.s0) {
    const float* p = a.s0 + (w.b * a.d + w.g0) * a.n;
#pragma unroll
    for (int s = 0; s < SPL; ++s) {
      const int i = w.blk * SPL + s;
      h[s] = (p + (i < a.n ? i : 0))[w.in * (uint32_t)a.n];
    }
#pragma unroll
    for (int s = 0; s < SPL; ++s) h[s] = w.blk * SPL + s < a.n ? h[s] : 0.f;
  } else {
#pragma unroll
    for (int s = 0; s < SPL; ++s) h[s] = 0.f;
  }
  Elem<T>* out = (Elem<T>*)a.y + ((w.b * a.l + w.t0) * a.d + w.g0);  // of token t
  int64_t t = w.t0;
  if (t < end) {
    const float bias = a.bias ? a.bias[w.c] : 0.f, skip = a.skip ? a.skip[w.c] : 0.f;
    constexpr int N = GATE ? 3 : 2;
    const char* ptr[N];
    int64_t step[N];
    ptr[0] = from<T>(a.u, a.u_stride, w, step[0]);
    ptr[1] = from<T>(a.delta, a.delta_stride, w, step[1]);
    if constexpr (GATE) ptr[2] = from<T>(a.z, a.z_stride, w, step[2]);
    const float* bc = lines<SPL>(a, w);
    const auto token = [&](const auto& x, int i) {
      const auto bb = load_scalar<SPL>(bc);
      const auto cc = load_scalar<SPL>(bc + SPL);
      const float dt = step_of(a.softplus, value<T>(x.v[1][i]) + bias), du = dt * value<T>(x.v[0][i]);
      float y = 0.f;
#pragma unroll
      for (int s = 0; s < SPL; ++s) {
        h[s] = fmaf(exp2_of(dt * a2[s]), h[s], du * bb[s]);
        y = fmaf(cc[s], h[s], y);
      }
      bc += 2 * SPL;
      return y;
    };
    const auto finish = [&](const auto& x, int i, float y) {
      y = fmaf(skip, value<T>(x.v[0][i]), y);
      if constexpr (GATE) {
        const float z = value<T>(x.v[2][i]);
        y *= z * sigmoid(z);
      }
      store1<T>(out + (int64_t)i * a.d, w.in, y);
    };
    Ahead<T, N, kAhead> now, next;
    if (t + kAhead <= end) now.load(ptr, step, w.in);
    int side = 0;
    for (; t + kAhead <= end; t += kAhead) {
      if (t + 2 * kAhead <= end) next.load(ptr, step, w.in);
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const float y = token(now, i);
        if constexpr (MULTI) lds[side][wave][i][lane] = y;
        else finish(now, i, y);
      }
      if constexpr (MULTI) {
        __syncthreads();  // (two sides: one barrier keeps readers and writers apart)
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
          if (i % a.nblk == wave) {
            float y = 0.f;
            for (int k = 0; k < a.nblk; ++k) y += lds[side][k][i][lane];
            finish(now, i, y);
          }
        }
        side ^= 1;
      }
      now = next;
      out += (int64_t)kAhead * a.d;
    }
    for (; t < end; ++t) {
      Ahead<T, N, 1> one;
      one.load(ptr, step, w.in);
      float y = token(one, 0);
      if constexpr (MULTI) {
        lds[side][wave][0][lane] = y;
        __syncthreads();
        if (wave == 0) {
          y = 0.f;
          for (int k = 0; k < a.nblk; ++k) y += lds[side][k][0][lane];
          finish(one, 0, y);
        }
        side ^= 1;
      } else {
        finish(one, 0, y);
      }
      out += a.d;
    }
  }
  if (wave == 0)
    for (; t < w.t1; ++t, out += a.d) store1<T>(out, w.in, 0.f);
  if (w.chunk + 1 == a.nc) {
    float* p = a.s1 + (w.b * a.d + w.g0) * a.n;
#pragma unroll
    for (int s = 0; s < SPL; ++s) {
      const int i = w.blk * SPL + s;
      if (i < a.n) (p + i)[w.in * (uint32_t)a.n] = h[s];
    }
  }
}

template <int T, bool FOURS>
void lay_out(const ScanArgs& a, hipStream_t st) {
  const int64_t lanes = a.b * a.lp * a.g * a.nblk * a.spl / 2 + (int64_t)a.nblk * a.spl * a.d;
  hipLaunchKernelGGL((scan_prep<T, FOURS>), dim3((uint32_t)((lanes + 255) / 256)), dim3(256), 0, st,
                     a);
}

template <int T, int SPL, bool BWD, bool GATE>
void prepare(const ScanArgs& a, hipStream_t st) {
  lay_out<T, BWD>(a, st);
  if (a.nc > 1) {
    const dim3 grid((uint32_t)(a.b * a.nc * a.g * a.cblk * a.nblk));
    hipLaunchKernelGGL((scan_chunk<T, SPL, BWD, GATE>), grid, dim3(64), 0, st, a);
    const int64_t rows = a.b * a.nblk * a.spl * ((a.d + 63) / 64);
    const dim3 blocks((uint32_t)rows, BWD ? 2 : 1);
    // one wave over all chunks where that fills the device
    if (rows >= 4096) hipLaunchKernelGGL(scan_combine<1>, blocks, dim3(64), 0, st, a);
    else hipLaunchKernelGGL(scan_combine<8>, blocks, dim3(512), 0, st, a);
  }
}

template <int T, int SPL, bool GATE>
void go(const ScanArgs& a, hipStream_t st) {
  prepare<T, SPL, false, false>(a, st);
  const dim3 grid((uint32_t)(a.b * a.nc * a.g * a.cblk));
  if (a.nblk > 1) {
    if constexpr (SPL == 16)
      hipLaunchKernelGGL((scan_out<T, 16, GATE, true>), grid, dim3(64 * a.nblk), 0, st, a);
  } else {
    hipLaunchKernelGGL((scan_out<T, SPL, GATE, false>), grid, dim3(64), 0, st, a);
  }
}

template <int T, int SPL>
void go_gate(const ScanArgs& a, hipStream_t st) {
  if (a.z) go<T, SPL, true>(a, st);
  else go<T, SPL, false>(a, st);
}

template <int T>
void go_states(const ScanArgs& a, hipStream_t st) {
  if (a.one) {
    lay_out<T, true>(a, st);
    launch_scan_wide(a, st);
  } else if (a.spl == 4) go_gate<T, 4>(a, st);
  else if (a.spl == 8) go_gate<T, 8>(a, st);
  else go_gate<T, 16>(a, st);
}

template <int T>
void prepare_bwd(const ScanArgs& a, hipStream_t st) {
  if (a.z) prepare<T, 16, true, true>(a, st);
  else prepare<T, 16, true, false>(a, st);
}

}  // namespace scan

// Whether one pass over all tokens is done before the chunks' three.  It takes
// one token's time (by the shape of its workgroups, see go_wide) while these
// have SIMDs to themselves, then kMore a token and 64 channels; the chunks take
// kTwo a token and 64 channels and kFixed besides, for their launches and the
// states between them.  bf16, us: 512 tokens of 2048 channels, 16 states: 50
// and 48 in chunks, 1024 tokens: 95 and 50; 4 sequences of 1024 tokens: 97 and
// 100, 16 of 2048: 359 and 499; 32 states, 700 tokens of 512 channels, 4
// sequences: 61 and 68, 16: 77 and 147; 64 states, 4 such: 83 and 84, one of 256
// channels: 80 and 49.
static bool one_pass(const ScanArgs& a) {
  if (a.n > 64) return false;
  const int blocks = (a.n + 15) / 16;
  const double groups = (double)(a.b * a.g * a.cblk);
  const int size = groups <= 64 ? 0 : (groups <= 128 ? 1 : 2);
  constexpr double kOnes[4][3] = {
      {0.092, 0.092, 0.106}, {0.083, 0.107, 0.13}, {0.083, 0.107, 0.146}, {0.118, 0.157, 0.22}};
  const double kOne = kOnes[a.n <= 16 ? 0 : (a.n <= 24 ? 1 : (a.n <= 32 ? 2 : 3))][size];
  const double kMore = 0.0003 * blocks;
  const double kTwo = 0.00043 * (blocks == 1 ? 1 : 1 + blocks), kFixed = 40.0;
  const double token = kMore * groups > kOne ? kMore * groups : kOne;
  return token * (double)a.l < kFixed + kTwo * groups * (double)a.l;
}

void scan_split(ScanArgs* a, bool bwd) {
  a->dg = a->d / a->g;
  a->cblk = (a->dg + 63) / 64;
  a->one = !bwd && one_pass(*a);
  // (the gradients' and the one pass' waves take fours of blocks of 16)
  a->spl = bwd || a->one ? 16 : (a->n <= 4 ? 4 : (a->n <= 8 ? 8 : 16));
  a->nblk = (a->n + a->spl - 1) / a->spl;
  // a workgroup of the gradients holds 16, 32 or 64 states
  if (bwd && a->nblk > 2) a->nblk = (a->nblk + 3) / 4 * 4;
  a->gblk = (a->nblk + 3) / 4;
  a->lp = (a->l + kGradChunk - 1) / kGradChunk * kGradChunk;
  if (a->one) {
    a->tc = (int)a->l;
    a->nc = 1;
    return;
  }
  if (bwd) {
    a->tc = kGradChunk;
  } else {
    const int64_t waves = a->b * a->g * a->cblk * a->nblk;
    // chunks for 8 waves a SIMD (2 sequences of 4096 tokens of 2048 channels: 147
    // us, 164 for 4)
    int64_t nc = waves >= 4096 || a->b == 0 ? 1 : 8192 / waves;
    const int64_t most = (a->l + 31) / 32;
    if (nc > most) nc = most;
    if (nc < 1) nc = 1;
    a->tc = (int)(((a->l + nc - 1) / nc + 7) / 8 * 8);
    if (a->tc < 8) a->tc = 8;
    // inside a chunk each decay is rounded: no more of them than 128
    if (a->tc > 128) a->tc = 128;
  }
  a->nc = (int)((a->l + a->tc - 1) / a->tc);
  if (a->nc < 1) a->nc = 1;
}

hipError_t launch_scan_prepare_bwd(const ScanArgs& a, hipStream_t st) {
  if (a.type == T_F32) scan::prepare_bwd<T_F32>(a, st);
  else if (a.type == T_BF16) scan::prepare_bwd<T_BF16>(a, st);
  else scan::prepare_bwd<T_F16>(a, st);
  return hipGetLastError();
}

hipError_t launch_scan_fwd(const ScanArgs& a, hipStream_t st) {
  if (a.type == T_F32) scan::go_states<T_F32>(a, st);
  else if (a.type == T_BF16) scan::go_states<T_BF16>(a, st);
  else scan::go_states<T_F16>(a, st);
  return hipGetLastError();
}

}  // namespace seq
}  // namespace dwc
