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
// Bound: the vector units.  A state of a token takes an exp and four other
// instructions, 20 us a pass at 4096 tokens of 2048 channels and 16 states.
#include "seq_scan.h"

namespace dwc {
namespace seq {
namespace scan {

template <int T>
__global__ void __launch_bounds__(256) scan_prep(ScanArgs a) {
  const int w = 2 * a.spl, line = a.nblk * w;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t token = i / ((int64_t)a.g * line);  // of b l
  if (token >= a.b * a.l) return;
  const int at = (int)(i - token * a.g * line), g = at / line, k = at - g * line;
  const int blk = k / w, j = k - blk * w, s = blk * a.spl + j % a.spl;
  const int64_t b = token / a.l, t = token - b * a.l;
  float v = 0.f;
  if (s < a.n && t < length_of(a, b))
    v = j < a.spl
            ? load1<T>(a.bm, b * a.b_stride[0] + t * a.b_stride[1] + g * a.b_stride[2] + s)
            : load1<T>(a.cm, b * a.c_stride[0] + t * a.c_stride[1] + g * a.c_stride[2] + s);
  a.bc[i] = v;
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
#pragma unroll
  for (int s = 0; s < SPL; ++s) {
    const int i = w.blk * SPL + s;
    v[s] = i < a.n ? kLog2e * a.a[(int64_t)w.c * a.n + i] : 0.f;
  }
}

constexpr int kAhead = 4;  // tokens whose loads are under way together

// Raw operands of kAhead tokens from t on; tokens from end on give the last
// one's again.
template <int T, int N>
struct Ahead {
  Raw<T> v[N][kAhead];
  // p: addresses that are the same in all lanes, of the group's first channel
  __device__ __forceinline__ void load(const void* const (&p)[N], const int64_t (&step)[N],
                                       uint32_t in, int64_t t, int64_t end) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int64_t at = t + i < end ? t + i : end - 1;
#pragma unroll
      for (int k = 0; k < N; ++k)
        if (p[k]) v[k][i] = ((const Raw<T>*)p[k] + at * step[k])[in];
    }
  }
};

// Each chunk's state from zero and the sum of its steps.  With BWD also, from
// zero at its end, the gradient that it hands to the state before it:
//   sum_t (a_t0 ... a_t) C_t do_t,  do = dy silu(z).
template <int T, int SPL, bool BWD>
__global__ void __launch_bounds__(64) scan_chunk(ScanArgs a) {
  const Where w = where(a, 0, blockIdx.x, a.nblk);
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
    constexpr int N = BWD ? 4 : 2;
    const int64_t e = sizeof(Raw<T>);
    const void* ptr[N];
    int64_t step[N];
    ptr[0] = (const char*)a.u + (w.b * a.u_stride[0] + w.g0) * e;
    step[0] = a.u_stride[1];
    ptr[1] = (const char*)a.delta + (w.b * a.delta_stride[0] + w.g0) * e;
    step[1] = a.delta_stride[1];
    if constexpr (BWD) {
      ptr[2] = (const char*)a.dy + (w.b * a.dy_stride[0] + w.g0) * e;
      step[2] = a.dy_stride[1];
      ptr[3] = a.z ? (const char*)a.z + (w.b * a.z_stride[0] + w.g0) * e : nullptr;
      step[3] = a.z_stride[1];
    }
    const int64_t line = (int64_t)a.g * a.nblk * 2 * SPL;
    const float* bc = a.bc + (w.b * a.l + w.t0) * line + (w.g * a.nblk + w.blk) * 2 * SPL;
    Ahead<T, N> now, next;
    now.load(ptr, step, w.in, w.t0, end);
    for (int64_t t = w.t0; t < end; t += kAhead) {
      next.load(ptr, step, w.in, t + kAhead, end);
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        if (t + i >= end) break;
        const auto bb = load_scalar<SPL>(bc);
        float dt = value<T>(now.v[1][i]) + bias;
        if (a.softplus) dt = softplus(dt);
        sum += dt;
        const float du = dt * value<T>(now.v[0][i]);
        float go = 0.f;
        typename VecOf<SPL>::type cc;
        if constexpr (BWD) {
          cc = load_scalar<SPL>(bc + SPL);
          go = value<T>(now.v[2][i]);
          if (a.z) {
            const float z = value<T>(now.v[3][i]);
            go *= z * sigmoid(z);
          }
        }
#pragma unroll
        for (int s = 0; s < SPL; ++s) {
          const float k = exp2_of(dt * a2[s]);
          h[s] = fmaf(k, h[s], du * bb[s]);
          if constexpr (BWD) {
            p[s] *= k;
            r[s] = fmaf(p[s], cc[s] * go, r[s]);
          }
        }
        bc += line;
      }
      now = next;
    }
  }
  if (!w.on) return;
  const int64_t at = ((w.b * a.nc + w.chunk) * a.nblk + w.blk) * SPL * a.d + w.c;
#pragma unroll
  for (int s = 0; s < SPL; ++s) {
    a.states[at + (int64_t)s * a.d] = h[s];
    if constexpr (BWD) a.rstates[at + (int64_t)s * a.d] = r[s];
  }
  if (w.blk == 0) a.dts[(w.b * a.nc + w.chunk) * a.d + w.c] = (float)sum;
}

// From each chunk's own part to the state that it starts from; blockIdx.y = 1:
// to the gradient that reaches its last state.
__global__ void __launch_bounds__(256) scan_combine(ScanArgs a) {
  const int np = a.nblk * a.spl;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= a.b * np * a.d) return;
  const int64_t row = i / a.d, b = row / np;
  const int c = (int)(i - row * a.d), s = (int)(row - b * np);
  const bool back = blockIdx.y == 1, in = s < a.n;
  const int64_t own = (b * a.d + c) * a.n + s, step = (int64_t)np * a.d;
  const float a2 = in ? kLog2e * a.a[(int64_t)c * a.n + s] : 0.f;
  const float* from = back ? a.ds1 : a.s0;
  float carry = from && in ? from[own] : 0.f;
  float* x = (back ? a.rstates : a.states) + (b * a.nc * np + s) * a.d + c;
  const float* dts = a.dts + b * a.nc * a.d + c;
  constexpr int U = 8;
  for (int k = 0; k < a.nc; k += U) {
    float v[U], p[U];
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const int q = back ? a.nc - 1 - k - j : k + j;
      if (k + j < a.nc) {
        v[j] = x[q * step];
        p[j] = dts[(int64_t)q * a.d];
      }
    }
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const int q = back ? a.nc - 1 - k - j : k + j;
      if (k + j < a.nc) {
        x[q * step] = carry;
        carry = fmaf(exp2_of(a2 * p[j]), carry, v[j]);
      }
    }
  }
}

// Outputs, a chunk from its first state on.  With MULTI a workgroup's waves
// hold the blocks of one channel block's states and their parts of C . h are
// joined in LDS, token i of each four by wave i.
template <int T, int SPL, bool MULTI>
__global__ void __launch_bounds__(MULTI ? 1024 : 64) scan_out(ScanArgs a) {
  __shared__ float lds[MULTI ? 2 : 1][MULTI ? 16 : 1][kAhead][64];
  const int wave = MULTI ? __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) : 0;
  const int lane = threadIdx.x & 63;
  const Where w = where(a, wave, blockIdx.x, 1);
  const int64_t end = w.t1 < w.len ? w.t1 : w.len;
  float a2[SPL], h[SPL];
  load_a<SPL>(a, w, a2);
#pragma unroll
  for (int s = 0; s < SPL; ++s) {
    const int i = w.blk * SPL + s;
    h[s] = 0.f;
    if (a.nc > 1)
      h[s] = a.states[(((w.b * a.nc + w.chunk) * a.nblk + w.blk) * SPL + s) * a.d + w.c];
    else if (a.s0 && i < a.n)
      h[s] = a.s0[(w.b * a.d + w.c) * a.n + i];
  }
  Raw<T>* const out = (Raw<T>*)a.y + w.b * a.l * a.d + w.g0;
  if (w.t0 < end) {
    const float bias = a.bias ? a.bias[w.c] : 0.f, skip = a.skip ? a.skip[w.c] : 0.f;
    const int64_t e = sizeof(Raw<T>);
    const void* ptr[3] = {(const char*)a.u + (w.b * a.u_stride[0] + w.g0) * e,
                          (const char*)a.delta + (w.b * a.delta_stride[0] + w.g0) * e,
                          a.z ? (const char*)a.z + (w.b * a.z_stride[0] + w.g0) * e : nullptr};
    const int64_t step[3] = {a.u_stride[1], a.delta_stride[1], a.z_stride[1]};
    const int64_t line = (int64_t)a.g * a.nblk * 2 * SPL;
    const float* bc = a.bc + (w.b * a.l + w.t0) * line + (w.g * a.nblk + w.blk) * 2 * SPL;
    const auto finish = [&](int64_t t, float y, float u, Raw<T> rz) {
      y = fmaf(skip, u, y);
      if (a.z) {
        const float z = value<T>(rz);
        y *= z * sigmoid(z);
      }
      if (w.on) store1<T>(out + t * a.d, w.in, y);
    };
    Ahead<T, 3> now, next;
    now.load(ptr, step, w.in, w.t0, end);
    int side = 0;
    for (int64_t t = w.t0; t < end; t += kAhead) {
      next.load(ptr, step, w.in, t + kAhead, end);
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        if (t + i >= end) break;
        const auto bb = load_scalar<SPL>(bc);
        const auto cc = load_scalar<SPL>(bc + SPL);
        float dt = value<T>(now.v[1][i]) + bias;
        if (a.softplus) dt = softplus(dt);
        const float u = value<T>(now.v[0][i]), du = dt * u;
        float y = 0.f;
#pragma unroll
        for (int s = 0; s < SPL; ++s) {
          h[s] = fmaf(exp2_of(dt * a2[s]), h[s], du * bb[s]);
          y = fmaf(cc[s], h[s], y);
        }
        if constexpr (MULTI) lds[side][wave][i][lane] = y;
        else finish(t + i, y, u, now.v[2][i]);
        bc += line;
      }
      if constexpr (MULTI) {
        __syncthreads();  // (two sides: one barrier keeps readers and writers apart)
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
          if (i % a.nblk == wave && t + i < end) {
            float y = 0.f;
            for (int k = 0; k < a.nblk; ++k) y += lds[side][k][i][lane];
            finish(t + i, y, value<T>(now.v[0][i]), now.v[2][i]);
          }
        }
        side ^= 1;
      }
      now = next;
    }
  }
  if (!w.on) return;
  if (wave == 0)
    for (int64_t t = end > w.t0 ? end : w.t0; t < w.t1; ++t) store1<T>(out + t * a.d, w.in, 0.f);
  if (w.chunk + 1 == a.nc) {
#pragma unroll
    for (int s = 0; s < SPL; ++s) {
      const int i = w.blk * SPL + s;
      if (i < a.n) a.s1[(w.b * a.d + w.c) * a.n + i] = h[s];
    }
  }
}

template <int T, int SPL, bool BWD>
void prepare(const ScanArgs& a, hipStream_t st) {
  if (a.l > 0) {
    const int64_t vals = a.b * a.l * a.g * a.nblk * 2 * a.spl;
    hipLaunchKernelGGL((scan_prep<T>), dim3((uint32_t)((vals + 255) / 256)), dim3(256), 0, st, a);
  }
  if (a.nc > 1) {
    const dim3 grid((uint32_t)(a.b * a.nc * a.g * a.cblk * a.nblk));
    hipLaunchKernelGGL((scan_chunk<T, SPL, BWD>), grid, dim3(64), 0, st, a);
    const int64_t vals = a.b * a.nblk * a.spl * a.d;
    hipLaunchKernelGGL(scan_combine, dim3((uint32_t)((vals + 255) / 256), BWD ? 2 : 1), dim3(256),
                       0, st, a);
  }
}

template <int T, int SPL>
void go(const ScanArgs& a, hipStream_t st) {
  prepare<T, SPL, false>(a, st);
  const dim3 grid((uint32_t)(a.b * a.nc * a.g * a.cblk));
  if (a.nblk > 1) {
    if constexpr (SPL == 16)
      hipLaunchKernelGGL((scan_out<T, 16, true>), grid, dim3(64 * a.nblk), 0, st, a);
  } else {
    hipLaunchKernelGGL((scan_out<T, SPL, false>), grid, dim3(64), 0, st, a);
  }
}

template <int T>
void go_states(const ScanArgs& a, hipStream_t st) {
  if (a.spl == 4) go<T, 4>(a, st);
  else if (a.spl == 8) go<T, 8>(a, st);
  else go<T, 16>(a, st);
}

}  // namespace scan

void scan_split(ScanArgs* a, bool bwd) {
  a->dg = a->d / a->g;
  // (the gradients' workgroups hold 16 states, four a wave)
  a->spl = bwd ? 16 : (a->n <= 4 ? 4 : (a->n <= 8 ? 8 : 16));
  a->nblk = (a->n + a->spl - 1) / a->spl;
  a->cblk = (a->dg + 63) / 64;
  if (bwd) {
    a->tc = 32;
  } else {
    const int64_t waves = a->b * a->g * a->cblk * a->nblk;
    int64_t nc = waves >= 2048 || a->b == 0 ? 1 : 4096 / waves;
    const int64_t most = (a->l + 31) / 32;
    if (nc > most) nc = most;
    if (nc < 1) nc = 1;
    a->tc = (int)(((a->l + nc - 1) / nc + 7) / 8 * 8);
    if (a->tc < 8) a->tc = 8;
  }
  a->nc = (int)((a->l + a->tc - 1) / a->tc);
  if (a->nc < 1) a->nc = 1;
}

hipError_t launch_scan_prepare_bwd(const ScanArgs& a, hipStream_t st) {
  if (a.type == T_F32) scan::prepare<T_F32, 16, true>(a, st);
  else if (a.type == T_BF16) scan::prepare<T_BF16, 16, true>(a, st);
  else scan::prepare<T_F16, 16, true>(a, st);
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
