// seq_conv.hip -- short causal depthwise convolution over tokens, forward,
// token by token and backward.
//
//   pre_t = bias + sum_j w_j x_(t-K+1+j),  y_t = pre_t or pre_t sigmoid(pre_t)
//   e_t = dy_t act'(pre_t),  dx_t = sum_j w_j e_(t+K-1-j)
//   dw_j = sum_t e_t x_(t-K+1+j),  dbias = sum_t e_t
// with x before token 0 from the state s0 and the last K - 1 inputs left in
// s1, whose gradient joins dx (and ds0, where the sequence is shorter).
//
// Bound: memory (2 K + 8 operations an element).  A lane owns VEC channels of
// a strip of tokens and keeps the K - 1 inputs behind the current one in
// registers, so x is read once but for the K - 1 tokens before each strip
// (from the caches: a neighbour reads them too).  8 sequences of 2048 tokens of
// 2048 channels, bf16, 4 taps: 32 us (4.2 TB/s), back 45 us (4.5 TB/s).
#include "seq_device.h"
#include "seq_space.h"

namespace dwc {
namespace seq {
namespace conv {

constexpr int kUnroll = 4;  // tokens whose loads are under way together

__device__ __forceinline__ float sigmoid(float x) {
  // exp of a large argument is inf, and 1 / inf 0: the limits come out right
  return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-1.44269504088896341f * x));
}

__device__ __forceinline__ int64_t length_of(const ConvArgs& a, int64_t b) {
  if (!a.lengths) return a.l;
  const int64_t n = a.lengths[b];
  return n < 0 ? 0 : (n < a.l ? n : a.l);
}

template <int VEC>
__device__ __forceinline__ void zero(float (&v)[VEC]) {
#pragma unroll
  for (int i = 0; i < VEC; ++i) v[i] = 0.f;
}

// VEC neighbouring channels as they stand in memory.
template <int T, int VEC> struct Row {
  uint32_t v[VEC / 2];
  __device__ __forceinline__ void load(const void* p, int64_t i) {
    const u32x2 t = *(const u32x2*)((const uint16_t*)p + i);
    v[0] = t[0];
    v[1] = t[1];
  }
  __device__ __forceinline__ void get(float (&x)[VEC]) const {
#pragma unroll
    for (int j = 0; j < VEC / 2; ++j) {
      x[2 * j] = from16<T>(v[j] & 0xffffu);
      x[2 * j + 1] = from16<T>(v[j] >> 16);
    }
  }
};
template <int T> struct Row<T, 1> {
  uint16_t v;
  __device__ __forceinline__ void load(const void* p, int64_t i) { v = ((const uint16_t*)p)[i]; }
  __device__ __forceinline__ void get(float (&x)[1]) const { x[0] = from16<T>(v); }
};
template <int VEC> struct Row<T_F32, VEC> {
  float v[VEC];
  __device__ __forceinline__ void load(const void* p, int64_t i) { load_vec<T_F32, VEC>(p, i, v); }
  __device__ __forceinline__ void get(float (&x)[VEC]) const {
#pragma unroll
    for (int j = 0; j < VEC; ++j) x[j] = v[j];
  }
};
template <> struct Row<T_F32, 1> {
  float v;
  __device__ __forceinline__ void load(const void* p, int64_t i) { v = ((const float*)p)[i]; }
  __device__ __forceinline__ void get(float (&x)[1]) const { x[0] = v; }
};

// Input of token t: of the state before the first one, nothing past len.
template <int T, int VEC>
__device__ __forceinline__ void input(const ConvArgs& a, int64_t b, int64_t t, int64_t len,
                                      int64_t c, float (&v)[VEC]) {
  if (t >= 0 && t < len) {
    load_vec<T, VEC>(a.x, b * a.x_stride[0] + t * a.x_stride[1] + c, v);
  } else if (t < 0 && t + a.taps > 0 && a.s0) {
    load_vec<T, VEC>(a.s0, (b * (a.taps - 1) + t + a.taps - 1) * a.d + c, v);
  } else {
    zero(v);
  }
}

template <int WT, int K, int VEC>
__device__ __forceinline__ void weights_of(const ConvArgs& a, int64_t c, float (&w)[K][VEC],
                                           float (&bias)[VEC]) {
#pragma unroll
  for (int j = 0; j < K; ++j) load_vec<WT, VEC>(a.w, j * a.d + c, w[j]);
  if (a.bias) load_vec<WT, VEC>(a.bias, c, bias);
}
template <int K, int VEC>
__device__ __forceinline__ void weights(const ConvArgs& a, int64_t c, float (&w)[K][VEC],
                                        float (&bias)[VEC]) {
  zero(bias);
  if (a.w_type == T_F32) weights_of<T_F32, K, VEC>(a, c, w, bias);
  else if (a.w_type == T_BF16) weights_of<T_BF16, K, VEC>(a, c, w, bias);
  else weights_of<T_F16, K, VEC>(a, c, w, bias);
}

template <int T, int K, int VEC>
__global__ void __launch_bounds__(256) conv_fwd(ConvArgs a) {
  constexpr int P = K - 1, U = kUnroll;
  const uint32_t vecs = (uint32_t)(a.d / VEC);
  const uint32_t at = blockIdx.x * 256u + threadIdx.x;
  const uint32_t rest = at / vecs;
  const int64_t c = (int64_t)(at - rest * vecs) * VEC;
  const uint32_t strip = rest % (uint32_t)a.strips;
  const int64_t b = rest / (uint32_t)a.strips;
  if (b >= a.b) return;
  const int64_t len = length_of(a, b);
  const int64_t t0 = (int64_t)strip * a.strip;
  const int64_t t1 = t0 + a.strip < a.l ? t0 + a.strip : a.l;
  const int64_t end = t1 < len ? t1 : len;
  const int64_t xb = b * a.x_stride[0] + c, xs = a.x_stride[1], yb = b * a.l * a.d + c;
  float w[K][VEC], bias[VEC], x[P + U][VEC], last[P > 0 ? P : 1][VEC];
  Row<T, VEC> now[U], next[U];
  int64_t t = t0;
  if (t + U <= end) {
#pragma unroll
    for (int i = 0; i < U; ++i) now[i].load(a.x, xb + (t + i) * xs);
  }
  weights<K, VEC>(a, c, w, bias);
#pragma unroll
  for (int j = 0; j < P; ++j) input<T, VEC>(a, b, t0 - P + j, len, c, x[j]);
  // the state left behind: read before any of it is written over
  if (strip == 0 && a.s1) {
#pragma unroll
    for (int j = 0; j < P; ++j) input<T, VEC>(a, b, len - P + j, len, c, last[j]);
  }
  const auto out = [&](int i, int64_t tt) {
    float y[VEC];
#pragma unroll
    for (int k = 0; k < VEC; ++k) {
      y[k] = bias[k];
#pragma unroll
      for (int j = 0; j < K; ++j) y[k] = fmaf(w[j][k], x[i + j][k], y[k]);
      const float s = y[k] * sigmoid(y[k]);
      y[k] = a.silu ? s : y[k];
    }
    store_vec<T, VEC>(a.y, yb + tt * a.d, y);
  };
  for (; t + U <= end; t += U) {
    if (t + 2 * U <= end) {
#pragma unroll
      for (int i = 0; i < U; ++i) next[i].load(a.x, xb + (t + U + i) * xs);
    }
#pragma unroll
    for (int i = 0; i < U; ++i) {
      now[i].get(x[P + i]);
      out(i, t + i);
    }
#pragma unroll
    for (int j = 0; j < P; ++j)
#pragma unroll
      for (int k = 0; k < VEC; ++k) x[j][k] = x[U + j][k];
#pragma unroll
    for (int i = 0; i < U; ++i) now[i] = next[i];
  }
  for (; t < end; ++t) {
    load_vec<T, VEC>(a.x, xb + t * xs, x[P]);
    out(0, t);
#pragma unroll
    for (int j = 0; j < P; ++j)
#pragma unroll
      for (int k = 0; k < VEC; ++k) x[j][k] = x[j + 1][k];
  }
  for (; t < t1; ++t) {
    zero(x[P]);
    store_vec<T, VEC>(a.y, yb + t * a.d, x[P]);
  }
  if (strip == 0 && a.s1) {
#pragma unroll
    for (int j = 0; j < P; ++j) store_vec<T, VEC>(a.s1, (b * P + j) * a.d + c, last[j]);
  }
}

// Four waves a workgroup take four strips of the same 64 VEC channels; their
// sums of dw and dbias are joined in LDS in order.
template <int T, int K, int VEC>
__global__ void __launch_bounds__(256) conv_bwd(ConvArgs a) {
  constexpr int P = K - 1, U = kUnroll;
  __shared__ float lds[3][64][VEC];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t blocks = (uint32_t)((a.d + 64 * VEC - 1) / (64 * VEC));
  const uint32_t quads = (uint32_t)((a.strips + 3) / 4);
  const uint32_t row = blockIdx.x / blocks;
  const int64_t c = ((int64_t)(blockIdx.x - row * blocks) * 64 + lane) * VEC;
  const int64_t b = row / quads;
  const int64_t strip = (int64_t)(row - (uint32_t)b * quads) * 4 + wave;
  const int64_t len = length_of(a, b);
  const int64_t t0 = strip * a.strip;
  const int64_t t1 = t0 + a.strip < a.l ? t0 + a.strip : a.l;
  const int64_t end = t1 < len ? t1 : len;
  float w[K][VEC], bias[VEC], dw[K][VEC], db[VEC];
#pragma unroll
  for (int k = 0; k < VEC; ++k) {
    db[k] = 0.f;
#pragma unroll
    for (int j = 0; j < K; ++j) dw[j][k] = 0.f;
  }
  if (c < a.d && strip < a.strips) {
    weights<K, VEC>(a, c, w, bias);
    // x[j]: input t - P + j, e[j]: e_(t - P + j)
    float x[P + U][VEC], e[P + U][VEC];
#pragma unroll
    for (int j = 0; j < P; ++j) {
      input<T, VEC>(a, b, t0 - P + j, len, c, x[j]);
      zero(e[j]);
    }
    // dy in e[P + i] to e of token t + i
    const auto slope = [&](int i) {
#pragma unroll
      for (int k = 0; k < VEC; ++k) {
        float pre = bias[k];
#pragma unroll
        for (int j = 0; j < K; ++j) pre = fmaf(w[j][k], x[i + j][k], pre);
        const float s = sigmoid(pre), g = e[P + i][k] * fmaf(pre * s, 1.f - s, s);
        e[P + i][k] = a.silu ? g : e[P + i][k];
      }
    };
    const auto sums = [&](int i) {
#pragma unroll
      for (int k = 0; k < VEC; ++k) {
        db[k] += e[P + i][k];
#pragma unroll
        for (int j = 0; j < K; ++j) dw[j][k] = fmaf(e[P + i][k], x[i + j][k], dw[j][k]);
      }
    };
    const auto back = [&](int i, float(&v)[VEC]) {
      zero(v);
#pragma unroll
      for (int k = 0; k < VEC; ++k)
#pragma unroll
        for (int j = 0; j < K; ++j) v[k] = fmaf(w[j][k], e[P + i - j][k], v[k]);
    };
    const auto shift = [&](int n) {
#pragma unroll
      for (int j = 0; j < P; ++j)
#pragma unroll
        for (int k = 0; k < VEC; ++k) {
          x[j][k] = x[n + j][k];
          e[j][k] = e[n + j][k];
        }
    };
    // one token, of whatever kind
    const auto one = [&](int64_t t) {
      input<T, VEC>(a, b, t, len, c, x[P]);
      zero(e[P]);
      if (t < len) {
        load_vec<T, VEC>(a.dy, b * a.dy_stride[0] + t * a.dy_stride[1] + c, e[P]);
        slope(0);
        if (t < t1) sums(0);
      }
      const int64_t s = t - P;  // every e that reads input s is known
      if (s >= t0 || (strip == 0 && s < 0)) {
        float v[VEC];
        zero(v);
        if (s < len) {
          back(0, v);
          if (s >= len - P && a.ds1) {
            float g[VEC];
            load_vec<T, VEC>(a.ds1, (b * P + s - len + P) * a.d + c, g);
#pragma unroll
            for (int k = 0; k < VEC; ++k) v[k] += g[k];
          }
        }
        if (s >= 0) store_vec<T, VEC>(a.y, (b * a.l + s) * a.d + c, v);
        else if (a.ds0) store_vec<T, VEC>(a.ds0, (b * P + s + P) * a.d + c, v);
      }
      shift(1);
    };
    int64_t t = t0;
    for (; t < t0 + P && t < t1 + P; ++t) one(t);
    // tokens inside the strip and the length, whose inputs s = t - P are too
    // and have no part in s1
    const int64_t xb = b * a.x_stride[0] + c, xs = a.x_stride[1];
    const int64_t gb = b * a.dy_stride[0] + c, gs = a.dy_stride[1];
    Row<T, VEC> xn[U], gn[U];
    const auto fetch = [&](int64_t at) {
#pragma unroll
      for (int i = 0; i < U; ++i) {
        xn[i].load(a.x, xb + (at + i) * xs);
        gn[i].load(a.dy, gb + (at + i) * gs);
      }
    };
    if (t + U <= end) fetch(t);
    for (; t + U <= end; t += U) {
#pragma unroll
      for (int i = 0; i < U; ++i) {
        xn[i].get(x[P + i]);
        gn[i].get(e[P + i]);
      }
      if (t + 2 * U <= end) fetch(t + U);
#pragma unroll
      for (int i = 0; i < U; ++i) {
        float v[VEC];
        slope(i);
        sums(i);
        back(i, v);
        store_vec<T, VEC>(a.y, (b * a.l + t + i - P) * a.d + c, v);
      }
      shift(U);
    }
    for (; t < t1 + P; ++t) one(t);
  }
#pragma unroll
  for (int j = 0; j <= K; ++j) {
    float(&v)[VEC] = j < K ? dw[j < K ? j : 0] : db;
    __syncthreads();
    if (wave > 0) {
#pragma unroll
      for (int k = 0; k < VEC; ++k) lds[wave - 1][lane][k] = v[k];
    }
    __syncthreads();
    if (wave == 0 && c < a.d) {
      float* out = a.part + ((int64_t)row * (K + 1) + j) * a.d + c;
#pragma unroll
      for (int k = 0; k < VEC; ++k) out[k] = v[k] + lds[0][lane][k] + lds[1][lane][k] + lds[2][lane][k];
    }
  }
}

static bool aligned(const void* p, size_t n) { return ((uintptr_t)p % n) == 0; }

// Whether a lane takes four channels: where sizes, strides and addresses
// allow loads of that.
static bool wide(const ConvArgs& a, bool bwd) {
  constexpr int vec = 4;
  const size_t n = a.type == T_F32 ? 16 : 8, m = a.w_type == T_F32 ? 16 : 8;
  bool ok = a.d % vec == 0 && a.x_stride[0] % vec == 0 && a.x_stride[1] % vec == 0 &&
            aligned(a.x, n) && aligned(a.y, n) && aligned(a.s0, n) && aligned(a.s1, n) &&
            aligned(a.w, m) && aligned(a.bias, m);
  if (bwd)
    ok = ok && a.dy_stride[0] % vec == 0 && a.dy_stride[1] % vec == 0 && aligned(a.dy, n) &&
         aligned(a.ds1, n) && aligned(a.ds0, n);
  return ok;
}

template <int T, int K, int VEC>
void go_fwd(const ConvArgs& a, hipStream_t st) {
  const int64_t lanes = a.b * a.strips * (a.d / VEC);
  hipLaunchKernelGGL((conv_fwd<T, K, VEC>), dim3((uint32_t)((lanes + 255) / 256)), dim3(256), 0, st,
                     a);
}

template <int T, int K, int VEC>
void go_bwd(const ConvArgs& a, hipStream_t st) {
  const int64_t blocks = (a.d + 64 * VEC - 1) / (64 * VEC);
  hipLaunchKernelGGL((conv_bwd<T, K, VEC>), dim3((uint32_t)(conv_rows(a) * blocks)), dim3(256), 0,
                     st, a);
}

template <int T, int K>
void go_width(bool bwd, const ConvArgs& a, hipStream_t st) {
  const bool w = wide(a, bwd);
  if (bwd) w ? go_bwd<T, K, 4>(a, st) : go_bwd<T, K, 1>(a, st);
  else w ? go_fwd<T, K, 4>(a, st) : go_fwd<T, K, 1>(a, st);
}

template <int T>
void go_taps(bool bwd, const ConvArgs& a, hipStream_t st) {
  switch (a.taps) {
    case 1: return go_width<T, 1>(bwd, a, st);
    case 2: return go_width<T, 2>(bwd, a, st);
    case 3: return go_width<T, 3>(bwd, a, st);
    case 4: return go_width<T, 4>(bwd, a, st);
    case 5: return go_width<T, 5>(bwd, a, st);
    case 6: return go_width<T, 6>(bwd, a, st);
    case 7: return go_width<T, 7>(bwd, a, st);
    case 8: return go_width<T, 8>(bwd, a, st);
  }
}

static void launch(bool bwd, const ConvArgs& a, hipStream_t st) {
  if (a.type == T_F32) go_taps<T_F32>(bwd, a, st);
  else if (a.type == T_BF16) go_taps<T_BF16>(bwd, a, st);
  else go_taps<T_F16>(bwd, a, st);
}

}  // namespace conv

int conv_strip(const ConvArgs& a, bool bwd) {
  // lanes for 8 waves a compute unit, in strips of 8 to 32 tokens (8 sequences
  // of 2048 tokens of 2048 channels, both ways: 82 us in strips of 32, 92 of 16,
  // 89 of 64, 90 of 128)
  const int64_t per = (a.d + 3) / 4 * a.b;
  int strip = 32;
  while (strip > 8 && per * ((a.l + strip - 1) / strip) < (int64_t)256 * 8 * 64) strip /= 2;
  return strip;
}

int64_t conv_rows(const ConvArgs& a) { return a.b * ((a.strips + 3) / 4); }

hipError_t launch_conv_fwd(const ConvArgs& a, hipStream_t st) {
  conv::launch(false, a, st);
  return hipGetLastError();
}

hipError_t launch_conv_bwd(const ConvArgs& a, float* dw, float* dbias, hipStream_t st) {
  if (a.b > 0) {  // (else the sums of no rows: zeros)
    conv::launch(true, a, st);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  const int64_t rows = conv_rows(a), stride = (a.taps + 1) * a.d;
  const ColumnSum jobs[kColumnJobs] = {{a.part, dw, rows, stride, a.taps * a.d, 0},
                                       {a.part + a.taps * a.d, dbias, rows, stride, a.d, 0},
                                       {nullptr, nullptr, 0, 0, 0, 0}};
  return launch_column_sums(jobs, st);
}

}  // namespace seq
}  // namespace dwc
