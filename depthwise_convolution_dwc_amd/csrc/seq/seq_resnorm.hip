// seq_resnorm.hip -- the norm behind a block, its gate and scale, the residual
// sum and the norm before the next block in one pass over the rows.
//
//   q1 = 1 / sqrt(mean(y^2) + eps), p = y q1 w_post  (or p = y)
//   r = x + scale act(gate) p
//   q2 = 1 / sqrt(mean(r^2) + eps), h = r q2 w_pre
// back, with e = dh w_pre and t the gradient that reaches r:
//   t = dr + q2 (e - r q2 mean(e r q2)),  dx = t
//   dscale = sum t act p,  dgate = t scale p act',  dp = t scale act
//   dw_post = sum dp y q1, dw_pre = sum dh r q2
//   dy = q1 (dp w_post - y q1 mean(dp w_post y q1))
// r is made again from x, y and the gate, as many bytes as reading it and
// without its rounding.
//
// Bound: memory.  A row is read once into registers; LPR lanes share it.
// 16384 rows of 2048, fp32 stream and bf16 blocks: 70 us (5.7 TB/s), back 120 us
// (5.0 TB/s) and 6 for the sums over the rows.  (Back, the next row read while
// this one is worked on: 225 us for both ways, then 203, for the registers.)
#include "seq_device.h"
#include "seq_space.h"

namespace dwc {
namespace seq {
namespace resnorm {

constexpr int kBlock = 256;

template <int LPR>
__device__ __forceinline__ float row_sum(float v, float* lds) {
  if constexpr (LPR <= 64) {
    return lane_sum<LPR>(v);
  } else {
    v = lane_sum<64>(v);
    constexpr int W = LPR / 64;
    __syncthreads();  // the previous sum's readers are done
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
    __syncthreads();
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < W; ++i) s += lds[i];
    return s;
  }
}

enum { A_NONE = 0, A_SILU = 1, A_SIGMOID = 2 };

// act(g) and its slope.
__device__ __forceinline__ f32x2 act_of(int act, float g) {
  if (act == A_NONE) return f32x2{g, 1.f};
  const float s =
      __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-1.44269504088896341f * g));
  if (act == A_SIGMOID) return f32x2{s, s * (1.f - s)};
  return f32x2{g * s, fmaf(g * s, 1.f - s, s)};
}

// The three rows of weights, 1 where one is not given; the type is decided
// once so that the loads are under way together.
template <int WT, int VEC, int LPR, int NV>
__device__ __forceinline__ void load_weights(const void* p, int64_t c, int lane,
                                             float (&w)[NV][VEC]) {
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int64_t col = (int64_t)(i * LPR + lane) * VEC;
#pragma unroll
    for (int j = 0; j < VEC; ++j) w[i][j] = 1.f;
    if (p && col < c) load_vec<WT, VEC>(p, col, w[i]);
  }
}

template <int VEC, int LPR, int NV>
__device__ __forceinline__ void weights(const ResNormArgs& a, int lane, float (&scale)[NV][VEC],
                                        float (&post)[NV][VEC], float (&pre)[NV][VEC]) {
  if (a.w_type == T_F32) {
    load_weights<T_F32, VEC, LPR, NV>(a.scale, a.c, lane, scale);
    load_weights<T_F32, VEC, LPR, NV>(a.w_post, a.c, lane, post);
    load_weights<T_F32, VEC, LPR, NV>(a.w_pre, a.c, lane, pre);
  } else if (a.w_type == T_BF16) {
    load_weights<T_BF16, VEC, LPR, NV>(a.scale, a.c, lane, scale);
    load_weights<T_BF16, VEC, LPR, NV>(a.w_post, a.c, lane, post);
    load_weights<T_BF16, VEC, LPR, NV>(a.w_pre, a.c, lane, pre);
  } else {
    load_weights<T_F16, VEC, LPR, NV>(a.scale, a.c, lane, scale);
    load_weights<T_F16, VEC, LPR, NV>(a.w_post, a.c, lane, post);
    load_weights<T_F16, VEC, LPR, NV>(a.w_pre, a.c, lane, pre);
  }
}

// A row, `none` where p is null, past the row's end and past the last row.
template <int T, int VEC, int LPR, int NV>
__device__ __forceinline__ void load_row(const void* p, int64_t row, int64_t stride, bool live,
                                         int64_t c, int lane, float none, float (&v)[NV][VEC]) {
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int64_t col = (int64_t)(i * LPR + lane) * VEC;
    if (p && live && col < c) {
      load_vec<T, VEC>(p, row * stride + col, v[i]);
    } else {
#pragma unroll
      for (int j = 0; j < VEC; ++j) v[i][j] = none;
    }
  }
}

// Each group of LPR lanes walks rows; the weights stay in registers and the
// next row is read while this one's sums are made (a workgroup a row with its
// weights read again: 88 us for 16384 rows of 2048, so 74 when both were tried).
template <int XT, int YT, int VEC, int LPR, int NV>
__global__ void __launch_bounds__(LPR <= 64 ? kBlock : LPR) resnorm_fwd(ResNormArgs a) {
  constexpr int ROWS = LPR <= 64 ? kBlock / LPR : 1;
  __shared__ float lds[LPR <= 64 ? 1 : LPR / 64];
  const int lane = threadIdx.x % LPR, sub = threadIdx.x / LPR;
  float yn[NV][VEC], xn[NV][VEC], gn[NV][VEC], scale[NV][VEC], post[NV][VEC], pre[NV][VEC];
  const auto fetch = [&](int64_t row) {
    const bool live = row < a.rows;
    load_row<YT, VEC, LPR, NV>(a.y, row, a.y_stride, live, a.c, lane, 0.f, yn);
    load_row<XT, VEC, LPR, NV>(a.x, row, a.x_stride, live, a.c, lane, 0.f, xn);
    load_row<YT, VEC, LPR, NV>(a.gate, row, a.gate_stride, live, a.c, lane, 1.f, gn);
  };
  const int64_t step = (int64_t)a.groups * ROWS, first = (int64_t)blockIdx.x * ROWS;
  fetch(first + sub);
  weights<VEC, LPR, NV>(a, lane, scale, post, pre);
  const float c = (float)a.c;
  const int act = a.gate ? a.act : A_NONE;
  for (int64_t row0 = first; row0 < a.rows; row0 += step) {  // (the same in all waves)
    const int64_t row = row0 + sub;
    const bool live = row < a.rows;
    float y[NV][VEC], x[NV][VEC], g[NV][VEC];
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        y[i][j] = yn[i][j];
        x[i][j] = xn[i][j];
        g[i][j] = gn[i][j];
      }
    if (row0 + step < a.rows) fetch(row + step);
    float q1 = 1.f;
    if (a.post) {
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < VEC; ++j) s = fmaf(y[i][j], y[i][j], s);
      q1 = 1.f / sqrtf(row_sum<LPR>(s, lds) / c + a.eps);
    }
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int64_t col = (int64_t)(i * LPR + lane) * VEC;
      const bool in = col < a.c;
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        const float p = y[i][j] * q1 * post[i][j];
        x[i][j] = fmaf(scale[i][j] * act_of(act, g[i][j])[0], p, x[i][j]);
        if (in) s = fmaf(x[i][j], x[i][j], s);
      }
      if (live && in) store_vec<XT, VEC>(a.r, row * a.c + col, x[i]);
    }
    float q2 = 1.f;
    if (a.pre) {
      q2 = 1.f / sqrtf(row_sum<LPR>(s, lds) / c + a.eps);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int64_t col = (int64_t)(i * LPR + lane) * VEC;
        if (!live || col >= a.c) continue;
#pragma unroll
        for (int j = 0; j < VEC; ++j) x[i][j] *= q2 * pre[i][j];
        store_vec<YT, VEC>(a.h, row * a.c + col, x[i]);
      }
    }
    if (live && lane == 0) {
      if (a.post_rstd) a.post_rstd[row] = q1;
      if (a.pre_rstd) a.pre_rstd[row] = q2;
    }
  }
}

// Each group of LPR lanes walks rows and keeps its columns' sums in registers;
// they are joined as layer norm's are, in a fixed order.
template <int XT, int YT, int VEC, int LPR, int NV>
__global__ void __launch_bounds__(LPR <= 64 ? kBlock : LPR) resnorm_bwd(ResNormArgs a) {
  constexpr int BLOCK = LPR <= 64 ? kBlock : LPR;
  constexpr int ROWS = BLOCK / LPR;
  __shared__ float lds[ROWS == 1 ? LPR / 64 : BLOCK * VEC];
  const int lane = threadIdx.x % LPR, sub = threadIdx.x / LPR;
  float scale[NV][VEC], post[NV][VEC], pre[NV][VEC];
  float ds[NV][VEC], dpost[NV][VEC], dpre[NV][VEC];
  weights<VEC, LPR, NV>(a, lane, scale, post, pre);
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < VEC; ++j) ds[i][j] = dpost[i][j] = dpre[i][j] = 0.f;
  const float inv_c = 1.f / (float)a.c;
  const int act = a.gate ? a.act : A_NONE;
  const int64_t steps = (a.rows + (int64_t)a.groups * ROWS - 1) / ((int64_t)a.groups * ROWS);
  for (int64_t it = 0; it < steps; ++it) {
    const int64_t row = (it * a.groups + blockIdx.x) * ROWS + sub;
    const bool live = row < a.rows;
    float y[NV][VEC], r[NV][VEC], g[NV][VEC], t[NV][VEC], e[NV][VEC];
    load_row<YT, VEC, LPR, NV>(a.y, row, a.y_stride, live, a.c, lane, 0.f, y);
    load_row<XT, VEC, LPR, NV>(a.x, row, a.x_stride, live, a.c, lane, 0.f, r);
    load_row<YT, VEC, LPR, NV>(a.gate, row, a.gate_stride, live, a.c, lane, 1.f, g);
    load_row<YT, VEC, LPR, NV>(a.dh, row, a.dh_stride, live, a.c, lane, 0.f, e);
    load_row<XT, VEC, LPR, NV>(a.dr, row, a.dr_stride, live, a.c, lane, 0.f, t);
    const float q1 = live && a.post ? a.post_rstd[row] : 1.f;
    const float q2 = live && a.pre ? a.pre_rstd[row] : 1.f;
    float s = 0.f;
    if (a.dh) {
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          // r^, the normalised row
          const float p = y[i][j] * q1 * post[i][j];
          r[i][j] = q2 * fmaf(scale[i][j] * act_of(act, g[i][j])[0], p, r[i][j]);
          dpre[i][j] = fmaf(e[i][j], r[i][j], dpre[i][j]);
          e[i][j] *= pre[i][j];
          s = fmaf(e[i][j], r[i][j], s);
        }
      s = row_sum<LPR>(s, lds) * inv_c;
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < VEC; ++j) t[i][j] = fmaf(q2, fmaf(-r[i][j], s, e[i][j]), t[i][j]);
    }
    s = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int64_t col = (int64_t)(i * LPR + lane) * VEC;
      const bool in = live && col < a.c;
      if (in && a.dx) store_vec<XT, VEC>(a.dx, row * a.c + col, t[i]);
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        const f32x2 k = act_of(act, g[i][j]);
        y[i][j] *= q1;  // y^
        const float p = y[i][j] * post[i][j], ts = t[i][j] * scale[i][j];
        ds[i][j] = fmaf(t[i][j], k[0] * p, ds[i][j]);
        g[i][j] = ts * p * k[1];
        t[i][j] = ts * k[0];  // dp
        dpost[i][j] = fmaf(t[i][j], y[i][j], dpost[i][j]);
        t[i][j] *= post[i][j];
        s = fmaf(t[i][j], y[i][j], s);
      }
      if (in && a.dgate) store_vec<YT, VEC>(a.dgate, row * a.c + col, g[i]);
    }
    s = a.post ? row_sum<LPR>(s, lds) * inv_c : 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int64_t col = (int64_t)(i * LPR + lane) * VEC;
      if (!live || col >= a.c) continue;
#pragma unroll
      for (int j = 0; j < VEC; ++j) t[i][j] = q1 * fmaf(-y[i][j], s, t[i][j]);
      store_vec<YT, VEC>(a.dy, row * a.c + col, t[i]);
    }
  }
  float* part = a.part + (int64_t)blockIdx.x * 3 * a.c;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      float* v = k == 0 ? ds[i] : (k == 1 ? dpost[i] : dpre[i]);
      if constexpr (ROWS > 1) {
        __syncthreads();
#pragma unroll
        for (int j = 0; j < VEC; ++j) lds[(sub * VEC + j) * LPR + lane] = v[j];
        __syncthreads();
        if (sub == 0) {
          for (int q = 1; q < ROWS; ++q) {
#pragma unroll
            for (int j = 0; j < VEC; ++j) v[j] += lds[(q * VEC + j) * LPR + lane];
          }
        }
      }
      const int64_t col = (int64_t)(i * LPR + lane) * VEC;
      if (sub == 0 && col < a.c) {
#pragma unroll
        for (int j = 0; j < VEC; ++j) part[k * a.c + col + j] = v[j];
      }
    }
  }
}

// One element of a row longer than the register forms.
struct One {
  float y, x, g, scale, post, pre;
};
template <int XT, int YT>
__device__ __forceinline__ One one(const ResNormArgs& a, int64_t row, int64_t c) {
  One v = {load1<YT>(a.y, row * a.y_stride + c), 0.f, 1.f, 1.f, 1.f, 1.f};
  if (a.x) v.x = load1<XT>(a.x, row * a.x_stride + c);
  if (a.gate) v.g = load1<YT>(a.gate, row * a.gate_stride + c);
  if (a.scale) load_any<1>(a.w_type, a.scale, c, &v.scale);
  if (a.w_post) load_any<1>(a.w_type, a.w_post, c, &v.post);
  if (a.w_pre) load_any<1>(a.w_type, a.w_pre, c, &v.pre);
  return v;
}
__device__ __forceinline__ float sum_of(const One& v, int act, float q1) {
  return fmaf(v.scale * act_of(act, v.g)[0], v.y * q1 * v.post, v.x);
}

// Such a row is read again for each sum.
template <int XT, int YT>
__global__ void __launch_bounds__(1024) resnorm_fwd_long(ResNormArgs a) {
  __shared__ float lds[16];
  const int64_t row = blockIdx.x;
  const float n = (float)a.c;
  const int act = a.gate ? a.act : A_NONE;
  float s = 0.f, q1 = 1.f, q2 = 1.f;
  if (a.post) {
    for (int64_t c = threadIdx.x; c < a.c; c += 1024) {
      const float y = load1<YT>(a.y, row * a.y_stride + c);
      s = fmaf(y, y, s);
    }
    q1 = 1.f / sqrtf(row_sum<1024>(s, lds) / n + a.eps);
  }
  s = 0.f;
  for (int64_t c = threadIdx.x; c < a.c; c += 1024) {
    const float r = sum_of(one<XT, YT>(a, row, c), act, q1);
    s = fmaf(r, r, s);
    store1<XT>(a.r, row * a.c + c, r);
  }
  if (a.pre) {
    q2 = 1.f / sqrtf(row_sum<1024>(s, lds) / n + a.eps);
    for (int64_t c = threadIdx.x; c < a.c; c += 1024) {
      const One v = one<XT, YT>(a, row, c);
      store1<YT>(a.h, row * a.c + c, sum_of(v, act, q1) * (q2 * v.pre));
    }
  }
  if (threadIdx.x == 0) {
    if (a.post_rstd) a.post_rstd[row] = q1;
    if (a.pre_rstd) a.pre_rstd[row] = q2;
  }
}

// The gradient that reaches r, from mean(e r^).
template <int XT, int YT>
__device__ __forceinline__ float reach(const ResNormArgs& a, int64_t row, int64_t c, const One& v,
                                       int act, float q1, float q2, float mean) {
  float t = a.dr ? load1<XT>(a.dr, row * a.dr_stride + c) : 0.f;
  if (a.dh) {
    const float e = load1<YT>(a.dh, row * a.dh_stride + c) * v.pre;
    t = fmaf(q2, fmaf(-q2 * sum_of(v, act, q1), mean, e), t);
  }
  return t;
}

// mean(e r^) of each row goes to a.part, behind the columns' partials, for
// resnorm_cols_long.
template <int XT, int YT>
__global__ void __launch_bounds__(1024) resnorm_bwd_long(ResNormArgs a) {
  __shared__ float lds[16];
  const int64_t row = blockIdx.x;
  const float inv_c = 1.f / (float)a.c;
  const int act = a.gate ? a.act : A_NONE;
  const float q1 = a.post ? a.post_rstd[row] : 1.f, q2 = a.pre ? a.pre_rstd[row] : 1.f;
  float s = 0.f, mean = 0.f;
  if (a.dh) {
    for (int64_t c = threadIdx.x; c < a.c; c += 1024) {
      const One v = one<XT, YT>(a, row, c);
      s = fmaf(load1<YT>(a.dh, row * a.dh_stride + c) * v.pre, q2 * sum_of(v, act, q1), s);
    }
    mean = row_sum<1024>(s, lds) * inv_c;
  }
  if (threadIdx.x == 0) a.part[(int64_t)a.groups * 3 * a.c + row] = mean;
  s = 0.f;
  for (int64_t c = threadIdx.x; c < a.c; c += 1024) {
    const One v = one<XT, YT>(a, row, c);
    const float t = reach<XT, YT>(a, row, c, v, act, q1, q2, mean);
    const f32x2 k = act_of(act, v.g);
    if (a.dx) store1<XT>(a.dx, row * a.c + c, t);
    const float p = v.y * q1 * v.post, ts = t * v.scale;
    if (a.dgate) store1<YT>(a.dgate, row * a.c + c, ts * p * k[1]);
    s = fmaf(ts * k[0] * v.post, v.y * q1, s);
  }
  s = a.post ? row_sum<1024>(s, lds) * inv_c : 0.f;
  for (int64_t c = threadIdx.x; c < a.c; c += 1024) {
    const One v = one<XT, YT>(a, row, c);
    const float t = reach<XT, YT>(a, row, c, v, act, q1, q2, mean);
    const float e = t * v.scale * act_of(act, v.g)[0] * v.post;
    store1<YT>(a.dy, row * a.c + c, q1 * fmaf(-v.y * q1, s, e));
  }
}

// Column partials of resnorm_bwd_long: one thread a column, rows by group.
template <int XT, int YT>
__global__ void __launch_bounds__(kBlock) resnorm_cols_long(ResNormArgs a) {
  const int64_t c = (int64_t)blockIdx.x * kBlock + threadIdx.x;
  if (c >= a.c) return;
  const int act = a.gate ? a.act : A_NONE;
  float ds = 0.f, dpost = 0.f, dpre = 0.f;
  for (int64_t row = blockIdx.y; row < a.rows; row += a.groups) {
    const float q1 = a.post ? a.post_rstd[row] : 1.f, q2 = a.pre ? a.pre_rstd[row] : 1.f;
    const One v = one<XT, YT>(a, row, c);
    const float t = reach<XT, YT>(a, row, c, v, act, q1, q2, a.part[(int64_t)a.groups * 3 * a.c + row]);
    const float k = act_of(act, v.g)[0];
    if (a.dh) dpre = fmaf(load1<YT>(a.dh, row * a.dh_stride + c), q2 * sum_of(v, act, q1), dpre);
    ds = fmaf(t, k * (v.y * q1 * v.post), ds);
    dpost = fmaf(t * v.scale * k, v.y * q1, dpost);
  }
  float* part = a.part + (int64_t)blockIdx.y * 3 * a.c;
  part[c] = ds;
  part[a.c + c] = dpost;
  part[2 * a.c + c] = dpre;
}

static bool aligned(const void* p) { return ((uintptr_t)p % 16) == 0; }

// Values of a row that a lane holds: nine registers a value forward, eleven
// backward, of 512 and of 128 in the 1024-lane form.
constexpr int most(int lpr) { return lpr == 1024 ? 8 : 16; }

}  // namespace resnorm

using namespace resnorm;

ResNormShape resnorm_shape(const ResNormArgs& a, bool bwd) {
  int vec = a.y_type == T_F32 ? 4 : 8;
  if (a.c % vec || a.x_stride % vec || a.y_stride % vec || (a.gate && a.gate_stride % vec) ||
      !aligned(a.x) || !aligned(a.y) || !aligned(a.gate) || !aligned(a.scale) ||
      !aligned(a.w_post) || !aligned(a.w_pre))
    vec = 1;
  if (!bwd && (!aligned(a.r) || !aligned(a.h))) vec = 1;
  if (bwd && ((a.dr && a.dr_stride % vec) || (a.dh && a.dh_stride % vec) || !aligned(a.dr) ||
              !aligned(a.dh) || !aligned(a.dx) || !aligned(a.dy) || !aligned(a.dgate)))
    vec = 1;
  const int64_t n = (a.c + vec - 1) / vec;
  for (int lpr : {8, 16, 32})
    if (n <= lpr) return {vec, lpr, 1};
  for (int lpr : {64, 256, 1024}) {
    const int64_t nv = (n + lpr - 1) / lpr;
    for (int v : {1, 2, 4, 8})
      if (nv <= v && v * vec <= most(lpr)) return {vec, lpr, v};
  }
  return {1, 0, 0};
}

int resnorm_groups(const ResNormArgs& a, const ResNormShape& s, bool bwd) {
  if (s.lpr == 0) return (int)(a.rows < 64 ? (a.rows > 0 ? a.rows : 1) : 64);
  const int64_t per = s.lpr <= 64 ? kBlock / s.lpr : 1;
  // (the backward pass leaves a row of partial sums each)
  int64_t most = (s.lpr <= 256 ? 1024 : 256) * (bwd ? 1 : 2);
  const int64_t need = (a.rows + per - 1) / per;
  if (s.vec == 1 && s.lpr == 256 && need > 0) {
    // as many as are resident, with the same number of rows each: seven waves a
    // SIMD forward and five back up to 1024 columns, four and three past them.
    // fp16, gated, us forward and back, by the rule above and so: 3333 rows of
    // 771: 17 and 39, 17 and 33; 16384 of 771: 78 and 123, 54 and 101; 3333 of
    // 1500: 33 and 86, 34 and 67; 16384 of 1500: 120 and 488, 118 and 358 (with
    // 1792 and 1280 there 142 and 419).  A wave a row does not gain.
    most = s.nv <= 4 ? (bwd ? 1280 : 1792) : (bwd ? 768 : 1024);
    const int64_t rounds = (need + most - 1) / most;
    most = (need + rounds - 1) / rounds;
  }
  return (int)(need < 1 ? 1 : (need < most ? need : most));
}

namespace resnorm {

template <int XT, int YT, int VEC, int LPR, int NV>
void go(bool bwd, const ResNormArgs& a, hipStream_t st) {
  constexpr int block = LPR <= 64 ? kBlock : LPR;
  if constexpr (NV * VEC <= most(LPR)) {
    auto* f = bwd ? &resnorm_bwd<XT, YT, VEC, LPR, NV> : &resnorm_fwd<XT, YT, VEC, LPR, NV>;
    hipLaunchKernelGGL(f, dim3(a.groups), dim3(block), 0, st, a);
  }
}

template <int XT, int YT, int VEC, int LPR>
void go_nv(int nv, bool bwd, const ResNormArgs& a, hipStream_t st) {
  switch (nv) {
    case 1: return go<XT, YT, VEC, LPR, 1>(bwd, a, st);
    case 2: return go<XT, YT, VEC, LPR, 2>(bwd, a, st);
    case 4: return go<XT, YT, VEC, LPR, 4>(bwd, a, st);
    case 8: return go<XT, YT, VEC, LPR, 8>(bwd, a, st);
  }
}

template <int XT, int YT, int VEC>
void go_lpr(const ResNormShape& s, bool bwd, const ResNormArgs& a, hipStream_t st) {
  switch (s.lpr) {
    case 8: return go<XT, YT, VEC, 8, 1>(bwd, a, st);
    case 16: return go<XT, YT, VEC, 16, 1>(bwd, a, st);
    case 32: return go<XT, YT, VEC, 32, 1>(bwd, a, st);
    case 64: return go_nv<XT, YT, VEC, 64>(s.nv, bwd, a, st);
    case 256: return go_nv<XT, YT, VEC, 256>(s.nv, bwd, a, st);
    case 1024: return go_nv<XT, YT, VEC, 1024>(s.nv, bwd, a, st);
  }
}

template <int XT, int YT>
void go_types(bool bwd, const ResNormArgs& a, hipStream_t st) {
  const ResNormShape s = resnorm_shape(a, bwd);
  if (s.lpr == 0) {
    if (bwd) {
      hipLaunchKernelGGL((resnorm_bwd_long<XT, YT>), dim3((uint32_t)a.rows), dim3(1024), 0, st, a);
      hipLaunchKernelGGL((resnorm_cols_long<XT, YT>),
                         dim3((uint32_t)((a.c + kBlock - 1) / kBlock), a.groups), dim3(kBlock), 0,
                         st, a);
    } else {
      hipLaunchKernelGGL((resnorm_fwd_long<XT, YT>), dim3((uint32_t)a.rows), dim3(1024), 0, st, a);
    }
    return;
  }
  if (s.vec == 1) go_lpr<XT, YT, 1>(s, bwd, a, st);
  else go_lpr<XT, YT, YT == T_F32 ? 4 : 8>(s, bwd, a, st);
}

static hipError_t launch(bool bwd, const ResNormArgs& a, hipStream_t st) {
  // the residual stream is fp32 or of the block's type
  if (a.x_type == T_F32) {
    if (a.y_type == T_F32) go_types<T_F32, T_F32>(bwd, a, st);
    else if (a.y_type == T_BF16) go_types<T_F32, T_BF16>(bwd, a, st);
    else go_types<T_F32, T_F16>(bwd, a, st);
  } else if (a.x_type == T_BF16) {
    go_types<T_BF16, T_BF16>(bwd, a, st);
  } else {
    go_types<T_F16, T_F16>(bwd, a, st);
  }
  return hipGetLastError();
}

}  // namespace resnorm

hipError_t launch_resnorm_fwd(ResNormArgs a, hipStream_t st) {
  a.groups = resnorm_groups(a, resnorm_shape(a, false), false);
  return launch(false, a, st);
}

hipError_t launch_resnorm_bwd(const ResNormArgs& a, float* dscale, float* dw_post, float* dw_pre,
                              hipStream_t st) {
  if (a.rows > 0) {
    const hipError_t e = launch(true, a, st);
    if (e != hipSuccess) return e;
  }
  const int64_t rows = a.rows > 0 ? a.groups : 0, stride = 3 * a.c;
  const ColumnSum jobs[kColumnJobs] = {{a.part, dscale, rows, stride, a.c, 0},
                                       {a.part + a.c, dw_post, rows, stride, a.c, 0},
                                       {a.part + 2 * a.c, dw_pre, rows, stride, a.c, 0}};
  return launch_column_sums(jobs, st);
}

}  // namespace seq
}  // namespace dwc
