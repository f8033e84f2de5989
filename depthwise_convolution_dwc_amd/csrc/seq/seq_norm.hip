// seq_norm.hip -- layer norm over the last axis, forward and backward.
//
//   m = mean(x), r = 1 / sqrt(mean((x - m)^2) + eps), h = (x - m) r
//   y = h w + b
//   e = dy w:  dx = r (e - mean(e) - h mean(e h)),
//   dw = sum over rows of dy h,  db = sum over rows of dy
//
// Bound: memory (8 to 14 operations an element).  So a row is read once into
// registers, in 16-byte loads where its length and address allow, and every
// sum runs over those registers: the mean first, then the squares of the
// differences from it, which loses nothing to cancellation the way
// mean(x^2) - m^2 does.  LPR lanes share a row; 8 to 64 of them lie inside a
// wave, so short rows leave no lane idle, and rows past 64 * VEC * NV
// elements take a whole workgroup.  MI355X: 200704 rows of 128, fp32 to bf16,
// in 27 us (5.7 TB/s); 100352 rows of 512, bf16, there in 35 us (5.9 TB/s) and
// back in 56 us (5.5 TB/s) and 5 us for the partials.
#include "seq_device.h"
#include "seq_launch.h"

namespace dwc {
namespace seq {
namespace norm {

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

template <int LPR>
__device__ __forceinline__ f32x2 row_sum2(float u, float v, float* lds) {
  if constexpr (LPR <= 64) {
    return f32x2{lane_sum<LPR>(u), lane_sum<LPR>(v)};
  } else {
    u = lane_sum<64>(u);
    v = lane_sum<64>(v);
    constexpr int W = LPR / 64;
    __syncthreads();
    if ((threadIdx.x & 63) == 0) {
      lds[threadIdx.x >> 6] = u;
      lds[W + (threadIdx.x >> 6)] = v;
    }
    __syncthreads();
    float s = 0.f, t = 0.f;
#pragma unroll
    for (int i = 0; i < W; ++i) {
      s += lds[i];
      t += lds[W + i];
    }
    return f32x2{s, t};
  }
}

// A row of x, zeros past its end and past the last row.
template <int XT, int VEC, int LPR, int NV>
__device__ __forceinline__ void load_row(const NormArgs& a, int64_t row, int lane,
                                         float (&x)[NV][VEC]) {
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int64_t col = (int64_t)(i * LPR + lane) * VEC;
    if (row < a.rows && col < a.c) {  // lanes of one row agree on the first
      load_vec<XT, VEC>(a.x, row * a.x_stride + col, x[i]);
    } else {
#pragma unroll
      for (int j = 0; j < VEC; ++j) x[i][j] = 0.f;
    }
  }
}

template <int VEC, int LPR, int NV>
__device__ __forceinline__ void norm_row(const NormArgs& a, int64_t row, int lane,
                                         float (&x)[NV][VEC], float* lds) {
  const bool live = row < a.rows;
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < VEC; ++j) s += x[i][j];
  const float c = (float)a.c;
  // divided, not multiplied by 1 / c: a constant row gives its own value back
  const float mean = row_sum<LPR>(s, lds) / c;
  s = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const bool in = (int64_t)(i * LPR + lane) * VEC < a.c;
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      x[i][j] = in ? x[i][j] - mean : 0.f;
      s = fmaf(x[i][j], x[i][j], s);
    }
  }
  const float rstd = 1.0f / sqrtf(row_sum<LPR>(s, lds) / c + a.eps);
  if (!live) return;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int64_t col = (int64_t)(i * LPR + lane) * VEC;
    if (col >= a.c) continue;
    float w[VEC], b[VEC];
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      w[j] = 1.f;
      b[j] = 0.f;
    }
    if (a.w) load_any<VEC>(a.w_type, a.w, col, w);
    if (a.b) load_any<VEC>(a.w_type, a.b, col, b);
#pragma unroll
    for (int j = 0; j < VEC; ++j) x[i][j] = fmaf(x[i][j] * rstd, w[j], b[j]);
    store_any<VEC>(a.y_type, a.y, row * a.c + col, x[i]);
  }
  if (lane == 0 && a.mean) {
    a.mean[row] = mean;
    a.rstd[row] = rstd;
  }
}

// Rows a lane group takes: two where a row is one load a lane, so that twice
// the bytes are under way (200704 rows of 128, fp32 to bf16: 27 us, 29 us
// one at a time).
template <int NV>
constexpr int kRows = NV == 1 ? 2 : 1;

template <int XT, int VEC, int LPR, int NV>
__global__ void __launch_bounds__(LPR <= 64 ? kBlock : LPR) norm_fwd(NormArgs a) {
  constexpr int ROWS = LPR <= 64 ? kBlock / LPR : 1, U = kRows<NV>;
  __shared__ float lds[2 * (LPR <= 64 ? 1 : LPR / 64)];
  const int lane = threadIdx.x % LPR;
  const int64_t row = (int64_t)blockIdx.x * ROWS * U + threadIdx.x / LPR;
  float x[U][NV][VEC];
#pragma unroll
  for (int u = 0; u < U; ++u) load_row<XT, VEC, LPR, NV>(a, row + u * ROWS, lane, x[u]);
#pragma unroll
  for (int u = 0; u < U; ++u) norm_row<VEC, LPR, NV>(a, row + u * ROWS, lane, x[u], lds);
}

// Each group of LPR lanes walks rows group, group + groups * ROWS, ... and
// keeps its columns' sums of dy h and dy in registers; a workgroup's row
// groups are joined in LDS in a fixed order and the workgroups' partials by
// norm_reduce, so the weight's gradient has the same bits every time.
template <int XT, int VEC, int LPR, int NV>
__global__ void __launch_bounds__(LPR <= 64 ? kBlock : LPR) norm_bwd(NormArgs a) {
  constexpr int BLOCK = LPR <= 64 ? kBlock : LPR;
  constexpr int ROWS = BLOCK / LPR;
  __shared__ float lds[ROWS == 1 ? 2 * (LPR / 64) : BLOCK * VEC];
  const int lane = threadIdx.x % LPR, sub = threadIdx.x / LPR;
  float w[NV][VEC], dw[NV][VEC], db[NV][VEC];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int64_t col = (int64_t)(i * LPR + lane) * VEC;
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      w[i][j] = 1.f;
      dw[i][j] = db[i][j] = 0.f;
    }
    if (a.w && col < a.c) load_any<VEC>(a.w_type, a.w, col, w[i]);
  }
  const float inv_c = 1.0f / (float)a.c;
  const int64_t steps = (a.rows + (int64_t)a.groups * ROWS - 1) / ((int64_t)a.groups * ROWS);
  // the next row is read before this one's sums are made
  float xn[NV][VEC], en[NV][VEC], mean_n, rstd_n;
  const auto fetch = [&](int64_t row) {
    const bool live = row < a.rows;
    mean_n = live ? a.mean[row] : 0.f;
    rstd_n = live ? a.rstd[row] : 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int64_t col = (int64_t)(i * LPR + lane) * VEC;
      if (live && col < a.c) {
        load_vec<XT, VEC>(a.x, row * a.x_stride + col, xn[i]);
        load_any<VEC>(a.y_type, a.dy, row * a.dy_stride + col, en[i]);
      } else {
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          xn[i][j] = mean_n;
          en[i][j] = 0.f;
        }
      }
    }
  };
  fetch((int64_t)blockIdx.x * ROWS + sub);
  for (int64_t it = 0; it < steps; ++it) {
    const int64_t row = (it * a.groups + blockIdx.x) * ROWS + sub;
    const bool live = row < a.rows;
    const float mean = mean_n, rstd = rstd_n;
    float h[NV][VEC], e[NV][VEC];
    float se = 0.f, sh = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        h[i][j] = xn[i][j];
        e[i][j] = en[i][j];
      }
    // (a wide row's registers are taken)
    if constexpr (NV * VEC <= 8) fetch(row + (int64_t)a.groups * ROWS);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        h[i][j] = (h[i][j] - mean) * rstd;
        dw[i][j] = fmaf(e[i][j], h[i][j], dw[i][j]);
        db[i][j] += e[i][j];
        e[i][j] *= w[i][j];
        se += e[i][j];
        sh = fmaf(e[i][j], h[i][j], sh);
      }
    }
    const f32x2 t = row_sum2<LPR>(se, sh, lds);
    const float me = t[0] * inv_c, mh = t[1] * inv_c;
    if (live) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int64_t col = (int64_t)(i * LPR + lane) * VEC;
        if (col >= a.c) continue;
#pragma unroll
        for (int j = 0; j < VEC; ++j) e[i][j] = rstd * (e[i][j] - me - h[i][j] * mh);
        store_vec<XT, VEC>(a.y, row * a.c + col, e[i]);
      }
    }
    if constexpr (NV * VEC > 8) fetch(row + (int64_t)a.groups * ROWS);
  }
  float* part = a.part + (int64_t)blockIdx.x * 2 * a.c;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      float* v = k == 0 ? dw[i] : db[i];
      if constexpr (ROWS > 1) {
        __syncthreads();
#pragma unroll
        for (int j = 0; j < VEC; ++j) lds[(sub * VEC + j) * LPR + lane] = v[j];
        __syncthreads();
        if (sub == 0) {
          for (int r = 1; r < ROWS; ++r) {
#pragma unroll
            for (int j = 0; j < VEC; ++j) v[j] += lds[(r * VEC + j) * LPR + lane];
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

// Rows longer than the register forms: the row is read again for each sum
// (from the caches while it fits them).
template <int XT>
__global__ void __launch_bounds__(1024) norm_fwd_long(NormArgs a) {
  __shared__ float lds[32];
  const int64_t row = blockIdx.x, base = row * a.x_stride;
  const float n = (float)a.c;
  float s = 0.f;
  for (int64_t c = threadIdx.x; c < a.c; c += 1024) s += load1<XT>(a.x, base + c);
  const float mean = row_sum<1024>(s, lds) / n;
  s = 0.f;
  for (int64_t c = threadIdx.x; c < a.c; c += 1024) {
    const float d = load1<XT>(a.x, base + c) - mean;
    s = fmaf(d, d, s);
  }
  const float rstd = 1.0f / sqrtf(row_sum<1024>(s, lds) / n + a.eps);
  for (int64_t c = threadIdx.x; c < a.c; c += 1024) {
    float w = 1.f, b = 0.f;
    if (a.w) load_any<1>(a.w_type, a.w, c, &w);
    if (a.b) load_any<1>(a.w_type, a.b, c, &b);
    const float y = fmaf((load1<XT>(a.x, base + c) - mean) * rstd, w, b);
    store_any<1>(a.y_type, a.y, row * a.c + c, &y);
  }
  if (threadIdx.x == 0 && a.mean) {
    a.mean[row] = mean;
    a.rstd[row] = rstd;
  }
}

template <int XT>
__global__ void __launch_bounds__(1024) norm_bwd_long(NormArgs a) {
  __shared__ float lds[32];
  const int64_t row = blockIdx.x;
  const float inv_c = 1.0f / (float)a.c, mean = a.mean[row], rstd = a.rstd[row];
  float se = 0.f, sh = 0.f;
  for (int pass = 0; pass < 2; ++pass) {
    float me = 0.f, mh = 0.f;
    if (pass) {
      const f32x2 t = row_sum2<1024>(se, sh, lds);
      me = t[0] * inv_c;
      mh = t[1] * inv_c;
    }
    for (int64_t c = threadIdx.x; c < a.c; c += 1024) {
      float w = 1.f, e;
      if (a.w) load_any<1>(a.w_type, a.w, c, &w);
      load_any<1>(a.y_type, a.dy, row * a.dy_stride + c, &e);
      e *= w;
      const float h = (load1<XT>(a.x, row * a.x_stride + c) - mean) * rstd;
      if (pass) {
        store1<XT>(a.y, row * a.c + c, rstd * (e - me - h * mh));
      } else {
        se += e;
        sh = fmaf(e, h, sh);
      }
    }
  }
}

// Column partials of norm_bwd_long: one thread a column, rows by group.
template <int XT>
__global__ void __launch_bounds__(kBlock) norm_cols_long(NormArgs a) {
  const int64_t c = (int64_t)blockIdx.x * kBlock + threadIdx.x;
  if (c >= a.c) return;
  float dw = 0.f, db = 0.f;
  for (int64_t row = blockIdx.y; row < a.rows; row += a.groups) {
    float e;
    load_any<1>(a.y_type, a.dy, row * a.dy_stride + c, &e);
    const float h = (load1<XT>(a.x, row * a.x_stride + c) - a.mean[row]) * a.rstd[row];
    dw = fmaf(e, h, dw);
    db += e;
  }
  float* part = a.part + (int64_t)blockIdx.y * 2 * a.c;
  part[c] = dw;
  part[a.c + c] = db;
}

// dw, db from the partials: 16 columns x 64 slices of the groups a
// workgroup, each slice's sum in order, the slices' sums in order.
__global__ void __launch_bounds__(1024) norm_reduce(const float* part, float* dw, float* db,
                                                    int64_t c, int groups) {
  __shared__ float lds[64][17];
  const int lane = threadIdx.x & 15, slice = threadIdx.x >> 4;
  const int64_t col = (int64_t)blockIdx.x * 16 + lane;
  float s = 0.f;
  if (col < 2 * c) {
#pragma unroll 8
    for (int g = slice; g < groups; g += 64) s += part[(int64_t)g * 2 * c + col];
  }
  lds[slice][lane] = s;
  __syncthreads();
  if (slice == 0 && col < 2 * c) {
    s = 0.f;
#pragma unroll
    for (int i = 0; i < 64; ++i) s += lds[i][lane];
    float* out = col < c ? dw : db;
    if (out) out[col < c ? col : col - c] = s;
  }
}

static bool aligned(const void* p, size_t n) { return ((uintptr_t)p % n) == 0; }

}  // namespace norm

using namespace norm;

NormShape norm_shape(const NormArgs& a, bool bwd) {
  // 16-byte loads of x where the row length, the strides and the addresses
  // of every tensor allow them
  int vec = a.x_type == T_F32 ? 4 : 8;
  if (a.c % vec || a.x_stride % vec || (bwd && a.dy_stride % vec) || !aligned(a.x, 16) ||
      !aligned(a.y, 16) || (a.w && !aligned(a.w, 16)) || (a.b && !aligned(a.b, 16)) ||
      (bwd && !aligned(a.dy, 16)))
    vec = 1;
  const int64_t n = (a.c + vec - 1) / vec;
  for (int lpr : {8, 16, 32}) {
    if (n <= lpr) return {vec, lpr, 1};
  }
  for (int lpr : {64, 256, 1024}) {
    // at most 32 values of a row in a lane, 12 in the 1024-lane form: the
    // backward pass keeps five registers a value, of 512 and of 128
    const int most = (lpr == 1024 ? 12 : 32) / vec;
    const int64_t nv = (n + lpr - 1) / lpr;
    if (nv > (most < 8 ? most : 8)) continue;
    for (int v : {1, 2, 3, 4, 6, 8}) {
      if (nv <= v) return {vec, lpr, v};
    }
  }
  return {1, 0, 0};
}

int norm_groups(const NormArgs& a, const NormShape& s) {
  if (s.lpr == 0) return (int)(a.rows < 64 ? (a.rows > 0 ? a.rows : 1) : 64);
  const int64_t per = s.lpr <= 64 ? kBlock / s.lpr : 1;
  const int64_t most = s.lpr <= 64 ? 1024 : (s.lpr == 256 ? 512 : 256);
  const int64_t need = (a.rows + per - 1) / per;
  return (int)(need < 1 ? 1 : (need < most ? need : most));
}

namespace norm {

template <int XT, int VEC, int LPR, int NV>
void go(bool bwd, const NormArgs& a, hipStream_t st) {
  constexpr int block = LPR <= 64 ? kBlock : LPR;
  constexpr int rows = block / LPR * kRows<NV>;
  if (bwd)
    hipLaunchKernelGGL((norm_bwd<XT, VEC, LPR, NV>), dim3(a.groups), dim3(block), 0, st, a);
  else
    hipLaunchKernelGGL((norm_fwd<XT, VEC, LPR, NV>), dim3((uint32_t)((a.rows + rows - 1) / rows)),
                       dim3(block), 0, st, a);
}

template <int XT, int VEC, int LPR, int NV>
bool go_one(bool bwd, const NormArgs& a, hipStream_t st) {
  // the forms norm_shape can return
  constexpr int most = (LPR == 1024 ? 12 : 32) / VEC;
  constexpr bool reached = NV <= most && (LPR == 64 || NV >= 2) &&
                           (LPR != 256 || NV * 4 > (most < 8 ? most : 8)) &&
                           (LPR != 1024 || NV * 4 > (32 / VEC < 8 ? 32 / VEC : 8));
  if constexpr (reached) go<XT, VEC, LPR, NV>(bwd, a, st);
  return reached;
}

template <int XT, int VEC, int LPR>
bool go_nv(int nv, bool bwd, const NormArgs& a, hipStream_t st) {
  switch (nv) {
    case 1: return go_one<XT, VEC, LPR, 1>(bwd, a, st);
    case 2: return go_one<XT, VEC, LPR, 2>(bwd, a, st);
    case 3: return go_one<XT, VEC, LPR, 3>(bwd, a, st);
    case 4: return go_one<XT, VEC, LPR, 4>(bwd, a, st);
    case 6: return go_one<XT, VEC, LPR, 6>(bwd, a, st);
    case 8: return go_one<XT, VEC, LPR, 8>(bwd, a, st);
  }
  return false;
}

template <int XT, int VEC>
bool go_lpr(const NormShape& s, bool bwd, const NormArgs& a, hipStream_t st) {
  switch (s.lpr) {
    case 8: go<XT, VEC, 8, 1>(bwd, a, st); return true;
    case 16: go<XT, VEC, 16, 1>(bwd, a, st); return true;
    case 32: go<XT, VEC, 32, 1>(bwd, a, st); return true;
    case 64: return go_nv<XT, VEC, 64>(s.nv, bwd, a, st);
    case 256: return go_nv<XT, VEC, 256>(s.nv, bwd, a, st);
    case 1024: return go_nv<XT, VEC, 1024>(s.nv, bwd, a, st);
  }
  return false;
}

template <int XT>
bool go_type(const NormShape& s, bool bwd, const NormArgs& a, hipStream_t st) {
  if (s.lpr == 0) {
    if (bwd) {
      hipLaunchKernelGGL((norm_bwd_long<XT>), dim3((uint32_t)a.rows), dim3(1024), 0, st, a);
      hipLaunchKernelGGL((norm_cols_long<XT>),
                         dim3((uint32_t)((a.c + kBlock - 1) / kBlock), a.groups), dim3(kBlock), 0,
                         st, a);
    } else {
      hipLaunchKernelGGL((norm_fwd_long<XT>), dim3((uint32_t)a.rows), dim3(1024), 0, st, a);
    }
    return true;
  }
  return s.vec == 1 ? go_lpr<XT, 1>(s, bwd, a, st)
                    : go_lpr<XT, XT == T_F32 ? 4 : 8>(s, bwd, a, st);
}

static hipError_t launch(bool bwd, const NormArgs& a, hipStream_t st) {
  const NormShape s = norm_shape(a, bwd);
  const bool ok = a.x_type == T_F32    ? go_type<T_F32>(s, bwd, a, st)
                  : a.x_type == T_BF16 ? go_type<T_BF16>(s, bwd, a, st)
                                       : go_type<T_F16>(s, bwd, a, st);
  return ok ? hipGetLastError() : hipErrorInvalidValue;
}

}  // namespace norm

hipError_t launch_norm_fwd(const NormArgs& a, hipStream_t st) { return launch(false, a, st); }

hipError_t launch_norm_bwd(const NormArgs& a, float* dw, float* db, hipStream_t st) {
  // no rows: norm_reduce over zero groups writes zeros
  if (a.rows > 0) {
    const hipError_t e = launch(true, a, st);
    if (e != hipSuccess) return e;
  }
  if (dw || db)
    hipLaunchKernelGGL(norm_reduce, dim3((uint32_t)((2 * a.c + 15) / 16)), dim3(1024), 0, st,
                       a.part, dw, db, a.c, a.rows > 0 ? a.groups : 0);
  return hipGetLastError();
}

}  // namespace seq
}  // namespace dwc
