// seq_columns.hip -- sums of columns over partial rows, in a fixed order.
#include "seq_space.h"

namespace dwc {
namespace seq {

struct ColumnJobs {
  ColumnSum job[kColumnJobs];
  uint32_t end[kColumnJobs];  // workgroups up to and with this job's
};

// WIDTH columns x 1024 / WIDTH slices of the rows a workgroup: each slice's sum
// in order, then the slices' sums in order, so that the result has the same
// bits every time.
template <int WIDTH>
__global__ void __launch_bounds__(1024) column_sums(ColumnJobs a) {
  constexpr int SLICES = 1024 / WIDTH;
  __shared__ float lds[SLICES][WIDTH + 1];
  int j = 0;
#pragma unroll
  for (int i = 0; i + 1 < kColumnJobs; ++i)
    if (blockIdx.x >= a.end[i]) j = i + 1;
  ColumnSum s = a.job[0];
  uint32_t first = 0;
#pragma unroll
  for (int i = 1; i < kColumnJobs; ++i)
    if (j == i) {
      s = a.job[i];
      first = a.end[i - 1];
    }
  const int lane = threadIdx.x % WIDTH, slice = threadIdx.x / WIDTH;
  const int64_t col = (int64_t)(blockIdx.x - first) * WIDTH + lane;
  float v = 0.f;
  if (col < s.cols) {
#pragma unroll 8
    for (int64_t r = slice; r < s.rows; r += SLICES) v += s.part[r * s.stride + col];
  }
  lds[slice][lane] = v;
  __syncthreads();
  if (slice == 0 && col < s.cols) {
    v = 0.f;
#pragma unroll
    for (int i = 0; i < SLICES; ++i) v += lds[i][lane];
    s.out[s.turn > 0 ? col % s.turn * (s.cols / s.turn) + col / s.turn : col] = v;
  }
}

hipError_t launch_column_sums(const ColumnSum (&jobs)[kColumnJobs], hipStream_t st) {
  int64_t cols = 0;
  for (const ColumnSum& s : jobs)
    if (s.out) cols += s.cols;
  if (cols == 0) return hipSuccess;
  // whole lines of the rows where there are columns for 64 workgroups (6144
  // columns of 1024 rows: 7 us, 11 by 16 columns when both were tried)
  const int width = cols >= 4096 ? 64 : 16;
  ColumnJobs a{};
  uint32_t blocks = 0;
  for (int i = 0; i < kColumnJobs; ++i) {
    a.job[i] = jobs[i];
    if (jobs[i].out) blocks += (uint32_t)((jobs[i].cols + width - 1) / width);
    a.end[i] = blocks;
  }
  if (width == 64) hipLaunchKernelGGL(column_sums<64>, dim3(blocks), dim3(1024), 0, st, a);
  else hipLaunchKernelGGL(column_sums<16>, dim3(blocks), dim3(1024), 0, st, a);
  return hipGetLastError();
}

}  // namespace seq
}  // namespace dwc
