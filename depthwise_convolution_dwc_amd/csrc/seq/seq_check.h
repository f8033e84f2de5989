// seq_check.h -- checks of arguments that the entry points of the
// sequence-layer operators share.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <string>

#include "../dwc_plan.h"

namespace dwc {
namespace seq {

inline int fail(int status, const char* what) {
  set_last_error(what);
  return status;
}

inline int hip_result(hipError_t e, const char* what) {
  if (e == hipSuccess) return DWC_OK;
  set_last_error(std::string(what) + ": " + hipGetErrorString(e));
  return DWC_ERR_HIP;
}

inline bool is_type(int t) { return t == DWC_F32 || t == DWC_BF16 || t == DWC_F16; }
inline int64_t bytes_of(int t) { return t == DWC_F32 ? 4 : 2; }

// A tensor as a range of addresses.
struct Span {
  const void* p;
  int64_t bytes;
  int64_t align;
};

inline bool overlap(const Span& a, const Span& b) {
  if (!a.p || !b.p || a.bytes <= 0 || b.bytes <= 0) return false;
  const uintptr_t x = (uintptr_t)a.p, y = (uintptr_t)b.p;
  return x < y + (uintptr_t)b.bytes && y < x + (uintptr_t)a.bytes;
}

// Alignment of every tensor; no output overlaps an input or another output.
template <int I, int O>
int check_spans(const Span (&in)[I], const Span (&out)[O]) {
  for (const Span& s : in)
    if ((uintptr_t)s.p % s.align)
      return fail(DWC_ERR_MISALIGNED, "input not aligned to its element size");
  for (const Span& s : out)
    if ((uintptr_t)s.p % s.align)
      return fail(DWC_ERR_MISALIGNED, "output not aligned to its element size");
  for (int o = 0; o < O; ++o) {
    for (const Span& s : in)
      if (overlap(out[o], s)) return fail(DWC_ERR_ALIAS, "output overlaps an input");
    for (int k = 0; k < o; ++k)
      if (overlap(out[o], out[k])) return fail(DWC_ERR_ALIAS, "outputs overlap each other");
  }
  return DWC_OK;
}

// Most elements a tensor may have: byte offsets stay far inside 64 bits.
constexpr int64_t kMost = (int64_t)1 << 48;

// Addresses from a strided tensor's first to past its last element; false
// for strides that are negative or past the index range.
inline bool strided_bytes(const int64_t* stride, int64_t b, int64_t l, int64_t h, int64_t d, int64_t e,
                   int64_t* bytes) {
  const int64_t n[3] = {b, l, h};
  int64_t last = d;
  for (int i = 0; i < 3; ++i) {
    if (n[i] <= 0) {
      *bytes = 0;
      return true;
    }
    if (stride[i] < 0 || (n[i] > 1 && stride[i] > kMost / n[i])) return false;
    last += (n[i] - 1) * stride[i];
  }
  *bytes = last * e;
  return last <= kMost;
}

}  // namespace seq
}  // namespace dwc
