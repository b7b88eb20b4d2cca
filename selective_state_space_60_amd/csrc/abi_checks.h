// Host-side checks shared by the C entry points (ssm_abi.cpp, layer_abi.cpp).
#pragma once

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>

#include "../../include/ssm.h"

namespace ssm {
namespace abi {

// hipError_t of the last SSM_ERR_HIP on this thread.
inline int& last_hip_error() {
  thread_local int e = 0;
  return e;
}

inline int64_t esize(int32_t dt) {
  return dt == SSM_BF16 || dt == SSM_F16 ? 2 : dt == SSM_E4M3 || dt == SSM_U8 ? 1 : 4;
}

struct Span {
  uintptr_t lo = 0, hi = 0;  // [lo, hi)
  bool valid = false;
};

inline Span span_of(const ssm_tensor_desc& t, const void* ptr) {
  Span s;
  if (!ptr) return s;
  int64_t last = 0;
  for (int i = 0; i < t.ndim; ++i) last += (t.shape[i] - 1) * t.stride[i];
  s.lo = (uintptr_t)ptr;
  s.hi = s.lo + (uintptr_t)((last + 1) * esize(t.dtype));
  s.valid = true;
  return s;
}

// The bytes [ptr, ptr + bytes) of a plain contiguous buffer.
inline Span span_bytes(const void* ptr, int64_t bytes) {
  Span s;
  if (!ptr) return s;
  s.lo = (uintptr_t)ptr;
  s.hi = s.lo + (uintptr_t)bytes;
  s.valid = true;
  return s;
}

inline bool overlap(const Span& a, const Span& b) { return a.valid && b.valid && a.lo < b.hi && b.lo < a.hi; }

// Shape, dtype and stride checks of one tensor.
inline ssm_status check_tensor(const ssm_tensor_desc& t, int ndim, const int64_t* shape, bool dtype_ok,
                               bool inner_unit, bool contiguous) {
  if (!dtype_ok) return SSM_ERR_DTYPE;
  if (t.ndim != ndim) return SSM_ERR_SHAPE;
  for (int i = 0; i < ndim; ++i)
    if (t.shape[i] != shape[i]) return SSM_ERR_SHAPE;
  for (int i = 0; i < ndim; ++i)
    if (t.stride[i] < 0) return SSM_ERR_STRIDE;
  if (inner_unit && t.stride[ndim - 1] != 1 && t.shape[ndim - 1] > 1) return SSM_ERR_STRIDE;
  if (contiguous) {
    int64_t expect = 1;
    for (int i = ndim - 1; i >= 0; --i) {
      if (t.shape[i] > 1 && t.stride[i] != expect) return SSM_ERR_STRIDE;
      expect *= t.shape[i];
    }
  }
  return SSM_OK;
}

// An output must not write one element twice: with dimensions sorted by
// stride, each stride must be at least the extent of the smaller ones.
inline bool non_overlapping(const ssm_tensor_desc& t) {
  int idx[SSM_MAX_DIMS];
  int n = 0;
  for (int i = 0; i < t.ndim; ++i)
    if (t.shape[i] > 1) idx[n++] = i;
  std::sort(idx, idx + n, [&](int a, int b) { return t.stride[a] < t.stride[b]; });
  int64_t extent = 1;
  for (int k = 0; k < n; ++k) {
    if (t.stride[idx[k]] < extent) return false;
    extent = t.stride[idx[k]] * (t.shape[idx[k]] - 1) + extent;
  }
  return true;
}

inline bool aligned(const void* p, int64_t bytes) { return ((uintptr_t)p % (uintptr_t)bytes) == 0; }

inline int64_t round256(int64_t n) { return (n + 255) / 256 * 256; }

inline ssm_status hip_status(hipError_t e) {
  if (e == hipSuccess) return SSM_OK;
  last_hip_error() = (int)e;
  return SSM_ERR_HIP;
}

}  // namespace abi
}  // namespace ssm
