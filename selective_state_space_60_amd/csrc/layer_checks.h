// Host-side checks of descriptors and pointers shared by the operators' entry
// points (layer_abi.cpp, serve_abi.cpp).
#pragma once

#include <cstdint>
#include <initializer_list>

#include "../../include/ssm.h"
#include "abi_checks.h"

namespace ssm {
namespace abi {

// a launch holds fewer than 2^32 threads: blocks of 1024, 512, 256
constexpr int64_t kMaxBlocks1024 = (int64_t)1 << 22, kMaxBlocks512 = (int64_t)1 << 23,
                  kMaxBlocks256 = (int64_t)1 << 24;
constexpr int64_t kMaxSpan = (int64_t)1 << 30;       // bytes a kernel addresses from one base

// Sizes whose products stay far from overflowing.
inline bool sizes_ok(std::initializer_list<int64_t> sizes) {
  __int128 n = 1;
  for (int64_t s : sizes) {
    if (s >= ((int64_t)1 << 40)) return false;
    n *= s;
    if (n >= ((__int128)1 << 56)) return false;
  }
  return true;
}

// The last element's offset must not overflow either.
inline bool strides_ok(const ssm_tensor_desc& t) {
  __int128 last = 0;
  for (int i = 0; i < t.ndim; ++i) last += (__int128)(t.shape[i] - 1) * t.stride[i];
  return last < ((__int128)1 << 56);
}

// The descriptor of one input (`on` false: left out), or of one output, which
// must not write an element twice.
inline ssm_status check_in(bool on, const ssm_tensor_desc& t, int ndim, const int64_t* shape, bool dtype_ok,
                    bool inner_unit, bool contiguous) {
  if (!on) return SSM_OK;
  const ssm_status s = check_tensor(t, ndim, shape, dtype_ok, inner_unit, contiguous);
  if (s) return s;
  return strides_ok(t) ? SSM_OK : SSM_ERR_UNSUPPORTED;
}

inline ssm_status check_out(bool on, const ssm_tensor_desc& t, int ndim, const int64_t* shape, bool dtype_ok,
                     bool inner_unit, bool contiguous) {
  const ssm_status s = check_in(on, t, ndim, shape, dtype_ok, inner_unit, contiguous);
  if (s || !on) return s;
  return non_overlapping(t) ? SSM_OK : SSM_ERR_STRIDE;
}

// One tensor of a call in memory.
struct Placed {
  const ssm_tensor_desc* t = nullptr;
  uintptr_t at = 0;
  Span span;
};

// Whether two tensors are different columns of one row-major buffer: all their
// outer strides are whole multiples of one row, and within a row they do not
// meet.  (Slices of one projection, or of its gradient, interleave so.)
inline bool different_columns(const Placed& a, const Placed& b) {
  int64_t row = 0;
  for (const Placed* p : {&a, &b}) {
    const ssm_tensor_desc& t = *p->t;
    if (t.ndim < 2 || (t.shape[t.ndim - 1] > 1 && t.stride[t.ndim - 1] != 1)) return false;
    for (int i = 0; i < t.ndim - 1; ++i)
      if (t.shape[i] > 1 && t.stride[i] > 0) {
        const int64_t bytes = t.stride[i] * esize(t.dtype);
        if (!row || bytes < row) row = bytes;
      }
  }
  if (!row) return false;
  for (const Placed* p : {&a, &b})
    for (int i = 0; i < p->t->ndim - 1; ++i)
      if (p->t->shape[i] > 1 && p->t->stride[i] * esize(p->t->dtype) % row) return false;
  const Placed& lo = a.at <= b.at ? a : b;
  const Placed& hi = a.at <= b.at ? b : a;
  const int64_t off = (int64_t)((hi.at - lo.at) % (uintptr_t)row);
  auto width = [](const Placed& p) { return p.t->shape[p.t->ndim - 1] * esize(p.t->dtype); };
  return off >= width(lo) && off + width(hi) <= row;
}

// The pointers of a call: presence, alignment, overlap.
class Ptrs {
 public:
  ssm_status in(bool on, const ssm_tensor_desc& t, const void* ptr, int64_t align = 0) {
    return add(on, t, ptr, align, ins_, nin_);
  }
  ssm_status out(bool on, const ssm_tensor_desc& t, const void* ptr, int64_t align = 0) {
    return add(on, t, ptr, align, outs_, nout_);
  }
  // Outputs (and the workspace) against everything else.
  ssm_status check(Span workspace = Span()) const {
    for (int i = 0; i < nout_; ++i) {
      for (int k = 0; k < nin_; ++k)
        if (meet(outs_[i], ins_[k])) return SSM_ERR_ALIAS;
      for (int k = i + 1; k < nout_; ++k)
        if (meet(outs_[i], outs_[k])) return SSM_ERR_ALIAS;
      if (overlap(outs_[i].span, workspace)) return SSM_ERR_ALIAS;
    }
    for (int k = 0; k < nin_; ++k)
      if (overlap(workspace, ins_[k].span)) return SSM_ERR_ALIAS;
    return SSM_OK;
  }

 private:
  static bool meet(const Placed& a, const Placed& b) { return overlap(a.span, b.span) && !different_columns(a, b); }
  static ssm_status add(bool on, const ssm_tensor_desc& t, const void* ptr, int64_t align, Placed* to, int& n) {
    if (!on) return SSM_OK;
    if (!ptr) return SSM_ERR_NULL;
    if (!aligned(ptr, align ? align : esize(t.dtype))) return SSM_ERR_ALIGN;
    to[n].t = &t;
    to[n].at = (uintptr_t)ptr;
    to[n++].span = span_of(t, ptr);
    return SSM_OK;
  }
  Placed ins_[16], outs_[12];
  int nin_ = 0, nout_ = 0;
};

#define SSM_TRY(call)                     \
  do {                                    \
    const ssm_status s_ = (call);         \
    if (s_ != SSM_OK) return s_;          \
  } while (0)

inline bool f32_or_bf16(int32_t dt) { return dt == SSM_F32 || dt == SSM_BF16; }

}  // namespace abi
}  // namespace ssm
