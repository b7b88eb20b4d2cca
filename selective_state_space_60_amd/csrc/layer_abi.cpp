// Host side of the recurrent layer's operators: the gated linear recurrence,
// the RMS norm and the product with 4-bit weights.  As in ssm_abi.cpp, every
// check runs before any HIP call.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>
#include <cstring>

#include "../../include/ssm.h"
#include "abi_checks.h"
#include "layer_internal.h"

using namespace ssm::abi;

namespace {

// a launch holds fewer than 2^32 threads: blocks of 1024, 512, 256
constexpr int64_t kMaxBlocks1024 = (int64_t)1 << 22, kMaxBlocks512 = (int64_t)1 << 23,
                  kMaxBlocks256 = (int64_t)1 << 24;
constexpr int64_t kMaxSpan = (int64_t)1 << 30;       // bytes a kernel addresses from one base

// Sizes whose products stay far from overflowing.
bool sizes_ok(std::initializer_list<int64_t> sizes) {
  __int128 n = 1;
  for (int64_t s : sizes) {
    if (s >= ((int64_t)1 << 40)) return false;
    n *= s;
    if (n >= ((__int128)1 << 56)) return false;
  }
  return true;
}

// The last element's offset must not overflow either.
bool strides_ok(const ssm_tensor_desc& t) {
  __int128 last = 0;
  for (int i = 0; i < t.ndim; ++i) last += (__int128)(t.shape[i] - 1) * t.stride[i];
  return last < ((__int128)1 << 56);
}

// The descriptor of one input (`on` false: left out), or of one output, which
// must not write an element twice.
ssm_status check_in(bool on, const ssm_tensor_desc& t, int ndim, const int64_t* shape, bool dtype_ok,
                    bool inner_unit, bool contiguous) {
  if (!on) return SSM_OK;
  const ssm_status s = check_tensor(t, ndim, shape, dtype_ok, inner_unit, contiguous);
  if (s) return s;
  return strides_ok(t) ? SSM_OK : SSM_ERR_UNSUPPORTED;
}

ssm_status check_out(bool on, const ssm_tensor_desc& t, int ndim, const int64_t* shape, bool dtype_ok,
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
bool different_columns(const Placed& a, const Placed& b) {
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

// -------------------------------------------------------------- gated scan

constexpr uint32_t kGatedInFlags = SSM_HAS_Z | SSM_HAS_H0 | SSM_HAS_BIAS_A | SSM_HAS_BIAS_X | SSM_HAS_LENS |
                                   SSM_NO_WAIT;
constexpr uint32_t kGatedFlags = kGatedInFlags | SSM_WANT_HLAST | SSM_WANT_CKPT;
constexpr uint32_t kGatedBwdFlags = kGatedInFlags | SSM_HAS_CKPT | SSM_HAS_DHLAST;

// The sequence is cut into segments of 8 chunks, one workgroup each for a
// tile of channels; with more than one, words pass the state on.
struct GatedPlan {
  int64_t nk = 0, fwd_seg = 0, bwd_seg = 0;
  bool fits = false;  // the grids and the words
};

GatedPlan plan_gated(int64_t batch, int64_t seqlen, int64_t dim) {
  GatedPlan pl;
  auto parts = [&](int64_t n) { return (seqlen + n - 1) / n; };
  pl.nk = parts(ssm::kGatedCkptSteps);
  pl.fwd_seg = parts(ssm::kGatedFwdChunks * ssm::kGatedFwdSteps);
  pl.bwd_seg = parts(ssm::kGatedBwdChunks * ssm::kGatedBwdSteps);
  const int64_t tiles = (dim + 31) / 32;  // at one channel per lane
  pl.fits = batch * tiles + 7 < kMaxBlocks256 && tiles < kMaxBlocks1024 && pl.bwd_seg < ((int64_t)1 << 30) &&
            (__int128)pl.bwd_seg * batch * dim * 12 < ((int64_t)1 << 35);
  return pl;
}

// Elements from one step to the next; a single step's stride addresses nothing.
int64_t time_stride(const ssm_tensor_desc& t) { return t.shape[1] > 1 ? t.stride[1] : 0; }

// A segment's rows must fit the 32-bit offsets of the kernel.
bool gated_fits(const ssm_tensor_desc& t) {
  return (ssm::kGatedSpanSteps * (__int128)time_stride(t) + 64) * esize(t.dtype) < kMaxSpan;
}

struct GatedShapes {
  int64_t bld[3], bd[2], d[1], b[1], ck[3];
  GatedShapes(int64_t batch, int64_t seqlen, int64_t dim)
      : bld{batch, seqlen, dim},
        bd{batch, dim},
        d{dim},
        b{batch},
        ck{batch, (seqlen + ssm::kGatedCkptSteps - 1) / ssm::kGatedCkptSteps, dim} {}
};

// The inputs that forward and backward share.
template <class D>
ssm_status check_gated_inputs(const D& d, const GatedShapes& sh) {
  const uint32_t f = d.flags;
  const int32_t io = d.x.dtype;
  if (io == SSM_F16) return SSM_ERR_UNSUPPORTED;
  SSM_TRY(check_in(true, d.x, 3, sh.bld, io == SSM_F32 || io == SSM_BF16, true, false));
  SSM_TRY(check_in(true, d.gate_a, 3, sh.bld, d.gate_a.dtype == io, true, false));
  SSM_TRY(check_in(true, d.gate_x, 3, sh.bld, d.gate_x.dtype == io, true, false));
  SSM_TRY(check_in(f & SSM_HAS_Z, d.z, 3, sh.bld, d.z.dtype == io, true, false));
  SSM_TRY(check_in(true, d.A, 1, sh.d, d.A.dtype == SSM_F32, false, false));
  SSM_TRY(check_in(f & SSM_HAS_BIAS_A, d.bias_a, 1, sh.d, d.bias_a.dtype == SSM_F32, false, false));
  SSM_TRY(check_in(f & SSM_HAS_BIAS_X, d.bias_x, 1, sh.d, d.bias_x.dtype == SSM_F32, false, false));
  SSM_TRY(check_in(f & SSM_HAS_H0, d.h0, 2, sh.bd, d.h0.dtype == SSM_F32, false, true));
  SSM_TRY(check_in(f & SSM_HAS_LENS, d.lens, 1, sh.b, d.lens.dtype == SSM_I32, false, true));
  if (!gated_fits(d.x) || !gated_fits(d.gate_a) || !gated_fits(d.gate_x) || ((f & SSM_HAS_Z) && !gated_fits(d.z)))
    return SSM_ERR_UNSUPPORTED;
  return SSM_OK;
}

template <class D, class P>
ssm_status take_gated_inputs(const D& d, const P& p, Ptrs& ptrs) {
  const uint32_t f = d.flags;
  SSM_TRY(ptrs.in(true, d.x, p.x));
  SSM_TRY(ptrs.in(true, d.gate_a, p.gate_a));
  SSM_TRY(ptrs.in(true, d.gate_x, p.gate_x));
  SSM_TRY(ptrs.in(true, d.A, p.A));
  SSM_TRY(ptrs.in(f & SSM_HAS_BIAS_A, d.bias_a, p.bias_a));
  SSM_TRY(ptrs.in(f & SSM_HAS_BIAS_X, d.bias_x, p.bias_x));
  SSM_TRY(ptrs.in(f & SSM_HAS_Z, d.z, p.z));
  SSM_TRY(ptrs.in(f & SSM_HAS_H0, d.h0, p.h0));
  SSM_TRY(ptrs.in(f & SSM_HAS_LENS, d.lens, p.lens));
  return SSM_OK;
}

ssm_status validate_gated(const ssm_gated_desc* d) {
  if (!d) return SSM_ERR_NULL;
  if (d->batch <= 0 || d->seqlen <= 0 || d->dim <= 0) return SSM_ERR_SHAPE;
  if (d->flags & ~kGatedFlags) return SSM_ERR_UNSUPPORTED;
  if (!sizes_ok({d->batch, d->seqlen, d->dim})) return SSM_ERR_UNSUPPORTED;
  const GatedShapes sh(d->batch, d->seqlen, d->dim);
  SSM_TRY(check_gated_inputs(*d, sh));
  SSM_TRY(check_out(true, d->y, 3, sh.bld, d->y.dtype == d->x.dtype || d->y.dtype == SSM_F32, true, false));
  SSM_TRY(check_out(d->flags & SSM_WANT_HLAST, d->h_last, 2, sh.bd, d->h_last.dtype == SSM_F32, false, true));
  SSM_TRY(check_out(d->flags & SSM_WANT_CKPT, d->ckpt, 3, sh.ck, d->ckpt.dtype == SSM_F32, false, true));
  if (!gated_fits(d->y)) return SSM_ERR_UNSUPPORTED;
  if (!plan_gated(d->batch, d->seqlen, d->dim).fits) return SSM_ERR_UNSUPPORTED;
  return SSM_OK;
}

// The kernel parameters of the inputs; what is left out stays null.
template <class D, class P>
ssm::GatedParams gated_params(const D& d, const P& p) {
  ssm::GatedParams q;
  std::memset(&q, 0, sizeof(q));
  const uint32_t f = d.flags;
  q.x = p.x; q.gate_a = p.gate_a; q.gate_x = p.gate_x; q.A = p.A;
  q.z = (f & SSM_HAS_Z) ? p.z : nullptr;
  q.bias_a = (f & SSM_HAS_BIAS_A) ? p.bias_a : nullptr;
  q.bias_x = (f & SSM_HAS_BIAS_X) ? p.bias_x : nullptr;
  q.h0 = (f & SSM_HAS_H0) ? p.h0 : nullptr;
  q.lens = (f & SSM_HAS_LENS) ? p.lens : nullptr;
  q.batch = d.batch; q.L = d.seqlen; q.D = d.dim;
  q.xs_b = d.x.stride[0]; q.xs_t = time_stride(d.x);
  q.gas_b = d.gate_a.stride[0]; q.gas_t = time_stride(d.gate_a);
  q.gxs_b = d.gate_x.stride[0]; q.gxs_t = time_stride(d.gate_x);
  if (q.z) { q.zs_b = d.z.stride[0]; q.zs_t = time_stride(d.z); }
  q.As_d = d.A.stride[0];
  if (q.bias_a) q.bas_d = d.bias_a.stride[0];
  if (q.bias_x) q.bxs_d = d.bias_x.stride[0];
  q.io_bf16 = d.x.dtype == SSM_BF16;
  q.polls = (f & SSM_NO_WAIT) ? 0 : ssm::kGatedPolls;
  return q;
}

// Gated backward workspace, in this order: checkpoints (unless given), the
// sums' partials, the segments' words (the checkpoint forward's first, then
// the carries': the forward is done with them by then).
struct GatedBwdPlan {
  int64_t ws_ckpt = 0, ws_part = 0, ws_chain = 0, ws_total = 0;
};

GatedBwdPlan plan_gated_bwd(const ssm_gated_bwd_desc& d) {
  GatedBwdPlan pl;
  const GatedPlan g = plan_gated(d.batch, d.seqlen, d.dim);
  pl.ws_ckpt = (d.flags & SSM_HAS_CKPT) ? 0 : round256(d.batch * g.nk * d.dim * 4);
  pl.ws_part = round256(d.batch * g.bwd_seg * 3 * d.dim * 4);
  pl.ws_chain = ssm::gated_chain_bytes(d.batch, d.dim, std::max(g.fwd_seg, g.bwd_seg));
  pl.ws_total = pl.ws_ckpt + pl.ws_part + pl.ws_chain;
  return pl;
}

ssm_status validate_gated_bwd(const ssm_gated_bwd_desc* d) {
  if (!d) return SSM_ERR_NULL;
  if (d->batch <= 0 || d->seqlen <= 0 || d->dim <= 0) return SSM_ERR_SHAPE;
  const uint32_t f = d->flags;
  if (f & ~kGatedBwdFlags) return SSM_ERR_UNSUPPORTED;
  if (!sizes_ok({d->batch, d->seqlen, d->dim})) return SSM_ERR_UNSUPPORTED;
  const GatedShapes sh(d->batch, d->seqlen, d->dim);
  SSM_TRY(check_gated_inputs(*d, sh));
  const int32_t g = d->dy.dtype;
  const bool g_ok = g == d->x.dtype || g == SSM_F32;
  SSM_TRY(check_in(true, d->dy, 3, sh.bld, g_ok, true, false));
  SSM_TRY(check_in(f & SSM_HAS_DHLAST, d->dh_last, 2, sh.bd, d->dh_last.dtype == SSM_F32, false, true));
  SSM_TRY(check_in(f & SSM_HAS_CKPT, d->ckpt, 3, sh.ck, d->ckpt.dtype == SSM_F32, false, true));
  SSM_TRY(check_out(true, d->dx, 3, sh.bld, d->dx.dtype == g, true, false));
  SSM_TRY(check_out(true, d->dgate_a, 3, sh.bld, d->dgate_a.dtype == g, true, false));
  SSM_TRY(check_out(true, d->dgate_x, 3, sh.bld, d->dgate_x.dtype == g, true, false));
  SSM_TRY(check_out(f & SSM_HAS_Z, d->dz, 3, sh.bld, d->dz.dtype == g, true, false));
  SSM_TRY(check_out(true, d->dA, 1, sh.d, d->dA.dtype == SSM_F32, false, true));
  SSM_TRY(check_out(f & SSM_HAS_BIAS_A, d->dbias_a, 1, sh.d, d->dbias_a.dtype == SSM_F32, false, true));
  SSM_TRY(check_out(f & SSM_HAS_BIAS_X, d->dbias_x, 1, sh.d, d->dbias_x.dtype == SSM_F32, false, true));
  SSM_TRY(check_out(f & SSM_HAS_H0, d->dh0, 2, sh.bd, d->dh0.dtype == SSM_F32, false, true));
  if (!gated_fits(d->dy) || !gated_fits(d->dx) || !gated_fits(d->dgate_a) || !gated_fits(d->dgate_x) ||
      ((f & SSM_HAS_Z) && !gated_fits(d->dz)))
    return SSM_ERR_UNSUPPORTED;
  if (!plan_gated(d->batch, d->seqlen, d->dim).fits) return SSM_ERR_UNSUPPORTED;
  return SSM_OK;
}

ssm_status validate_gated_bwd_ptrs(const ssm_gated_bwd_desc* d, const ssm_gated_bwd_ptrs* p, Span ws) {
  if (!p) return SSM_ERR_NULL;
  const uint32_t f = d->flags;
  Ptrs a;
  SSM_TRY(take_gated_inputs(*d, *p, a));
  SSM_TRY(a.in(true, d->dy, p->dy));
  SSM_TRY(a.in(f & SSM_HAS_DHLAST, d->dh_last, p->dh_last));
  SSM_TRY(a.in(f & SSM_HAS_CKPT, d->ckpt, p->ckpt));
  SSM_TRY(a.out(true, d->dx, p->dx));
  SSM_TRY(a.out(true, d->dgate_a, p->dgate_a));
  SSM_TRY(a.out(true, d->dgate_x, p->dgate_x));
  SSM_TRY(a.out(f & SSM_HAS_Z, d->dz, p->dz));
  SSM_TRY(a.out(true, d->dA, p->dA));
  SSM_TRY(a.out(f & SSM_HAS_BIAS_A, d->dbias_a, p->dbias_a));
  SSM_TRY(a.out(f & SSM_HAS_BIAS_X, d->dbias_x, p->dbias_x));
  SSM_TRY(a.out(f & SSM_HAS_H0, d->dh0, p->dh0));
  return a.check(ws);
}

// ------------------------------------------------------------ gated decode

constexpr uint32_t kGatedUpdateFlags = SSM_HAS_Z | SSM_HAS_BIAS_A | SSM_HAS_BIAS_X | SSM_HAS_STATE_OUT;

ssm_status validate_gated_update(const ssm_gated_update_desc* d, const ssm_gated_update_ptrs* p) {
  if (!d || !p) return SSM_ERR_NULL;
  if (d->batch <= 0 || d->dim <= 0) return SSM_ERR_SHAPE;
  const uint32_t f = d->flags;
  if (f & ~kGatedUpdateFlags) return SSM_ERR_UNSUPPORTED;
  if (!sizes_ok({d->batch, d->dim})) return SSM_ERR_UNSUPPORTED;
  if (d->batch * ((d->dim + 255) / 256) >= kMaxBlocks256) return SSM_ERR_UNSUPPORTED;
  const int32_t io = d->x.dtype;
  if (io == SSM_F16) return SSM_ERR_UNSUPPORTED;
  const int64_t bd[2] = {d->batch, d->dim}, dd[1] = {d->dim};
  const bool apart = f & SSM_HAS_STATE_OUT;
  SSM_TRY(check_in(true, d->x, 2, bd, io == SSM_F32 || io == SSM_BF16, true, false));
  SSM_TRY(check_in(true, d->gate_a, 2, bd, d->gate_a.dtype == io, true, false));
  SSM_TRY(check_in(true, d->gate_x, 2, bd, d->gate_x.dtype == io, true, false));
  SSM_TRY(check_in(f & SSM_HAS_Z, d->z, 2, bd, d->z.dtype == io, true, false));
  SSM_TRY(check_in(true, d->A, 1, dd, d->A.dtype == SSM_F32, false, false));
  SSM_TRY(check_in(f & SSM_HAS_BIAS_A, d->bias_a, 1, dd, d->bias_a.dtype == SSM_F32, false, false));
  SSM_TRY(check_in(f & SSM_HAS_BIAS_X, d->bias_x, 1, dd, d->bias_x.dtype == SSM_F32, false, false));
  SSM_TRY(check_out(true, d->y, 2, bd, d->y.dtype == io || d->y.dtype == SSM_F32, true, false));
  SSM_TRY(check_in(true, d->state, 2, bd, d->state.dtype == SSM_F32, false, true));
  SSM_TRY(check_out(apart, d->state_out, 2, bd, d->state_out.dtype == SSM_F32, false, true));
  Ptrs t;
  SSM_TRY(t.in(true, d->x, p->x));
  SSM_TRY(t.in(true, d->gate_a, p->gate_a));
  SSM_TRY(t.in(true, d->gate_x, p->gate_x));
  SSM_TRY(t.in(true, d->A, p->A));
  SSM_TRY(t.in(f & SSM_HAS_BIAS_A, d->bias_a, p->bias_a));
  SSM_TRY(t.in(f & SSM_HAS_BIAS_X, d->bias_x, p->bias_x));
  SSM_TRY(t.in(f & SSM_HAS_Z, d->z, p->z));
  SSM_TRY(apart ? t.in(true, d->state, p->state) : t.out(true, d->state, p->state));
  SSM_TRY(t.out(apart, d->state_out, p->state_out));
  SSM_TRY(t.out(true, d->y, p->y));
  return t.check();
}

// -------------------------------------------------------------------- norm

bool f32_or_bf16(int32_t dt) { return dt == SSM_F32 || dt == SSM_BF16; }

int norm_type(int32_t dt) {
  return dt == SSM_F32 ? ssm::kNormF32 : dt == SSM_BF16 ? ssm::kNormBF16 : ssm::kNormE4M3;
}

ssm_status check_norm_sizes(int64_t batch, int64_t seqlen, int64_t dim, float eps) {
  if (batch <= 0 || seqlen <= 0 || dim <= 0) return SSM_ERR_SHAPE;
  if (!(eps >= 0.f)) return SSM_ERR_UNSUPPORTED;
  if (dim > SSM_NORM_MAX_DIM || !sizes_ok({batch, seqlen, dim}) || batch * seqlen >= kMaxBlocks256)
    return SSM_ERR_UNSUPPORTED;
  return SSM_OK;
}

bool same_layout(const ssm_tensor_desc& a, const ssm_tensor_desc& b) {
  if (a.dtype != b.dtype || a.ndim != b.ndim) return false;
  for (int i = 0; i < a.ndim; ++i)
    if (a.shape[i] > 1 && a.stride[i] != b.stride[i]) return false;
  return true;
}

ssm_status validate_norm(const ssm_norm_desc* d, const ssm_norm_ptrs* p) {
  if (!d || !p) return SSM_ERR_NULL;
  SSM_TRY(check_norm_sizes(d->batch, d->seqlen, d->dim, d->eps));
  const uint32_t f = d->flags;
  if (f & ~SSM_HAS_RESIDUAL) return SSM_ERR_UNSUPPORTED;
  const int32_t io = d->x.dtype;
  if (io == SSM_F16) return SSM_ERR_UNSUPPORTED;
  const bool quant = d->y.dtype == SSM_E4M3, res = f & SSM_HAS_RESIDUAL;
  if (d->group != 0 && (!quant || (d->group != 32 && d->group != 64 && d->group != 128))) return SSM_ERR_UNSUPPORTED;
  const int64_t bld[3] = {d->batch, d->seqlen, d->dim}, dd[1] = {d->dim};
  const int64_t sc[3] = {d->batch, d->seqlen, d->group ? (d->dim + d->group - 1) / d->group : 1};
  SSM_TRY(check_in(true, d->x, 3, bld, f32_or_bf16(io), true, false));
  SSM_TRY(check_in(res, d->residual, 3, bld, d->residual.dtype == io || d->residual.dtype == SSM_F32, true, false));
  SSM_TRY(check_out(res, d->residual_out, 3, bld, d->residual_out.dtype == io || d->residual_out.dtype == SSM_F32, true,
                false));
  SSM_TRY(check_in(true, d->weight, 1, dd, d->weight.dtype == SSM_F32, false, true));
  SSM_TRY(check_out(true, d->y, 3, bld, quant || d->y.dtype == io || d->y.dtype == SSM_F32, true, false));
  SSM_TRY(check_out(quant, d->scale, 3, sc, d->scale.dtype == SSM_F32, false, true));
  const bool in_place = res && p->residual == p->residual_out && same_layout(d->residual, d->residual_out);
  Ptrs t;
  SSM_TRY(t.in(true, d->x, p->x));
  if (res && !p->residual) return SSM_ERR_NULL;
  SSM_TRY(t.in(res && !in_place, d->residual, p->residual));
  SSM_TRY(t.in(true, d->weight, p->weight));
  SSM_TRY(t.out(res, d->residual_out, p->residual_out));
  SSM_TRY(t.out(true, d->y, p->y));
  SSM_TRY(t.out(quant, d->scale, p->scale));
  return t.check();
}

ssm_status validate_norm_bwd(const ssm_norm_bwd_desc* d) {
  if (!d) return SSM_ERR_NULL;
  SSM_TRY(check_norm_sizes(d->batch, d->seqlen, d->dim, d->eps));
  if (d->flags & ~SSM_HAS_RESIDUAL) return SSM_ERR_UNSUPPORTED;
  if (d->row.dtype == SSM_F16 || d->dy.dtype == SSM_F16) return SSM_ERR_UNSUPPORTED;
  const bool res = d->flags & SSM_HAS_RESIDUAL;
  const int64_t bld[3] = {d->batch, d->seqlen, d->dim}, dd[1] = {d->dim};
  SSM_TRY(check_in(true, d->dy, 3, bld, f32_or_bf16(d->dy.dtype), true, false));
  SSM_TRY(check_in(true, d->row, 3, bld, f32_or_bf16(d->row.dtype), true, false));
  SSM_TRY(check_in(res, d->dres, 3, bld, f32_or_bf16(d->dres.dtype), true, false));
  SSM_TRY(check_in(true, d->weight, 1, dd, d->weight.dtype == SSM_F32, false, true));
  SSM_TRY(check_out(true, d->dx, 3, bld, f32_or_bf16(d->dx.dtype), true, false));
  SSM_TRY(check_out(true, d->dweight, 1, dd, d->dweight.dtype == SSM_F32, false, true));
  return SSM_OK;
}

int64_t norm_bwd_bytes(const ssm_norm_bwd_desc& d) {
  return round256((int64_t)ssm::norm_bwd_parts(d.batch * d.seqlen, d.dim) * d.dim * 4);
}

// ----------------------------------------------------------- 4-bit weights

ssm_status validate_w4(const ssm_w4_desc* d, const ssm_w4_ptrs* p) {
  if (!d || !p) return SSM_ERR_NULL;
  if (d->rows <= 0 || d->ins <= 0 || d->outs <= 0 || d->group <= 0) return SSM_ERR_SHAPE;
  const uint32_t f = d->flags;
  if (f & ~(SSM_HAS_ZERO | SSM_HAS_BIAS)) return SSM_ERR_UNSUPPORTED;
  if ((d->group != 32 && d->group != 64 && d->group != 128) || d->rows > SSM_W4_MAX_ROWS) return SSM_ERR_UNSUPPORTED;
  if (d->ins % d->group) return SSM_ERR_SHAPE;
  // 32 outputs' weights and all rows of x are addressed from one base each
  if (d->ins >= ((int64_t)1 << 26) || !sizes_ok({d->outs, d->ins}) || (d->outs + 15) / 16 >= kMaxBlocks512)
    return SSM_ERR_UNSUPPORTED;
  const int64_t mk[2] = {d->rows, d->ins}, nh[2] = {d->outs, d->ins / 2}, ng[2] = {d->outs, d->ins / d->group};
  const int64_t mn[2] = {d->rows, d->outs}, n[1] = {d->outs};
  SSM_TRY(check_in(true, d->x, 2, mk, d->x.dtype == SSM_BF16, true, false));
  SSM_TRY(check_in(true, d->weight, 2, nh, d->weight.dtype == SSM_U8, false, true));
  SSM_TRY(check_in(true, d->scale, 2, ng, f32_or_bf16(d->scale.dtype), false, true));
  SSM_TRY(check_in(f & SSM_HAS_ZERO, d->zero, 2, ng, d->zero.dtype == SSM_U8, false, true));
  SSM_TRY(check_in(f & SSM_HAS_BIAS, d->bias, 1, n, d->bias.dtype == SSM_F32, false, false));
  SSM_TRY(check_out(true, d->y, 2, mn, f32_or_bf16(d->y.dtype), true, false));
  if (((d->rows - 1) * (__int128)d->x.stride[0] + d->ins) * 2 >= kMaxSpan) return SSM_ERR_UNSUPPORTED;
  if (p->x && d->rows > 1 && d->x.stride[0] % 8) return SSM_ERR_ALIGN;
  Ptrs t;
  SSM_TRY(t.in(true, d->x, p->x, 16));
  SSM_TRY(t.in(true, d->weight, p->weight, 16));
  SSM_TRY(t.in(true, d->scale, p->scale));
  SSM_TRY(t.in(f & SSM_HAS_ZERO, d->zero, p->zero));
  SSM_TRY(t.in(f & SSM_HAS_BIAS, d->bias, p->bias));
  SSM_TRY(t.out(true, d->y, p->y));
  return t.check();
}

}  // namespace

extern "C" {

ssm_status ssm_gated_scan_workspace_size(const ssm_gated_desc* d, size_t* bytes) {
  if (!bytes) return SSM_ERR_NULL;
  SSM_TRY(validate_gated(d));
  *bytes = (size_t)ssm::gated_chain_bytes(d->batch, d->dim, plan_gated(d->batch, d->seqlen, d->dim).fwd_seg);
  return SSM_OK;
}

ssm_status ssm_gated_scan_fwd(const ssm_gated_desc* d, const ssm_gated_ptrs* p, void* workspace,
                              size_t workspace_bytes, void* hip_stream) {
  SSM_TRY(validate_gated(d));
  if (!p) return SSM_ERR_NULL;
  const int64_t need = ssm::gated_chain_bytes(d->batch, d->dim, plan_gated(d->batch, d->seqlen, d->dim).fwd_seg);
  Ptrs a;
  SSM_TRY(take_gated_inputs(*d, *p, a));
  SSM_TRY(a.out(true, d->y, p->y));
  SSM_TRY(a.out(d->flags & SSM_WANT_HLAST, d->h_last, p->h_last));
  SSM_TRY(a.out(d->flags & SSM_WANT_CKPT, d->ckpt, p->ckpt));
  SSM_TRY(a.check(need ? span_bytes(workspace, need) : Span()));
  if (need && (!workspace || workspace_bytes < (size_t)need)) return SSM_ERR_WORKSPACE;
  if (need && !aligned(workspace, 256)) return SSM_ERR_ALIGN;
  ssm::GatedParams q = gated_params(*d, *p);
  q.y = p->y;
  q.ys_b = d->y.stride[0]; q.ys_t = time_stride(d->y);
  q.y_f32 = d->y.dtype == SSM_F32;
  q.h_last = (d->flags & SSM_WANT_HLAST) ? p->h_last : nullptr;
  q.ckpt = (d->flags & SSM_WANT_CKPT) ? p->ckpt : nullptr;
  q.chain = workspace;
  return hip_status(ssm::launch_gated_scan(q, (hipStream_t)hip_stream));
}

ssm_status ssm_gated_scan_bwd_workspace_size(const ssm_gated_bwd_desc* d, size_t* bytes) {
  if (!bytes) return SSM_ERR_NULL;
  SSM_TRY(validate_gated_bwd(d));
  *bytes = (size_t)plan_gated_bwd(*d).ws_total;
  return SSM_OK;
}

ssm_status ssm_gated_scan_bwd(const ssm_gated_bwd_desc* d, const ssm_gated_bwd_ptrs* p, void* workspace,
                              size_t workspace_bytes, void* hip_stream) {
  SSM_TRY(validate_gated_bwd(d));
  const GatedBwdPlan pl = plan_gated_bwd(*d);
  SSM_TRY(validate_gated_bwd_ptrs(d, p, span_bytes(workspace, pl.ws_total)));
  if (!workspace || workspace_bytes < (size_t)pl.ws_total) return SSM_ERR_WORKSPACE;
  if (!aligned(workspace, 256)) return SSM_ERR_ALIGN;
  const uint32_t f = d->flags;
  const hipStream_t st = (hipStream_t)hip_stream;
  char* w = (char*)workspace;
  ssm::GatedBwdParams q;
  std::memset(&q, 0, sizeof(q));
  q.f = gated_params(*d, *p);
  q.f.ckpt = (f & SSM_HAS_CKPT) ? const_cast<float*>(p->ckpt) : (float*)w;  // given checkpoints are only read
  q.part = (float*)(w + pl.ws_ckpt);
  q.f.chain = w + pl.ws_ckpt + pl.ws_part;
  q.dy = p->dy;
  q.dh_last = (f & SSM_HAS_DHLAST) ? p->dh_last : nullptr;
  q.dx = p->dx; q.dgate_a = p->dgate_a; q.dgate_x = p->dgate_x;
  q.dz = (f & SSM_HAS_Z) ? p->dz : nullptr;
  q.dA = p->dA;
  q.dbias_a = (f & SSM_HAS_BIAS_A) ? p->dbias_a : nullptr;
  q.dbias_x = (f & SSM_HAS_BIAS_X) ? p->dbias_x : nullptr;
  q.dh0 = (f & SSM_HAS_H0) ? p->dh0 : nullptr;
  q.dys_b = d->dy.stride[0]; q.dys_t = time_stride(d->dy);
  q.dxs_b = d->dx.stride[0]; q.dxs_t = time_stride(d->dx);
  q.dgas_b = d->dgate_a.stride[0]; q.dgas_t = time_stride(d->dgate_a);
  q.dgxs_b = d->dgate_x.stride[0]; q.dgxs_t = time_stride(d->dgate_x);
  if (q.dz) { q.dzs_b = d->dz.stride[0]; q.dzs_t = time_stride(d->dz); }
  q.g_f32 = d->dy.dtype == SSM_F32;
  if (!(f & SSM_HAS_CKPT)) {
    const hipError_t e = ssm::launch_gated_scan(q.f, st);  // y is null: checkpoints only
    if (e != hipSuccess) return hip_status(e);
  }
  return hip_status(ssm::launch_gated_scan_bwd(q, st));
}

ssm_status ssm_gated_state_update(const ssm_gated_update_desc* d, const ssm_gated_update_ptrs* p, void* hip_stream) {
  SSM_TRY(validate_gated_update(d, p));
  const uint32_t f = d->flags;
  ssm::GatedUpdateParams q;
  std::memset(&q, 0, sizeof(q));
  q.x = p->x; q.gate_a = p->gate_a; q.gate_x = p->gate_x; q.y = p->y; q.A = p->A;
  q.z = (f & SSM_HAS_Z) ? p->z : nullptr;
  q.bias_a = (f & SSM_HAS_BIAS_A) ? p->bias_a : nullptr;
  q.bias_x = (f & SSM_HAS_BIAS_X) ? p->bias_x : nullptr;
  q.state = p->state;
  q.state_out = (f & SSM_HAS_STATE_OUT) ? p->state_out : p->state;
  q.batch = d->batch; q.D = d->dim;
  q.xs_b = d->x.stride[0]; q.gas_b = d->gate_a.stride[0]; q.gxs_b = d->gate_x.stride[0];
  if (q.z) q.zs_b = d->z.stride[0];
  q.ys_b = d->y.stride[0];
  q.As_d = d->A.stride[0];
  if (q.bias_a) q.bas_d = d->bias_a.stride[0];
  if (q.bias_x) q.bxs_d = d->bias_x.stride[0];
  q.io_bf16 = d->x.dtype == SSM_BF16;
  q.y_f32 = d->y.dtype == SSM_F32;
  return hip_status(ssm::launch_gated_state_update(q, (hipStream_t)hip_stream));
}

ssm_status ssm_rms_norm_fwd(const ssm_norm_desc* d, const ssm_norm_ptrs* p, void* hip_stream) {
  SSM_TRY(validate_norm(d, p));
  ssm::NormParams q;
  std::memset(&q, 0, sizeof(q));
  q.x = p->x; q.weight = p->weight; q.y = p->y;
  q.batch = d->batch; q.L = d->seqlen; q.D = d->dim; q.group = d->group; q.eps = d->eps;
  q.xs_b = d->x.stride[0]; q.xs_t = d->x.stride[1];
  q.ys_b = d->y.stride[0]; q.ys_t = d->y.stride[1];
  q.x_type = norm_type(d->x.dtype);
  q.y_type = norm_type(d->y.dtype);
  if (d->flags & SSM_HAS_RESIDUAL) {
    q.residual = p->residual;
    q.residual_out = p->residual_out;
    q.rs_b = d->residual.stride[0]; q.rs_t = d->residual.stride[1];
    q.ros_b = d->residual_out.stride[0]; q.ros_t = d->residual_out.stride[1];
    q.r_type = norm_type(d->residual.dtype);
    q.ro_type = norm_type(d->residual_out.dtype);
  }
  q.scale = d->y.dtype == SSM_E4M3 ? p->scale : nullptr;
  return hip_status(ssm::launch_rms_norm(q, (hipStream_t)hip_stream));
}

ssm_status ssm_rms_norm_bwd_workspace_size(const ssm_norm_bwd_desc* d, size_t* bytes) {
  if (!bytes) return SSM_ERR_NULL;
  SSM_TRY(validate_norm_bwd(d));
  *bytes = (size_t)norm_bwd_bytes(*d);
  return SSM_OK;
}

ssm_status ssm_rms_norm_bwd(const ssm_norm_bwd_desc* d, const ssm_norm_bwd_ptrs* p, void* workspace,
                            size_t workspace_bytes, void* hip_stream) {
  SSM_TRY(validate_norm_bwd(d));
  if (!p) return SSM_ERR_NULL;
  const bool res = d->flags & SSM_HAS_RESIDUAL;
  const int64_t need = norm_bwd_bytes(*d);
  Ptrs a;
  SSM_TRY(a.in(true, d->dy, p->dy));
  SSM_TRY(a.in(true, d->row, p->row));
  SSM_TRY(a.in(true, d->weight, p->weight));
  SSM_TRY(a.in(res, d->dres, p->dres));
  SSM_TRY(a.out(true, d->dx, p->dx));
  SSM_TRY(a.out(true, d->dweight, p->dweight));
  SSM_TRY(a.check(span_bytes(workspace, need)));
  if (!workspace || workspace_bytes < (size_t)need) return SSM_ERR_WORKSPACE;
  if (!aligned(workspace, 256)) return SSM_ERR_ALIGN;
  ssm::NormBwdParams q;
  std::memset(&q, 0, sizeof(q));
  q.dy = p->dy; q.row = p->row; q.weight = p->weight; q.dx = p->dx; q.dweight = p->dweight;
  q.part = (float*)workspace;
  q.parts = ssm::norm_bwd_parts(d->batch * d->seqlen, d->dim);
  q.batch = d->batch; q.L = d->seqlen; q.D = d->dim; q.eps = d->eps;
  q.dys_b = d->dy.stride[0]; q.dys_t = d->dy.stride[1];
  q.rs_b = d->row.stride[0]; q.rs_t = d->row.stride[1];
  q.dxs_b = d->dx.stride[0]; q.dxs_t = d->dx.stride[1];
  q.dy_type = norm_type(d->dy.dtype);
  q.row_type = norm_type(d->row.dtype);
  q.dx_type = norm_type(d->dx.dtype);
  if (res) {
    q.dres = p->dres;
    q.drs_b = d->dres.stride[0]; q.drs_t = d->dres.stride[1];
    q.dres_type = norm_type(d->dres.dtype);
  }
  return hip_status(ssm::launch_rms_norm_bwd(q, (hipStream_t)hip_stream));
}

ssm_status ssm_w4_matvec(const ssm_w4_desc* d, const ssm_w4_ptrs* p, void* hip_stream) {
  SSM_TRY(validate_w4(d, p));
  ssm::W4Params q;
  std::memset(&q, 0, sizeof(q));
  q.x = p->x; q.weight = (const uint8_t*)p->weight; q.scale = p->scale; q.y = p->y;
  q.zero = (d->flags & SSM_HAS_ZERO) ? (const uint8_t*)p->zero : nullptr;
  q.bias = (d->flags & SSM_HAS_BIAS) ? p->bias : nullptr;
  q.rows = d->rows; q.ins = d->ins; q.outs = d->outs; q.group = d->group;
  q.xs_m = d->x.stride[0]; q.ys_m = d->y.stride[0];
  q.bs_n = q.bias ? d->bias.stride[0] : 0;
  q.scale_f32 = d->scale.dtype == SSM_F32;
  q.y_f32 = d->y.dtype == SSM_F32;
  return hip_status(ssm::launch_w4_matvec(q, (hipStream_t)hip_stream));
}

}  // extern "C"
