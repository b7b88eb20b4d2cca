// Host side of the operators over packed sequences and pools of states, of the
// convolution's backward, of the beam selection and of the slot moves.  As in
// ssm_abi.cpp, every check runs before any HIP call.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>
#include <cstring>

#include "../../include/ssm.h"
#include "abi_checks.h"
#include "layer_checks.h"
#include "packed_pieces.h"
#include "serve_internal.h"

using namespace ssm::abi;

namespace {

// `rows` rows of a tensor, addressed from one base; a single row's stride addresses nothing.
bool rows_fit(const ssm_tensor_desc& t, int dim, int64_t rows) {
  const int64_t st = t.shape[dim] > 1 ? t.stride[dim] : 0;
  return (rows * (__int128)st + 64) * esize(t.dtype) < kMaxSpan;
}

// The same for rows of `width` elements that lie `sn` apart.
bool rows_fit(const ssm_tensor_desc& t, int dim, int64_t rows, int64_t width, int64_t sn) {
  const int64_t st = t.shape[dim] > 1 ? t.stride[dim] : 0;
  return (rows * (__int128)st + (__int128)width * sn + 64) * esize(t.dtype) < kMaxSpan;
}

// The row stride of an output that a kernel drops rows behind the last from.
int64_t out_stride(const ssm_tensor_desc& t, int dim, int64_t width) {
  return t.shape[dim] > 1 ? t.stride[dim] : width;
}

// ---------------------------------------------------------- packed sequences

constexpr uint32_t kPackedFlags = SSM_HAS_STARTS | SSM_HAS_STATES | SSM_HAS_SRC | SSM_HAS_DST;

template <class D>
ssm_status check_packed(const D& d) {
  const uint32_t f = d.flags;
  if (!(f & SSM_HAS_STATES) && (f & (SSM_HAS_SRC | SSM_HAS_DST))) return SSM_ERR_UNSUPPORTED;
  if (!(f & SSM_HAS_STARTS) && d.seqs != d.tokens) return SSM_ERR_SHAPE;
  if ((f & SSM_HAS_STATES) && d.slots <= 0) return SSM_ERR_SHAPE;
  if ((f & SSM_HAS_STATES) && !(f & SSM_HAS_SRC) && d.seqs > d.slots) return SSM_ERR_SHAPE;
  const int64_t n[1] = {d.seqs}, n1[1] = {d.seqs + 1};
  SSM_TRY(check_in(f & SSM_HAS_STARTS, d.starts, 1, n1, d.starts.dtype == SSM_I32, false, true));
  SSM_TRY(check_in(f & SSM_HAS_SRC, d.src, 1, n, d.src.dtype == SSM_I32, false, true));
  SSM_TRY(check_in(f & SSM_HAS_DST, d.dst, 1, n, d.dst.dtype == SSM_I32, false, true));
  return SSM_OK;
}

template <class D, class P>
ssm_status take_packed(const D& d, const P& p, Ptrs& a) {
  SSM_TRY(a.in(d.flags & SSM_HAS_STARTS, d.starts, p.starts));
  SSM_TRY(a.in(d.flags & SSM_HAS_SRC, d.src, p.src));
  SSM_TRY(a.in(d.flags & SSM_HAS_DST, d.dst, p.dst));
  return SSM_OK;
}

template <class D, class P>
ssm::PackedSeqs packed_seqs(const D& d, const P& p) {
  const uint32_t f = d.flags;
  ssm::PackedSeqs q;
  q.starts = (f & SSM_HAS_STARTS) ? p.starts : nullptr;
  q.src = (f & SSM_HAS_SRC) ? p.src : nullptr;
  q.dst = (f & SSM_HAS_DST) ? p.dst : nullptr;
  q.tokens = (int)d.tokens;
  q.seqs = (int)d.seqs;
  q.slots = (f & SSM_HAS_STATES) ? d.slots : 0;
  return q;
}

// -------------------------------------------------------------- packed conv

ssm_status validate_conv_packed(const ssm_conv_packed_desc* d, const ssm_conv_packed_ptrs* p) {
  if (!d || !p) return SSM_ERR_NULL;
  if (d->tokens <= 0 || d->seqs <= 0 || d->dim <= 0 || d->width <= 0) return SSM_ERR_SHAPE;
  const uint32_t f = d->flags;
  if (f & ~(kPackedFlags | SSM_HAS_BIAS | SSM_SILU)) return SSM_ERR_UNSUPPORTED;
  if (d->width > 8 || d->tokens >= ((int64_t)1 << 30) || d->seqs >= ((int64_t)1 << 30)) return SSM_ERR_UNSUPPORTED;
  const bool pool = f & SSM_HAS_STATES;
  if (pool && d->width == 1) return SSM_ERR_UNSUPPORTED;
  if (!sizes_ok({d->tokens, d->dim}) || (pool && !sizes_ok({d->slots, d->width, d->dim}))) return SSM_ERR_UNSUPPORTED;
  if ((d->seqs + d->tokens / ssm::kConvPackedStep + 1) * ((d->dim + 255) / 256) >= kMaxBlocks256)
    return SSM_ERR_UNSUPPORTED;
  const int32_t io = d->x.dtype;
  if (io == SSM_F16) return SSM_ERR_UNSUPPORTED;
  SSM_TRY(check_packed(*d));
  const int64_t td[2] = {d->tokens, d->dim}, dw[2] = {d->dim, d->width}, dd[1] = {d->dim};
  const int64_t win[3] = {d->slots, d->width - 1, d->dim};
  SSM_TRY(check_in(true, d->x, 2, td, f32_or_bf16(io), true, false));
  SSM_TRY(check_in(true, d->weight, 2, dw, d->weight.dtype == SSM_F32, false, false));
  SSM_TRY(check_in(f & SSM_HAS_BIAS, d->bias, 1, dd, d->bias.dtype == SSM_F32, false, false));
  SSM_TRY(check_out(true, d->y, 2, td, d->y.dtype == io || d->y.dtype == SSM_F32, true, false));
  SSM_TRY(check_out(pool, d->windows, 3, win, d->windows.dtype == io, true, false));
  if (!rows_fit(d->x, 0, 64) || !rows_fit(d->y, 0, 64) || (pool && !rows_fit(d->windows, 1, 64)) ||
      d->dim >= ((int64_t)1 << 28))
    return SSM_ERR_UNSUPPORTED;
  Ptrs a;
  SSM_TRY(a.in(true, d->x, p->x));
  SSM_TRY(a.in(true, d->weight, p->weight));
  SSM_TRY(a.in(f & SSM_HAS_BIAS, d->bias, p->bias));
  SSM_TRY(take_packed(*d, *p, a));
  SSM_TRY(a.out(true, d->y, p->y));
  SSM_TRY(a.out(pool, d->windows, p->windows));
  return a.check();
}

// -------------------------------------------------------------- packed scan

constexpr uint32_t kScanPackedFlags = kPackedFlags | SSM_HAS_Z | SSM_HAS_D | SSM_DISC_EULER | SSM_DELTA_SOFTPLUS |
                                      SSM_HAS_DELTA_BIAS;

ssm::ScanPackedPlan plan_packed(const ssm_scan_packed_desc& d) {
  return ssm::plan_scan_packed(d.tokens, d.seqs, d.dim, d.dstate, !(d.flags & SSM_HAS_STARTS));
}

ssm_status validate_scan_packed(const ssm_scan_packed_desc* d) {
  if (!d) return SSM_ERR_NULL;
  if (d->tokens <= 0 || d->seqs <= 0 || d->dim <= 0 || d->dstate <= 0) return SSM_ERR_SHAPE;
  const uint32_t f = d->flags;
  if (f & ~kScanPackedFlags) return SSM_ERR_UNSUPPORTED;
  if ((f & SSM_HAS_DELTA_BIAS) && !(f & SSM_DELTA_SOFTPLUS)) return SSM_ERR_UNSUPPORTED;
  if (d->dstate > SSM_SCAN_MAX_DSTATE || d->tokens >= ((int64_t)1 << 30) || d->seqs >= ((int64_t)1 << 30))
    return SSM_ERR_UNSUPPORTED;
  const bool pool = f & SSM_HAS_STATES;
  if (!sizes_ok({d->tokens, d->dim}) || (pool && !sizes_ok({d->slots, d->dim, d->dstate})) ||
      d->dim * d->dstate >= ((int64_t)1 << 28) || (d->seqs + 256) * ((d->dim + 63) / 64) >= kMaxBlocks256)
    return SSM_ERR_UNSUPPORTED;
  const int32_t io = d->x.dtype;
  if (io == SSM_F16) return SSM_ERR_UNSUPPORTED;
  SSM_TRY(check_packed(*d));
  const int64_t td[2] = {d->tokens, d->dim}, tn[2] = {d->tokens, d->dstate}, dn[2] = {d->dim, d->dstate};
  const int64_t dd[1] = {d->dim}, st[3] = {d->slots, d->dim, d->dstate};
  SSM_TRY(check_in(true, d->x, 2, td, f32_or_bf16(io), true, false));
  SSM_TRY(check_in(true, d->delta, 2, td, d->delta.dtype == io, true, false));
  SSM_TRY(check_in(true, d->A, 2, dn, d->A.dtype == SSM_F32, false, false));
  SSM_TRY(check_in(true, d->B, 2, tn, d->B.dtype == io, false, false));
  SSM_TRY(check_in(true, d->C, 2, tn, d->C.dtype == io, false, false));
  SSM_TRY(check_in(f & SSM_HAS_D, d->D, 1, dd, d->D.dtype == SSM_F32, false, false));
  SSM_TRY(check_in(f & SSM_HAS_Z, d->z, 2, td, d->z.dtype == io, true, false));
  SSM_TRY(check_in(f & SSM_HAS_DELTA_BIAS, d->delta_bias, 1, dd, d->delta_bias.dtype == SSM_F32, false, false));
  SSM_TRY(check_out(true, d->y, 2, td, d->y.dtype == io || d->y.dtype == SSM_F32, true, false));
  SSM_TRY(check_out(pool, d->states, 3, st, d->states.dtype == SSM_F32, false, false));
  // a slot is one contiguous (dim, dstate) block
  if (pool && ((d->dstate > 1 && d->states.stride[2] != 1) || (d->dim > 1 && d->states.stride[1] != d->dstate)))
    return SSM_ERR_STRIDE;
  for (const ssm_tensor_desc* t : {&d->x, &d->delta, &d->y})
    if (!rows_fit(*t, 0, 64)) return SSM_ERR_UNSUPPORTED;
  if ((f & SSM_HAS_Z) && !rows_fit(d->z, 0, 64)) return SSM_ERR_UNSUPPORTED;
  if (!rows_fit(d->B, 0, 64, d->dstate, d->B.stride[1]) || !rows_fit(d->C, 0, 64, d->dstate, d->C.stride[1]))
    return SSM_ERR_UNSUPPORTED;
  return SSM_OK;
}

// ------------------------------------------------------------ conv backward

ssm_status validate_conv_bwd(const ssm_conv_bwd_desc* d) {
  if (!d) return SSM_ERR_NULL;
  if (d->batch <= 0 || d->seqlen <= 0 || d->dim <= 0 || d->width <= 0) return SSM_ERR_SHAPE;
  const uint32_t f = d->flags;
  if (f & ~(SSM_HAS_BIAS | SSM_SILU)) return SSM_ERR_UNSUPPORTED;
  if (d->width > 8 || d->dim >= ((int64_t)1 << 28) || !sizes_ok({d->batch, d->seqlen, d->dim}))
    return SSM_ERR_UNSUPPORTED;
  if ((__int128)d->batch * ((d->seqlen + 127) / 128) * ((d->dim + 63) / 64) >= kMaxBlocks256) return SSM_ERR_UNSUPPORTED;
  const int32_t io = d->x.dtype;
  if (io == SSM_F16) return SSM_ERR_UNSUPPORTED;
  const int64_t bld[3] = {d->batch, d->seqlen, d->dim}, dw[2] = {d->dim, d->width}, dd[1] = {d->dim};
  SSM_TRY(check_in(true, d->dy, 3, bld, d->dy.dtype == io || d->dy.dtype == SSM_F32, true, false));
  SSM_TRY(check_in(true, d->x, 3, bld, f32_or_bf16(io), true, false));
  SSM_TRY(check_in(true, d->weight, 2, dw, d->weight.dtype == SSM_F32, false, false));
  SSM_TRY(check_in(f & SSM_HAS_BIAS, d->bias, 1, dd, d->bias.dtype == SSM_F32, false, false));
  SSM_TRY(check_out(true, d->dx, 3, bld, d->dx.dtype == io || d->dx.dtype == SSM_F32, true, false));
  SSM_TRY(check_out(true, d->dweight, 2, dw, d->dweight.dtype == SSM_F32, false, true));
  SSM_TRY(check_out(f & SSM_HAS_BIAS, d->dbias, 1, dd, d->dbias.dtype == SSM_F32, false, true));
  if (!rows_fit(d->dy, 1, 128) || !rows_fit(d->x, 1, 128) || !rows_fit(d->dx, 1, 128)) return SSM_ERR_UNSUPPORTED;
  return SSM_OK;
}

int64_t conv_bwd_bytes(const ssm_conv_bwd_desc& d) {
  return round256(ssm::conv_bwd_parts(d.batch, d.seqlen) * (d.width + 1) * d.dim * 4);
}

// ----------------------------------------------------------- beam selection

ssm_status validate_beam(const ssm_beam_desc* d) {
  if (!d) return SSM_ERR_NULL;
  if (d->batch <= 0 || d->beams <= 0 || d->vocab <= 0 || d->k <= 0) return SSM_ERR_SHAPE;
  if (d->flags) return SSM_ERR_UNSUPPORTED;
  const int64_t pieces = (d->vocab + 4095) / 4096;
  if (d->k > SSM_BEAM_MAX_K || d->beams > 1024 || d->vocab >= ((int64_t)1 << 31) ||
      d->beams * d->vocab >= ((int64_t)1 << 31) || d->batch >= ((int64_t)1 << 24) || d->beams * pieces > 4096 ||
      d->batch * d->beams * pieces >= ((int64_t)1 << 24))
    return SSM_ERR_UNSUPPORTED;
  if (d->k > d->beams * d->vocab) return SSM_ERR_SHAPE;
  const int32_t io = d->logits.dtype;
  if (io == SSM_F16) return SSM_ERR_UNSUPPORTED;
  const int64_t bnv[3] = {d->batch, d->beams, d->vocab}, bn[2] = {d->batch, d->beams}, bk[2] = {d->batch, d->k};
  SSM_TRY(check_in(true, d->logits, 3, bnv, f32_or_bf16(io), true, false));
  SSM_TRY(check_in(true, d->scores, 2, bn, d->scores.dtype == SSM_F32, false, false));
  SSM_TRY(check_out(true, d->out_scores, 2, bk, d->out_scores.dtype == SSM_F32, false, true));
  SSM_TRY(check_out(true, d->tokens, 2, bk, d->tokens.dtype == SSM_I32, false, true));
  SSM_TRY(check_out(true, d->parents, 2, bk, d->parents.dtype == SSM_I32, false, true));
  return SSM_OK;
}

struct BeamPlan {
  ssm::BeamPieces cut;
  int64_t ws_cand, ws_total;
};

BeamPlan plan_beam(const ssm_beam_desc& d) {
  BeamPlan pl;
  pl.cut = ssm::beam_pieces(d.batch * d.beams, d.vocab);
  const int64_t n = d.batch * d.beams * pl.cut.parts;
  pl.ws_cand = round256(n * d.k * 8);
  pl.ws_total = pl.ws_cand + round256(n * 8);
  return pl;
}

// --------------------------------------------------------------- slot moves

ssm_status validate_move(const ssm_move_desc* d, const ssm_move_ptrs* p) {
  if (!d || !p) return SSM_ERR_NULL;
  if (d->slots <= 0 || d->row <= 0 || d->moves <= 0) return SSM_ERR_SHAPE;
  const bool dst = d->flags & SSM_HAS_DST;
  if (d->flags & ~SSM_HAS_DST) return SSM_ERR_UNSUPPORTED;
  if (d->moves > SSM_MOVE_MAX_MOVES || d->row >= ((int64_t)1 << 27) || !sizes_ok({d->slots, d->row}))
    return SSM_ERR_UNSUPPORTED;
  if (!dst && d->moves > d->slots) return SSM_ERR_SHAPE;
  const int64_t sr[2] = {d->slots, d->row}, m[1] = {d->moves};
  if (d->pool.dtype == SSM_F16) return SSM_ERR_UNSUPPORTED;
  SSM_TRY(check_out(true, d->pool, 2, sr, f32_or_bf16(d->pool.dtype), true, false));
  SSM_TRY(check_in(true, d->src, 1, m, d->src.dtype == SSM_I32, false, true));
  SSM_TRY(check_in(dst, d->dst, 1, m, d->dst.dtype == SSM_I32, false, true));
  Ptrs a;
  SSM_TRY(a.out(true, d->pool, p->pool));
  SSM_TRY(a.in(true, d->src, p->src));
  SSM_TRY(a.in(dst, d->dst, p->dst));
  return a.check();
}

}  // namespace

extern "C" {

ssm_status ssm_causal_conv1d_packed(const ssm_conv_packed_desc* d, const ssm_conv_packed_ptrs* p, void* hip_stream) {
  SSM_TRY(validate_conv_packed(d, p));
  ssm::ConvPackedParams q;
  std::memset(&q, 0, sizeof(q));
  q.q = packed_seqs(*d, *p);
  q.x = p->x; q.w = p->weight; q.y = p->y;
  q.bias = (d->flags & SSM_HAS_BIAS) ? p->bias : nullptr;
  q.D = d->dim; q.W = d->width;
  q.xs_t = d->tokens > 1 ? d->x.stride[0] : 0;
  q.ys_t = out_stride(d->y, 0, d->dim);
  q.ws_d = d->weight.stride[0]; q.ws_k = d->weight.stride[1];
  if (q.bias) q.bs_d = d->bias.stride[0];
  if (d->flags & SSM_HAS_STATES) {
    q.windows = p->windows;
    q.wins_s = d->slots > 1 ? d->windows.stride[0] : 0;
    q.wins_t = out_stride(d->windows, 1, d->dim);
  }
  q.io_bf16 = d->x.dtype == SSM_BF16;
  q.y_f32 = d->y.dtype == SSM_F32;
  q.silu = (d->flags & SSM_SILU) != 0;
  return hip_status(ssm::launch_conv_packed(q, (hipStream_t)hip_stream));
}

ssm_status ssm_causal_conv1d_bwd_workspace_size(const ssm_conv_bwd_desc* d, size_t* bytes) {
  if (!bytes) return SSM_ERR_NULL;
  SSM_TRY(validate_conv_bwd(d));
  *bytes = (size_t)conv_bwd_bytes(*d);
  return SSM_OK;
}

ssm_status ssm_causal_conv1d_bwd(const ssm_conv_bwd_desc* d, const ssm_conv_bwd_ptrs* p, void* workspace,
                                 size_t workspace_bytes, void* hip_stream) {
  SSM_TRY(validate_conv_bwd(d));
  if (!p) return SSM_ERR_NULL;
  const bool bias = d->flags & SSM_HAS_BIAS;
  const int64_t need = conv_bwd_bytes(*d);
  Ptrs a;
  SSM_TRY(a.in(true, d->dy, p->dy));
  SSM_TRY(a.in(true, d->x, p->x));
  SSM_TRY(a.in(true, d->weight, p->weight));
  SSM_TRY(a.in(bias, d->bias, p->bias));
  SSM_TRY(a.out(true, d->dx, p->dx));
  SSM_TRY(a.out(true, d->dweight, p->dweight));
  SSM_TRY(a.out(bias, d->dbias, p->dbias));
  SSM_TRY(a.check(span_bytes(workspace, need)));
  if (!workspace || workspace_bytes < (size_t)need) return SSM_ERR_WORKSPACE;
  if (!aligned(workspace, 256)) return SSM_ERR_ALIGN;
  ssm::ConvBwdParams q;
  std::memset(&q, 0, sizeof(q));
  auto time = [](const ssm_tensor_desc& t) { return t.shape[1] > 1 ? t.stride[1] : 0; };
  auto batch = [](const ssm_tensor_desc& t) { return t.shape[0] > 1 ? t.stride[0] : 0; };
  q.dy = p->dy; q.x = p->x; q.w = p->weight; q.dx = p->dx; q.dweight = p->dweight;
  q.bias = bias ? p->bias : nullptr;
  q.dbias = bias ? p->dbias : nullptr;
  q.part = (float*)workspace;
  q.batch = d->batch; q.L = d->seqlen; q.D = d->dim; q.W = d->width;
  q.dys_b = batch(d->dy); q.dys_t = time(d->dy);
  q.xs_b = batch(d->x); q.xs_t = time(d->x);
  q.dxs_b = batch(d->dx); q.dxs_t = time(d->dx);
  q.ws_d = d->weight.stride[0]; q.ws_k = d->weight.stride[1];
  if (bias) q.bs_d = d->bias.stride[0];
  q.io_bf16 = d->x.dtype == SSM_BF16;
  q.dy_f32 = d->dy.dtype == SSM_F32;
  q.dx_f32 = d->dx.dtype == SSM_F32;
  q.silu = (d->flags & SSM_SILU) != 0;
  return hip_status(ssm::launch_conv_bwd(q, (hipStream_t)hip_stream));
}

ssm_status ssm_selective_scan_packed_workspace_size(const ssm_scan_packed_desc* d, size_t* bytes) {
  if (!bytes) return SSM_ERR_NULL;
  SSM_TRY(validate_scan_packed(d));
  *bytes = (size_t)plan_packed(*d).ws_total;
  return SSM_OK;
}

ssm_status ssm_selective_scan_packed(const ssm_scan_packed_desc* d, const ssm_scan_packed_ptrs* p, void* workspace,
                                     size_t workspace_bytes, void* hip_stream) {
  SSM_TRY(validate_scan_packed(d));
  if (!p) return SSM_ERR_NULL;
  const uint32_t f = d->flags;
  const ssm::ScanPackedPlan pl = plan_packed(*d);
  Ptrs a;
  SSM_TRY(a.in(true, d->x, p->x));
  SSM_TRY(a.in(true, d->delta, p->delta));
  SSM_TRY(a.in(true, d->A, p->A));
  SSM_TRY(a.in(true, d->B, p->B));
  SSM_TRY(a.in(true, d->C, p->C));
  SSM_TRY(a.in(f & SSM_HAS_D, d->D, p->D));
  SSM_TRY(a.in(f & SSM_HAS_Z, d->z, p->z));
  SSM_TRY(a.in(f & SSM_HAS_DELTA_BIAS, d->delta_bias, p->delta_bias));
  SSM_TRY(take_packed(*d, *p, a));
  SSM_TRY(a.out(true, d->y, p->y));
  SSM_TRY(a.out(f & SSM_HAS_STATES, d->states, p->states));
  SSM_TRY(a.check(pl.ws_total ? span_bytes(workspace, pl.ws_total) : Span()));
  if (pl.ws_total && (!workspace || workspace_bytes < (size_t)pl.ws_total)) return SSM_ERR_WORKSPACE;
  if (pl.ws_total && !aligned(workspace, 256)) return SSM_ERR_ALIGN;
  ssm::ScanPackedParams q;
  std::memset(&q, 0, sizeof(q));
  auto row = [](const ssm_tensor_desc& t) { return t.shape[0] > 1 ? t.stride[0] : 0; };
  q.q = packed_seqs(*d, *p);
  q.x = p->x; q.delta = p->delta; q.A = p->A; q.B = p->B; q.C = p->C; q.y = p->y;
  q.D = d->dim; q.N = d->dstate;
  q.xs_t = row(d->x); q.ds_t = row(d->delta);
  q.ys_t = out_stride(d->y, 0, d->dim);
  q.Bs_t = row(d->B); q.Bs_n = d->B.stride[1];
  q.Cs_t = row(d->C); q.Cs_n = d->C.stride[1];
  q.As_d = d->A.stride[0]; q.As_n = d->A.stride[1];
  if (f & SSM_HAS_Z) { q.z = p->z; q.zs_t = row(d->z); }
  if (f & SSM_HAS_D) { q.Dskip = p->D; q.Ds_d = d->D.stride[0]; }
  if (f & SSM_HAS_DELTA_BIAS) { q.dbias = p->delta_bias; q.dbs_d = d->delta_bias.stride[0]; }
  if (f & SSM_HAS_STATES) { q.states = p->states; q.sts_s = d->slots > 1 ? d->states.stride[0] : 0; }
  q.io_bf16 = d->x.dtype == SSM_BF16;
  q.y_f32 = d->y.dtype == SSM_F32;
  q.euler = (f & SSM_DISC_EULER) != 0;
  q.dsoftplus = (f & SSM_DELTA_SOFTPLUS) != 0;
  q.step = (int)pl.step;
  q.lines = (int)pl.lines;
  char* const w = (char*)workspace;
  if (pl.ws_order) q.order = (int*)(w + pl.ws_H + pl.ws_E + pl.ws_S);
  if (pl.lines) {
    q.H = (float*)w;
    q.E = (float*)(w + pl.ws_H);
    q.dsum = (float*)(w + pl.ws_H + pl.ws_E);
    q.esum = q.dsum + pl.lines * d->dim;
  }
  return hip_status(ssm::launch_scan_packed(q, (hipStream_t)hip_stream));
}

ssm_status ssm_beam_select_workspace_size(const ssm_beam_desc* d, size_t* bytes) {
  if (!bytes) return SSM_ERR_NULL;
  SSM_TRY(validate_beam(d));
  *bytes = (size_t)plan_beam(*d).ws_total;
  return SSM_OK;
}

ssm_status ssm_beam_select(const ssm_beam_desc* d, const ssm_beam_ptrs* p, void* workspace, size_t workspace_bytes,
                           void* hip_stream) {
  SSM_TRY(validate_beam(d));
  if (!p) return SSM_ERR_NULL;
  const BeamPlan pl = plan_beam(*d);
  Ptrs a;
  SSM_TRY(a.in(true, d->logits, p->logits));
  SSM_TRY(a.in(true, d->scores, p->scores));
  SSM_TRY(a.out(true, d->out_scores, p->out_scores));
  SSM_TRY(a.out(true, d->tokens, p->tokens));
  SSM_TRY(a.out(true, d->parents, p->parents));
  SSM_TRY(a.check(span_bytes(workspace, pl.ws_total)));
  if (!workspace || workspace_bytes < (size_t)pl.ws_total) return SSM_ERR_WORKSPACE;
  if (!aligned(workspace, 256)) return SSM_ERR_ALIGN;
  ssm::BeamParams q;
  std::memset(&q, 0, sizeof(q));
  q.logits = p->logits; q.scores = p->scores;
  q.out_scores = p->out_scores; q.tokens = p->tokens; q.parents = p->parents;
  q.batch = d->batch; q.beams = d->beams; q.V = d->vocab; q.k = (int)d->k;
  q.ls_b = d->logits.stride[0]; q.ls_n = d->logits.stride[1];
  q.ss_b = d->scores.stride[0]; q.ss_n = d->scores.stride[1];
  q.f32 = d->logits.dtype == SSM_F32;
  q.values = pl.cut.values;
  q.parts = (int)pl.cut.parts;
  q.cand = (uint64_t*)workspace;
  q.stat = (float2*)((char*)workspace + pl.ws_cand);
  return hip_status(ssm::launch_beam_select(q, (hipStream_t)hip_stream));
}

ssm_status ssm_state_move(const ssm_move_desc* d, const ssm_move_ptrs* p, void* hip_stream) {
  SSM_TRY(validate_move(d, p));
  ssm::MoveParams q;
  std::memset(&q, 0, sizeof(q));
  const int64_t e = esize(d->pool.dtype);
  q.pool = p->pool;
  q.src = p->src;
  q.dst = (d->flags & SSM_HAS_DST) ? p->dst : nullptr;
  q.slots = d->slots;
  q.row_bytes = d->row * e;
  q.slot_bytes = (d->slots > 1 ? d->pool.stride[0] : 0) * e;
  q.moves = (int)d->moves;
  return hip_status(ssm::launch_state_move(q, (hipStream_t)hip_stream));
}

}  // extern "C"
