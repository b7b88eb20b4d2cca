// Gated linear recurrence for gfx950: forward, backward and one-token step.
//
//   r = sigmoid(gate_a + bias_a), i = sigmoid(gate_x + bias_x)
//   a = exp(A r), s = sqrt(1 - a^2), h_t = a h_{t-1} + s i x, y = h silu(z)
//
// One fp32 state per channel and 6-8 transcendentals per element, so memory
// and VALU issue are close: every stream is read once and written once, and
// nothing is recomputed across workgroups unless the sequence is split.
//
// Time is parallel inside a workgroup.  A workgroup owns 64 channels (32
// lanes of two) and walks the sequence in rounds of 16 chunks; each half-wave
// holds one chunk of T consecutive steps in registers.  It scans its chunk
// from zero to the pair (P, H) = (product of decays, end state), the pairs of
// the 16 chunks are exchanged through LDS, every lane folds them in order
//   h <- P h + H
// to the state that enters its chunk (and the state after the round), and the
// chunk is walked again from registers with the true state.  One barrier a
// round: the exchange buffer alternates.
//
// The backward runs the rounds from the end.  Forward states come from the
// checkpoints (every 64th step) and the same fold; the adjoint
//   lam_t = g_t + m_t,  m_{t-1} = a_t lam_t
// is affine in the carry m as well, with the same product P, and is folded
// from the other end in the same exchange.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "ssm_internal.h"

namespace ssm {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int LC = kGatedLanes;
constexpr int NCH = kGatedChunks;
constexpr int NT = LC * NCH;
constexpr int kFwdT = kGatedFwdSteps;
constexpr int kBwdT = kGatedBwdSteps;
constexpr int kBwdRound = NCH * kBwdT;
static_assert(kGatedCkptSteps % kFwdT == 0 && (NCH * kFwdT) % kGatedCkptSteps == 0, "checkpoints fall on chunks");
static_assert(kBwdRound % kGatedCkptSteps == 0, "every backward round starts at a checkpoint");
static_assert(kGatedRound % kBwdRound == 0, "segments hold whole rounds of both passes");

constexpr uint32_t kRsrcWord3 = 0x00020000u;  // raw (unformatted) buffer access
constexpr uint32_t kMaxRange = 0x40000000u;   // the host keeps a round's rows below this
constexpr uint32_t kFar = 0x7FFFFFF0u;        // past every range: loads give 0, stores are dropped

__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc(const void* p, int64_t bytes) {
  const uint32_t range = bytes < (int64_t)kMaxRange ? (uint32_t)bytes : kMaxRange;
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), (short)0, (int)range, (int)kRsrcWord3);
}

// The rows [t, L) of channels [c, D) of batch row b, as one buffer.  A round
// that lies inside the sequence addresses only rows of it; one that crosses
// its end sends the rows behind it to kFar.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rows_from(const void* p, int64_t sb, int64_t st, int64_t b,
                                                            int64_t t, int64_t c, int64_t L, int64_t D, int e) {
  return rsrc((const char*)p + (b * sb + t * st + c) * e, ((L - 1 - t) * st + (D - c)) * e);
}

// V channels of one row as loaded: bf16 pairs or fp32.
template <bool BF16, int V>
struct Raw {
  uint32_t w[BF16 ? (V + 1) / 2 : V];
};

// Byte offset of a row of the round: the lane's own offset `off` and the row's
// `row` (block-uniform, in a scalar register).
template <bool BF16, int V>
__device__ __forceinline__ Raw<BF16, V> load(__amdgpu_buffer_rsrc_t r, uint32_t off, uint32_t row) {
  Raw<BF16, V> o;
  if constexpr (BF16 && V == 1) {
    o.w[0] = __builtin_amdgcn_raw_buffer_load_b16(r, (int)off, (int)row, 0);
  } else if constexpr (BF16 || V == 1) {
    o.w[0] = __builtin_amdgcn_raw_buffer_load_b32(r, (int)off, (int)row, 0);
  } else {
    const auto v = __builtin_amdgcn_raw_buffer_load_b64(r, (int)off, (int)row, 0);
    o.w[0] = v[0];
    o.w[1] = v[1];
  }
  return o;
}

template <bool BF16, int V>
__device__ __forceinline__ float elem(const Raw<BF16, V>& r, int v) {
  if constexpr (BF16) return __uint_as_float(v ? (r.w[0] & 0xFFFF0000u) : (r.w[0] << 16));
  else return __uint_as_float(r.w[v]);
}

typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef float f32x2_t __attribute__((ext_vector_type(2)));
typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));

template <bool F32, int V>
__device__ __forceinline__ void store(__amdgpu_buffer_rsrc_t r, uint32_t off, uint32_t row, const float (&o)[V]) {
  if constexpr (F32 && V == 2) {
    const u32x2_t w = {__float_as_uint(o[0]), __float_as_uint(o[1])};
    __builtin_amdgcn_raw_buffer_store_b64(w, r, (int)off, (int)row, 0);
  } else if constexpr (F32) {
    __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(o[0]), r, (int)off, (int)row, 0);
  } else if constexpr (V == 2) {
    const f32x2_t w = {o[0], o[1]};
    __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(uint32_t, __builtin_convertvector(w, bf16x2_t)), r,
                                          (int)off, (int)row, 0);
  } else {
    __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(uint16_t, (__bf16)o[0]), r, (int)off, (int)row, 0);
  }
}

// sigmoid(g + bias) with nb = -bias log2(e); both ends are reached exactly
// (exp2 overflows to infinity, whose reciprocal is 0).
__device__ __forceinline__ float gate(float g, float nb) {
  return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(__builtin_fmaf(g, -kLog2e, nb)));
}

// 1 - a^2 for a = 2^t, at least 0.  Near a = 1 the difference cancels, so for
// |t| < 1/4 it is t q(t), q the degree-4 polynomial through (1 - 4^t) / t at
// the Chebyshev nodes of [-1/4, 0] (relative error 2.7e-8); beyond, the
// difference loses less than two bits.
__device__ __forceinline__ float one_minus_sq(float t, float a) {
  float q = -0.03698064f;
  q = __builtin_fmaf(q, t, -0.15267968f);
  q = __builtin_fmaf(q, t, -0.44392627f);
  q = __builtin_fmaf(q, t, -0.96090275f);
  q = __builtin_fmaf(q, t, -1.38629436f);
  const float d = __builtin_fmaf(-a, a, 1.f);
  return fmaxf(fabsf(t) < 0.25f ? t * q : d, 0.f);
}

// The per-channel constants of a lane.
template <int V>
struct Chan {
  float al2[V], nba[V], nbx[V];  // A log2(e), -bias_a log2(e), -bias_x log2(e)

  template <class P>
  __device__ __forceinline__ void load(const P& p, int64_t c, bool ok) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      al2[v] = ok ? p.A[(c + v) * p.As_d] * kLog2e : 0.f;
      nba[v] = ok && p.bias_a ? p.bias_a[(c + v) * p.bas_d] * -kLog2e : 0.f;
      nbx[v] = ok && p.bias_x ? p.bias_x[(c + v) * p.bxs_d] * -kLog2e : 0.f;
    }
  }
};

__device__ __forceinline__ int clamp_steps(int64_t n, int T) { return n < 0 ? 0 : n > T ? T : (int)n; }

__device__ __forceinline__ int64_t row_len(const GatedParams& p, int64_t b) {
  if (!p.lens) return p.L;
  const int64_t n = p.lens[b];
  return n < 0 ? 0 : n > p.L ? p.L : n;
}

// One stream of a tile: its buffer for a round, the lane's offset of the first
// row of its chunk and the row stride, in bytes.
struct Stream {
  __amdgpu_buffer_rsrc_t r;
  uint32_t off, row;

  // T: steps per chunk, e: bytes per element; `ok` is false for the lanes
  // behind the last channel
  __device__ __forceinline__ void set(const void* p, int64_t sb, int64_t st, int64_t b, int64_t t0, int64_t c0,
                                      int64_t L, int64_t D, int e, int T, int chunk, int lane_elem, bool ok) {
    r = rows_from(p, sb, st, b, t0, c0, L, D, e);
    row = (uint32_t)(st * e);
    off = ok ? (uint32_t)(chunk * T) * row + (uint32_t)(lane_elem * e) : kFar;
  }
};

// Row j of the chunk; with MASK rows from `n` on are sent out of range.
template <bool MASK, bool BF16, int V>
__device__ __forceinline__ Raw<BF16, V> load_row(const Stream& s, int j, int n) {
  if constexpr (MASK) return load<BF16, V>(s.r, j < n ? s.off + (uint32_t)j * s.row : kFar, 0);
  else return load<BF16, V>(s.r, s.off, (uint32_t)j * s.row);
}

template <bool MASK, bool F32, int V>
__device__ __forceinline__ void store_row(const Stream& s, int j, int n, const float (&o)[V]) {
  if constexpr (MASK) store<F32, V>(s.r, j < n && s.off != kFar ? s.off + (uint32_t)j * s.row : kFar, 0, o);
  else store<F32, V>(s.r, s.off, (uint32_t)j * s.row, o);
}

// ------------------------------------------------------------------- forward
// kOut writes y (and h_last, checkpoints); kCkpt only the checkpoints; kAgg
// only the pair (P, H) of segments 0 .. n_seg-2 of a split sequence.
enum Mode { kOut, kCkpt, kAgg };

template <bool BF16, bool YF32, bool Z, int V, Mode M>
struct Fwd {
  static constexpr int E = BF16 ? 2 : 4;
  static constexpr int YE = (YF32 || !BF16) ? 4 : 2;
  static constexpr int T = kFwdT;
  typedef float2 Pairs[NCH][LC * V];

  const GatedParams& p;
  int64_t b, c0, c, len;
  int lane, chunk;
  bool ok;
  Chan<V> ch;
  float h[V], P[V];  // state at the start of the round; product of the decays so far (kAgg)

  __device__ __forceinline__ Fwd(const GatedParams& q) : p(q) {}

  template <bool MASK>
  __device__ __forceinline__ void round(int64_t t0, Pairs& lds) {
    Stream sx, sa, sg, sz, sy;
    sx.set(p.x, p.xs_b, p.xs_t, b, t0, c0, p.L, p.D, E, T, chunk, lane * V, ok);
    sa.set(p.gate_a, p.gas_b, p.gas_t, b, t0, c0, p.L, p.D, E, T, chunk, lane * V, ok);
    sg.set(p.gate_x, p.gxs_b, p.gxs_t, b, t0, c0, p.L, p.D, E, T, chunk, lane * V, ok);
    const int64_t t = t0 + chunk * T;
    const int rows = MASK ? clamp_steps(p.L - t, T) : T;   // rows of the chunk inside the sequence
    const int live = MASK ? clamp_steps(len - t, T) : T;   // steps that count
    Raw<BF16, V> xr[T], ar[T], gr[T], zr[Z && M == kOut ? T : 1];
#pragma unroll
    for (int j = 0; j < T; ++j) {
      ar[j] = load_row<MASK, BF16, V>(sa, j, live);
      gr[j] = load_row<MASK, BF16, V>(sg, j, live);
      xr[j] = load_row<MASK, BF16, V>(sx, j, live);
    }
    if constexpr (Z && M == kOut) {
      sz.set(p.z, p.zs_b, p.zs_t, b, t0, c0, p.L, p.D, E, T, chunk, lane * V, ok);
#pragma unroll
      for (int j = 0; j < T; ++j) zr[j] = load_row<MASK, BF16, V>(sz, j, live);
    }
    float a[T][V], u[T][V], cp[V], cH[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      cp[v] = 1.f;
      cH[v] = 0.f;
    }
#pragma unroll
    for (int j = 0; j < T; ++j)
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const float r = gate(elem(ar[j], v), ch.nba[v]);
        const float i = gate(elem(gr[j], v), ch.nbx[v]);
        const float e = r * ch.al2[v];
        a[j][v] = __builtin_amdgcn_exp2f(e);
        u[j][v] = __builtin_amdgcn_sqrtf(one_minus_sq(e, a[j][v])) * (i * elem(xr[j], v));
        if (MASK && j >= live) {
          a[j][v] = 1.f;
          u[j][v] = 0.f;
        }
        cp[v] *= a[j][v];
        cH[v] = __builtin_fmaf(a[j][v], cH[v], u[j][v]);
      }
#pragma unroll
    for (int v = 0; v < V; ++v) lds[chunk][lane * V + v] = make_float2(cp[v], cH[v]);
    __syncthreads();
    float in[V];
#pragma unroll
    for (int k = 0; k < NCH; ++k)
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const float2 w = lds[k][lane * V + v];
        if (k == chunk) in[v] = h[v];
        h[v] = __builtin_fmaf(w.x, h[v], w.y);
        if constexpr (M == kAgg) P[v] *= w.x;
      }
    if constexpr (M != kAgg) {
      if (p.ckpt && (chunk * T) % kGatedCkptSteps == 0 && ok && rows > 0) {
        const int64_t nk = (p.L + kGatedCkptSteps - 1) / kGatedCkptSteps;
#pragma unroll
        for (int v = 0; v < V; ++v) p.ckpt[(b * nk + t / kGatedCkptSteps) * p.D + c + v] = in[v];
      }
    }
    if constexpr (M == kOut) {
      sy.set(p.y, p.ys_b, p.ys_t, b, t0, c0, p.L, p.D, YE, T, chunk, lane * V, ok);
#pragma unroll
      for (int j = 0; j < T; ++j) {
        float o[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
          in[v] = __builtin_fmaf(a[j][v], in[v], u[j][v]);
          o[v] = in[v];
          if constexpr (Z) {
            const float z = elem(zr[j], v);
            o[v] *= z * gate(z, 0.f);
          }
          if (MASK && j >= live) o[v] = 0.f;
        }
        store_row<MASK, YF32 || !BF16, V>(sy, j, rows, o);
      }
    }
  }
};

template <bool BF16, bool YF32, bool Z, int V, Mode M>
__global__ __launch_bounds__(NT) void gated_fwd_kernel(GatedParams p, unsigned tiles) {
  typedef Fwd<BF16, YF32, Z, V, M> F;
  constexpr int R = NCH * kFwdT;
  __shared__ typename F::Pairs lds[2];
  const int nseg = M == kAgg ? p.n_seg - 1 : p.n_seg;
  const unsigned tile = blockIdx.x % tiles;
  const int64_t rest = blockIdx.x / tiles;
  const int seg = (int)(rest % nseg);
  F f(p);
  f.b = rest / nseg;
  f.lane = threadIdx.x % LC;
  f.chunk = threadIdx.x / LC;
  f.c0 = (int64_t)tile * LC * V;
  f.c = f.c0 + f.lane * V;
  f.ok = f.c < p.D;  // with V == 2 the channels are even: a lane is all in or all out
  f.len = row_len(p, f.b);
  f.ch.load(p, f.c, f.ok);
#pragma unroll
  for (int v = 0; v < V; ++v) {
    f.P[v] = 1.f;
    f.h[v] = M != kAgg && p.h0 && f.ok ? p.h0[f.b * p.D + f.c + v] : 0.f;
  }
  if constexpr (M != kAgg) {
    for (int s = 0; s < seg; ++s)  // the state that enters the segment
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (f.ok) {
          const float2 w = p.agg[(f.b * (p.n_seg - 1) + s) * p.D + f.c + v];
          f.h[v] = __builtin_fmaf(w.x, f.h[v], w.y);
        }
  }
  const int64_t ts = (int64_t)seg * p.seg_len;
  const int64_t te = min(p.L, ts + p.seg_len);
  int buf = 0;
  for (int64_t t0 = ts; t0 < te; t0 += R, buf ^= 1) {
    if (t0 + R <= f.len) f.template round<false>(t0, lds[buf]);
    else f.template round<true>(t0, lds[buf]);
  }
  if (f.chunk == 0 && f.ok) {
    if constexpr (M == kAgg) {
#pragma unroll
      for (int v = 0; v < V; ++v)
        p.agg[(f.b * (p.n_seg - 1) + seg) * p.D + f.c + v] = make_float2(f.P[v], f.h[v]);
    } else if (p.h_last && seg == p.n_seg - 1) {
#pragma unroll
      for (int v = 0; v < V; ++v) p.h_last[f.b * p.D + f.c + v] = f.h[v];
    }
  }
}

// ------------------------------------------------------------------ backward
// kGrads writes the gradients; kCarry only (P, O) of segments 1 .. n_seg-1 of
// a split sequence: the carry out of a segment is P carry_in + O.
enum BwdMode { kGrads, kCarry };

template <bool BF16, bool GF32, bool Z, int V, BwdMode M>
struct Bwd {
  static constexpr int E = BF16 ? 2 : 4;
  static constexpr bool G32 = GF32 || !BF16;
  static constexpr int GE = G32 ? 4 : 2;
  static constexpr int T = kBwdT;
  // decay product, end state from zero, carry out from a zero carry in
  struct Agg {
    float P[NCH][LC * V], H[NCH][LC * V], O[NCH][LC * V];
  };

  const GatedBwdParams& q;
  const GatedParams& p;
  int64_t b, c0, c, len;
  int lane, chunk;
  bool ok;
  Chan<V> ch;
  float A[V];
  float m[V], P[V];                 // carry into the round's last step; decay product so far (kCarry)
  float sA[V], sba[V], sbx[V];      // sums of dA, dgate_a, dgate_x over the lane's steps

  __device__ __forceinline__ Bwd(const GatedBwdParams& w) : q(w), p(w.f) {}

  template <bool MASK>
  __device__ __forceinline__ void round(int64_t t0, Agg& lds) {
    Stream sx, sa, sg, sz, sd;
    const int64_t t = t0 + chunk * T;
    const int rows = MASK ? clamp_steps(p.L - t, T) : T;
    const int live = MASK ? clamp_steps(len - t, T) : T;
    sa.set(p.gate_a, p.gas_b, p.gas_t, b, t0, c0, p.L, p.D, E, T, chunk, lane * V, ok);
    sd.set(q.dy, q.dys_b, q.dys_t, b, t0, c0, p.L, p.D, GE, T, chunk, lane * V, ok);
    if constexpr (Z) sz.set(p.z, p.zs_b, p.zs_t, b, t0, c0, p.L, p.D, E, T, chunk, lane * V, ok);
    Raw<BF16, V> xr[T], ar[T], gr[T], zr[Z ? T : 1];
    Raw<!G32, V> dr[T];
#pragma unroll
    for (int j = 0; j < T; ++j) {
      ar[j] = load_row<MASK, BF16, V>(sa, j, live);
      dr[j] = load_row<MASK, !G32, V>(sd, j, live);
      if constexpr (Z) zr[j] = load_row<MASK, BF16, V>(sz, j, live);
    }
    float c_in[V];  // state that enters the round
    if constexpr (M == kGrads) {
      sx.set(p.x, p.xs_b, p.xs_t, b, t0, c0, p.L, p.D, E, T, chunk, lane * V, ok);
      sg.set(p.gate_x, p.gxs_b, p.gxs_t, b, t0, c0, p.L, p.D, E, T, chunk, lane * V, ok);
#pragma unroll
      for (int j = 0; j < T; ++j) {
        gr[j] = load_row<MASK, BF16, V>(sg, j, live);
        xr[j] = load_row<MASK, BF16, V>(sx, j, live);
      }
      const int64_t nk = (p.L + kGatedCkptSteps - 1) / kGatedCkptSteps;
#pragma unroll
      for (int v = 0; v < V; ++v) c_in[v] = ok ? p.ckpt[(b * nk + t0 / kGatedCkptSteps) * p.D + c + v] : 0.f;
    }
    // a, the input s i x (later the state before the step), g, r, i, 1 / s and 1 - a^2 of every step
    float a[T][V], u[T][V], g[T][V], r[T][V], i[T][V], is[T][V], om[T][V], zf[Z && M == kGrads ? T : 1][V];
    float cp[V], cH[V], cM[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      cp[v] = 1.f;
      cH[v] = cM[v] = 0.f;
    }
#pragma unroll
    for (int j = 0; j < T; ++j)
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const bool dead = MASK && j >= live;
        r[j][v] = gate(elem(ar[j], v), ch.nba[v]);
        const float e = r[j][v] * ch.al2[v];
        a[j][v] = __builtin_amdgcn_exp2f(e);
        const float dy = elem(dr[j], v);
        g[j][v] = dy;
        if constexpr (Z) {
          const float z = elem(zr[j], v), sz_ = gate(z, 0.f);
          g[j][v] = dy * (z * sz_);
          if constexpr (M == kGrads) zf[j][v] = dy * (sz_ * __builtin_fmaf(z, 1.f - sz_, 1.f));
        }
        if constexpr (M == kGrads) {
          i[j][v] = gate(elem(gr[j], v), ch.nbx[v]);
          om[j][v] = one_minus_sq(e, a[j][v]);
          is[j][v] = om[j][v] > 0.f ? __builtin_amdgcn_rsqf(om[j][v]) : 0.f;
          u[j][v] = om[j][v] * is[j][v] * (i[j][v] * elem(xr[j], v));
        }
        if (dead) {
          a[j][v] = 1.f;
          g[j][v] = 0.f;
          if constexpr (M == kGrads) u[j][v] = 0.f;
        }
        cp[v] *= a[j][v];
        if constexpr (M == kGrads) cH[v] = __builtin_fmaf(a[j][v], cH[v], u[j][v]);
      }
#pragma unroll
    for (int j = T - 1; j >= 0; --j)
#pragma unroll
      for (int v = 0; v < V; ++v) cM[v] = a[j][v] * (g[j][v] + cM[v]);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      lds.P[chunk][lane * V + v] = cp[v];
      lds.O[chunk][lane * V + v] = cM[v];
      if constexpr (M == kGrads) lds.H[chunk][lane * V + v] = cH[v];
    }
    __syncthreads();
    float mi[V];  // carry into the chunk's last step
#pragma unroll
    for (int k = NCH - 1; k >= 0; --k)
#pragma unroll
      for (int v = 0; v < V; ++v) {
        if (k == chunk) mi[v] = m[v];
        const float w = lds.P[k][lane * V + v];
        m[v] = __builtin_fmaf(w, m[v], lds.O[k][lane * V + v]);
        if constexpr (M == kCarry) P[v] *= w;
      }
    if constexpr (M == kGrads) {
      float h[V];
#pragma unroll
      for (int k = 0; k < NCH; ++k)
#pragma unroll
        for (int v = 0; v < V; ++v) {
          if (k == chunk) h[v] = c_in[v];
          c_in[v] = __builtin_fmaf(lds.P[k][lane * V + v], c_in[v], lds.H[k][lane * V + v]);
        }
      Stream so;
      if constexpr (Z) so.set(q.dz, q.dzs_b, q.dzs_t, b, t0, c0, p.L, p.D, GE, T, chunk, lane * V, ok);
#pragma unroll
      for (int j = 0; j < T; ++j) {
        float o[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const float hn = __builtin_fmaf(a[j][v], h[v], u[j][v]);
          u[j][v] = h[v];
          h[v] = hn;
          if constexpr (Z) o[v] = MASK && j >= live ? 0.f : hn * zf[j][v];
        }
        if constexpr (Z) store_row<MASK, G32, V>(so, j, rows, o);
      }
      Stream dx, da, dg;
      dx.set(q.dx, q.dxs_b, q.dxs_t, b, t0, c0, p.L, p.D, GE, T, chunk, lane * V, ok);
      da.set(q.dgate_a, q.dgas_b, q.dgas_t, b, t0, c0, p.L, p.D, GE, T, chunk, lane * V, ok);
      dg.set(q.dgate_x, q.dgxs_b, q.dgxs_t, b, t0, c0, p.L, p.D, GE, T, chunk, lane * V, ok);
#pragma unroll
      for (int j = T - 1; j >= 0; --j) {
        float ox[V], oa[V], og[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const float x = elem(xr[j], v);
          const float lam = g[j][v] + mi[v];
          mi[v] = a[j][v] * lam;
          // du = lam (a h_{t-1} - i x a^2 / s)
          const float du = mi[v] * (u[j][v] - i[j][v] * x * a[j][v] * is[j][v]);
          const float dv = lam * (om[j][v] * is[j][v]);
          ox[v] = dv * i[j][v];
          oa[v] = du * A[v] * __builtin_fmaf(-r[j][v], r[j][v], r[j][v]);
          og[v] = dv * x * __builtin_fmaf(-i[j][v], i[j][v], i[j][v]);
          float dA = du * r[j][v];
          if (MASK && j >= live) ox[v] = oa[v] = og[v] = dA = 0.f;
          sA[v] += dA;
          sba[v] += oa[v];
          sbx[v] += og[v];
        }
        store_row<MASK, G32, V>(dx, j, rows, ox);
        store_row<MASK, G32, V>(da, j, rows, oa);
        store_row<MASK, G32, V>(dg, j, rows, og);
      }
    }
  }
};

template <bool BF16, bool GF32, bool Z, int V, BwdMode M>
__global__ __launch_bounds__(NT) void gated_bwd_kernel(GatedBwdParams q, unsigned tiles) {
  typedef Bwd<BF16, GF32, Z, V, M> F;
  constexpr int R = kBwdRound;
  __shared__ typename F::Agg lds[2];
  const GatedParams& p = q.f;
  const int nseg = M == kCarry ? p.n_seg - 1 : p.n_seg;
  const unsigned tile = blockIdx.x % tiles;
  const int64_t rest = blockIdx.x / tiles;
  const int part = (int)(rest % nseg);
  const int seg = M == kCarry ? part + 1 : part;
  F f(q);
  f.b = rest / nseg;
  f.lane = threadIdx.x % LC;
  f.chunk = threadIdx.x / LC;
  f.c0 = (int64_t)tile * LC * V;
  f.c = f.c0 + f.lane * V;
  f.ok = f.c < p.D;
  f.len = row_len(p, f.b);
  f.ch.load(p, f.c, f.ok);
#pragma unroll
  for (int v = 0; v < V; ++v) {
    f.A[v] = f.ok ? p.A[(f.c + v) * p.As_d] : 0.f;
    f.P[v] = 1.f;
    f.m[v] = M == kGrads && q.dh_last && f.ok ? q.dh_last[f.b * p.D + f.c + v] : 0.f;
    f.sA[v] = f.sba[v] = f.sbx[v] = 0.f;
  }
  if constexpr (M == kGrads) {
    for (int s = p.n_seg - 1; s > seg; --s)  // the carry that comes in from the later segments
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (f.ok) {
          const float2 w = q.agg[(f.b * (p.n_seg - 1) + s - 1) * p.D + f.c + v];
          f.m[v] = __builtin_fmaf(w.x, f.m[v], w.y);
        }
  }
  const int64_t ts = (int64_t)seg * p.seg_len;
  const int64_t te = min(p.L, ts + p.seg_len);
  int buf = 0;
  for (int64_t t0 = ts + (te - 1 - ts) / R * R; t0 >= ts; t0 -= R, buf ^= 1) {
    if (t0 + R <= f.len) f.template round<false>(t0, lds[buf]);
    else f.template round<true>(t0, lds[buf]);
  }
  if constexpr (M == kCarry) {
    if (f.chunk == 0 && f.ok)
#pragma unroll
      for (int v = 0; v < V; ++v)
        q.agg[(f.b * (p.n_seg - 1) + part) * p.D + f.c + v] = make_float2(f.P[v], f.m[v]);
  } else {
    if (q.dh0 && seg == 0 && f.chunk == 0 && f.ok)
#pragma unroll
      for (int v = 0; v < V; ++v) q.dh0[f.b * p.D + f.c + v] = f.m[v];
    // the 16 chunks' sums, added in order by the first chunk's lanes
    __syncthreads();
    typename F::Agg& w = lds[0];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      w.P[f.chunk][f.lane * V + v] = f.sA[v];
      w.H[f.chunk][f.lane * V + v] = f.sba[v];
      w.O[f.chunk][f.lane * V + v] = f.sbx[v];
    }
    __syncthreads();
    if (f.chunk < 3 && f.ok) {
      const auto& from = f.chunk == 0 ? w.P : f.chunk == 1 ? w.H : w.O;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        float sum = 0.f;
#pragma unroll
        for (int k = 0; k < NCH; ++k) sum += from[k][f.lane * V + v];
        q.part[((f.b * p.n_seg + seg) * 3 + f.chunk) * p.D + f.c + v] = sum;
      }
    }
  }
}

// dA, dbias_a, dbias_x: the partial sums of every (row, segment) in a fixed
// order: 8 interleaved runs per channel, then the runs.
__global__ __launch_bounds__(256) void gated_sums_kernel(const float* part, int64_t parts, int64_t D, float* dA,
                                                         float* dba, float* dbx) {
  __shared__ float lds[8][32];
  const int lane = threadIdx.x % 32, run = threadIdx.x / 32;
  const int64_t c = (int64_t)blockIdx.x * 32 + lane;
  float* const out = blockIdx.y == 0 ? dA : blockIdx.y == 1 ? dba : dbx;
  if (!out) return;  // block-uniform
  float sum = 0.f;
  if (c < D)
    for (int64_t k = run; k < parts; k += 8) sum += part[(k * 3 + blockIdx.y) * D + c];
  lds[run][lane] = sum;
  __syncthreads();
  if (run == 0 && c < D) {
#pragma unroll
    for (int k = 1; k < 8; ++k) sum += lds[k][lane];
    out[c] = sum;
  }
}

// ---------------------------------------------------------------- one token
// A thread owns V channels of one batch row: latency is everything, the
// traffic is one state in and out and four or five elements per channel.
template <bool BF16, bool YF32, int V>
__global__ __launch_bounds__(256) void gated_update_kernel(GatedUpdateParams p, unsigned tiles) {
  constexpr int E = BF16 ? 2 : 4;
  const int64_t b = blockIdx.x / tiles;
  const int64_t c = ((int64_t)(blockIdx.x % tiles) * 256 + threadIdx.x) * V;
  if (c >= p.D) return;
  auto read = [&](const void* base, int64_t sb) {
    Raw<BF16, V> o;
    const char* at = (const char*)base + (b * sb + c) * E;
    if constexpr (BF16 && V == 1) o.w[0] = *(const uint16_t*)at;
    else if constexpr (BF16 || V == 1) o.w[0] = *(const uint32_t*)at;
    else {
      const uint2 w = *(const uint2*)at;
      o.w[0] = w.x;
      o.w[1] = w.y;
    }
    return o;
  };
  const Raw<BF16, V> xr = read(p.x, p.xs_b), ar = read(p.gate_a, p.gas_b), gr = read(p.gate_x, p.gxs_b);
  Raw<BF16, V> zr = {};
  if (p.z) zr = read(p.z, p.zs_b);
  Chan<V> ch;
  ch.load(p, c, true);
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const float r = gate(elem(ar, v), ch.nba[v]), i = gate(elem(gr, v), ch.nbx[v]);
    const float e = r * ch.al2[v], a = __builtin_amdgcn_exp2f(e);
    const float u = __builtin_amdgcn_sqrtf(one_minus_sq(e, a)) * (i * elem(xr, v));
    const float h = __builtin_fmaf(a, p.state[b * p.D + c + v], u);
    p.state_out[b * p.D + c + v] = h;
    float o = h;
    if (p.z) {
      const float z = elem(zr, v);
      o *= z * gate(z, 0.f);
    }
    if constexpr (YF32 || !BF16) ((float*)p.y)[b * p.ys_b + c + v] = o;
    else ((__bf16*)p.y)[b * p.ys_b + c + v] = (__bf16)o;
  }
}

// -------------------------------------------------------------------- launch
bool pair_rows(const void* ptr, int e, int64_t sb, int64_t st) {
  return (uintptr_t)ptr % (2 * e) == 0 && sb % 2 == 0 && st % 2 == 0;
}

template <bool BF16, bool YF32, bool Z, int V>
void launch_fwd(const GatedParams& p, hipStream_t stream) {
  const unsigned tiles = (unsigned)((p.D + LC * V - 1) / (LC * V));
  const unsigned rows = (unsigned)(tiles * p.batch);
  if (p.n_seg > 1)
    hipLaunchKernelGGL((gated_fwd_kernel<BF16, false, false, V, kAgg>), dim3(rows * (p.n_seg - 1)), dim3(NT), 0,
                       stream, p, tiles);
  if (p.y)
    hipLaunchKernelGGL((gated_fwd_kernel<BF16, YF32, Z, V, kOut>), dim3(rows * p.n_seg), dim3(NT), 0, stream, p,
                       tiles);
  else
    hipLaunchKernelGGL((gated_fwd_kernel<BF16, false, false, V, kCkpt>), dim3(rows * p.n_seg), dim3(NT), 0, stream,
                       p, tiles);
}

template <bool BF16, bool YF32, int V>
void launch_fwd_z(const GatedParams& p, hipStream_t stream) {
  if (p.z) launch_fwd<BF16, YF32, true, V>(p, stream);
  else launch_fwd<BF16, YF32, false, V>(p, stream);
}

template <int V>
void launch_fwd_io(const GatedParams& p, hipStream_t stream) {
  if (!p.io_bf16) launch_fwd_z<false, true, V>(p, stream);
  else if (p.y_f32) launch_fwd_z<true, true, V>(p, stream);
  else launch_fwd_z<true, false, V>(p, stream);
}

template <bool BF16, bool GF32, bool Z, int V>
void launch_bwd(const GatedBwdParams& q, hipStream_t stream) {
  const GatedParams& p = q.f;
  const unsigned tiles = (unsigned)((p.D + LC * V - 1) / (LC * V));
  const unsigned rows = (unsigned)(tiles * p.batch);
  if (p.n_seg > 1)
    hipLaunchKernelGGL((gated_bwd_kernel<BF16, GF32, Z, V, kCarry>), dim3(rows * (p.n_seg - 1)), dim3(NT), 0, stream,
                       q, tiles);
  hipLaunchKernelGGL((gated_bwd_kernel<BF16, GF32, Z, V, kGrads>), dim3(rows * p.n_seg), dim3(NT), 0, stream, q,
                     tiles);
  hipLaunchKernelGGL(gated_sums_kernel, dim3((unsigned)((p.D + 31) / 32), 3), dim3(256), 0, stream, q.part,
                     p.batch * p.n_seg, p.D, q.dA, q.dbias_a, q.dbias_x);
}

template <bool BF16, bool GF32, int V>
void launch_bwd_z(const GatedBwdParams& q, hipStream_t stream) {
  if (q.f.z) launch_bwd<BF16, GF32, true, V>(q, stream);
  else launch_bwd<BF16, GF32, false, V>(q, stream);
}

template <int V>
void launch_bwd_io(const GatedBwdParams& q, hipStream_t stream) {
  if (!q.f.io_bf16) launch_bwd_z<false, true, V>(q, stream);
  else if (q.g_f32) launch_bwd_z<true, true, V>(q, stream);
  else launch_bwd_z<true, false, V>(q, stream);
}

template <int V>
void launch_update(const GatedUpdateParams& p, hipStream_t stream) {
  const unsigned tiles = (unsigned)((p.D + 256 * V - 1) / (256 * V));
  const dim3 grid((unsigned)(tiles * p.batch));
  if (!p.io_bf16) hipLaunchKernelGGL((gated_update_kernel<false, true, V>), grid, dim3(256), 0, stream, p, tiles);
  else if (p.y_f32) hipLaunchKernelGGL((gated_update_kernel<true, true, V>), grid, dim3(256), 0, stream, p, tiles);
  else hipLaunchKernelGGL((gated_update_kernel<true, false, V>), grid, dim3(256), 0, stream, p, tiles);
}

}  // namespace

bool gated_pairs(const GatedParams& p) {
  const int e = p.io_bf16 ? 2 : 4, ye = p.y_f32 || !p.io_bf16 ? 4 : 2;
  return p.D % 2 == 0 && pair_rows(p.x, e, p.xs_b, p.xs_t) && pair_rows(p.gate_a, e, p.gas_b, p.gas_t) &&
         pair_rows(p.gate_x, e, p.gxs_b, p.gxs_t) && pair_rows(p.z, e, p.zs_b, p.zs_t) &&
         pair_rows(p.y, ye, p.ys_b, p.ys_t);
}

hipError_t launch_gated_scan(const GatedParams& p, hipStream_t stream) {
  if (gated_pairs(p)) launch_fwd_io<2>(p, stream);
  else launch_fwd_io<1>(p, stream);
  return hipGetLastError();
}

hipError_t launch_gated_scan_bwd(const GatedBwdParams& q, hipStream_t stream) {
  const int ge = q.g_f32 || !q.f.io_bf16 ? 4 : 2;
  const bool pairs = gated_pairs(q.f) && pair_rows(q.dy, ge, q.dys_b, q.dys_t) &&
                     pair_rows(q.dx, ge, q.dxs_b, q.dxs_t) && pair_rows(q.dgate_a, ge, q.dgas_b, q.dgas_t) &&
                     pair_rows(q.dgate_x, ge, q.dgxs_b, q.dgxs_t) && pair_rows(q.dz, ge, q.dzs_b, q.dzs_t);
  if (pairs) launch_bwd_io<2>(q, stream);
  else launch_bwd_io<1>(q, stream);
  return hipGetLastError();
}

hipError_t launch_gated_state_update(const GatedUpdateParams& p, hipStream_t stream) {
  const int e = p.io_bf16 ? 2 : 4;
  const bool pairs = p.D % 2 == 0 && pair_rows(p.x, e, p.xs_b, 0) && pair_rows(p.gate_a, e, p.gas_b, 0) &&
                     pair_rows(p.gate_x, e, p.gxs_b, 0) && pair_rows(p.z, e, p.zs_b, 0);
  if (pairs) launch_update<2>(p, stream);
  else launch_update<1>(p, stream);
  return hipGetLastError();
}

}  // namespace ssm
