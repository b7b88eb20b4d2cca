// Gated linear recurrence for gfx950: forward, backward and one-token step.
//
//   r = sigmoid(gate_a + bias_a), i = sigmoid(gate_x + bias_x)
//   a = exp(A r), s = sqrt(1 - a^2), h_t = a h_{t-1} + s i x, y = h silu(z)
//
// One fp32 state per channel and 6-8 transcendentals per element, so memory
// and VALU issue are close: every stream is read once and written once, and
// nothing is computed twice.
//
// A workgroup owns 64 channels (32 lanes of two) over one segment of 8
// chunks.  Each half-wave holds one chunk of T consecutive steps in registers
// and scans it from zero to the pair (P, H) = (product of decays, end state).
// The first wave, a channel a lane, folds the 8 pairs through LDS
//   h <- P h + H
// to the segment's own pair, finds the state that enters the segment, and
// hands every chunk the state that enters it; the chunks are then walked again
// from registers with the true state.
//
// The segments of one sequence run side by side.  A workgroup publishes its
// pair as soon as it has it and its end state once it knows the state that
// enters it, each in a word that says by itself whether it has been written.
// To find the entering state a workgroup goes back over its predecessors,
// four at a time, to the nearest published end state and folds the pairs
// since then forward from it: the same operations in the same order whichever
// state it finds, so the result does not depend on timing.  Workgroups are
// dispatched in order (a layer of all tiles after another, a tile always on
// the same XCD), so those waited for are running or done.  The wait is bounded
// all the same: a workgroup that runs out of polls computes the entering state
// itself, from the start of the sequence, by the same operations.
//
// The backward takes the segments from the end.  Forward states come from the
// checkpoints (every 64th step) and the same fold; the adjoint
//   lam_t = g_t + m_t,  m_{t-1} = a_t lam_t
// is affine in the carry m as well, with the same product P, and its carry is
// found among the later segments in the same way.
//
// Times here and below are of calls in a captured graph, replayed over sets of
// inputs that together exceed the last-level cache; a call is its fill, its
// kernel and, backward, its sums.  Forward 4 x 4096 x 5120 bf16 with z 196 us (4.3
// TB/s; VALU 55 % busy; 243 us with 16 chunks a segment and fewer waves), 1 x
// 131072 x 1536 fp32 634 us (5.1 TB/s); backward 8 x 2048 x 1536 bf16 with z 121 us
// (3.7 TB/s).
#include <hip/hip_runtime.h>

#include <algorithm>

#include "column_sums.h"
#include "layer_internal.h"

// A segment's pair comes out the same from every variant of a kernel: products
// and sums are contracted where an fma is written, nowhere else.
#pragma clang fp contract(off)

namespace ssm {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int LC = 32;  // lanes per chunk
constexpr int kFwdT = kGatedFwdSteps;
constexpr int kBwdT = kGatedBwdSteps;
constexpr int kFwdNT = LC * kGatedFwdChunks, kFwdSeg = kGatedFwdChunks * kFwdT;
constexpr int kBwdNT = LC * kGatedBwdChunks, kBwdSeg = kGatedBwdChunks * kBwdT;
// Waves per SIMD that the registers are cut to: 128 and 168 hold a chunk of
// two channels without a spill (4 x 4096 x 5120 forward at 3 waves: 247 us
// against 197); four streams of fp32 do not fit 128 (8 x 2048 x 1536 with z at 4
// waves: 114 us, at 3: 109).
constexpr int kFwdWaves = 4, kFwdWaves32 = 3, kBwdWaves = 3;
static_assert(kGatedCkptSteps % kFwdT == 0 && kFwdSeg % kGatedCkptSteps == 0, "checkpoints fall on chunks");
static_assert(kBwdSeg % kGatedCkptSteps == 0, "every backward segment starts at a checkpoint");
static_assert(kFwdSeg <= kGatedSpanSteps && kBwdSeg <= kGatedSpanSteps, "a segment's rows fit the offsets");

constexpr uint32_t kRsrcWord3 = 0x00020000u;  // raw (unformatted) buffer access
constexpr uint32_t kMaxRange = 0x40000000u;   // the host keeps a segment's rows below this
constexpr uint32_t kFar = 0x7FFFFFF0u;        // past every range: loads give 0, stores are dropped

__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc(const void* p, int64_t bytes) {
  const uint32_t range = bytes < (int64_t)kMaxRange ? (uint32_t)bytes : kMaxRange;
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), (short)0, (int)range, (int)kRsrcWord3);
}

// The rows [t, L) of channels [c, D) of batch row b, as one buffer.  A segment
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

// Byte offset of a row of the segment: the lane's own offset `off` and the row's
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
  // the clamps to [0, 1] are modifiers of the product and of the fma
  const float n = __builtin_amdgcn_fmed3f(t * q, 0.f, 1.f);
  const float d = __builtin_amdgcn_fmed3f(__builtin_fmaf(-a, a, 1.f), 0.f, 1.f);
  return fabsf(t) < 0.25f ? n : d;
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

// One stream of a tile: its buffer for a segment, the lane's offset of the first
// row of its chunk and the row stride, in bytes.
struct Stream {
  __amdgpu_buffer_rsrc_t r;
  uint32_t off, row, at;

  // T: steps per chunk, e: bytes per element; `ok` is false for the lanes
  // behind the last channel
  __device__ __forceinline__ void set(const void* p, int64_t sb, int64_t st, int64_t b, int64_t t0, int64_t c0,
                                      int64_t L, int64_t D, int e, int T, int chunk, int lane_elem, bool ok) {
    r = rows_from(p, sb, st, b, t0, c0, L, D, e);
    row = (uint32_t)(st * e);
    off = ok ? (uint32_t)(chunk * T) * row + (uint32_t)(lane_elem * e) : kFar;
    at = 0;
  }
  // The rows are walked one after another: `at` is the current one's offset.
  // Opaque to the compiler, which would otherwise compute the offsets of all
  // rows of all streams at once and spill the scalar registers.
  __device__ __forceinline__ void next() {
    at += row;
    asm volatile("" : "+s"(at));
  }
  __device__ __forceinline__ void last(int T) {
    at = (uint32_t)(T - 1) * row;
    asm volatile("" : "+s"(at));
  }
  __device__ __forceinline__ void prev() {
    at -= row;
    asm volatile("" : "+s"(at));
  }
};

// The current row, number j of the chunk, and on to the next; with MASK rows
// from `n` on are sent out of range.  The range check takes the scalar offset
// off the range, so that offset must stay below it: it does where the whole
// segment lies inside the sequence, and with MASK it is 0.
template <bool MASK, bool BF16, int V>
__device__ __forceinline__ Raw<BF16, V> load_row(Stream& s, int j, int n) {
  Raw<BF16, V> o;
  if constexpr (MASK) o = load<BF16, V>(s.r, j < n ? s.off + s.at : kFar, 0);
  else o = load<BF16, V>(s.r, s.off, s.at);
  s.next();
  return o;
}

template <bool MASK, bool F32, int V>
__device__ __forceinline__ void store_row(const Stream& s, int j, int n, const float (&o)[V]) {
  if constexpr (MASK) store<F32, V>(s.r, j < n ? s.off + s.at : kFar, 0, o);
  else store<F32, V>(s.r, s.off, s.at, o);
}

// What leaves a chunk or a segment with the pair (P, H) that h enters.  The
// product P of up to 128 decays passes the largest fp32 where A > 0 (no decay
// of A <= 0 does); a state of zero, which such decays leave at zero, stays so.
__device__ __forceinline__ float pass_on(float P, float h, float H) {
  return h == 0.f ? H : __builtin_fmaf(P, h, H);
}

// ------------------------------------------------------------------ segments
// Words of the segments of one sequence: agg holds (P, H) of a segment, inc
// its end state.  All bits set means not yet written (the launch fills them);
// a NaN that is published has other bits.
struct Chain {
  unsigned long long* agg;
  uint32_t* inc;
  int64_t step;  // words from one segment to the next
  int polls;     // bound of the wait
};

constexpr int kBack = 4;    // predecessors read at once
constexpr int kStack = 32;  // pairs kept while going back; a multiple of kBack

__device__ __forceinline__ uint32_t bits_of(float v) { return v != v ? 0x7FC00000u : __float_as_uint(v); }

__device__ __forceinline__ void publish_pair(const Chain& q, int64_t at, float P, float H) {
  const unsigned long long w = (unsigned long long)bits_of(H) << 32 | bits_of(P);
  __hip_atomic_store(q.agg + at, w, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

__device__ __forceinline__ void publish_state(const Chain& q, int64_t at, float h) {
  __hip_atomic_store(q.inc + at, bits_of(h), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// One wave, a channel per lane (`ok`: the lane has one): the state that enters
// segment k >= 1, whose word index is `at`.  False when the polls ran out.
template <int CW>
__device__ __forceinline__ bool entering(const Chain& q, int64_t k, int64_t at, bool ok, float2 (&stack)[kStack][CW],
                                         int lane, float& h) {
  int depth = 0, polls = q.polls;
  int64_t j = k - 1;
  at -= q.step;
  while (true) {
    uint32_t s[kBack];
    unsigned long long w[kBack];
#pragma unroll
    for (int i = 0; i < kBack; ++i) {
      const bool in = ok && j - i >= 0;
      s[i] = in ? __hip_atomic_load(q.inc + at - i * q.step, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) : 0u;
      w[i] = in ? __hip_atomic_load(q.agg + at - i * q.step, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) : 0ull;
    }
    int used = 0;
    bool found = false, stop = false;
#pragma unroll
    for (int i = 0; i < kBack; ++i)
      if (!found && !stop) {  // wave-uniform
        if (__all(s[i] != 0xFFFFFFFFu)) {
          found = true;
          h = __uint_as_float(s[i]);
        } else if (depth + used < kStack && __all((uint32_t)w[i] != 0xFFFFFFFFu)) {
          if (lane < CW)
            stack[depth + used][lane] = make_float2(__uint_as_float((uint32_t)w[i]),
                                                    __uint_as_float((uint32_t)(w[i] >> 32)));
          ++used;
        } else {
          stop = true;
        }
      }
    depth += used;
    j -= used;
    at -= used * q.step;
    if (found) break;
    if (used == 0) {
      if (--polls <= 0) return false;
      __builtin_amdgcn_s_sleep(2);
    }
  }
  // own writes of this lane: no barrier between them and these reads
  for (int d = depth - 1; d >= 0; --d)
    if (lane < CW) h = pass_on(stack[d][lane].x, h, stack[d][lane].y);
  return true;
}

// Fills the words: 16 bytes a thread.
__global__ __launch_bounds__(256) void gated_fill_kernel(uint4* words, int64_t n) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i < n) words[i] = uint4{0xFFFFFFFFu, 0xFFFFFFFFu, 0xFFFFFFFFu, 0xFFFFFFFFu};
}

// Where a workgroup is: tile, batch row, segment, and the lane's place in it.
// grid.x holds all tiles of all rows (padded to a multiple of 8, so that a
// tile keeps its XCD from segment to segment), grid.y and z the segments.
template <int V>
struct Place {
  static constexpr int CW = LC * V;  // channels of the tile
  int64_t b, c0, c, len;             // c: the lane's first channel
  int64_t k;                         // the segment's place in the order of work
  int lane, chunk;
  bool ok;

  __device__ __forceinline__ bool set(const GatedParams& p, unsigned tiles, int64_t nseg) {
    const unsigned tile = blockIdx.x % tiles;
    b = blockIdx.x / tiles;
    k = (int64_t)blockIdx.z * gridDim.y + blockIdx.y;
    if (b >= p.batch || k >= nseg) return false;  // block-uniform
    lane = threadIdx.x % LC;
    chunk = threadIdx.x / LC;
    c0 = (int64_t)tile * CW;
    c = c0 + lane * V;
    ok = c < p.D;  // with V == 2 the channels are even: a lane is all in or all out
    len = row_len(p, b);
    return true;
  }
};

// The kernel's first argument read anew: what only a rare or a late part needs
// is loaded there, not held in (or spilled from) scalar registers until then.
template <class P>
__device__ __forceinline__ const P& args_anew() {
  auto at = (uint64_t)__builtin_amdgcn_kernarg_segment_ptr();
  asm volatile("" : "+s"(at));
  return *(const P*)(const __attribute__((address_space(4))) P*)at;
}

// ------------------------------------------------------------------- forward
template <bool BF16, bool YF32, bool Z, int V, bool Y>
struct Fwd : Place<V> {
  using Place<V>::CW;
  using Place<V>::b;
  using Place<V>::c0;
  using Place<V>::c;
  using Place<V>::len;
  using Place<V>::k;
  using Place<V>::lane;
  using Place<V>::chunk;
  using Place<V>::ok;
  static constexpr int E = BF16 ? 2 : 4;
  static constexpr int YE = (YF32 || !BF16) ? 4 : 2;
  static constexpr int T = kFwdT, NCH = kGatedFwdChunks;
  static constexpr bool kZ = Z && Y;
  struct Shared {
    float2 pair[NCH][CW];
    float2 stack[kStack][CW];
    float in[NCH][CW];
    int found;
  };

  const GatedParams& p;
  Chan<V> ch;
  Raw<BF16, V> zr[kZ ? T : 1];
  float a[T][V], u[T][V];

  __device__ __forceinline__ Fwd(const GatedParams& q) : p(q) {}

  // Decays and inputs of the chunk of the segment at t0 into a, u, and its pair into LDS.
  template <bool MASK, bool WITH_Z>
  __device__ __forceinline__ void scan_chunk(int64_t t0, Shared& sh) {
    Stream sx, sa, sg, sz;
    const int live = MASK ? clamp_steps(len - t0 - chunk * T, T) : T;  // steps that count
    sa.set(p.gate_a, p.gas_b, p.gas_t, b, t0, c0, p.L, p.D, E, T, chunk, lane * V, ok);
    sg.set(p.gate_x, p.gxs_b, p.gxs_t, b, t0, c0, p.L, p.D, E, T, chunk, lane * V, ok);
    sx.set(p.x, p.xs_b, p.xs_t, b, t0, c0, p.L, p.D, E, T, chunk, lane * V, ok);
    Raw<BF16, V> xr[T], ar[T], gr[T];
#pragma unroll
    for (int j = 0; j < T; ++j) {
      ar[j] = load_row<MASK, BF16, V>(sa, j, live);
      gr[j] = load_row<MASK, BF16, V>(sg, j, live);
      xr[j] = load_row<MASK, BF16, V>(sx, j, live);
    }
    if constexpr (kZ && WITH_Z) {
      sz.set(p.z, p.zs_b, p.zs_t, b, t0, c0, p.L, p.D, E, T, chunk, lane * V, ok);
#pragma unroll
      for (int j = 0; j < T; ++j) zr[j] = load_row<MASK, BF16, V>(sz, j, live);
    }
    float cp[V], cH[V];
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
    for (int v = 0; v < V; ++v) sh.pair[chunk][lane * V + v] = make_float2(cp[v], cH[v]);
  }

  // The segment's pair, by the first wave.
  __device__ __forceinline__ float2 fold(const Shared& sh, int ch_lane) const {
    float2 f = make_float2(1.f, 0.f);
#pragma unroll 4
    for (int q = 0; q < NCH; ++q) {
      const float2 w = sh.pair[q][ch_lane];
      f.x *= w.x;
      f.y = pass_on(w.x, f.y, w.y);
    }
    return f;
  }

  // The whole segment.  `known`: h is the entering state (in the first wave's
  // lanes); otherwise it is looked for, and false returned if it is not found.
  template <bool MASK>
  __device__ __forceinline__ bool segment(const Chain& q, Shared& sh, bool known, float h) {
    const int64_t t0 = k * kFwdSeg, t = t0 + chunk * T;
    const int rows = MASK ? clamp_steps(p.L - t, T) : T;  // rows of the chunk inside the sequence
    const int live = MASK ? clamp_steps(len - t, T) : T;
    scan_chunk<MASK, true>(t0, sh);
    __syncthreads();
    if (threadIdx.x < 64) {
      const int l = threadIdx.x;
      const bool mine = l < CW && c0 + l < p.D;
      const int64_t at = (k * p.batch + b) * p.D + c0 + l;
      const float2 f = fold(sh, l < CW ? l : 0);
      const bool more = (k + 1) * kFwdSeg < p.L;
      if (more && k > 0 && mine) publish_pair(q, at, f.x, f.y);
      bool found = known || k == 0;
      if (!found) found = entering<CW>(q, k, at, mine, sh.stack, l, h);
      if (found) {
        if (mine) {
          const float end = pass_on(f.x, h, f.y);
          if (more) publish_state(q, at, end);
          else if (Y && p.h_last) p.h_last[b * p.D + c0 + l] = end;
        }
        // read the pairs again rather than hold them over the wait
        asm volatile("" ::: "memory");
        if (l < CW)
#pragma unroll 4
          for (int i = 0; i < NCH; ++i) {
            sh.in[i][l] = h;
            h = pass_on(sh.pair[i][l].x, h, sh.pair[i][l].y);
          }
      }
      if (l == 0) sh.found = found;
    }
    __syncthreads();
    if (!sh.found) return false;
    float in[V];
#pragma unroll
    for (int v = 0; v < V; ++v) in[v] = sh.in[chunk][lane * V + v];
    if (p.ckpt && (chunk * T) % kGatedCkptSteps == 0 && ok && rows > 0) {
      const int64_t nk = (p.L + kGatedCkptSteps - 1) / kGatedCkptSteps;
#pragma unroll
      for (int v = 0; v < V; ++v) p.ckpt[(b * nk + t / kGatedCkptSteps) * p.D + c + v] = in[v];
    }
    if constexpr (Y) {
      Stream sy;
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
        sy.next();
      }
    }
    return true;
  }
};

template <bool BF16, bool YF32, bool Z, int V, bool Y>
__global__ __launch_bounds__(kFwdNT, !BF16 && Z && V == 2 ? kFwdWaves32 : kFwdWaves) void gated_fwd_kernel(
    GatedParams p, Chain q, unsigned tiles, int64_t nseg) {
  typedef Fwd<BF16, YF32, Z, V, Y> F;
  __shared__ typename F::Shared sh;
  F f(p);
  if (!f.set(p, tiles, nseg)) return;
  f.ch.load(p, f.c, f.ok);
  const int l = threadIdx.x;  // the first wave's channels
  const float h0 = p.h0 && l < F::CW && f.c0 + l < p.D ? p.h0[f.b * p.D + f.c0 + l] : 0.f;
  if (q.polls > 0 || f.k == 0) {
    if ((f.k + 1) * kFwdSeg <= f.len ? f.template segment<false>(q, sh, false, h0)
                                     : f.template segment<true>(q, sh, false, h0))
      return;
  }
  // Not found in time: the segments before this one, from the start.
  F late(args_anew<GatedParams>());
  late.set(late.p, tiles, nseg);
  late.ch.load(late.p, late.c, late.ok);
  float h = late.p.h0 && l < F::CW && late.c0 + l < late.p.D ? late.p.h0[late.b * late.p.D + late.c0 + l] : 0.f;
  for (int64_t k = 0; k < late.k; ++k) {
    __syncthreads();  // the last fold has read the pairs
    late.template scan_chunk<true, false>(k * kFwdSeg, sh);
    __syncthreads();
    if (l < 64) {
      const float2 w = late.fold(sh, l < F::CW ? l : 0);
      h = pass_on(w.x, h, w.y);
    }
  }
  __syncthreads();
  late.template segment<true>(q, sh, true, h);
}

// ------------------------------------------------------------------ backward
template <bool BF16, bool GF32, bool Z, int V>
struct Bwd : Place<V> {
  using Place<V>::CW;
  using Place<V>::b;
  using Place<V>::c0;
  using Place<V>::c;
  using Place<V>::len;
  using Place<V>::k;
  using Place<V>::lane;
  using Place<V>::chunk;
  using Place<V>::ok;
  static constexpr int E = BF16 ? 2 : 4;
  static constexpr bool G32 = GF32 || !BF16;
  static constexpr int GE = G32 ? 4 : 2;
  static constexpr int T = kBwdT, NCH = kGatedBwdChunks;
  struct Shared {
    float P[NCH][CW], H[NCH][CW], O[NCH][CW];  // decay product, end state from zero, carry out from a zero carry
    float2 stack[kStack][CW];
    float h[NCH][CW], m[NCH][CW];              // state and carry that enter each chunk
    int found;
  };

  const GatedBwdParams& q;
  const GatedParams& p;
  Chan<V> ch;
  // a, g, r, i, s, x of every step; zf = dy silu'(z), later the state before the step less i x a / s
  float a[T][V], g[T][V], r[T][V], i[T][V], s[T][V], zf[T][V];
  Raw<BF16, V> xr[T];

  __device__ __forceinline__ Bwd(const GatedBwdParams& w) : q(w), p(w.f) {}

  // What step j adds to the state.
  __device__ __forceinline__ float input(int j, int v) const { return s[j][v] * (i[j][v] * elem(xr[j], v)); }

  // GRADS: everything of the chunk of the segment at t0; else only what the carry needs (a, g).
  template <bool MASK, bool GRADS>
  __device__ __forceinline__ void scan_chunk(int64_t t0, Shared& sh) {
    Stream sx, sa, sg, sz, sd;
    const int live = MASK ? clamp_steps(len - t0 - chunk * T, T) : T;
    sa.set(p.gate_a, p.gas_b, p.gas_t, b, t0, c0, p.L, p.D, E, T, chunk, lane * V, ok);
    sd.set(q.dy, q.dys_b, q.dys_t, b, t0, c0, p.L, p.D, GE, T, chunk, lane * V, ok);
    if constexpr (Z) sz.set(p.z, p.zs_b, p.zs_t, b, t0, c0, p.L, p.D, E, T, chunk, lane * V, ok);
    Raw<BF16, V> ar[T], gr[T], zr[Z ? T : 1];
    Raw<!G32, V> dr[T];
#pragma unroll
    for (int j = 0; j < T; ++j) {
      ar[j] = load_row<MASK, BF16, V>(sa, j, live);
      dr[j] = load_row<MASK, !G32, V>(sd, j, live);
      if constexpr (Z) zr[j] = load_row<MASK, BF16, V>(sz, j, live);
    }
    if constexpr (GRADS) {
      sx.set(p.x, p.xs_b, p.xs_t, b, t0, c0, p.L, p.D, E, T, chunk, lane * V, ok);
      sg.set(p.gate_x, p.gxs_b, p.gxs_t, b, t0, c0, p.L, p.D, E, T, chunk, lane * V, ok);
#pragma unroll
      for (int j = 0; j < T; ++j) {
        gr[j] = load_row<MASK, BF16, V>(sg, j, live);
        xr[j] = load_row<MASK, BF16, V>(sx, j, live);
      }
    }
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
        r[j][v] = gate(elem(ar[j], v), ch.nba[v]);
        const float e = r[j][v] * ch.al2[v];
        a[j][v] = __builtin_amdgcn_exp2f(e);
        const float dy = elem(dr[j], v);
        g[j][v] = dy;
        if constexpr (Z) {
          // dy silu(z) and dy silu'(z) = dy sig(z) + dy silu(z) (1 - sig(z))
          const float z = elem(zr[j], v), sz = gate(z, 0.f), ds = dy * sz;
          g[j][v] = ds * z;
          if constexpr (GRADS) zf[j][v] = __builtin_fmaf(g[j][v], 1.f - sz, ds);
        }
        if constexpr (GRADS) {
          i[j][v] = gate(elem(gr[j], v), ch.nbx[v]);
          s[j][v] = __builtin_amdgcn_sqrtf(one_minus_sq(e, a[j][v]));
        }
        if (MASK && j >= live) {
          a[j][v] = 1.f;
          g[j][v] = 0.f;
        }
        cp[v] *= a[j][v];
        if constexpr (GRADS) cH[v] = __builtin_fmaf(a[j][v], cH[v], MASK && j >= live ? 0.f : input(j, v));
        // finished here: left for after the barriers, its factors would be held instead
        if constexpr (GRADS && Z) asm volatile("" : "+v"(zf[j][v]));
        if constexpr (GRADS) asm volatile("" : "+v"(g[j][v]));
      }
#pragma unroll
    for (int j = T - 1; j >= 0; --j)
#pragma unroll
      for (int v = 0; v < V; ++v) cM[v] = a[j][v] * (g[j][v] + cM[v]);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      sh.P[chunk][lane * V + v] = cp[v];
      sh.O[chunk][lane * V + v] = cM[v];
      if constexpr (GRADS) sh.H[chunk][lane * V + v] = cH[v];
    }
  }

  // The segment's pair for the carry, by the first wave.
  __device__ __forceinline__ float2 fold(const Shared& sh, int l) const {
    float2 f = make_float2(1.f, 0.f);
#pragma unroll 4
    for (int w = NCH - 1; w >= 0; --w) {
      f.x *= sh.P[w][l];
      f.y = pass_on(sh.P[w][l], f.y, sh.O[w][l]);
    }
    return f;
  }

  // Segment seg = nseg - 1 - k.  `known`: m is the carry into its last step.
  template <bool MASK>
  __device__ __forceinline__ bool segment(const Chain& cn, Shared& sh, int64_t seg, bool known, float m) {
    const int64_t t0 = seg * kBwdSeg, t = t0 + chunk * T;
    const int rows = MASK ? clamp_steps(p.L - t, T) : T;
    const int live = MASK ? clamp_steps(len - t, T) : T;
    scan_chunk<MASK, true>(t0, sh);
    __syncthreads();
    if (threadIdx.x < 64) {
      const int l = threadIdx.x;
      const bool mine = l < CW && c0 + l < p.D;
      const int64_t nk = (p.L + kGatedCkptSteps - 1) / kGatedCkptSteps;
      float h = mine ? p.ckpt[(b * nk + t0 / kGatedCkptSteps) * p.D + c0 + l] : 0.f;
      const int64_t at = (k * p.batch + b) * p.D + c0 + l;
      const float2 f = fold(sh, l < CW ? l : 0);
      if (seg > 0 && k > 0 && mine) publish_pair(cn, at, f.x, f.y);
      bool found = known || k == 0;
      if (!found) found = entering<CW>(cn, k, at, mine, sh.stack, l, m);
      if (found) {
        if (mine) {
          const float end = pass_on(f.x, m, f.y);
          if (seg > 0) publish_state(cn, at, end);
          else if (q.dh0) q.dh0[b * p.D + c0 + l] = end;
        }
        // read the pairs again rather than hold them over the wait
        asm volatile("" ::: "memory");
        if (l < CW) {
#pragma unroll 4
          for (int w = 0; w < NCH; ++w) {
            sh.h[w][l] = h;
            h = pass_on(sh.P[w][l], h, sh.H[w][l]);
          }
#pragma unroll 4
          for (int w = NCH - 1; w >= 0; --w) {
            sh.m[w][l] = m;
            m = pass_on(sh.P[w][l], m, sh.O[w][l]);
          }
        }
      }
      if (l == 0) sh.found = found;
    }
    __syncthreads();
    if (!sh.found) return false;
    // Products of these made before the barriers are made again: held over
    // them they cost twice the registers that the factors do.
#pragma unroll
    for (int j = 0; j < T; ++j) {
#pragma unroll
      for (int v = 0; v < V; ++v) asm volatile("" : "+v"(r[j][v]), "+v"(i[j][v]), "+v"(s[j][v]));
#pragma unroll
      for (uint32_t& x : xr[j].w) asm volatile("" : "+v"(x));
    }
    // bf16 with z: four outputs' addresses on top of the inputs' spill (8 x 2048 x
    // 1536 127 us, read anew 124; but held fp32 203 against 237, bf16 without z 106
    // against 109)
    constexpr bool kAnew = BF16 && Z;
    const GatedBwdParams& q = kAnew ? args_anew<GatedBwdParams>() : this->q;
    const GatedParams& p = q.f;
    float h[V], mi[V], A[V], sA[V], sba[V], sbx[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      h[v] = sh.h[chunk][lane * V + v];
      mi[v] = sh.m[chunk][lane * V + v];
      A[v] = ok ? p.A[(c + v) * p.As_d] : 0.f;
      sA[v] = sba[v] = sbx[v] = 0.f;
    }
    Stream so, dx, da, dg;
    if constexpr (Z) so.set(q.dz, q.dzs_b, q.dzs_t, b, t0, c0, p.L, p.D, GE, T, chunk, lane * V, ok);
#pragma unroll
    for (int j = 0; j < T; ++j) {
      float o[V];
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const float hn = __builtin_fmaf(a[j][v], h[v], MASK && j >= live ? 0.f : input(j, v));
        if constexpr (Z) o[v] = MASK && j >= live ? 0.f : hn * zf[j][v];
        const float is = s[j][v] > 0.f ? __builtin_amdgcn_rcpf(s[j][v]) : 0.f;
        zf[j][v] = __builtin_fmaf(-(i[j][v] * elem(xr[j], v)) * a[j][v], is, h[v]);
        h[v] = hn;
      }
      if constexpr (Z) {
        store_row<MASK, G32, V>(so, j, rows, o);
        so.next();
      }
    }
    dx.set(q.dx, q.dxs_b, q.dxs_t, b, t0, c0, p.L, p.D, GE, T, chunk, lane * V, ok);
    da.set(q.dgate_a, q.dgas_b, q.dgas_t, b, t0, c0, p.L, p.D, GE, T, chunk, lane * V, ok);
    dg.set(q.dgate_x, q.dgxs_b, q.dgxs_t, b, t0, c0, p.L, p.D, GE, T, chunk, lane * V, ok);
    dx.last(T);
    da.last(T);
    dg.last(T);
#pragma unroll
    for (int j = T - 1; j >= 0; --j) {
      float ox[V], oa[V], og[V];
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const float x = elem(xr[j], v);
        const float lam = g[j][v] + mi[v];
        mi[v] = a[j][v] * lam;
        const float du = mi[v] * zf[j][v];  // lam (a h_{t-1} - i x a^2 / s)
        ox[v] = lam * s[j][v] * i[j][v];
        // dA = du r, dgate_a = dA A (1 - r), dgate_x = dx x (1 - i)
        float dA = du * r[j][v];
        const float ga = dA * A[v], gx = ox[v] * x;
        oa[v] = __builtin_fmaf(-r[j][v], ga, ga);
        og[v] = __builtin_fmaf(-i[j][v], gx, gx);
        if (MASK && j >= live) ox[v] = oa[v] = og[v] = dA = 0.f;
        sA[v] += dA;
        sba[v] += oa[v];
        sbx[v] += og[v];
      }
      store_row<MASK, G32, V>(dx, j, rows, ox);
      dx.prev();
      store_row<MASK, G32, V>(da, j, rows, oa);
      da.prev();
      store_row<MASK, G32, V>(dg, j, rows, og);
      dg.prev();
    }
    // The chunks' sums, added in order.  P, H and O were last read before
    // the barrier.
#pragma unroll
    for (int v = 0; v < V; ++v) {
      sh.P[chunk][lane * V + v] = sA[v];
      sh.H[chunk][lane * V + v] = sba[v];
      sh.O[chunk][lane * V + v] = sbx[v];
    }
    __syncthreads();
    if (chunk < 3 && ok) {
      const auto& from = chunk == 0 ? sh.P : chunk == 1 ? sh.H : sh.O;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        float sum = 0.f;
#pragma unroll
        for (int w = 0; w < NCH; ++w) sum += from[w][lane * V + v];
        q.part[((k * p.batch + b) * 3 + chunk) * p.D + c + v] = sum;
      }
    }
    return true;
  }
};

template <bool BF16, bool GF32, bool Z, int V>
__global__ __launch_bounds__(kBwdNT, kBwdWaves) void gated_bwd_kernel(GatedBwdParams q, Chain cn, unsigned tiles,
                                                                        int64_t nseg) {
  typedef Bwd<BF16, GF32, Z, V> F;
  __shared__ typename F::Shared sh;
  const GatedParams& p = q.f;
  F f(q);
  if (!f.set(p, tiles, nseg)) return;
  f.ch.load(p, f.c, f.ok);
  const int l = threadIdx.x;
  const int64_t seg = nseg - 1 - f.k;
  const float m0 = q.dh_last && l < F::CW && f.c0 + l < p.D ? q.dh_last[f.b * p.D + f.c0 + l] : 0.f;
  if (cn.polls > 0 || f.k == 0) {
    if ((seg + 1) * kBwdSeg <= f.len ? f.template segment<false>(cn, sh, seg, false, m0)
                                     : f.template segment<true>(cn, sh, seg, false, m0))
      return;
  }
  // Not found in time: the segments behind this one, from the end.
  F late(args_anew<GatedBwdParams>());
  late.set(late.p, tiles, nseg);
  late.ch.load(late.p, late.c, late.ok);
  float m = late.q.dh_last && l < F::CW && late.c0 + l < late.p.D ? late.q.dh_last[late.b * late.p.D + late.c0 + l]
                                                                  : 0.f;
  const int64_t last = nseg - 1 - late.k;
  for (int64_t s = nseg - 1; s > last; --s) {
    __syncthreads();
    late.template scan_chunk<true, false>(s * kBwdSeg, sh);
    __syncthreads();
    if (l < 64) {
      const float2 w = late.fold(sh, l < F::CW ? l : 0);
      m = pass_on(w.x, m, w.y);
    }
  }
  __syncthreads();
  late.template segment<true>(cn, sh, last, true, m);
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

// The grid of all tiles and segments, and the chain's words in `ws`, filled.
template <int V>
dim3 seg_grid(const GatedParams& p, int64_t nseg, unsigned& tiles) {
  tiles = (unsigned)((p.D + LC * V - 1) / (LC * V));
  const int64_t y = std::min<int64_t>(nseg, 32768);
  return dim3((unsigned)((tiles * p.batch + 7) / 8 * 8), (unsigned)y, (unsigned)((nseg + y - 1) / y));
}

Chain make_chain(const GatedParams& p, void* ws, int64_t nseg, hipStream_t stream) {
  Chain q = {nullptr, nullptr, p.batch * p.D, p.polls};
  if (nseg > 1) {
    const int64_t words = nseg * q.step;
    q.agg = (unsigned long long*)ws;
    q.inc = (uint32_t*)(q.agg + words);
    const int64_t n = gated_chain_bytes(p.batch, p.D, nseg) / 16;
    hipLaunchKernelGGL(gated_fill_kernel, dim3((unsigned)((n + 255) / 256)), dim3(256), 0, stream, (uint4*)ws, n);
  }
  return q;
}

template <bool BF16, bool YF32, bool Z, int V>
void launch_fwd(const GatedParams& p, hipStream_t stream) {
  const int64_t nseg = (p.L + kFwdSeg - 1) / kFwdSeg;
  unsigned tiles;
  const dim3 grid = seg_grid<V>(p, nseg, tiles);
  const Chain q = make_chain(p, p.chain, nseg, stream);
  if (p.y)
    hipLaunchKernelGGL((gated_fwd_kernel<BF16, YF32, Z, V, true>), grid, dim3(kFwdNT), 0, stream, p, q, tiles, nseg);
  else
    hipLaunchKernelGGL((gated_fwd_kernel<BF16, false, false, V, false>), grid, dim3(kFwdNT), 0, stream, p, q, tiles, nseg);
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
  const int64_t nseg = (p.L + kBwdSeg - 1) / kBwdSeg;
  unsigned tiles;
  const dim3 grid = seg_grid<V>(p, nseg, tiles);
  const Chain cn = make_chain(p, p.chain, nseg, stream);
  hipLaunchKernelGGL((gated_bwd_kernel<BF16, GF32, Z, V>), grid, dim3(kBwdNT), 0, stream, q, cn, tiles, nseg);
  launch_column_sums(q.part, p.batch * nseg, 3 * p.D, p.D, q.dA, q.dbias_a, q.dbias_x, stream);
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

// Two channels per lane when every row starts on a whole pair (4 x 4096 x 5120:
// 198 us, with one channel per lane 271 us).
bool gated_pairs(const GatedParams& p) {
  const int e = p.io_bf16 ? 2 : 4, ye = p.y_f32 || !p.io_bf16 ? 4 : 2;
  return p.D % 2 == 0 && pair_rows(p.x, e, p.xs_b, p.xs_t) && pair_rows(p.gate_a, e, p.gas_b, p.gas_t) &&
         pair_rows(p.gate_x, e, p.gxs_b, p.gxs_t) && pair_rows(p.z, e, p.zs_b, p.zs_t) &&
         pair_rows(p.y, ye, p.ys_b, p.ys_t);
}

}  // namespace

// Two channels a lane, unless so few workgroups come of it that latency is all:
// with one, a wave has half the work.  bf16 forward, one against two channels:
// 1 x 16 x 2560 (40 workgroups of two) 6.0 us against 7.5, 1 x 300 x 2560 (120)
// 10.0 against 10.6, 1 x 2048 x 640 (160) 13.4 against 12.9; fp32 with z 1 x 2048
// x 1536 (384) 17.9 against 19.5, 2 x 2048 x 1536 (768) 32.5 against 30.0;
// backward in step.
bool wide_tiles(const GatedParams& p, int64_t segment) {
  const int64_t workgroups = (p.D + 2 * LC - 1) / (2 * LC) * p.batch * ((p.L + segment - 1) / segment);
  return workgroups > (p.io_bf16 ? 128 : 384);
}

hipError_t launch_gated_scan(const GatedParams& p, hipStream_t stream) {
  if (gated_pairs(p) && wide_tiles(p, kFwdSeg)) launch_fwd_io<2>(p, stream);
  else launch_fwd_io<1>(p, stream);
  return hipGetLastError();
}

hipError_t launch_gated_scan_bwd(const GatedBwdParams& q, hipStream_t stream) {
  const int ge = q.g_f32 || !q.f.io_bf16 ? 4 : 2;
  const bool pairs = gated_pairs(q.f) && pair_rows(q.dy, ge, q.dys_b, q.dys_t) &&
                     pair_rows(q.dx, ge, q.dxs_b, q.dxs_t) && pair_rows(q.dgate_a, ge, q.dgas_b, q.dgas_t) &&
                     pair_rows(q.dgate_x, ge, q.dgxs_b, q.dgxs_t) && pair_rows(q.dz, ge, q.dzs_b, q.dzs_t);
  if (pairs && wide_tiles(q.f, kBwdSeg)) launch_bwd_io<2>(q, stream);
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
