// Selective scan of packed sequences over a pool of states, for gfx950.
//
// For every sequence, channel d and state n (h from slot src, or 0):
//   Abar = exp(delta A),  Bbar = expm1(delta A) / A * B   (or delta B, simplified)
//   h_t = Abar h_{t-1} + Bbar x_t,  y_t = (C_t . h_t + D x_t) silu(z_t);  slot dst <- h
//
// Prompts are bound by VALU issue (an exp2 and about eight fp32 operations for
// each state, step and channel against 8 bytes of HBM traffic for each step and
// channel); single tokens by the state's traffic.
//
// Layout.  Four lanes hold a channel, NS consecutive states each, in registers
// for the whole walk; a wave has 16 channels and walks alone: no barrier, no
// state outside registers.  Steps are walked in tiles of 16.  Lane j of a
// channel's four also holds delta, x and z of the tile's steps 4i + j: a step
// takes delta and x from that lane by a DPP quad broadcast folded into the
// multiply, its readout is summed over the four lanes by two DPP adds that end
// in the lane that holds the step's x and z, and that lane stores y.  B and C
// of a tile lie in the wave's own LDS, 16 bytes a read for four states, the same
// address for the 16 channels.  The next tile's values are asked for a tile
// ahead.
//
// Pieces (packed_pieces.h).  A sequence is cut at grid lines, so that a long one
// does not walk alone.  The first pass walks every piece, the later ones of a
// sequence from zeros, and keeps each piece's end state and sum of delta.  The
// second pass walks the later pieces again from their true states -- chained
// from the kept ones by each wave for itself -- next to a twin from zeros, and
// stops at the end of the tile where every state equals its twin bit for bit:
// what follows is what the first pass wrote.  States that decay are walked again
// over a short stretch only.
//
// Forms, chosen for each tile of a wave (delta A of its steps and channels):
//   small   all |delta A| < 1/8: expm1(u)/u by its Taylor polynomial; right for A = 0
//   fast    bf16 input, no A = 0: h <- Abar (h + q) - q, q = B x / A (the update
//           multiplied out): 8 issue slots a state and step
//   any     otherwise: (Abar - 1) / A, or the polynomial where |u| < 1/4
#include <hip/hip_runtime.h>

#include <algorithm>

#include "serve_device.h"

namespace ssm {
namespace {

using namespace dev;

constexpr int kWaves = 4;           // of a workgroup; they share nothing
constexpr int kCh = 16;             // channels of a wave
constexpr int kTile = 16;           // steps

// Value of lane J of each four lanes.
template <int J>
__device__ __forceinline__ float quad(float v) {
  return __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), J * 0x55, 0xF, 0xF, true));
}

// v of the lane whose number within its four differs in the bits M (1 or 2).
template <int M>
__device__ __forceinline__ float other(float v) {
  return __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), M == 1 ? 0xB1 : 0x4E, 0xF, 0xF,
                                                           true));
}

// expm1(u) / u for |u| < 1/4 (through u^5; the next term is u^6 / 5040 < 5e-8).
__device__ __forceinline__ float phi(float u) {
  float q = 1.f / 720.f;
  q = __builtin_fmaf(q, u, 1.f / 120.f);
  q = __builtin_fmaf(q, u, 1.f / 24.f);
  q = __builtin_fmaf(q, u, 1.f / 6.f);
  q = __builtin_fmaf(q, u, 0.5f);
  return __builtin_fmaf(q, u, 1.f);
}

enum Form : int { kSmall = 0, kFast = 1, kAny = 2, kEuler = 3 };

// A lane's constants of its states.
template <int NS>
struct Lane {
  float A[NS], A2[NS], iA[NS];  // A, A log2(e), 1/A (0 where A is 0)
};

// The state, its input and its decay of one step: h <- the next state; with a
// twin, it takes the same factors through the same operations.  No implicit
// fusing: the broadcast multiplies have to stay multiplies (an fma takes no DPP).
template <int NS, int FORM, bool TWIN, int J>
__device__ __forceinline__ float step(float (&h)[NS], float (&h2)[NS], const Lane<NS>& ln, float dt, float x,
                                      const float (&B)[NS], const float (&C)[NS]) {
#pragma clang fp contract(off)
  float yp = 0.f;
#pragma unroll
  for (int k = 0; k < NS; ++k) {
    if constexpr (FORM == kFast) {
      const float Ab = __builtin_amdgcn_exp2f(quad<J>(dt) * ln.A2[k]);
      const float q = (quad<J>(x) * ln.iA[k]) * B[k];
      h[k] = __builtin_fmaf(Ab, h[k] + q, -q);
      if constexpr (TWIN) h2[k] = __builtin_fmaf(Ab, h2[k] + q, -q);
    } else if constexpr (FORM == kEuler) {
      const float Ab = __builtin_amdgcn_exp2f(quad<J>(dt) * ln.A2[k]);
      const float q = quad<J>(x) * B[k];  // x is delta x here
      h[k] = __builtin_fmaf(Ab, h[k], q);
      if constexpr (TWIN) h2[k] = __builtin_fmaf(Ab, h2[k], q);
    } else {
      const float u = quad<J>(dt) * ln.A[k];
      float c = quad<J>(dt) * phi(u), Ab;
      if constexpr (FORM == kSmall) {
        Ab = __builtin_fmaf(c, ln.A[k], 1.f);
      } else {
        Ab = __builtin_amdgcn_exp2f(quad<J>(dt) * ln.A2[k]);
        const float far = (Ab - 1.f) * ln.iA[k];
        c = fabsf(u) < 0.25f ? c : far;
      }
      const float q = c * (quad<J>(x) * B[k]);
      h[k] = __builtin_fmaf(Ab, h[k], q);
      if constexpr (TWIN) h2[k] = __builtin_fmaf(Ab, h2[k], q);
    }
    yp = k == 0 ? C[k] * h[k] : __builtin_fmaf(C[k], h[k], yp);
  }
  return yp;
}

// Steps 4i .. 4i+3 of a tile; returns the readout of step 4i + (lane % 4).
// bc: the tile's B and C in LDS from this lane's first state on.
template <int NS, int FORM, bool TWIN>
__device__ __forceinline__ float four_steps(float (&h)[NS], float (&h2)[NS], const Lane<NS>& ln, float dt, float x,
                                            const float* bc) {
  constexpr int NP = 4 * NS;
  float B[4][NS], C[4][NS];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
#pragma unroll
    for (int k = 0; k < NS; ++k) {
      B[j][k] = bc[(2 * j) * NP + k];
      C[j][k] = bc[(2 * j + 1) * NP + k];
    }
  }
  const float y0 = step<NS, FORM, TWIN, 0>(h, h2, ln, dt, x, B[0], C[0]);
  const float y1 = step<NS, FORM, TWIN, 1>(h, h2, ln, dt, x, B[1], C[1]);
  const float y2 = step<NS, FORM, TWIN, 2>(h, h2, ln, dt, x, B[2], C[2]);
  const float y3 = step<NS, FORM, TWIN, 3>(h, h2, ln, dt, x, B[3], C[3]);
  // lane j: the sum of step j over the four lanes, by exchanging what the other needs
  const bool odd = threadIdx.x & 1, up = threadIdx.x & 2;
  const float a = (odd ? y1 : y0) + other<1>(odd ? y0 : y1);
  const float b = (odd ? y3 : y2) + other<1>(odd ? y2 : y3);
  return (up ? b : a) + other<2>(up ? a : b);
}

// One tile of a lane's values, as loaded (converted where they are used, so that
// nothing waits for them before): x, delta, z of steps 4i + lane % 4 of its
// channel; row lane / 4 of B and C, states NS (lane % 4) and on.
template <bool BF16, int NS, bool VEC>
struct Tile {
  static constexpr int kWords = BF16 && VEC ? (NS + 1) / 2 : NS;
  uint32_t x[4], dt[4], z[4], B[kWords], C[kWords];

  __device__ __forceinline__ static float state(const uint32_t (&w)[kWords], int k) {
    if constexpr (!BF16) return __uint_as_float(w[k]);
    else if constexpr (!VEC || NS == 1) return __uint_as_float(w[k] << 16);
    else return __uint_as_float((k & 1) ? (w[k >> 1] & 0xFFFF0000u) : (w[k >> 1] << 16));
  }
};

template <bool BF16>
__device__ __forceinline__ uint32_t load_raw(__amdgpu_buffer_rsrc_t r, uint32_t off) {
  if constexpr (BF16) return __builtin_amdgcn_raw_buffer_load_b16(r, (int)off, 0, 0);
  else return __builtin_amdgcn_raw_buffer_load_b32(r, (int)off, 0, 0);
}

// A wave's streams over one piece.
template <bool BF16, int NS, bool VEC>
struct Streams {
  static constexpr int E = BF16 ? 2 : 4;
  using T = Tile<BF16, NS, VEC>;
  const ScanPackedParams& p;
  int64_t d0;     // first channel of the wave
  uint32_t lch;   // this lane's channel within the wave's
  bool ch_ok;
  int j, r, n0;   // lane % 4, lane / 4, first state
  int end;        // of the piece

  // Rows t .. t + left - 1 from the wave's first channel on.
  __device__ __forceinline__ __amdgpu_buffer_rsrc_t rows(const void* base, int64_t st, int t, int left) const {
    return rsrc((const char*)base + ((int64_t)t * st + d0) * E, row_range(left, st, p.D - d0, E));
  }

  // The tile at row t; rows past the piece and channels and states that do not exist read zeros.
  __device__ __forceinline__ void load(int t, T& o) const {
    const int left = end - t < kTile ? end - t : kTile;
    const auto rx = rows(p.x, p.xs_t, t, left), rd = rows(p.delta, p.ds_t, t, left);
    const auto rz = rows(p.z ? p.z : p.x, p.zs_t, t, p.z ? left : 0);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = 4 * i + j;
      const bool ok = ch_ok && row < left;
      o.x[i] = load_raw<BF16>(rx, ok ? ((uint32_t)row * (uint32_t)p.xs_t + lch) * E : kFar);
      o.dt[i] = load_raw<BF16>(rd, ok ? ((uint32_t)row * (uint32_t)p.ds_t + lch) * E : kFar);
      o.z[i] = load_raw<BF16>(rz, ok ? ((uint32_t)row * (uint32_t)p.zs_t + lch) * E : kFar);
    }
    load_states(p.B, p.Bs_t, p.Bs_n, t, left, o.B);
    load_states(p.C, p.Cs_t, p.Cs_n, t, left, o.C);
  }

  __device__ __forceinline__ void load_states(const void* base, int64_t st, int64_t sn, int t, int left,
                                              uint32_t (&o)[T::kWords]) const {
    const auto rb = rsrc((const char*)base + (int64_t)t * st * E, row_range(left, st, (p.N - 1) * sn + 1, E));
    const uint32_t row = (uint32_t)r * (uint32_t)st;
    if constexpr (VEC) {  // this lane's NS states lie side by side, all in or all out
      const uint32_t off = r < left && n0 < p.N ? (row + (uint32_t)n0) * E : kFar;
      if constexpr (T::kWords == 1) {
        if constexpr (BF16 && NS == 1) o[0] = load_raw<true>(rb, off);
        else o[0] = __builtin_amdgcn_raw_buffer_load_b32(rb, (int)off, 0, 0);
      } else if constexpr (T::kWords == 2) {
        const auto v = __builtin_amdgcn_raw_buffer_load_b64(rb, (int)off, 0, 0);
        o[0] = v[0]; o[1] = v[1];
      } else {
#pragma unroll
        for (int i = 0; i < T::kWords / 4; ++i) {
          const auto v = __builtin_amdgcn_raw_buffer_load_b128(rb, (int)(off + 16u * i), 0, 0);
          o[4 * i] = v[0]; o[4 * i + 1] = v[1]; o[4 * i + 2] = v[2]; o[4 * i + 3] = v[3];
        }
      }
    } else {
#pragma unroll
      for (int k = 0; k < NS; ++k)
        o[k] = load_raw<BF16>(rb, r < left && n0 + k < p.N ? (row + (uint32_t)(n0 + k) * (uint32_t)sn) * E : kFar);
    }
  }
};

// A lane's states of one (D, N) block in memory, as 16-byte words where they
// are aligned (NS of them exist then), else one by one.
template <int NS>
__device__ __forceinline__ void load_block(const float* at, int nk, bool vec, float (&h)[NS]) {
  if constexpr (NS >= 4) {
    if (vec) {
#pragma unroll
      for (int i = 0; i < NS / 4; ++i) {
        const float4 v = nk ? ((const float4*)at)[i] : make_float4(0.f, 0.f, 0.f, 0.f);
        h[4 * i] = v.x; h[4 * i + 1] = v.y; h[4 * i + 2] = v.z; h[4 * i + 3] = v.w;
      }
      return;
    }
  }
#pragma unroll
  for (int k = 0; k < NS; ++k) h[k] = k < nk ? at[k] : 0.f;
}

template <int NS>
__device__ __forceinline__ void store_block(float* at, int nk, bool vec, const float (&h)[NS]) {
  if constexpr (NS >= 4) {
    if (vec) {
      if (nk)
#pragma unroll
        for (int i = 0; i < NS / 4; ++i) ((float4*)at)[i] = make_float4(h[4 * i], h[4 * i + 1], h[4 * i + 2], h[4 * i + 3]);
      return;
    }
  }
#pragma unroll
  for (int k = 0; k < NS; ++k)
    if (k < nk) at[k] = h[k];
}

__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// One piece of one sequence for 16 channels.  TWIN: the second pass over a later
// piece (packed_pieces.h).
template <bool BF16, int NS, bool EULER, bool TWIN, bool VEC>
__global__ __launch_bounds__(64 * kWaves) void scan_packed_kernel(ScanPackedParams p, unsigned nblk, int vec_state) {
  constexpr int NP = 4 * NS;
  __shared__ __align__(16) float lds[kWaves][2][kTile][2][NP];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), lane = threadIdx.x % 64;
  const int piece = (int)(blockIdx.x / nblk);
  const int64_t d0 = ((int64_t)(blockIdx.x % nblk) * kWaves + wave) * kCh;
  if (d0 >= p.D) return;
  // the piece: rows [begin, end) of sequence s; `line` > 0: from that grid line on
  int s = piece, line = 0;
  packed::Run seq, run;
  if (!TWIN && piece < p.q.seqs) {
    seq = sequence_of(p.q, s);
    run = p.lines ? packed::first_piece(seq, p.step) : seq;
  } else {
    line = TWIN ? piece + 1 : piece - p.q.seqs + 1;
    s = find_sequence(p.q, line * p.step);
    if (s < 0) return;
    seq = sequence_of(p.q, s);
    run = packed::later_piece(seq, line * p.step, p.step);
    if (run.end <= run.begin) return;
  }
  const int j = lane % 4, n0 = j * NS;
  const int64_t d = d0 + lane / 4;
  const bool ch_ok = d < p.D;
  const int64_t dd = ch_ok ? d : d0;
  const int nk = !ch_ok || n0 >= p.N ? 0 : (p.N - n0 < NS ? (int)(p.N - n0) : NS);  // states that exist
  const int64_t own = dd * p.N + (n0 < p.N ? n0 : 0);  // of the lane's first state in a (D, N) block

  Lane<NS> ln;
  float h[NS], h2[NS];
  float amax = 0.f;
  bool zero = false;
#pragma unroll
  for (int k = 0; k < NS; ++k) {
    const float a = k < nk ? p.A[dd * p.As_d + (n0 + k) * p.As_n] : -1.f;
    ln.A[k] = a;
    ln.A2[k] = a * kLog2e;
    ln.iA[k] = a != 0.f ? 1.f / a : 0.f;
    zero = zero || a == 0.f;
    amax = k < nk ? fmaxf(amax, fabsf(a)) : amax;
    h[k] = h2[k] = 0.f;
  }
  const bool any_zero = __ballot(zero) != 0;
  const float Dk = p.Dskip && ch_ok ? p.Dskip[dd * p.Ds_d] : 0.f;
  const float bias = p.dbias && ch_ok ? p.dbias[dd * p.dbs_d] : 0.f;
  const int64_t block = p.D * p.N;
  const bool vec = vec_state != 0;
  if constexpr (TWIN) {
    // the state at the line: from the sequence's first line on, each piece's end state, the decay over
    // it applied to the state before it
    const int first = seq.begin / p.step + 1;
    load_block<NS>(p.H + (int64_t)(first - 1) * block + own, nk, vec, h);
    for (int l = first + 1; l <= line; ++l) {
      float e[NS];
      load_block<NS>(p.H + (int64_t)(l - 1) * block + own, nk, vec, e);
      const float sum = p.dsum[(int64_t)(l - 1) * p.D + dd];
#pragma unroll
      for (int k = 0; k < NS; ++k) h[k] = __builtin_fmaf(__builtin_amdgcn_exp2f(ln.A2[k] * sum), h[k], e[k]);
    }
  } else if (line == 0) {
    const int64_t from = src_slot(p.q, s);
    if (from >= 0) load_block<NS>(p.states + from * p.sts_s + own, nk, vec, h);
  }

  Streams<BF16, NS, VEC> st = {p, d0, (uint32_t)(lane / 4), ch_ok, j, lane / 4, n0, run.end};
  const int YE = p.y_f32 ? 4 : 2;
  Tile<BF16, NS, VEC> tile;
  auto stage = [&](int buf) {
    float* row = lds[wave][buf][lane / 4][0] + n0;
#pragma unroll
    for (int k = 0; k < NS; ++k) {
      row[k] = tile.state(tile.B, k);
      row[NP + k] = tile.state(tile.C, k);
    }
  };
  float sum_dt = 0.f;
  bool met = false;
  st.load(run.begin, tile);
  stage(0);
  int buf = 0;
  for (int t = run.begin; t < run.end; t += kTile, buf ^= 1) {
    const int left = run.end - t < kTile ? run.end - t : kTile;
    float x[4], dt[4], z[4], xs[4];
    float umax = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[i] = raw2f<BF16>(tile.x[i]);
      z[i] = raw2f<BF16>(tile.z[i]);
      float v = raw2f<BF16>(tile.dt[i]);
      if (p.dsoftplus) v = 4 * i + j < left ? softplus(v + bias) : 0.f;  // past the piece nothing changes
      dt[i] = v;
      umax = fmaxf(umax, fabsf(v));
      if constexpr (!TWIN) sum_dt += v;
      xs[i] = EULER ? v * x[i] : x[i];
    }
    st.load(t + kTile, tile);
    wave_sync();
    const float* bc = lds[wave][buf][0][0] + n0;
    float y[4];
    // the four lanes hold different steps and states: each one's largest delta and |A|
    umax = fmaxf(umax, other<1>(umax));
    umax = fmaxf(umax, other<2>(umax));
    const int form = EULER ? kEuler : __ballot(!(umax * amax < 0.125f)) == 0 ? kSmall : BF16 && !any_zero ? kFast : kAny;
    if constexpr (EULER) {
#pragma unroll
      for (int i = 0; i < 4; ++i) y[i] = four_steps<NS, kEuler, TWIN>(h, h2, ln, dt[i], xs[i], bc + i * 8 * NP);
    } else if (form == kSmall) {
#pragma unroll
      for (int i = 0; i < 4; ++i) y[i] = four_steps<NS, kSmall, TWIN>(h, h2, ln, dt[i], xs[i], bc + i * 8 * NP);
    } else if (form == kFast) {
#pragma unroll
      for (int i = 0; i < 4; ++i) y[i] = four_steps<NS, kFast, TWIN>(h, h2, ln, dt[i], xs[i], bc + i * 8 * NP);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) y[i] = four_steps<NS, kAny, TWIN>(h, h2, ln, dt[i], xs[i], bc + i * 8 * NP);
    }
    const auto ry = rsrc((char*)p.y + ((int64_t)t * p.ys_t + d0) * YE, row_range(left, p.ys_t, p.D - d0, YE));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float v = __builtin_fmaf(Dk, x[i], y[i]);
      if (p.z) v *= z[i] * sigmoid(z[i]);
      const int row = 4 * i + j;
      store1(ry, ch_ok && row < left ? ((uint32_t)row * (uint32_t)p.ys_t + st.lch) * (uint32_t)YE : kFar, v, p.y_f32);
    }
    stage(buf ^ 1);
    if constexpr (TWIN) {
      bool same = true;
#pragma unroll
      for (int k = 0; k < NS; ++k) same = same && __float_as_uint(h[k]) == __float_as_uint(h2[k]);
      if (__ballot(!same) == 0) {
        met = t + kTile < run.end;
        break;
      }
    }
  }

  if (run.end < seq.end) {  // the piece ends at a line inside the sequence
    if constexpr (!TWIN) {
      const int64_t l = run.end / p.step - 1;
      store_block<NS>(p.H + l * block + own, nk, vec, h);
      sum_dt += other<1>(sum_dt);
      sum_dt += other<2>(sum_dt);
      if (j == 0 && ch_ok) p.dsum[l * p.D + d] = sum_dt;
    }
    return;
  }
  // the sequence's end: the first pass keeps that of a later piece aside (another workgroup may not have read
  // the slot yet, and it is not the true state)
  if (!TWIN && line > 0) {
    store_block<NS>(p.E + (int64_t)(line - 1) * block + own, nk, vec, h);
    return;
  }
  const int64_t to = dst_slot(p.q, s);
  if (to < 0) return;
  if (TWIN && met) load_block<NS>(p.E + (int64_t)(line - 1) * block + own, nk, vec, h);
  store_block<NS>(p.states + to * p.sts_s + own, nk, vec, h);
}

// ------------------------------------------------------------ single tokens

// One token of each sequence: a wave has 16 channels of it, a lane NS states of
// one channel, read and written 16 bytes at a time.  Bound by that traffic, so
// every state takes the accurate form.
template <bool BF16, int NS, bool EULER>
__global__ __launch_bounds__(64 * kWaves) void step_packed_kernel(ScanPackedParams p, unsigned nblk, int vec_state) {
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), lane = threadIdx.x % 64;
  const int s = (int)(blockIdx.x / nblk);
  const int64_t d0 = ((int64_t)(blockIdx.x % nblk) * kWaves + wave) * kCh;
  if (d0 >= p.D) return;
  const int j = lane % 4, n0 = j * NS;
  const int64_t d = d0 + lane / 4;
  const bool ch_ok = d < p.D;
  const int64_t dd = ch_ok ? d : d0;
  const int nk = !ch_ok || n0 >= p.N ? 0 : (p.N - n0 < NS ? (int)(p.N - n0) : NS);
  const int64_t own = dd * p.N + (n0 < p.N ? n0 : 0);
  const bool vec = vec_state != 0;
  const int64_t from = src_slot(p.q, s), to = dst_slot(p.q, s);
  float h[NS], A[NS], B[NS], C[NS];
#pragma unroll
  for (int k = 0; k < NS; ++k) h[k] = 0.f;
  if (from >= 0) load_block<NS>(p.states + from * p.sts_s + own, nk, vec, h);
  auto at = [&](const void* base, int64_t i) {
    if constexpr (BF16) return raw2f<true>(((const uint16_t*)base)[i]);
    else return ((const float*)base)[i];
  };
  const float x = at(p.x, s * p.xs_t + dd);
  float dt = at(p.delta, s * p.ds_t + dd);
  const float z = p.z ? at(p.z, s * p.zs_t + dd) : 0.f;
#pragma unroll
  for (int k = 0; k < NS; ++k) {
    const int64_t n = k < nk ? n0 + k : 0;
    A[k] = p.A[dd * p.As_d + n * p.As_n];
    B[k] = at(p.B, s * p.Bs_t + n * p.Bs_n);
    C[k] = at(p.C, s * p.Cs_t + n * p.Cs_n);
  }
  const float Dk = p.Dskip ? p.Dskip[dd * p.Ds_d] : 0.f;
  if (p.dsoftplus) dt = softplus(dt + (p.dbias ? p.dbias[dd * p.dbs_d] : 0.f));
  float y = 0.f;
#pragma unroll
  for (int k = 0; k < NS; ++k) {
    const float u = dt * A[k], Ab = __builtin_amdgcn_exp2f(u * kLog2e);
    const float c = EULER ? dt : fabsf(u) < 0.25f ? dt * phi(u) : (Ab - 1.f) / A[k];
    h[k] = __builtin_fmaf(Ab, h[k], c * (x * B[k]));
    if (k < nk) y = __builtin_fmaf(C[k], h[k], y);
  }
  if (to >= 0) store_block<NS>(p.states + to * p.sts_s + own, nk, vec, h);
  y += other<1>(y);
  y += other<2>(y);
  if (j == 0 && ch_ok) {
    float v = __builtin_fmaf(Dk, x, y);
    if (p.z) v *= z * sigmoid(z);
    if (p.y_f32) ((float*)p.y)[s * p.ys_t + d] = v;
    else ((__bf16*)p.y)[s * p.ys_t + d] = (__bf16)v;
  }
}

template <bool BF16, int NS, bool EULER>
void launch_ns(const ScanPackedParams& p, hipStream_t stream) {
  const unsigned nblk = (unsigned)((p.D + kWaves * kCh - 1) / (kWaves * kCh));
  auto al = [](const void* ptr, int64_t bytes) { return ((uintptr_t)ptr % (uintptr_t)bytes) == 0; };
  // whole 16-byte words of a lane's states (the workspace's blocks are aligned and follow (D, N))
  const int vec_state = NS >= 4 && p.N % NS == 0 && al(p.states, 16) && p.sts_s % 4 == 0;
  if (!p.q.starts) {
    hipLaunchKernelGGL((step_packed_kernel<BF16, NS, EULER>), dim3(nblk * (unsigned)p.q.seqs), dim3(64 * kWaves), 0,
                       stream, p, nblk, vec_state);
    return;
  }
  // B and C: a lane's NS states by 16-byte words (or one smaller)
  const int64_t word = std::min<int64_t>(16, NS * (BF16 ? 2 : 4)), e = BF16 ? 2 : 4;
  const bool vec = p.N % NS == 0 && p.Bs_n == 1 && p.Cs_n == 1 && al(p.B, word) && al(p.C, word) &&
                   p.Bs_t * e % word == 0 && p.Cs_t * e % word == 0;
  const unsigned n = (unsigned)p.q.seqs + (unsigned)p.lines;
  const dim3 block(64 * kWaves);
  if (vec) {
    hipLaunchKernelGGL((scan_packed_kernel<BF16, NS, EULER, false, true>), dim3(nblk * n), block, 0, stream, p, nblk,
                       vec_state);
    if (p.lines)
      hipLaunchKernelGGL((scan_packed_kernel<BF16, NS, EULER, true, true>), dim3(nblk * (unsigned)p.lines), block, 0,
                         stream, p, nblk, vec_state);
  } else {
    hipLaunchKernelGGL((scan_packed_kernel<BF16, NS, EULER, false, false>), dim3(nblk * n), block, 0, stream, p, nblk,
                       vec_state);
    if (p.lines)
      hipLaunchKernelGGL((scan_packed_kernel<BF16, NS, EULER, true, false>), dim3(nblk * (unsigned)p.lines), block, 0,
                         stream, p, nblk, vec_state);
  }
}

template <bool BF16, bool EULER>
void launch_n(const ScanPackedParams& p, hipStream_t stream) {
  if (p.N <= 4) launch_ns<BF16, 1, EULER>(p, stream);
  else if (p.N <= 8) launch_ns<BF16, 2, EULER>(p, stream);
  else if (p.N <= 16) launch_ns<BF16, 4, EULER>(p, stream);
  else if (p.N <= 32) launch_ns<BF16, 8, EULER>(p, stream);
  else launch_ns<BF16, 16, EULER>(p, stream);
}

}  // namespace

ScanPackedPlan plan_scan_packed(int64_t tokens, int64_t seqs, int64_t dim, int64_t dstate, bool single) {
  ScanPackedPlan pl = {0, 0, 0, 0, 0, 0};
  (void)seqs;
  if (single) return pl;
  auto round256 = [](int64_t n) { return (n + 255) / 256 * 256; };
  // pieces of 16 channels that fill the card
  const int64_t waves = (dim + kCh - 1) / kCh;
  int64_t step = (tokens * waves / 4096 + kTile - 1) / kTile * kTile;
  step = std::max<int64_t>(step, 256);
  step = std::max<int64_t>(step, ((tokens + 254) / 255 + kTile - 1) / kTile * kTile);  // at most 255 lines
  pl.step = step;
  pl.lines = (tokens - 1) / step;
  pl.ws_H = pl.ws_E = round256(pl.lines * dim * dstate * 4);
  pl.ws_S = round256(pl.lines * dim * 4);
  pl.ws_total = pl.ws_H + pl.ws_E + pl.ws_S;
  return pl;
}

hipError_t launch_scan_packed(const ScanPackedParams& p, hipStream_t stream) {
  if (p.io_bf16) {
    if (p.euler) launch_n<true, true>(p, stream);
    else launch_n<true, false>(p, stream);
  } else {
    if (p.euler) launch_n<false, true>(p, stream);
    else launch_n<false, false>(p, stream);
  }
  return hipGetLastError();
}

}  // namespace ssm
