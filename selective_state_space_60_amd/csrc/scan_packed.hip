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
// sequence from zeros, and keeps each piece's end state and sum of delta; true end
// states follow from those without another walk.  The second pass corrects y: it
// walks a later piece again from its true state -- chained from the kept ones by
// each wave for itself -- and carries along what is left of that state, its product
// with the decays so far, which is what the first pass's states lack.  It stops at
// the end of the tile where that has come down to 2^-24 of every state where y is
// fp32 (half a step of the state: the walk itself holds no more of it), 2^-16 where y
// is bf16 (half a step is 2^-9); it decays on from there, but the state may shrink
// faster where later inputs cancel it: what y lacks is that part of the sum of its
// absolute terms, and a caller who needs more of it asks for an fp32 y.  States that
// decay are walked again over a short stretch only.  (16384 x 5120 bf16 in 24
// sequences, y bf16: 493 us, 521 with 2^-24; y fp32: 512, 498 with 2^-20.)
//
// Measured in a captured graph: 16384 x 5120 bf16 in 24 sequences, z, N 16: 491 us
// (traced from a cold cache: order 5, first pass 466, second 69).  The first pass's
// VALU issue is 95 % busy at 2.15 GHz: a tile's walk is 484 VALU operations in the fast
// form, of which the formula's seven a state and step are 448, and step sizes, forms,
// gate, loads and stores are 160; 713 in the mixed form, 1090 in the general one.  Where
// states are forgotten slowly every later piece is walked twice: delta around 7 10^-3
// 916 us, around 10^-3 1026.  1111 x 1536 fp32 in 37 sequences: 49 us, passes of few
// tiles each (33 and 21); 16384 x 5120 fp32: 916 us.
//
// Forms, chosen for each tile of a wave (delta A of its steps and channels):
//   small   all |delta A| < 1/8: expm1(u)/u by its Taylor polynomial; right for A = 0
//   fast    bf16 only: h <- Abar (h + q) - q, q = B x / A (the update multiplied out), 8
//           issue slots a state and step with the readout.  A step is off by the
//           roundings of q, 2^-22 |q|, whatever it adds, so it takes that every step of
//           every channel has |u| >= 2^-11 (its smallest delta and smallest |A|): then
//           that is 2^-11 of what the step adds, as its x and B are rounded to 2^-9.  One
//           step next to zero sends its tile to the next form, and a step of zero
//           leaves the state to the bit.
//   mixed   bf16 otherwise, A = 0 among it: (Abar - 1) / A, or delta where |delta A| <
//           2^-11, both to 2^-12; 11 issue slots (16384 x 5120 in 24 sequences with delta
//           around 10^-3: 1028 us, 1345 in the next form)
//   any     fp32 otherwise: (Abar - 1) / A, or the polynomial where |delta A| < 1/4; 17
//           issue slots
// fp32 has no fast form: it would keep its terms to 2^-14 where |u| >= 2^-8, and hardly
// any tile of common step sizes holds no smaller one (1111 x 1536 in 37 sequences, called:
// 51-53 us with it, 52-55 without; 38 where the largest step chose the form, and small ones
// lost up to a percent of the state).
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>

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

// (2^t - 1) / t for |t| < 1/4 log2(e): the Taylor series of expm1(u) / u, u = t ln 2,
// times ln 2, through u^5 (the next term is u^6 / 5040 < 5e-8).
__device__ __forceinline__ float ratio(float t) {
  constexpr float l1 = kLn2, l2 = l1 * kLn2, l3 = l2 * kLn2, l4 = l3 * kLn2, l5 = l4 * kLn2, l6 = l5 * kLn2;
  float q = l6 / 720.f;
  q = __builtin_fmaf(q, t, l5 / 120.f);
  q = __builtin_fmaf(q, t, l4 / 24.f);
  q = __builtin_fmaf(q, t, l3 / 6.f);
  q = __builtin_fmaf(q, t, l2 / 2.f);
  return __builtin_fmaf(q, t, l1);
}

enum Form : int { kSmall = 0, kFast = 1, kAny = 2, kEuler = 3, kMixed = 4 };

// A lane's constants of its states.
template <int NS>
struct Lane {
  float A[NS], iA[NS];  // A, 1/A (0 where A is 0)
};

// One step of a lane's states; returns its part of the readout.  dt: delta
// log2(e); x: x, or delta x (kEuler).  AGAIN (the second pass): `old`, what is
// left of the states that the piece started from, decays along.  No implicit fusing: the broadcast multiplies have
// to stay multiplies (an fma takes no DPP), and side by side (the compiler looks
// for a broadcast's uses over some twenty instructions only).
template <int NS, int FORM, bool AGAIN, int J>
__device__ __forceinline__ float step(float (&h)[NS], float (&old)[NS], const Lane<NS>& ln, float dt, float x,
                                      const float* bc) {
#pragma clang fp contract(off)
  constexpr int NP = 4 * NS;
  float t[NS], q[NS], B[NS], yp = 0.f;
#pragma unroll
  for (int k = 0; k < NS; ++k) t[k] = quad<J>(dt) * ln.A[k];
#pragma unroll
  for (int k = 0; k < NS; ++k) B[k] = bc[2 * J * NP + k];
#pragma unroll
  for (int k = 0; k < NS; ++k) q[k] = quad<J>(x) * (FORM == kFast ? ln.iA[k] : B[k]);
  const float d = quad<J>(dt) * kLn2;  // delta
#pragma unroll
  for (int k = 0; k < NS; ++k) {
    if constexpr (FORM == kFast) {
      // (as h + (Ab - 1)(h + q) a state that a large delta wipes out would leave its rounding behind)
      const float Ab = __builtin_amdgcn_exp2f(t[k]);
      q[k] *= B[k];
      h[k] = __builtin_fmaf(Ab, h[k] + q[k], -q[k]);
      if constexpr (AGAIN) old[k] *= Ab;
    } else {
      float Ab;
      if constexpr (FORM == kEuler) {
        Ab = __builtin_amdgcn_exp2f(t[k]);
      } else if constexpr (FORM == kMixed) {
        Ab = __builtin_amdgcn_exp2f(t[k]);
        const float far = (Ab - 1.f) * ln.iA[k];  // off by 2^-24 / |u| of itself (A > 0: twice that), delta by |u| / 2
        q[k] *= fabsf(t[k]) < 0x1p-11f * kLog2e ? d : far;
      } else {
        const float r = ratio(t[k]);
        float c = quad<J>(dt) * r;  // expm1(delta A) / A
        if constexpr (FORM == kSmall) {
          Ab = __builtin_fmaf(t[k], r, 1.f);
        } else {
          Ab = __builtin_amdgcn_exp2f(t[k]);
          const float far = (Ab - 1.f) * ln.iA[k];
          c = fabsf(t[k]) < 0.25f * kLog2e ? c : far;
        }
        q[k] *= c;
      }
      h[k] = __builtin_fmaf(Ab, h[k], q[k]);
      if constexpr (AGAIN) old[k] *= Ab;
    }
  }
#pragma unroll
  for (int k = 0; k < NS; ++k) {
    const float C = bc[(2 * J + 1) * NP + k];
    yp = k == 0 ? C * h[k] : __builtin_fmaf(C, h[k], yp);
  }
  return yp;
}

// Steps 4i .. 4i+3 of a tile; returns the readout of step 4i + (lane % 4).
// bc: the tile's B and C in LDS from this lane's first state on.
template <int NS, int FORM, bool AGAIN>
__device__ __forceinline__ float four_steps(float (&h)[NS], float (&old)[NS], const Lane<NS>& ln, float dt, float x,
                                            const float* bc) {
  // operands of later steps are not read ahead of these: that costs registers
  __builtin_amdgcn_sched_barrier(0);
  const float y0 = step<NS, FORM, AGAIN, 0>(h, old, ln, dt, x, bc);
  const float y1 = step<NS, FORM, AGAIN, 1>(h, old, ln, dt, x, bc);
  const float y2 = step<NS, FORM, AGAIN, 2>(h, old, ln, dt, x, bc);
  const float y3 = step<NS, FORM, AGAIN, 3>(h, old, ln, dt, x, bc);
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

// One stream of a wave: the address of the current tile's first row at the wave's
// first channel (or state), the bytes of four rows, and this lane's place in a tile.
// That place is fixed and the rows 4i are scalar offsets, so a whole tile's loads
// and stores cost no vector arithmetic, and the walk few scalar registers.  What
// does not exist -- channels, states, rows behind the piece -- goes out of range by
// the lane's offset.
struct Stream {
  const char* at;
  uint32_t four;
  uint32_t off;

  __device__ __forceinline__ void set(const void* base, int64_t st, int row, int64_t first, int e, uint32_t lane_off) {
    at = (const char*)base + ((int64_t)row * st + first) * e;
    four = 4 * (uint32_t)st * (uint32_t)e;
    off = lane_off;
  }
  __device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer() const { return rsrc(at, kFar); }
  __device__ __forceinline__ void advance() { at += 4 * (int64_t)four; }
};

// A wave's streams over one piece.
template <bool BF16, int NS, bool VEC>
struct Streams {
  static constexpr int E = BF16 ? 2 : 4;
  using T = Tile<BF16, NS, VEC>;
  Stream x, dt, z, y, B, C;
  uint32_t nB, nC;   // bytes from state to state
  int j, r, kn;      // lane % 4, lane / 4, states of the lane that exist
  bool has_z, y_f32;

  __device__ __forceinline__ Streams(const ScanPackedParams& p, int64_t d0, int lane, int t)
      : j(lane % 4), r(lane / 4), has_z(p.z != nullptr), y_f32(p.y_f32) {
    const int64_t ch = lane / 4, n0 = NS * j;
    const bool ok = d0 + ch < p.D, in = n0 < p.N;
    kn = in ? (int)(p.N - n0) : 0;
    auto place = [&](int64_t st, uint32_t e) { return ok ? ((uint32_t)j * (uint32_t)st + (uint32_t)ch) * e : kFar; };
    auto states = [&](int64_t st, int64_t sn) {
      return in ? ((uint32_t)r * (uint32_t)st + (uint32_t)n0 * (uint32_t)sn) * E : kFar;
    };
    x.set(p.x, p.xs_t, t, d0, E, place(p.xs_t, E));
    dt.set(p.delta, p.ds_t, t, d0, E, place(p.ds_t, E));
    z.set(has_z ? p.z : p.x, p.zs_t, t, d0, E, place(p.zs_t, E));
    const int ye = 2 << p.y_f32;  // y_f32 is 0 or 1 (a select would move the address to vector registers)
    y.set(p.y, p.ys_t, t, d0, ye, place(p.ys_t, (uint32_t)ye));
    B.set(p.B, p.Bs_t, t, 0, E, states(p.Bs_t, p.Bs_n));
    C.set(p.C, p.Cs_t, t, 0, E, states(p.Cs_t, p.Cs_n));
    nB = (uint32_t)p.Bs_n * E;
    nC = (uint32_t)p.Cs_n * E;
  }

  template <bool FULL>
  __device__ __forceinline__ void load_rows(const Stream& s, int left, uint32_t (&v)[4]) const {
    const auto b = s.buffer();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t off = FULL ? s.off : 4 * i + j < left ? s.off + i * s.four : kFar;
      const int so = FULL ? (int)(i * s.four) : 0;
      if constexpr (BF16) v[i] = __builtin_amdgcn_raw_buffer_load_b16(b, (int)off, so, 0);
      else v[i] = __builtin_amdgcn_raw_buffer_load_b32(b, (int)off, so, 0);
    }
  }

  // Row r of B or C.
  __device__ __forceinline__ void load_states(const Stream& s, uint32_t sn, uint32_t off, uint32_t (&o)[T::kWords]) const {
    const auto b = s.buffer();
    if constexpr (VEC) {  // this lane's NS states lie side by side, all in or all out
      if constexpr (T::kWords == 1) {
        if constexpr (BF16 && NS == 1) o[0] = load_raw<true>(b, off);
        else o[0] = __builtin_amdgcn_raw_buffer_load_b32(b, (int)off, 0, 0);
      } else if constexpr (T::kWords == 2) {
        const auto v = __builtin_amdgcn_raw_buffer_load_b64(b, (int)off, 0, 0);
        o[0] = v[0]; o[1] = v[1];
      } else {
#pragma unroll
        for (int i = 0; i < T::kWords / 4; ++i) {
          const auto v = __builtin_amdgcn_raw_buffer_load_b128(b, (int)(off + 16u * i), 0, 0);
          o[4 * i] = v[0]; o[4 * i + 1] = v[1]; o[4 * i + 2] = v[2]; o[4 * i + 3] = v[3];
        }
      }
    } else {
#pragma unroll
      for (int k = 0; k < NS; ++k) o[k] = load_raw<BF16>(b, k < kn ? off + (uint32_t)k * sn : kFar);
    }
  }

  template <bool FULL>
  __device__ __forceinline__ void load_tile(int left, T& o) const {
    load_rows<FULL>(x, left, o.x);
    load_rows<FULL>(dt, left, o.dt);
    if (has_z) load_rows<FULL>(z, left, o.z);
    load_states(B, nB, FULL || r < left ? B.off : kFar, o.B);
    load_states(C, nC, FULL || r < left ? C.off : kFar, o.C);
  }

  // The next tile, `left` of whose rows belong to the piece (<= 0: none); what does not exist reads zeros.
  __device__ __forceinline__ void load(int left, T& o) {
    if (left >= kTile) load_tile<true>(kTile, o);
    else load_tile<false>(left, o);
    x.advance();
    dt.advance();
    z.advance();
    B.advance();
    C.advance();
  }

  template <bool FULL, bool F32>
  __device__ __forceinline__ void store_rows(int left, const float (&v)[4]) const {
    const auto b = y.buffer();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t off = FULL ? y.off : 4 * i + j < left ? y.off + i * y.four : kFar;
      const int so = FULL ? (int)(i * y.four) : 0;
      if constexpr (F32) __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(v[i]), b, (int)off, so, 0);
      else __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(uint16_t, (__bf16)v[i]), b, (int)off, so, 0);
    }
  }

  // y of the next tile.
  __device__ __forceinline__ void store(int left, const float (&v)[4]) {
    if (left >= kTile) {
      if (!BF16 || y_f32) store_rows<true, true>(left, v);
      else store_rows<true, false>(left, v);
    } else {
      if (!BF16 || y_f32) store_rows<false, true>(left, v);
      else store_rows<false, false>(left, v);
    }
    y.advance();
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

// The state behind a piece: 2^t h + e.  Where A > 0 the product of a piece's decays
// can pass the largest fp32 next to a state that is zero or small: 2^t in halves, and
// a zero state stays one (4000 x 128 fp32, 62 lines: 33.8 -> 35.2 us).  An infinite
// state stays infinite, also where 2^t is below the smallest fp32 (no decay is zero):
// the halves end at 2^-126, which leaves at most 2^-124 of a finite one.  (Asking
// whether h is infinite stands in the chain from line to line: 500 x 64 bf16 17.3 ->
// 21.3 us.)
__device__ __forceinline__ float passed(float h, float t, float e) {
  const float half = fmaxf(__builtin_amdgcn_exp2f(0.5f * t), 0x1p-126f);
  return h != 0.f ? __builtin_fmaf(half, half * h, e) : e;
}

// The state at grid line `line` of a sequence that crosses line `first` first:
// from that line's state on, each piece's end state and the decay over the piece
// applied to the state before it.  Latency is all there is: several lines are
// asked for at a time.
template <int NS>
__device__ __forceinline__ void enter(const ScanPackedParams& p, const Lane<NS>& ln, int first, int line, int64_t own,
                                      int64_t d, int nk, bool vec, float (&h)[NS]) {
  constexpr int kLines = NS <= 4 ? 12 : 8;
  const int64_t words = p.D * p.N;
  load_block<NS>(p.H + (int64_t)(first - 1) * words + own, nk, vec, h);
#pragma unroll 1
  for (int l0 = first + 1; l0 <= line; l0 += kLines) {
    float e[kLines][NS], sum[kLines];
#pragma unroll
    for (int i = 0; i < kLines; ++i) {
      const int64_t l = (l0 + i < line ? l0 + i : line) - 1;
      load_block<NS>(p.H + l * words + own, nk, vec, e[i]);
      sum[i] = p.dsum[l * p.D + d];
    }
#pragma unroll
    for (int i = 0; i < kLines; ++i)
      if (l0 + i <= line)
#pragma unroll
        for (int k = 0; k < NS; ++k) h[k] = passed(h[k], ln.A[k] * sum[i], e[i][k]);
  }
}

// One piece of one sequence for 16 channels.  AGAIN: the second pass over a later
// piece (packed_pieces.h).
template <bool BF16, int NS, bool EULER, bool AGAIN, bool VEC>
__global__ __launch_bounds__(64 * kWaves, NS <= 4 ? 4 : NS == 8 ? 2 : 1) void scan_packed_kernel(ScanPackedParams p, unsigned nblk, int vec_state) {
  constexpr int NP = 4 * NS;
  constexpr bool kMultiplied = BF16 && !EULER;  // kFast is one of the forms
  constexpr int kRest = BF16 ? kMixed : kAny;   // what is left
  __shared__ __align__(16) float lds[kWaves][2][kTile][2][NP];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), lane = threadIdx.x % 64;
  const int64_t d0 = ((int64_t)(blockIdx.x % nblk) * kWaves + wave) * kCh;
  if (d0 >= p.D) return;
  // the piece: rows [begin, end) of sequence s; `line` > 0: from that grid line on
  int piece = (int)(blockIdx.x / nblk);
  if (!AGAIN && p.order) piece = p.order[piece];
  int s = piece - p.lines, line = 0;
  packed::Run seq, run;
  if (!AGAIN && s >= 0) {
    seq = sequence_of(p.q, s);
    run = p.lines ? packed::first_piece(seq, p.step) : seq;
  } else {
    line = piece + 1;
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
  float h[NS], old[NS];
  float amax = 0.f, amin = __builtin_inff();  // of |A|
#pragma unroll
  for (int k = 0; k < NS; ++k) {
    const float a = k < nk ? p.A[dd * p.As_d + (n0 + k) * p.As_n] : -1.f;
    ln.A[k] = a;
    ln.iA[k] = a != 0.f ? 1.f / a : 0.f;
    amax = k < nk ? fmaxf(amax, fabsf(a)) : amax;
    amin = k < nk ? fminf(amin, fabsf(a)) : amin;
    h[k] = old[k] = 0.f;
  }
  // of the channel
  amax = fmaxf(amax, other<1>(amax));
  amax = fmaxf(amax, other<2>(amax));
  amin = fminf(amin, other<1>(amin));
  amin = fminf(amin, other<2>(amin));
  const float Dk = p.Dskip && ch_ok ? p.Dskip[dd * p.Ds_d] : 0.f;
  const float bias = p.dbias && ch_ok ? p.dbias[dd * p.dbs_d] : 0.f;
  const uint64_t alive = __ballot(ch_ok);
  const bool vec = vec_state != 0;
  if constexpr (AGAIN) {
    enter<NS>(p, ln, seq.begin / p.step + 1, line, own, dd, nk, vec, h);
#pragma unroll
    for (int k = 0; k < NS; ++k) old[k] = h[k];
  } else if (line == 0) {
    const int64_t from = slots_of(p.q, s, p.A).from;
    if (from >= 0) load_block<NS>(p.states + from * p.sts_s + own, nk, vec, h);
  }

  Streams<BF16, NS, VEC> st(p, d0, lane, run.begin);
  const bool has_z = st.has_z, dsoftplus = p.dsoftplus;
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
  const float close = p.y_f32 ? 0x1p-24f : 0x1p-16f;
  int left = run.end - run.begin;
  st.load(left, tile);
  stage(0);
  int buf = 0;
  for (; left > 0; left -= kTile, buf ^= 1) {
    float x[4], dt[4], xs[4], gate[4];
    float tmax = 0.f, tmin = __builtin_inff();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[i] = raw2f<BF16>(tile.x[i]);
      dt[i] = raw2f<BF16>(tile.dt[i]);
    }
    if (dsoftplus) {
#pragma unroll
      for (int i = 0; i < 4; ++i) dt[i] = softplus(dt[i] + bias);
      if (left < kTile) {  // uniform; past the piece nothing changes
#pragma unroll
        for (int i = 0; i < 4; ++i) dt[i] = 4 * i + j < left ? dt[i] : 0.f;
      }
    }
    if (has_z) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float z = raw2f<BF16>(tile.z[i]);
        gate[i] = z * sigmoid(z);
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      xs[i] = EULER ? dt[i] * x[i] : x[i];
      dt[i] *= kLog2e;
      tmax = fmaxf(tmax, fabsf(dt[i]));
      if constexpr (kMultiplied) tmin = fminf(tmin, fabsf(dt[i]));
      if constexpr (!AGAIN) sum_dt += dt[i];
    }
    if constexpr (kMultiplied) {
      if (left < kTile) {  // uniform; what is past the piece is no step, and changes nothing in any form
        tmin = __builtin_inff();
#pragma unroll
        for (int i = 0; i < 4; ++i) tmin = 4 * i + j < left ? fminf(tmin, fabsf(dt[i])) : tmin;
      }
    }
    st.load(left - kTile, tile);
    wave_sync();
    const float* bc = lds[wave][buf][0][0] + n0;
    float y[4];
    // the four lanes hold different steps
    tmax = fmaxf(tmax, other<1>(tmax));
    tmax = fmaxf(tmax, other<2>(tmax));
    int form = EULER ? kEuler : __ballot(!(tmax * amax < 0.125f * kLog2e)) == 0 ? kSmall : kRest;
    if constexpr (kMultiplied) {
      tmin = fminf(tmin, other<1>(tmin));
      tmin = fminf(tmin, other<2>(tmin));
      if (form == kRest && (__ballot(!(tmin * amin >= 0x1p-11f * kLog2e)) & alive) == 0) form = kFast;
    }
    if constexpr (EULER) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        y[i] = four_steps<NS, kEuler, AGAIN>(h, old, ln, dt[i], xs[i], bc + i * 8 * NP);
        // a tile is one block of code here, and all its factors would be formed first, and spilled
        if (AGAIN && i < 3) asm volatile("" : "+v"(h[0]), "+v"(dt[i + 1]), "+v"(xs[i + 1]));
      }
    } else if (form == kSmall) {
#pragma unroll
      for (int i = 0; i < 4; ++i) y[i] = four_steps<NS, kSmall, AGAIN>(h, old, ln, dt[i], xs[i], bc + i * 8 * NP);
    } else if (kMultiplied && form == kFast) {
      constexpr int kForm = kMultiplied ? kFast : kAny;  // (no other variant holds that code)
#pragma unroll
      for (int i = 0; i < 4; ++i) y[i] = four_steps<NS, kForm, AGAIN>(h, old, ln, dt[i], xs[i], bc + i * 8 * NP);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) y[i] = four_steps<NS, kRest, AGAIN>(h, old, ln, dt[i], xs[i], bc + i * 8 * NP);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) y[i] = __builtin_fmaf(Dk, x[i], y[i]);
    if (has_z) {
#pragma unroll
      for (int i = 0; i < 4; ++i) y[i] *= gate[i];
    }
    st.store(left, y);
    stage(buf ^ 1);
    if constexpr (AGAIN) {
      bool same = true;
#pragma unroll
      for (int k = 0; k < NS; ++k)  // (an infinite state, whose old part is infinite too, is never met)
        same = same && fabsf(old[k]) <= close * fabsf(h[k]) && fabsf(h[k]) < __builtin_inff();
      if (__ballot(!same) == 0) {
        met = left > kTile;
        break;
      }
    }
  }

  const ScanPackedParams& q = args_anew<ScanPackedParams>();
  const int64_t words = q.D * q.N;
  const bool inside = run.end < seq.end;  // the piece ends at a line inside the sequence
  if constexpr (!AGAIN) {
    if (inside || line > 0) {
      // the sequence's end after a line is not the true one yet, and another workgroup may not have read the slot
      const int64_t at = inside ? run.end / q.step - 1 : line - 1;
      store_block<NS>((inside ? q.H : q.E) + at * words + own, nk, vec, h);
      sum_dt += other<1>(sum_dt);
      sum_dt += other<2>(sum_dt);
      if (j == 0 && ch_ok) (inside ? q.dsum : q.esum)[at * q.D + d] = sum_dt;
      return;
    }
  }
  const int64_t to = inside ? -1 : slots_of(q.q, s, q.A).to;
  if (to < 0) return;
  if (AGAIN && met) {
    float e[NS];
    load_block<NS>(q.E + (int64_t)(line - 1) * words + own, nk, vec, e);
    const float sum = q.esum[(int64_t)(line - 1) * q.D + dd];
    enter<NS>(q, ln, seq.begin / q.step + 1, line, own, dd, nk, vec, h);
#pragma unroll
    for (int k = 0; k < NS; ++k) h[k] = passed(h[k], ln.A[k] * sum, e[k]);
  }
  store_block<NS>(q.states + to * q.sts_s + own, nk, vec, h);
}

// The pieces of the first pass by their length, the longest first: one workgroup,
// a piece for each thread.
__global__ __launch_bounds__(kScanOrdered) void order_kernel(ScanPackedParams p) {
  __shared__ int len[kScanOrdered], starts[kScanOrdered + 1];
  const int i = (int)threadIdx.x, n = p.lines + p.q.seqs;
  for (int k = i; k <= p.q.seqs; k += kScanOrdered) starts[k] = p.q.starts[k];
  __syncthreads();
  int mine = -1;
  auto rows = [&](int s) { return packed::sequence(starts[s], starts[s + 1], p.q.tokens); };
  if (i < n) {
    packed::Run r;
    if (i < p.lines) {
      const int at = (i + 1) * p.step;
      const int s = packed::last_start(p.q.seqs, [&](int lo, int stride, int count) {
        int c = 0;
        for (int k = 0; k < count; ++k) c += starts[lo + k * stride] <= at;
        return c;
      });
      r = s < 0 ? packed::Run{0, 0} : packed::later_piece(rows(s), at, p.step);
    } else {
      r = packed::first_piece(rows(i - p.lines), p.step);
    }
    mine = r.end - r.begin;
  }
  len[i] = mine;
  __syncthreads();
  int rank = 0;
  for (int k = 0; k < n; ++k) rank += len[k] > mine || (len[k] == mine && k < i);
  if (i < n) p.order[rank] = i;
}

// ------------------------------------------------------------ single tokens

// A lane's NS states of a row: by words where `vec` says that they lie side by
// side and aligned (all of them in or all out), else one by one.
template <bool BF16, int NS>
__device__ __forceinline__ void load_row(const void* base, int64_t at, int64_t sn, int n0, int nk, bool vec,
                                         float (&o)[NS]) {
  constexpr int E = BF16 ? 2 : 4;
  const char* const p = (const char*)base + (at + (nk > 0 ? n0 : 0) * sn) * E;
  if (NS > 1 && vec) {
    uint32_t w[NS * E / 4 > 0 ? NS * E / 4 : 1];
    if constexpr (NS * E % 16 == 0) {
#pragma unroll
      for (int i = 0; i < NS * E / 16; ++i) {
        const uint4 v = ((const uint4*)p)[i];
        w[4 * i] = v.x; w[4 * i + 1] = v.y; w[4 * i + 2] = v.z; w[4 * i + 3] = v.w;
      }
    } else if constexpr (NS * E == 8) {
      const uint2 v = *(const uint2*)p;
      w[0] = v.x; w[1] = v.y;
    } else {
      w[0] = *(const uint32_t*)p;
    }
#pragma unroll
    for (int k = 0; k < NS; ++k)
      o[k] = BF16 ? __uint_as_float((k & 1) ? (w[k >> 1] & 0xFFFF0000u) : (w[k >> 1] << 16)) : __uint_as_float(w[BF16 ? 0 : k]);
    return;
  }
#pragma unroll
  for (int k = 0; k < NS; ++k) {
    const char* const q = p + (k < nk ? k : 0) * sn * E;
    o[k] = BF16 ? raw2f<true>(*(const uint16_t*)q) : *(const float*)q;
  }
}

// One token of each sequence.  A wave has 16 channels of U sequences, a lane NS
// states of one channel of each, read and written 16 bytes at a time, all U asked
// for at once.  Bound by that traffic (64 x 5120 x 16 bf16: 13.2 us for 45 MB), so every
// state takes the accurate form.
template <bool BF16, int NS, bool EULER, int U>
__global__ __launch_bounds__(64 * kWaves) void step_packed_kernel(ScanPackedParams p, unsigned nblk, int vec_state,
                                                                  int vec_bc, int vec_a) {
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), lane = threadIdx.x % 64;
  const int s0 = (int)(blockIdx.x / nblk) * U;
  const int64_t d0 = ((int64_t)(blockIdx.x % nblk) * kWaves + wave) * kCh;
  if (d0 >= p.D) return;
  const int j = lane % 4, n0 = j * NS;
  const int64_t d = d0 + lane / 4;
  const bool ch_ok = d < p.D;
  const int64_t dd = ch_ok ? d : d0;
  const int nk = !ch_ok || n0 >= p.N ? 0 : (p.N - n0 < NS ? (int)(p.N - n0) : NS);
  const int64_t own = dd * p.N + (n0 < p.N ? n0 : 0);
  const bool vec = vec_state != 0;
  auto at = [&](const void* base, int64_t i) {
    if constexpr (BF16) return raw2f<true>(((const uint16_t*)base)[i]);
    else return ((const float*)base)[i];
  };
  float h[U][NS], B[U][NS], C[U][NS], x[U], dt[U], z[U], A[NS];
  int64_t to[U];
  Slots slot[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    // the last sequence again where there are no U left: its results are not stored twice
    const int s = s0 + u < p.q.seqs ? s0 + u : p.q.seqs - 1;
    slot[u] = slots_of(p.q, s, p.A);
    to[u] = s0 + u < p.q.seqs ? slot[u].to : -1;
    x[u] = at(p.x, s * p.xs_t + dd);
    dt[u] = at(p.delta, s * p.ds_t + dd);
    z[u] = p.z ? at(p.z, s * p.zs_t + dd) : 0.f;
    load_row<BF16, NS>(p.B, s * p.Bs_t, p.Bs_n, n0, nk, vec_bc, B[u]);
    load_row<BF16, NS>(p.C, s * p.Cs_t, p.Cs_n, n0, nk, vec_bc, C[u]);
  }
  load_row<false, NS>(p.A, dd * p.As_d, p.As_n, n0, nk, vec_a, A);
  const float Dk = p.Dskip ? p.Dskip[dd * p.Ds_d] : 0.f;
  const float bias = p.dbias ? p.dbias[dd * p.dbs_d] : 0.f;
  // all that needs no slot is on its way by now
#pragma unroll
  for (int u = 0; u < U; ++u) {
#pragma unroll
    for (int k = 0; k < NS; ++k) h[u][k] = 0.f;
    if (slot[u].from >= 0) load_block<NS>(p.states + slot[u].from * p.sts_s + own, nk, vec, h[u]);
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    float v = dt[u];
    if (p.dsoftplus) v = softplus(v + bias);
    const float dte = v * kLog2e;
    float y = 0.f;
#pragma unroll
    for (int k = 0; k < NS; ++k) {
      const float t = dte * A[k], Ab = __builtin_amdgcn_exp2f(t);
      const float far = (Ab - 1.f) * __builtin_amdgcn_rcpf(A[k]), near = dte * ratio(t);
      const float c = EULER ? v : fabsf(t) < 0.25f * kLog2e ? near : far;
      h[u][k] = __builtin_fmaf(Ab, h[u][k], c * (x[u] * B[u][k]));
      y = __builtin_fmaf(k < nk ? C[u][k] : 0.f, k < nk ? h[u][k] : 0.f, y);
    }
    if (to[u] >= 0) store_block<NS>(p.states + to[u] * p.sts_s + own, nk, vec, h[u]);
    y += other<1>(y);
    y += other<2>(y);
    if (j == 0 && ch_ok && s0 + u < p.q.seqs) {
      float o = __builtin_fmaf(Dk, x[u], y);
      if (p.z) o *= z[u] * sigmoid(z[u]);
      const int64_t i = (int64_t)(s0 + u) * p.ys_t + d;
      if (p.y_f32) ((float*)p.y)[i] = o;
      else ((__bf16*)p.y)[i] = (__bf16)o;
    }
  }
}

template <bool BF16, int NS, bool EULER>
void launch_ns(const ScanPackedParams& p, hipStream_t stream) {
  const unsigned nblk = (unsigned)((p.D + kWaves * kCh - 1) / (kWaves * kCh));
  auto al = [](const void* ptr, int64_t bytes) { return ((uintptr_t)ptr % (uintptr_t)bytes) == 0; };
  // whole 16-byte words of a lane's states (the workspace's blocks are aligned and follow (D, N))
  const int vec_state = NS >= 4 && p.N % NS == 0 && al(p.states, 16) && p.sts_s % 4 == 0;
  // B and C: a lane's NS states by 16-byte words (or one smaller)
  const int64_t word = std::min<int64_t>(16, NS * (BF16 ? 2 : 4)), e = BF16 ? 2 : 4;
  const bool vec = p.N % NS == 0 && p.Bs_n == 1 && p.Cs_n == 1 && al(p.B, word) && al(p.C, word) &&
                   p.Bs_t * e % word == 0 && p.Cs_t * e % word == 0;
  if (!p.q.starts) {
    const int vec_a = p.N % NS == 0 && p.As_n == 1 && al(p.A, std::min(16, 4 * NS)) && p.As_d % std::min(4, NS) == 0;
    // two sequences a wave where that leaves two workgroups a compute unit: 64 x 5120
    // fp32 16.3 us one at a time, 13.2 with two, 13.6 with four
    constexpr int U = NS <= 4 ? 2 : 1;
    const unsigned groups = ((unsigned)p.q.seqs + U - 1) / U;
    if (U > 1 && nblk * groups >= 512)
      hipLaunchKernelGGL((step_packed_kernel<BF16, NS, EULER, U>), dim3(nblk * groups), dim3(64 * kWaves), 0, stream, p,
                         nblk, vec_state, vec, vec_a);
    else
      hipLaunchKernelGGL((step_packed_kernel<BF16, NS, EULER, 1>), dim3(nblk * (unsigned)p.q.seqs), dim3(64 * kWaves), 0,
                         stream, p, nblk, vec_state, vec, vec_a);
    return;
  }
  const unsigned n = (unsigned)p.q.seqs + (unsigned)p.lines;
  const dim3 block(64 * kWaves);
  if (p.order) hipLaunchKernelGGL(order_kernel, dim3(1), dim3(kScanOrdered), 0, stream, p);
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
  ScanPackedPlan pl = {};
  if (single) return pl;
  auto round256 = [](int64_t n) { return (n + 255) / 256 * 256; };
  // Three waves for each SIMD (four are resident).  Fewer, longer pieces leave them
  // idle at the end, more are walked again: 16384 x 5120 bf16 at 2 waves a SIMD
  // 646 us, 2.5 492, 3 495, 4 498.
  constexpr int64_t kSimds = 256 * 4;
  const int64_t waves = (dim + kCh - 1) / kCh;
  int64_t step = (tokens * waves / (3 * kSimds) + kTile - 1) / kTile * kTile;
  // Where that many waves are not to be had, the rows that a wave walks in either pass
  // (16 in 2.2 us) stand against the lines that it chains a state over: about
  // sqrt(0.8 tokens) rows a piece.  Measured before states were passed on in halves and
  // fp32 lost its fast form: 4000 x 128 fp32 33.8 us at its 64 rows, 32.8 at 48; 2000 x
  // 768 bf16 35.3 at its 48, 38.0 at 32; 500 x 64 bf16 16.3 at its 16, and 26.7 at 64
  // (chained four lines at a time).  Now, at the rule's rows: 43.1, 37.8 and 17.6.
  step = std::max(step, ((int64_t)std::sqrt(0.8 * (double)tokens) + kTile / 2) / kTile * kTile);
  step = std::max<int64_t>(step, kTile);
  step = std::max<int64_t>(step, ((tokens + 254) / 255 + kTile - 1) / kTile * kTile);  // at most 255 lines
  pl.step = step;
  pl.lines = (tokens - 1) / step;
  const int64_t n = pl.lines + seqs;
  pl.ws_H = pl.ws_E = round256(pl.lines * dim * dstate * 4);
  pl.ws_S = round256(2 * pl.lines * dim * 4);
  // The longest first where they do not run all at once (16384 x 5120 in 24
  // sequences: 740 -> 590 us), unless the 4 us that this takes are too many.
  pl.ws_order = n <= kScanOrdered && n * waves > 4096 && tokens * waves >= (1 << 20) ? round256(n * 4) : 0;
  pl.ws_total = pl.ws_H + pl.ws_E + pl.ws_S + pl.ws_order;
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
