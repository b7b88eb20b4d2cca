// Beam search's selection for gfx950: of every batch element's beams x vocab
// continuations the k of the highest score, score = scores[n] + logits[n, v] -
// log sum exp logits[n, :].
//
// One pass over the logits: a wave holds a stretch of one row in registers and
// finds its largest logit, its sum of exp(logit - largest) and its k best (logit,
// index) in falling order.  A lower bound for the k-th best is the k-th of the 64
// lanes' largest values, found bit by bit with ballots; the few values that reach it
// go to LDS, where each one's rank is counted.  The four waves of a workgroup, a
// piece of the row, join theirs (the fewer lists, the shorter the second kernel).  A
// second kernel, one wave for each batch element, adds the pieces' sums
// to each row's normaliser and chooses among all pieces' candidates in the same
// way.  Each logit is read once.  64 x 4 beams x 50281 bf16, k 8: 19 us, of which
// the bytes are 5.3; most is the first kernel's VALU issue (17 operations a value, 9 us)
// with the latency of its loads and of its selection around it, since all waves are
// resident at once.  5 beams x 32000 fp32: 11 us, two kernels of one pass of latencies
// each.  Not kept: candidates taken from the registers by an unrolled loop instead of
// read again (22 us: a branch for each of the 64 values).
//
// The normaliser: a lane adds at most 64 exponentials in fp32, six levels join a wave's
// lanes, four additions the workgroup's waves: up to 16384 tokens.  The pieces are added
// up in fp64.  With 17 ulp of the exponentials (arguments down to -32 count) and three of
// the weights that waves and pieces are joined with, that is within 57 2^-23 of itself.
//
// Order: logits are compared as integers that rise with the value (-0 as +0),
// with the index behind, lower first; scores in fp64, then the index.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "serve_device.h"

namespace ssm {
namespace {

using namespace dev;

constexpr int kWaves = 4;
constexpr int kSmall = 16, kLarge = 64;  // values of a lane
constexpr int kHeld = 128;               // candidates in LDS: k <= 64 kept, and 64 more
constexpr uint32_t kBanned = 0x007FFFFFu;  // order(-inf)

// Rises with the value; -0 counts as +0; 0 stands for no value (no float maps to it but a NaN).
__device__ __forceinline__ uint32_t order(float v) {
  const uint32_t b = __float_as_uint(v + 0.f);
  return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float value(uint32_t o) {
  return __uint_as_float((o & 0x80000000u) ? o & 0x7FFFFFFFu : ~o);
}
__device__ __forceinline__ uint64_t order64(double v) {
  const uint64_t b = (uint64_t)__double_as_longlong(v + 0.0);
  return (b >> 63) ? ~b : b | (1ull << 63);
}
__device__ __forceinline__ double value64(uint64_t o) {
  return __longlong_as_double((long long)((o >> 63) ? o & ~(1ull << 63) : ~o));
}

__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// The k-th largest of the lanes' values (0 where fewer than k are not 0), of
// whose lowest `low` bits only zeros are kept.
__device__ __forceinline__ uint32_t kth_largest(uint32_t v, int k, int low) {
  uint32_t t = 0;
  for (int bit = 31; bit >= low; --bit) {
    const uint32_t c = t | 1u << bit;
    if (__popcll(__ballot(v >= c)) >= k) t = c;
  }
  return t;
}

// A wave's candidates in LDS, an order and an index each; the k best in falling
// order after keep().  All lanes call together; held and bar are uniform.
template <class T>
struct Held {
  T* hi;         // kHeld
  uint32_t* lo;  // kHeld: ~index
  int k, held;
  T bar_hi;      // the k-th best so far: what does not pass it is none of the k
  uint32_t bar_lo;

  __device__ __forceinline__ Held(T* h, uint32_t* l, int n) : hi(h), lo(l), k(n), held(0), bar_hi(0), bar_lo(0) {}

  __device__ __forceinline__ bool passes(T h, uint32_t l) const { return h > bar_hi || (h == bar_hi && l > bar_lo); }

  __device__ __forceinline__ void keep() {
    const int lane = (int)__lane_id();
    wave_sync();
    T h[2];
    uint32_t l[2];
    int rank[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const bool in = 64 * i + lane < held;
      h[i] = in ? hi[64 * i + lane] : 0;
      l[i] = in ? lo[64 * i + lane] : 0;
    }
    // four at a time: the reads' latency is all there is (what lies behind `held` counts as nothing)
#pragma unroll 1
    for (int j0 = 0; j0 < held; j0 += 4) {
      T oh[4];
      uint32_t ol[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        oh[j] = hi[j0 + j];
        ol[j] = lo[j0 + j];
      }
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int i = 0; i < 2; ++i)
          rank[i] += j0 + j < held && (oh[j] > h[i] || (oh[j] == h[i] && ol[j] > l[i]));
    }
    wave_sync();
#pragma unroll
    for (int i = 0; i < 2; ++i)
      if (64 * i + lane < held && rank[i] < k) {
        hi[rank[i]] = h[i];
        lo[rank[i]] = l[i];
      }
    wave_sync();
    held = held < k ? held : k;
    if (held == k) {
      bar_hi = hi[k - 1];
      bar_lo = lo[k - 1];
    }
  }

  // The candidates of the lanes in `mask`; there is room for them.
  __device__ __forceinline__ void append(uint64_t mask, T h, uint32_t l) {
    const int lane = (int)__lane_id();
    if (mask >> lane & 1) {
      const int at = held + __popcll(mask & ((1ull << lane) - 1));
      hi[at] = h;
      lo[at] = l;
    }
    held += __popcll(mask);
  }

  // The candidates of the lanes where `in`.
  __device__ __forceinline__ void add(bool in, T h, uint32_t l) {
    uint64_t mask = __ballot(in && passes(h, l));
    if (held + __popcll(mask) > kHeld) {  // uniform
      keep();
      mask = __ballot(in && passes(h, l));
    }
    append(mask, h, l);
  }
};

// Value g of a 16-byte load.
template <bool F32>
__device__ __forceinline__ float unpack(const uint32_t (&raw)[4], int g) {
  if constexpr (F32) return __uint_as_float(raw[g]);
  else return __uint_as_float((g & 1) ? (raw[g >> 1] & 0xFFFF0000u) : (raw[g >> 1] << 16));
}

// E values of each thread are a piece; lane l holds G values side by side of every
// run of 64 G of its wave's stretch.
template <bool F32, int E>
__global__ __launch_bounds__(64 * kWaves) void beam_piece_kernel(BeamParams p) {
  constexpr int G = F32 ? 4 : 8;  // values of a 16-byte load
  constexpr int NL = E / G;       // loads
  __shared__ uint32_t hi[kWaves][kHeld], lo[kWaves][kHeld];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), lane = threadIdx.x % 64;
  __shared__ float2 stat[kWaves];
  __shared__ int count[kWaves];
  // (32-bit quotients: a 64-bit one is a hundred operations in front of the loads)
  const uint32_t job = blockIdx.x, row = job / (uint32_t)p.parts;
  const int part = (int)(job - row * (uint32_t)p.parts) * kWaves + wave;
  const int64_t b = row / (uint32_t)p.beams, n = row - (uint32_t)b * (uint32_t)p.beams;
  constexpr int ES = F32 ? 4 : 2;
  const char* const at = (const char*)p.logits + (b * p.ls_b + n * p.ls_n) * ES;
  const int V = (int)p.V, base = part * (64 * E);
  // 16-byte loads whatever the row's alignment; the last, incomplete ones value by value
  uint32_t raw[NL][4];
#pragma unroll
  for (int i = 0; i < NL; ++i) {
    const int v0 = base + (i * 64 + lane) * G;
    if (v0 + G <= V) {
      __builtin_memcpy(raw[i], at + (int64_t)v0 * ES, 16);
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if constexpr (F32) {
          raw[i][k] = v0 + k < V ? ((const uint32_t*)at)[v0 + k] : 0xFF800000u;
        } else {
          const uint32_t l = v0 + 2 * k < V ? ((const uint16_t*)at)[v0 + 2 * k] : 0xFF80u;
          const uint32_t h = v0 + 2 * k + 1 < V ? ((const uint16_t*)at)[v0 + 2 * k + 1] : 0xFF80u;
          raw[i][k] = l | h << 16;
        }
      }
    }
  }
  float top = -__builtin_inff();
#pragma unroll
  for (int i = 0; i < NL; ++i)
#pragma unroll
    for (int g = 0; g < G; ++g) top = fmaxf(top, unpack<F32>(raw[i], g));
  top = fmaxf(top, -__builtin_inff());  // -inf for a NaN, which reaches the sum instead
  float high = top;
#pragma unroll
  for (int m = 1; m < 64; m *= 2) high = fmaxf(high, __shfl_xor(high, m, 64));
  // Banned tokens are no candidates (where nothing else is left the merge looks for them itself), nor is what
  // lies behind the row.
  const uint32_t kth = kth_largest(base + lane * G < V ? order(top) : 0u, p.k, F32 ? 12 : 16);
  const float least = value(kth > kBanned ? kth : kBanned + 1);
  // An empty or fully banned piece: largest -inf, sum 0; +inf and NaN end in a sum that is not finite.  (x - high
  // rounds relative to itself, so that a token without rivals has the sum 1 exactly and its beam's score; as
  // x log2(e) - high log2(e) in one fma it would be off by the exponent's rounding.)
  const float shift = high == -__builtin_inff() ? 0.f : high;
  float sum = 0.f;
  uint64_t mask = 0;
#pragma unroll
  for (int i = 0; i < NL; ++i)
#pragma unroll
    for (int g = 0; g < G; ++g) {
      const float v = unpack<F32>(raw[i], g);
      sum += __builtin_amdgcn_exp2f((v - shift) * kLog2e);
      mask |= v >= least ? 1ull << (i * G + g) : 0;
    }
#pragma unroll
  for (int m = 1; m < 64; m *= 2) sum += __shfl_xor(sum, m, 64);
  if (lane == 0) stat[wave] = make_float2(high, sum);
  Held<uint32_t> held(hi[wave], lo[wave], p.k);
#pragma unroll 1
  while (__ballot(mask != 0)) {
    const bool in = mask != 0;
    const int e = in ? __builtin_ctzll(mask) : 0;
    const int v = in ? base + ((e / G) * 64 + lane) * G + e % G : 0;  // one of the row's
    mask &= mask - 1;
    const float f = F32 ? ((const float*)at)[v] : __uint_as_float((uint32_t)((const uint16_t*)at)[v] << 16);
    held.add(in, order(f), ~(uint32_t)v);
  }
  held.keep();
  if (lane == 0) count[wave] = held.held;
  __syncthreads();
  // the place of this lane's candidate among all four waves': its own, and how many of each other's are before it
  const uint32_t mh = hi[wave][lane], ml = lo[wave][lane];
  int rank = lane;
#pragma unroll
  for (int o = 1; o < kWaves; ++o) {
    const int w = wave ^ o, m = count[w];
#pragma unroll 4
    for (int i = 0; i < m; ++i) rank += hi[w][i] > mh || (hi[w][i] == mh && lo[w][i] > ml);
  }
  uint64_t* const cand = p.cand + (int64_t)job * p.k;
  if (lane < held.held && rank < p.k) cand[rank] = (uint64_t)mh << 32 | ml;
  if (threadIdx.x < 64) {
    int all = 0;
    float h = -__builtin_inff(), s = 0.f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      all += count[w];
      h = fmaxf(h, stat[w].x);
    }
#pragma unroll
    for (int w = 0; w < kWaves; ++w)  // an empty stretch adds nothing; a sum that is no number reaches the piece's
      if (stat[w].y != 0.f) s += stat[w].y * __builtin_amdgcn_exp2f((stat[w].x - h) * kLog2e);
    if (lane == 0) p.stat[job] = make_float2(h, s);
    if (lane >= all && lane < p.k) cand[lane] = 0;
  }
}

// One wave for each batch element.  A list is one piece's candidates.  Latency is
// all there is: loads and LDS reads go out together, candidates stay in registers.
template <bool F32>
__global__ __launch_bounds__(64) void beam_merge_kernel(BeamParams p) {
  constexpr int R = 8;  // candidates of a lane at a time
  extern __shared__ __align__(8) char smem[];
  __shared__ uint64_t hi[kHeld];
  __shared__ uint32_t lo[kHeld];
  const int lists = (int)p.beams * p.parts;
  float2* const stat = (float2*)smem;                              // (lists): largest logit and sum,
  double* const term = (double*)smem;                              // then the sum's part of its row's
  double* const offset = (double*)(smem + (int64_t)lists * 8);     // (beams): what a row's logits are raised by
  float* const most = (float*)(offset + p.beams);                  // (beams): largest logit
  const int lane = threadIdx.x;
  const int64_t b = blockIdx.x;
  const uint64_t* const cand = p.cand + b * lists * p.k;
  const int total = lists * p.k;
  // the first candidates are on their way while the normalisers are formed
  uint64_t c[R];
#pragma unroll
  for (int r = 0; r < R; ++r) c[r] = r * 64 + lane < total ? cand[r * 64 + lane] : 0;
  for (int l = lane; l < lists; l += 64) stat[l] = p.stat[b * lists + l];
  __syncthreads();
#pragma unroll 1
  for (int n = lane; n < (int)p.beams; n += 64) {
    float h = -__builtin_inff();
#pragma unroll 8
    for (int i = 0; i < p.parts; ++i) h = fmaxf(h, stat[n * p.parts + i].x);
    most[n] = h;
  }
  __syncthreads();
  // i / n for i < 2^21 (the quotient's error stays below half of 1 / n)
  auto quotient = [](int i, float inverse) { return (int)(((float)i + 0.5f) * inverse); };
  const float per_beam = 1.f / (float)p.parts, per_row = 1.f / (float)(p.parts * p.k);
#pragma unroll 1
  for (int l = lane; l < lists; l += 64) {
    const float2 s = stat[l];
    // an empty piece adds nothing; a sum that is no number reaches the row's
    const float w = __builtin_amdgcn_exp2f((s.x - most[quotient(l, per_beam)]) * kLog2e);
    term[l] = s.y != 0.f ? (double)s.y * (double)w : 0.0;
  }
  __syncthreads();
#pragma unroll 1
  for (int n = lane; n < (int)p.beams; n += 64) {
    double sum = 0;
#pragma unroll 8
    for (int i = 0; i < p.parts; ++i) sum += term[n * p.parts + i];
    const double off = (double)p.scores[b * p.ss_b + n * p.ss_n] - ((double)most[n] + log(sum));
    offset[n] = off - off == 0 ? off : -__builtin_inf();  // not finite: the row offers nothing
  }
  __syncthreads();
  Held<uint64_t> held(hi, lo, p.k);
#pragma unroll 1
  for (int c0 = 0; c0 < total; c0 += 64 * R) {
    uint64_t score[R];
    uint32_t index[R], top = 0;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int n = c[r] != 0 ? quotient(c0 + r * 64 + lane, per_row) : 0;
      const double off = offset[n];
      const bool in = c[r] != 0 && off != -__builtin_inf();
      score[r] = in ? order64(off + (double)value((uint32_t)(c[r] >> 32))) : 0;
      index[r] = (uint32_t)n * (uint32_t)p.V + (uint32_t)~(uint32_t)c[r];
      top = (uint32_t)(score[r] >> 32) > top ? (uint32_t)(score[r] >> 32) : top;
    }
    const int next = c0 + 64 * R;
    if (next < total)
#pragma unroll
      for (int r = 0; r < R; ++r) c[r] = next + r * 64 + lane < total ? cand[next + r * 64 + lane] : 0;
    const uint32_t kth = kth_largest(top, p.k, 0);
    uint64_t mask[R];
    int count = held.held;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      mask[r] = __ballot(score[r] != 0 && (uint32_t)(score[r] >> 32) >= kth && held.passes(score[r], ~index[r]));
      count += __popcll(mask[r]);
    }
    if (count <= kHeld) {  // uniform, and the rule
#pragma unroll
      for (int r = 0; r < R; ++r)
        if (mask[r]) held.append(mask[r], score[r], ~index[r]);
    } else {
#pragma unroll 1
      for (int r = 0; r < R; ++r) {  // one copy of the code: the candidates come by
        held.add(mask[0] >> lane & 1, score[0], ~index[0]);
#pragma unroll
        for (int i = 0; i + 1 < R; ++i) {
          mask[i] = mask[i + 1];
          score[i] = score[i + 1];
          index[i] = index[i + 1];
        }
      }
    }
  }
  held.keep();
  auto put = [&](int i, float score, uint32_t index) {
    const uint32_t n = index / (uint32_t)p.V;
    p.out_scores[b * p.k + i] = score;
    p.tokens[b * p.k + i] = (int32_t)(index - n * (uint32_t)p.V);
    p.parents[b * p.k + i] = (int32_t)n;
  };
  int done = held.held;
  if (lane < done) put(lane, (float)value64(hi[lane]), ~lo[lane]);
  // what is left scores -inf: banned tokens, and all of the rows that offer nothing, by their index
  for (int64_t at = 0; done < p.k && at < p.beams * p.V; at += 64) {
    const int64_t i = at + lane;
    bool in = i < p.beams * p.V;
    if (in) {
      const int64_t n = i / p.V, e = b * p.ls_b + n * p.ls_n + i % p.V;
      in = offset[n] == -__builtin_inf() ||
           (F32 ? ((const float*)p.logits)[e] == -__builtin_inff() : ((const uint16_t*)p.logits)[e] == 0xFF80u);
    }
    const uint64_t mask = __ballot(in);
    const int slot = done + __popcll(mask & ((1ull << lane) - 1));
    if (in && slot < p.k) put(slot, -__builtin_inff(), (uint32_t)i);
    done += __popcll(mask);
  }
}

template <bool F32>
void launch_io(const BeamParams& p, hipStream_t stream) {
  const int64_t lists = p.beams * p.parts;
  const dim3 grid((unsigned)(p.batch * lists)), block(64 * kWaves);
  if (p.values == kSmall) hipLaunchKernelGGL((beam_piece_kernel<F32, kSmall>), grid, block, 0, stream, p);
  else hipLaunchKernelGGL((beam_piece_kernel<F32, kLarge>), grid, block, 0, stream, p);
  hipLaunchKernelGGL(beam_merge_kernel<F32>, dim3((unsigned)p.batch), dim3(64), (unsigned)(lists * 8 + p.beams * 12),
                     stream, p);
}

}  // namespace

// Pieces of 4096 values spread a small call over more compute units (5 x 32000 fp32:
// 40 of them); where more than four such pieces come on each compute unit, of 16384,
// whose lists are a quarter as many.
BeamPieces beam_pieces(int64_t rows, int64_t vocab) {
  const int64_t small = (vocab + 256 * kSmall - 1) / (256 * kSmall), large = (vocab + 256 * kLarge - 1) / (256 * kLarge);
  return rows * small <= 1024 ? BeamPieces{kSmall, small} : BeamPieces{kLarge, large};
}

hipError_t launch_beam_select(const BeamParams& p, hipStream_t stream) {
  if (p.f32) launch_io<true>(p, stream);
  else launch_io<false>(p, stream);
  return hipGetLastError();
}

}  // namespace ssm
