// Beam search's selection for gfx950: of every batch element's beams x vocab
// continuations the k of the highest score, score = scores[n] + logits[n, v] -
// log sum exp logits[n, :].
//
// One pass over the logits: a wave takes one piece of one row, holds it in
// registers and leaves the piece's largest logit, its sum of exp(logit -
// largest) and its k best (logit, index) in falling order.  For those it sorts
// the 64 lanes' largest values; whatever reaches the k-th of them is a candidate
// (k lanes hold one, so nothing below can be among the k best; few more do as a
// rule), is collected in LDS and sorted 64 at a time.  A second kernel adds the
// pieces' sums to each row's normaliser and takes k times the best of all
// pieces' first remaining candidates.
// Bound by HBM for large batches (each logit is read once), by the two launches'
// latency for small ones.
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
constexpr int kList = 64;  // a wave's sorted candidates
constexpr uint32_t kBanned = 0x007FFFFFu;  // order(-inf)

// Rises with the value; -0 counts as +0; 0 stands for no value (no float maps to it but a NaN).
__device__ __forceinline__ uint32_t order(float v) {
  const uint32_t b = __float_as_uint(v + 0.f);
  return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float value(uint32_t o) {
  return __uint_as_float((o & 0x80000000u) ? o & 0x7FFFFFFFu : ~o);
}

__device__ __forceinline__ uint32_t lane_xor(uint32_t v, int m) { return (uint32_t)__shfl_xor((int)v, m, 64); }
__device__ __forceinline__ uint64_t lane_xor64(uint64_t v, int m) {
  return (uint64_t)lane_xor((uint32_t)(v >> 32), m) << 32 | lane_xor((uint32_t)v, m);
}

// The 64 lanes' values in falling order (bitonic).
template <class T, class X>
__device__ __forceinline__ T sort_down(T v, int lane, X x) {
#pragma unroll
  for (int size = 2; size <= 64; size *= 2) {
#pragma unroll
    for (int m = size / 2; m >= 1; m /= 2) {
      const T o = x(v, m);
      const bool want_max = ((lane & m) == 0) == ((lane & size) == 0 || size == 64);
      v = want_max ? (v > o ? v : o) : (v < o ? v : o);
    }
  }
  return v;
}

// The 64 largest of two falling lists, falling.
__device__ __forceinline__ uint64_t merge_down(uint64_t a, uint64_t b, int lane) {
  const uint64_t rev = (uint64_t)(uint32_t)__shfl((int)(uint32_t)(b >> 32), 63 - lane, 64) << 32 |
                       (uint32_t)__shfl((int)(uint32_t)b, 63 - lane, 64);
  uint64_t v = a > rev ? a : rev;  // bitonic: the larger halves
#pragma unroll
  for (int m = 32; m >= 1; m /= 2) {
    const uint64_t o = lane_xor64(v, m);
    v = (lane & m) == 0 ? (v > o ? v : o) : (v < o ? v : o);
  }
  return v;
}

__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// E values of 64 lanes each are a piece; lane l holds G values side by side of
// every run of 64 G.
template <bool F32, int E>
__global__ __launch_bounds__(64 * kWaves) void beam_piece_kernel(BeamParams p) {
  constexpr int G = F32 ? 4 : 8;  // values of a 16-byte load
  constexpr int NL = E / G;       // loads
  __shared__ uint64_t lds[kWaves][kList];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), lane = threadIdx.x % 64;
  const int64_t job = (int64_t)blockIdx.x * kWaves + wave;
  if (job >= p.batch * p.beams * p.parts) return;
  const int part = (int)(job % p.parts);
  const int64_t row = job / p.parts, b = row / p.beams, n = row % p.beams;
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
          const uint32_t lo = v0 + 2 * k < V ? ((const uint16_t*)at)[v0 + 2 * k] : 0xFF80u;
          const uint32_t hi = v0 + 2 * k + 1 < V ? ((const uint16_t*)at)[v0 + 2 * k + 1] : 0xFF80u;
          raw[i][k] = lo | hi << 16;
        }
      }
    }
  }
  auto get = [&](int i, int g) {
    if constexpr (F32) return __uint_as_float(raw[i][g]);
    else return __uint_as_float((g & 1) ? (raw[i][g >> 1] & 0xFFFF0000u) : (raw[i][g >> 1] << 16));
  };
  // the lane's largest (a NaN reaches the sum instead), then the piece's
  float top = -__builtin_inff();
#pragma unroll
  for (int i = 0; i < NL; ++i)
#pragma unroll
    for (int g = 0; g < G; ++g) top = fmaxf(top, get(i, g));
  // the k-th of the lanes' largest values
  const uint32_t mine = base + lane * G < V ? order(top) : 0u;
  const uint32_t sorted = sort_down(mine, lane, lane_xor);
  const float high = value((uint32_t)__builtin_amdgcn_readfirstlane((int)sorted));
  const uint32_t kth = (uint32_t)__shfl((int)sorted, p.k - 1, 64);
  // banned tokens are no candidates: where nothing else is left the merge looks for them itself
  uint32_t least = kth > kBanned ? kth : kBanned + 1;
  float sum = 0.f;
  // an empty or fully banned piece: largest -inf, sum 0; +inf and NaN end in a sum that is not finite
  const float shift = high == -__builtin_inff() ? 0.f : high;
#pragma unroll
  for (int i = 0; i < NL; ++i)
#pragma unroll
    for (int g = 0; g < G; ++g) sum += __builtin_amdgcn_exp2f((get(i, g) - shift) * kLog2e);
#pragma unroll
  for (int m = 1; m < 64; m *= 2) sum += __shfl_xor(sum, m, 64);
  if (lane == 0) p.stat[job] = make_float2(high, sum);

  uint64_t list = 0;  // lane l: the l-th best so far
  uint64_t bar = 0;   // the k-th best so far: what does not pass it is none of the k
  int held = 0;       // in LDS
  auto flush = [&]() {
    wave_sync();
    const uint64_t key = lane < held ? lds[wave][lane] : 0;
    list = merge_down(list, sort_down(key, lane, lane_xor64), lane);
    bar = (uint64_t)(uint32_t)__shfl((int)(uint32_t)(list >> 32), p.k - 1, 64) << 32 |
          (uint32_t)__shfl((int)(uint32_t)list, p.k - 1, 64);
    if ((uint32_t)(bar >> 32) > least) least = (uint32_t)(bar >> 32);
    held = 0;
    wave_sync();
  };
#pragma unroll
  for (int i = 0; i < NL; ++i) {
#pragma unroll
    for (int g = 0; g < G; ++g) {
      const int v = base + (i * 64 + lane) * G + g;
      const uint32_t o = order(get(i, g));
      bool in = o >= least && v < V;
      if (__ballot(in) == 0) continue;  // uniform, and the rule
      const uint64_t key = (uint64_t)o << 32 | (uint32_t)~(uint32_t)v;
      in = in && key > bar;
      uint64_t mask = __ballot(in);
      if (held + __popcll(mask) > kList) {
        flush();
        in = in && key > bar;
        mask = __ballot(in);
      }
      if (in) lds[wave][held + __popcll(mask & ((1ull << lane) - 1))] = key;
      held += __popcll(mask);
    }
  }
  flush();
  if (lane < p.k) p.cand[job * p.k + lane] = list;
}

// Falling by score, then rising by index.
struct Best {
  double score;
  uint32_t index;  // n V + v
};
constexpr uint32_t kNothing = 0xFFFFFFFFu;

__device__ __forceinline__ bool before(const Best& a, const Best& b) {
  if (a.index == kNothing || b.index == kNothing) return a.index < b.index;
  return a.score > b.score || (a.score == b.score && a.index < b.index);
}

// One workgroup for each batch element; its first wave chooses.  A list is one
// piece's candidates, in LDS where they fit (`cached`); lane l takes lists l, l +
// 64, ..
template <bool F32>
__global__ __launch_bounds__(256) void beam_merge_kernel(BeamParams p, int cached) {
  extern __shared__ char smem[];
  const int lists = (int)p.beams * p.parts;
  double* const offset = (double*)smem;                        // (beams): what a row's logits are raised by
  float2* const stat = (float2*)(smem + p.beams * 8);          // (lists)
  uint64_t* const keys = (uint64_t*)(stat + lists);            // (lists, k), if cached
  int* const taken = (int*)(keys + (cached ? lists * p.k : 0));  // (lists): candidates taken from each
  const int64_t b = blockIdx.x;
  const uint64_t* const cand = p.cand + b * lists * p.k;
  for (int l = threadIdx.x; l < lists; l += 256) {
    stat[l] = p.stat[b * lists + l];
    taken[l] = 0;
  }
  if (cached)
    for (int i = threadIdx.x; i < lists * p.k; i += 256) keys[i] = cand[i];
  __syncthreads();
  for (int n = threadIdx.x; n < (int)p.beams; n += 256) {
    const float2* st = stat + n * p.parts;
    float high = -__builtin_inff();
    for (int i = 0; i < p.parts; ++i) high = fmaxf(high, st[i].x);
    double sum = 0;
    for (int i = 0; i < p.parts; ++i)  // an empty piece adds nothing; a sum that is no number reaches the row's
      if (st[i].y != 0.f) sum += (double)st[i].y * exp((double)st[i].x - (double)high);
    const double off = (double)p.scores[b * p.ss_b + n * p.ss_n] - ((double)high + log(sum));
    offset[n] = off - off == 0 ? off : -__builtin_inf();  // not finite: the row offers nothing
  }
  __syncthreads();
  if (threadIdx.x >= 64) return;
  const int lane = threadIdx.x;
  auto head = [&](int l) {
    Best r = {0, kNothing};
    const int n = l / p.parts, i = taken[l];
    const double off = offset[n];
    if (i >= p.k || off == -__builtin_inf()) return r;
    const uint64_t c = cached ? keys[l * p.k + i] : cand[l * p.k + i];
    if (c != 0) r = {off + (double)value((uint32_t)(c >> 32)), (uint32_t)((int64_t)n * p.V + (uint32_t)~(uint32_t)c)};
    return r;
  };
  Best mine = {0, kNothing};
  int from = 0;
  auto look = [&]() {
    mine.index = kNothing;
    for (int l = lane; l < lists; l += 64) {
      const Best h = head(l);
      if (before(h, mine)) {
        mine = h;
        from = l;
      }
    }
  };
  auto put = [&](int i, float score, uint32_t index) {
    const uint32_t n = index / (uint32_t)p.V;
    p.out_scores[b * p.k + i] = score;
    p.tokens[b * p.k + i] = (int32_t)(index - n * (uint32_t)p.V);
    p.parents[b * p.k + i] = (int32_t)n;
  };
  look();
  int done = 0;
  for (; done < p.k; ++done) {
    Best best = mine;
#pragma unroll
    for (int m = 1; m < 64; m *= 2) {
      Best o;
      o.score = __shfl_xor(best.score, m, 64);
      o.index = (uint32_t)__shfl_xor((int)best.index, m, 64);
      if (before(o, best)) best = o;
    }
    if (best.index == kNothing) break;  // uniform
    if (lane == 0) put(done, (float)best.score, best.index);
    if (mine.index == best.index) {  // one lane: indexes differ
      ++taken[from];
      look();
    }
  }
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
  const int64_t waves = p.batch * p.beams * p.parts, lists = p.beams * p.parts;
  const dim3 grid((unsigned)((waves + kWaves - 1) / kWaves)), block(64 * kWaves);
  const int64_t e = (p.V + p.parts * 64 - 1) / (p.parts * 64);  // values of a lane
  if (e <= kSmall) hipLaunchKernelGGL((beam_piece_kernel<F32, kSmall>), grid, block, 0, stream, p);
  else hipLaunchKernelGGL((beam_piece_kernel<F32, kLarge>), grid, block, 0, stream, p);
  const int64_t bytes = p.beams * 8 + lists * 12, all = bytes + lists * p.k * 8;
  const int cached = all <= 65536;
  hipLaunchKernelGGL(beam_merge_kernel<F32>, dim3((unsigned)p.batch), dim3(256), (unsigned)(cached ? all : bytes),
                     stream, p, cached);
}

}  // namespace

int64_t beam_parts(int64_t rows, int64_t vocab) {
  const int64_t small = (vocab + 64 * kSmall - 1) / (64 * kSmall), large = (vocab + 64 * kLarge - 1) / (64 * kLarge);
  return rows * small <= 4096 ? small : large;
}

hipError_t launch_beam_select(const BeamParams& p, hipStream_t stream) {
  if (p.f32) launch_io<true>(p, stream);
  else launch_io<false>(p, stream);
  return hipGetLastError();
}

}  // namespace ssm
