// Causal depthwise convolution (+ bias, + SiLU) of packed sequences with a
// window of the last W - 1 inputs for each, for gfx950:
//   y_t = silu(bias + sum_k w_k r_{t-W+1+k}),  r = the sequence's rows, in front
//   of them the window of slot src (zeros without one); the window of slot dst
//   <- the last W - 1 rows of [window, sequence].
// Bound by HBM: each x is read once, each y written once (16384 x 5120 bf16 in 24
// sequences, W 4: 75 us, 4.5 TB/s).  One token of each of 64 sequences of 5120
// channels takes 6.5 us, of which a launch is 2.2 and the bytes 1.1.  A workgroup
// takes one piece (packed_pieces.h) of up to TS rows and NT * V channels; a thread owns V
// consecutive channels, loads its rows and the W - 1 in front of them at once
// and slides the window in registers.  Rows of other sequences and rows that do
// not exist come back as zeros from the buffer's range, so no load sits behind
// a branch.
// Only the workgroup of a sequence's first piece touches windows: where the
// piece is shorter than W - 1 rows (the next one would need the window, too) it
// takes the next piece as well.  So a thread reads a channel's old window before
// it writes the new one, and no other does either.
#include <hip/hip_runtime.h>

#include "serve_device.h"

namespace ssm {
namespace {

using namespace dev;

constexpr int NT = 256;
constexpr int kTS = kConvPackedStep;

template <bool BF16, int V>
struct Row {
  uint32_t w[BF16 ? (V + 1) / 2 : V];
};

template <bool BF16, int V>
__device__ __forceinline__ Row<BF16, V> load_row(__amdgpu_buffer_rsrc_t r, uint32_t off) {
  Row<BF16, V> o;
  if constexpr (BF16 && V == 4) {
    const auto v = __builtin_amdgcn_raw_buffer_load_b64(r, (int)off, 0, 0);
    o.w[0] = v[0]; o.w[1] = v[1];
  } else if constexpr (!BF16 && V == 4) {
    const auto v = __builtin_amdgcn_raw_buffer_load_b128(r, (int)off, 0, 0);
    o.w[0] = v[0]; o.w[1] = v[1]; o.w[2] = v[2]; o.w[3] = v[3];
  } else if constexpr (BF16) {
    o.w[0] = __builtin_amdgcn_raw_buffer_load_b16(r, (int)off, 0, 0);
  } else {
    o.w[0] = __builtin_amdgcn_raw_buffer_load_b32(r, (int)off, 0, 0);
  }
  return o;
}

// A row as it was loaded.
template <bool BF16, int V>
__device__ __forceinline__ void store_raw(__amdgpu_buffer_rsrc_t r, uint32_t off, const Row<BF16, V>& o) {
  if constexpr (BF16 && V == 4) {
    const u32x2 w = {o.w[0], o.w[1]};
    __builtin_amdgcn_raw_buffer_store_b64(w, r, (int)off, 0, 0);
  } else if constexpr (!BF16 && V == 4) {
    const u32x4 w = {o.w[0], o.w[1], o.w[2], o.w[3]};
    __builtin_amdgcn_raw_buffer_store_b128(w, r, (int)off, 0, 0);
  } else if constexpr (BF16) {
    __builtin_amdgcn_raw_buffer_store_b16((uint16_t)o.w[0], r, (int)off, 0, 0);
  } else {
    __builtin_amdgcn_raw_buffer_store_b32(o.w[0], r, (int)off, 0, 0);
  }
}

template <bool BF16, int V>
__device__ __forceinline__ float elem(const Row<BF16, V>& r, int v) {
  if constexpr (!BF16) return __uint_as_float(r.w[v]);
  else if constexpr (V == 1) return __uint_as_float(r.w[0] << 16);
  else return __uint_as_float((v & 1) ? (r.w[v >> 1] & 0xFFFF0000u) : (r.w[v >> 1] << 16));
}

template <int V>
__device__ __forceinline__ void store_y(__amdgpu_buffer_rsrc_t r, uint32_t off, const float (&o)[V], bool f32) {
  if constexpr (V == 1) {
    store1(r, off, o[0], f32);
  } else if (f32) {
    const u32x4 w = {__float_as_uint(o[0]), __float_as_uint(o[1]), __float_as_uint(o[2]), __float_as_uint(o[3])};
    __builtin_amdgcn_raw_buffer_store_b128(w, r, (int)off, 0, 0);
  } else {
    const u32x2 w = {pack2(o[0], o[1]), pack2(o[2], o[3])};
    __builtin_amdgcn_raw_buffer_store_b64(w, r, (int)off, 0, 0);
  }
}

// One workgroup's channels.
template <int V, int W>
struct Chan {
  int64_t c0;      // first channel of the workgroup
  int lane;        // first channel of the thread, from c0 on
  float w[V][W], b[V];
};

// A window's slot as a buffer from the workgroup's first channel on; no slot: of no bytes.
template <bool BF16, int W>
__device__ __forceinline__ __amdgpu_buffer_rsrc_t window_buffer(const ConvPackedParams& p, int64_t slot, int64_t c0) {
  constexpr int E = BF16 ? 2 : 4;
  const char* at = (const char*)p.windows + ((slot < 0 ? 0 : slot) * p.wins_s + c0) * E;
  return rsrc(at, slot < 0 ? 0 : row_range(W - 1, p.wins_t, p.D - c0, E));
}

// Rows [t0, end) of the sequence that begins at `begin`, at most TS of them.
// win: the slot that it starts from, needed where t0 - begin < W - 1.
template <bool BF16, int V, int W, int TS>
__device__ __forceinline__ void convolve(const ConvPackedParams& p, const Chan<V, W>& ch, int begin, int t0, int end,
                                         __amdgpu_buffer_rsrc_t win) {
  constexpr int E = BF16 ? 2 : 4;
  const int YE = p.y_f32 ? 4 : 2;
  constexpr int R = TS + W - 1;
  // the first row read, and the rows in front of it that lie in the window
  const int tb = t0 - (W - 1) > begin ? t0 - (W - 1) : begin;
  const int skip = W - 1 - (t0 - tb);
  const __amdgpu_buffer_rsrc_t rx =
      rsrc((const char*)p.x + ((int64_t)tb * p.xs_t + ch.c0) * E, row_range(end - tb, p.xs_t, p.D - ch.c0, E));
  const uint32_t lane_x = (uint32_t)(ch.lane * E), row_x = (uint32_t)(p.xs_t * E);
  Row<BF16, V> rows[R];
#pragma unroll
  for (int j = 0; j < R; ++j)
    rows[j] = load_row<BF16, V>(rx, j < skip ? kFar : lane_x + (uint32_t)(j - skip) * row_x);
  if constexpr (W > 1) {
    if (skip > 0) {  // uniform
      const uint32_t row_w = (uint32_t)(p.wins_t * E);
#pragma unroll
      for (int j = 0; j < W - 1; ++j) {
        const Row<BF16, V> v = load_row<BF16, V>(win, j < skip ? lane_x + (uint32_t)(t0 - begin + j) * row_w : kFar);
#pragma unroll
        for (int i = 0; i < (int)(sizeof(v.w) / 4); ++i) rows[j].w[i] |= v.w[i];  // one of them is zero
      }
    }
  }
  const __amdgpu_buffer_rsrc_t ry = rsrc((char*)p.y + ((int64_t)t0 * p.ys_t + ch.c0) * YE,
                                         row_range(end - t0, p.ys_t, p.D - ch.c0, YE));
  const uint32_t lane_y = (uint32_t)(ch.lane * YE), row_y = (uint32_t)(p.ys_t * YE);
#pragma unroll
  for (int j = 0; j < TS; ++j) {
    if (j % 8 == 0 && t0 + j >= end) break;  // uniform
    float o[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      float acc = ch.b[v];
#pragma unroll
      for (int k = 0; k < W; ++k) acc = __builtin_fmaf(ch.w[v][k], elem<BF16, V>(rows[j + k], v), acc);
      o[v] = p.silu ? acc * sigmoid(acc) : acc;
    }
    store_y<V>(ry, lane_y + (uint32_t)j * row_y, o, p.y_f32);
  }
}

// TS rows of a piece at most.
template <bool BF16, int V, int W, int TS>
__global__ __launch_bounds__(NT) void conv_packed_kernel(ConvPackedParams p, unsigned nchb) {
  constexpr int E = BF16 ? 2 : 4;
  const int piece = (int)(blockIdx.x / nchb);
  Chan<V, W> ch;
  ch.c0 = (int64_t)(blockIdx.x % nchb) * (NT * V);
  ch.lane = (int)threadIdx.x * V;
  const bool first = piece < p.q.seqs;
  int s = piece, t0, end;
  packed::Run seq;
  if (first) {
    seq = sequence_of(p.q, s);
    const packed::Run r = packed::first_piece(seq, TS);
    t0 = r.begin;
    end = r.end;
  } else {
    const int at = (piece - p.q.seqs + 1) * TS;
    s = find_sequence(p.q, at);
    if (s < 0) return;
    seq = sequence_of(p.q, s);
    if (p.windows && at - seq.begin < W - 1) return;  // the first piece's workgroup takes it
    const packed::Run r = packed::later_piece(seq, at, TS);
    t0 = r.begin;
    end = r.end;
    if (t0 >= end) return;
  }
  if (ch.c0 + ch.lane >= p.D) return;  // V divides D where it is 4, so a thread is all in or all out
  const bool pool = W > 1 && p.windows && first;
  const Slots slot = slots_of(p.q, s, p.w);  // no pool: no slots
  const int64_t from = pool ? slot.from : -1, to = pool ? slot.to : -1;
  load_taps<V, W>(p.w, ch.c0 + ch.lane, p.ws_d, p.ws_k, ch.w);
#pragma unroll
  for (int v = 0; v < V; ++v) ch.b[v] = p.bias ? p.bias[(ch.c0 + ch.lane + v) * p.bs_d] : 0.f;
  const __amdgpu_buffer_rsrc_t win = window_buffer<BF16, W>(p, from, ch.c0);
  // the new window: its row i is row n - (W - 1) + i of the sequence, or one of the old window
  Row<BF16, V> next[W > 1 ? W - 1 : 1];
  if (to >= 0) {
    const int n = seq.end - seq.begin, e0 = n - (W - 1);
    const int t1 = seq.begin + (e0 > 0 ? e0 : 0);
    const __amdgpu_buffer_rsrc_t rx = rsrc((const char*)p.x + ((int64_t)t1 * p.xs_t + ch.c0) * E,
                                           row_range(seq.end - t1, p.xs_t, p.D - ch.c0, E));
#pragma unroll
    for (int i = 0; i < W - 1; ++i) {
      const uint32_t off = (uint32_t)(ch.lane * E);
      if (e0 + i >= 0) next[i] = load_row<BF16, V>(rx, off + (uint32_t)(i + (e0 > 0 ? 0 : e0)) * (uint32_t)(p.xs_t * E));
      else next[i] = load_row<BF16, V>(win, off + (uint32_t)(n + i) * (uint32_t)(p.wins_t * E));
    }
  }
  if (end > t0) convolve<BF16, V, W, TS>(p, ch, seq.begin, t0, end, win);
  if (pool && end < seq.end && end - seq.begin < W - 1)
    convolve<BF16, V, W, TS>(p, ch, seq.begin, end, seq.end < end + TS ? seq.end : end + TS, win);
  if (to >= 0) {
    const __amdgpu_buffer_rsrc_t out = window_buffer<BF16, W>(p, to, ch.c0);
#pragma unroll
    for (int i = 0; i < W - 1; ++i)
      store_raw<BF16, V>(out, (uint32_t)(ch.lane * E) + (uint32_t)i * (uint32_t)(p.wins_t * E), next[i]);
  }
}

// One token of each sequence.  The slot is asked for first, then all that does not
// depend on it, so that the window is the only load that waits for another (64 x 5120
// bf16: 6.5 us; as pieces of one row each, 6.7).
template <bool BF16, int V, int W>
__global__ __launch_bounds__(NT) void conv_token_kernel(ConvPackedParams p, unsigned nchb) {
  constexpr int E = BF16 ? 2 : 4;
  const int s = (int)(blockIdx.x / nchb);
  Chan<V, W> ch;
  ch.c0 = (int64_t)(blockIdx.x % nchb) * (NT * V);
  ch.lane = (int)threadIdx.x * V;
  if (ch.c0 + ch.lane >= p.D) return;
  const Slots slot = slots_of(p.q, s, p.w);  // no pool: no slots
  Row<BF16, V> rows[W];
  rows[W - 1] = load_row<BF16, V>(rsrc((const char*)p.x + ((int64_t)s * p.xs_t + ch.c0) * E, kFar), (uint32_t)(ch.lane * E));
  load_taps<V, W>(p.w, ch.c0 + ch.lane, p.ws_d, p.ws_k, ch.w);
#pragma unroll
  for (int v = 0; v < V; ++v) ch.b[v] = p.bias ? p.bias[(ch.c0 + ch.lane + v) * p.bs_d] : 0.f;
  const uint32_t lane_w = (uint32_t)(ch.lane * E), row_w = (uint32_t)(p.wins_t * E);
  const __amdgpu_buffer_rsrc_t win = window_buffer<BF16, W>(p, slot.from, ch.c0);
#pragma unroll
  for (int k = 0; k < W - 1; ++k) rows[k] = load_row<BF16, V>(win, lane_w + (uint32_t)k * row_w);
  float o[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    float acc = ch.b[v];
#pragma unroll
    for (int k = 0; k < W; ++k) acc = __builtin_fmaf(ch.w[v][k], elem<BF16, V>(rows[k], v), acc);
    o[v] = p.silu ? acc * sigmoid(acc) : acc;
  }
  const int YE = p.y_f32 ? 4 : 2;
  store_y<V>(rsrc((char*)p.y + ((int64_t)s * p.ys_t + ch.c0) * YE, kFar), (uint32_t)(ch.lane * YE), o, p.y_f32);
  // what has no slot goes out of the buffer's range
  const __amdgpu_buffer_rsrc_t out = window_buffer<BF16, W>(p, slot.to, ch.c0);
#pragma unroll
  for (int k = 0; k < W - 1; ++k) store_raw<BF16, V>(out, lane_w + (uint32_t)k * row_w, rows[k + 1]);
}

template <bool BF16, int V, int W>
void launch_w(const ConvPackedParams& p, hipStream_t stream) {
  const unsigned nchb = (unsigned)((p.D + (int64_t)NT * V - 1) / ((int64_t)NT * V));
  if (!p.q.starts) {
    hipLaunchKernelGGL((conv_token_kernel<BF16, V, W>), dim3(nchb * (unsigned)p.q.seqs), dim3(NT), 0, stream, p, nchb);
  } else {
    const unsigned n = (unsigned)packed::pieces(p.q.tokens, p.q.seqs, kTS);
    hipLaunchKernelGGL((conv_packed_kernel<BF16, V, W, kTS>), dim3(nchb * n), dim3(NT), 0, stream, p, nchb);
  }
}

template <bool BF16, int V>
void launch_v(const ConvPackedParams& p, hipStream_t stream) {
  switch (p.W) {
    case 1: launch_w<BF16, V, 1>(p, stream); break;
    case 2: launch_w<BF16, V, 2>(p, stream); break;
    case 3: launch_w<BF16, V, 3>(p, stream); break;
    case 4: launch_w<BF16, V, 4>(p, stream); break;
    case 5: launch_w<BF16, V, 5>(p, stream); break;
    case 6: launch_w<BF16, V, 6>(p, stream); break;
    case 7: launch_w<BF16, V, 7>(p, stream); break;
    default: launch_w<BF16, V, 8>(p, stream); break;
  }
}

template <bool BF16>
void launch_io(const ConvPackedParams& p, hipStream_t stream) {
  const int64_t e = BF16 ? 2 : 4, ye = p.y_f32 ? 4 : 2;
  auto al = [](const void* ptr, int64_t bytes) { return ((uintptr_t)ptr % (uintptr_t)bytes) == 0; };
  const bool vec = p.D % 4 == 0 && al(p.x, 4 * e) && al(p.y, 4 * ye) && p.xs_t % 4 == 0 && p.ys_t % 4 == 0 &&
                   (!p.windows || (al(p.windows, 4 * e) && p.wins_s % 4 == 0 && p.wins_t % 4 == 0));
  if (vec) launch_v<BF16, 4>(p, stream);
  else launch_v<BF16, 1>(p, stream);
}

}  // namespace

hipError_t launch_conv_packed(const ConvPackedParams& p, hipStream_t stream) {
  if (p.io_bf16) launch_io<true>(p, stream);
  else launch_io<false>(p, stream);
  return hipGetLastError();
}

}  // namespace ssm
