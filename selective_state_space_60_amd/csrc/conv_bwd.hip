// Backward of the causal depthwise convolution (+ bias, + SiLU) for gfx950:
//   a_t = bias + sum_k w_k x_{t-W+1+k},  g_t = dy_t silu'(a_t)
//   dx_t = sum_k w_k g_{t+W-1-k},  dw_k = sum g_t x_{t-W+1+k},  dbias = sum g_t
// with a recomputed.  Bound by HBM, and VALU issue not far below (25 operations an
// element): x and dy are read once, dx is written once (8 x 2048 x 1536 bf16, W 4:
// 38.5 us, the second kernel among it, 3.9 TB/s).  A wave walks the steps of one stretch for 64 * V channels: x and
// g slide through registers, so a step costs one load of x and one of dy (asked for U
// steps ahead, their rows scalar offsets) and stores the dx of W - 1 steps before.
// A stretch starts W - 1 steps early in x and runs W - 1 steps over in x and dy,
// whose g only reach dx: that is 2 (W - 1) rows of x and W - 1 of dy read twice,
// from the L2.  32 steps a wave: 16 cost 3 us more, 64 as much.  Two channels a lane:
// four take twice the registers, and 3 to 6 us more.
// The four waves of a workgroup take consecutive stretches; their sums of dw
// and dbias are added in LDS, and a second kernel adds the workgroups' in a
// fixed order.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "column_sums.h"
#include "serve_device.h"

namespace ssm {
namespace {

using namespace dev;

constexpr int NW = 4;  // waves
constexpr int U = 8;   // steps asked for at a time

// V (1 or 2) values side by side, as loaded.
template <bool BF16, int V>
struct Vals {
  static constexpr int kWords = BF16 ? (V + 1) / 2 : V;
  uint32_t w[kWords];
};

template <bool BF16, int V>
__device__ __forceinline__ Vals<BF16, V> load_vals(__amdgpu_buffer_rsrc_t r, uint32_t off, uint32_t so) {
  Vals<BF16, V> o;
  if constexpr (BF16 && V == 1) {
    o.w[0] = __builtin_amdgcn_raw_buffer_load_b16(r, (int)off, (int)so, 0);
  } else if constexpr (o.kWords == 1) {
    o.w[0] = __builtin_amdgcn_raw_buffer_load_b32(r, (int)off, (int)so, 0);
  } else {
    const auto v = __builtin_amdgcn_raw_buffer_load_b64(r, (int)off, (int)so, 0);
    o.w[0] = v[0]; o.w[1] = v[1];
  }
  return o;
}

template <bool BF16, int V>
__device__ __forceinline__ float val(const Vals<BF16, V>& r, int v) {
  if constexpr (!BF16) return __uint_as_float(r.w[v]);
  else if constexpr (V == 1) return __uint_as_float(r.w[0] << 16);
  else return __uint_as_float((v & 1) ? (r.w[v >> 1] & 0xFFFF0000u) : (r.w[v >> 1] << 16));
}

template <int V>
__device__ __forceinline__ void store_vals(__amdgpu_buffer_rsrc_t r, uint32_t off, uint32_t so, const float (&o)[V],
                                           bool f32) {
  if constexpr (V == 1) {
    if (f32) __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(o[0]), r, (int)off, (int)so, 0);
    else __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(uint16_t, (__bf16)o[0]), r, (int)off, (int)so, 0);
  } else if (f32) {
    const u32x2 w = {__float_as_uint(o[0]), __float_as_uint(o[1])};
    __builtin_amdgcn_raw_buffer_store_b64(w, r, (int)off, (int)so, 0);
  } else {
    __builtin_amdgcn_raw_buffer_store_b32(pack2(o[0], o[1]), r, (int)off, (int)so, 0);
  }
}

// One stretch of a wave: `own` steps (a multiple of U) from t0 on.
template <bool BF16, bool DYF, int V, int W>
struct Stretch {
  static constexpr int E = BF16 ? 2 : 4, DE = DYF ? 4 : 2;
  __amdgpu_buffer_rsrc_t rx, rd, ro;  // x from row tb on, dy and dx from row t0 on
  uint32_t lx, ld, lo;                // the lane's channels in a row (kFar: it has none)
  uint32_t row_x, row_d, row_o;
  int skip;                           // steps in front of row 0 among the W - 1 before t0
  int rows, ends;                     // steps from t0 on that have a dy; whose dx this wave stores
  bool silu, f32;                     // f32: dx
  float wk[V][W], bv[V], dw[V][W], db[V];
  float xh[V][W - 1 + U], gh[V][W - 1 + U];
  Vals<BF16, V> xn[U];
  Vals<!DYF, V> dn[U];

  // The loads of steps s .. s + U - 1.  A whole block's rows are scalar offsets; past the end: zeros.
  __device__ __forceinline__ void ask(int s) {
    const int before = W - 1 - skip;  // rows of x in front of t0
    if (s + U <= rows) {
#pragma unroll
      for (int i = 0; i < U; ++i) {
        xn[i] = load_vals<BF16, V>(rx, lx, (uint32_t)(before + s + i) * row_x);
        dn[i] = load_vals<!DYF, V>(rd, ld, (uint32_t)(s + i) * row_d);
      }
    } else {
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const bool in = s + i < rows;
        xn[i] = load_vals<BF16, V>(rx, in ? lx + (uint32_t)(before + s + i) * row_x : kFar, 0);
        dn[i] = load_vals<!DYF, V>(rd, in ? ld + (uint32_t)(s + i) * row_d : kFar, 0);
      }
    }
  }

  __device__ __forceinline__ void begin() {
    Vals<BF16, V> h[W > 1 ? W - 1 : 1];
#pragma unroll
    for (int i = 0; i < W - 1; ++i)
      h[i] = load_vals<BF16, V>(rx, i >= skip ? lx + (uint32_t)(i - skip) * row_x : kFar, 0);
    ask(0);
#pragma unroll
    for (int v = 0; v < V; ++v) {
#pragma unroll
      for (int i = 0; i < W - 1; ++i) {
        xh[v][i] = val<BF16, V>(h[i], v);
        gh[v][i] = 0.f;
      }
#pragma unroll
      for (int k = 0; k < W; ++k) dw[v][k] = 0.f;
      db[v] = 0.f;
    }
  }

  // N steps from s on: the dx of W - 1 steps before them, and, if SUM, their part of dw and dbias.
  template <int N, bool SUM>
  __device__ __forceinline__ void block(int s) {
    float dy[N][V], out[N][V];
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
      for (int v = 0; v < V; ++v) {
        xh[v][W - 1 + i] = val<BF16, V>(xn[i], v);
        dy[i][v] = val<!DYF, V>(dn[i], v);
      }
    if constexpr (SUM) ask(s + U);
    if (silu) {  // uniform
#pragma unroll
      for (int i = 0; i < N; ++i)
#pragma unroll
        for (int v = 0; v < V; ++v) {
          float a = bv[v];
#pragma unroll
          for (int k = 0; k < W; ++k) a = __builtin_fmaf(wk[v][k], xh[v][i + k], a);
          const float sg = sigmoid(a);
          dy[i][v] *= sg * __builtin_fmaf(a, 1.f - sg, 1.f);
        }
    }
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const float g = dy[i][v];
        gh[v][W - 1 + i] = g;
        float o = 0.f;
#pragma unroll
        for (int k = 0; k < W; ++k) o = __builtin_fmaf(wk[v][k], gh[v][W - 1 + i - k], o);
        out[i][v] = o;
        if constexpr (SUM) {
#pragma unroll
          for (int k = 0; k < W; ++k) dw[v][k] = __builtin_fmaf(g, xh[v][i + k], dw[v][k]);
          db[v] += g;
        }
      }
    if (f32) store<N>(s, out, true);
    else store<N>(s, out, false);
#pragma unroll
    for (int i = 0; i < W - 1; ++i)
#pragma unroll
      for (int v = 0; v < V; ++v) {
        xh[v][i] = xh[v][N + i];
        gh[v][i] = gh[v][N + i];
      }
  }

  template <int N>
  __device__ __forceinline__ void store(int s, const float (&out)[N][V], bool wide) const {
    const int first = s - (W - 1);
    if (first >= 0 && first + N <= ends) {
#pragma unroll
      for (int i = 0; i < N; ++i) store_vals<V>(ro, lo, (uint32_t)(first + i) * row_o, out[i], wide);
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const bool in = first + i >= 0 && first + i < ends;
        store_vals<V>(ro, in ? lo + (uint32_t)(first + i) * row_o : kFar, 0, out[i], wide);
      }
    }
  }
};

// Workgroup (channel block, part of a row's steps, row).
template <bool BF16, bool DYF, int V, int W>
__global__ __launch_bounds__(64 * NW) void conv_bwd_kernel(ConvBwdParams p, unsigned nchb, unsigned nparts) {
  __shared__ float lds[NW][W + 1][64 * V];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), lane = threadIdx.x % 64;
  const unsigned blk = blockIdx.x;
  const int64_t c0 = (int64_t)(blk % nchb) * (64 * V);
  const int64_t pt = (blk / nchb) % nparts, b = blk / (nchb * nparts);
  const int64_t d0 = c0 + lane * V;
  const bool on = d0 < p.D;  // V divides D where it is not 1
  constexpr int own = (int)kConvBwdSteps / NW;
  const int64_t t0 = (pt * NW + wave) * own;
  Stretch<BF16, DYF, V, W> q;
  load_taps<V, W>(p.w, on ? d0 : c0, p.ws_d, p.ws_k, q.wk);
#pragma unroll
  for (int v = 0; v < V; ++v) {
    q.bv[v] = on && p.bias ? p.bias[(d0 + v) * p.bs_d] : 0.f;
#pragma unroll
    for (int k = 0; k < W; ++k) q.dw[v][k] = 0.f;
    q.db[v] = 0.f;
  }
  if (t0 < p.L) {  // uniform in the wave
    constexpr int E = BF16 ? 2 : 4, DE = DYF ? 4 : 2;
    const int XE = 2 << p.dx_f32;  // dx_f32 is 0 or 1
    const int64_t t1 = t0 + own < p.L ? t0 + own : p.L, tend = t1 + W - 1 < p.L ? t1 + W - 1 : p.L;
    const int64_t tb = t0 > W - 1 ? t0 - (W - 1) : 0;
    q.skip = (int)(W - 1 - (t0 - tb));
    q.rows = (int)(tend - t0);
    q.ends = (int)(t1 - t0);
    q.silu = p.silu;
    q.f32 = p.dx_f32;
    // what does not exist goes out of range by the lane's offset
    q.rx = rsrc((const char*)p.x + (b * p.xs_b + tb * p.xs_t + c0) * E, kFar);
    q.rd = rsrc((const char*)p.dy + (b * p.dys_b + t0 * p.dys_t + c0) * DE, kFar);
    q.ro = rsrc((char*)p.dx + (b * p.dxs_b + t0 * p.dxs_t + c0) * XE, kFar);
    q.lx = on ? (uint32_t)(lane * V * E) : kFar;
    q.ld = on ? (uint32_t)(lane * V * DE) : kFar;
    q.lo = on ? (uint32_t)(lane * V * XE) : kFar;
    q.row_x = (uint32_t)(p.xs_t * E);
    q.row_d = (uint32_t)(p.dys_t * DE);
    q.row_o = (uint32_t)(p.dxs_t * XE);
    q.begin();
    int s = 0;
    for (; s < q.ends; s += U) q.template block<U, true>(s);
    if constexpr (W > 1) q.template block<W - 1, false>(s);  // the g of the next stretch, for the last dx
  }
#pragma unroll
  for (int v = 0; v < V; ++v) {
#pragma unroll
    for (int k = 0; k < W; ++k) lds[wave][k][lane * V + v] = q.dw[v][k];
    lds[wave][W][lane * V + v] = q.db[v];
  }
  __syncthreads();
  float* const part = p.part + (b * nparts + pt) * (W + 1) * p.D;
  for (int i = threadIdx.x; i < (W + 1) * 64 * V; i += 64 * NW) {
    const int k = i / (64 * V), c = i % (64 * V);
    if (c0 + c < p.D) part[k * p.D + c0 + c] = (lds[0][k][c] + lds[1][k][c]) + (lds[2][k][c] + lds[3][k][c]);
  }
}

// dweight[d][k], dbias[d] = the parts' sums, in a fixed order.  A workgroup
// takes 32 of the (W + 1) D columns, from column c0 on; 32 threads share a column's
// parts.
__global__ __launch_bounds__(1024) void conv_bwd_sum_kernel(const float* part, int64_t parts, int64_t D, int64_t W,
                                                            float* dweight, float* dbias, int64_t c0) {
  __shared__ float lds[32][33];
  const int lane = threadIdx.x % 32, run = threadIdx.x / 32;
  const int64_t c = c0 + (int64_t)blockIdx.x * 32 + lane, cols = (W + 1) * D;
  float sum = 0.f;
  if (c < cols) {
    if (parts <= 32 * 4) sum = column_run<4>(part + c, run, parts, cols, sum);
    else
      for (int64_t k = run; k < parts; k += 32 * 16) sum = column_run<16>(part + c, k, parts, cols, sum);
  }
  lds[run][lane] = sum;
  __syncthreads();
  if (run == 0 && c < cols) {
#pragma unroll
    for (int k = 1; k < 32; ++k) sum += lds[k][lane];
    const int64_t k = c / D, d = c % D;
    if (k < W) dweight[d * W + k] = sum;
    else if (dbias) dbias[d] = sum;
  }
}

template <bool BF16, bool DYF, int V, int W>
void launch_w(const ConvBwdParams& p, hipStream_t stream) {
  const unsigned nchb = (unsigned)((p.D + 64 * V - 1) / (64 * V));
  const int64_t parts = conv_bwd_parts(p.batch, p.L);
  const unsigned nparts = (unsigned)(parts / p.batch);
  hipLaunchKernelGGL((conv_bwd_kernel<BF16, DYF, V, W>), dim3((unsigned)(nchb * parts)), dim3(64 * NW), 0, stream, p,
                     nchb, nparts);
  const int64_t groups = ((W + 1) * p.D + 31) / 32;
  for (int64_t g = 0; g < groups; g += kLaunchBlocks1024)  // one launch up to 64 M columns
    hipLaunchKernelGGL(conv_bwd_sum_kernel, dim3((unsigned)std::min(groups - g, kLaunchBlocks1024)), dim3(1024), 0,
                       stream, p.part, parts, p.D, p.W, p.dweight, p.dbias, g * 32);
}

template <bool BF16, bool DYF, int V>
void launch_v(const ConvBwdParams& p, hipStream_t stream) {
  switch (p.W) {
    case 1: launch_w<BF16, DYF, V, 1>(p, stream); break;
    case 2: launch_w<BF16, DYF, V, 2>(p, stream); break;
    case 3: launch_w<BF16, DYF, V, 3>(p, stream); break;
    case 4: launch_w<BF16, DYF, V, 4>(p, stream); break;
    case 5: launch_w<BF16, DYF, V, 5>(p, stream); break;
    case 6: launch_w<BF16, DYF, V, 6>(p, stream); break;
    case 7: launch_w<BF16, DYF, V, 7>(p, stream); break;
    default: launch_w<BF16, DYF, V, 8>(p, stream); break;
  }
}

template <bool BF16, bool DYF>
void launch_io(const ConvBwdParams& p, hipStream_t stream) {
  const int64_t e = BF16 ? 2 : 4, de = DYF ? 4 : 2, xe = p.dx_f32 ? 4 : 2;
  auto al = [](const void* ptr, int64_t bytes) { return ((uintptr_t)ptr % (uintptr_t)bytes) == 0; };
  const bool vec = p.D % 2 == 0 && al(p.x, 2 * e) && al(p.dy, 2 * de) && al(p.dx, 2 * xe) && p.xs_b % 2 == 0 &&
                   p.xs_t % 2 == 0 && p.dys_b % 2 == 0 && p.dys_t % 2 == 0 && p.dxs_b % 2 == 0 && p.dxs_t % 2 == 0;
  if (vec) launch_v<BF16, DYF, 2>(p, stream);
  else launch_v<BF16, DYF, 1>(p, stream);
}

}  // namespace

hipError_t launch_conv_bwd(const ConvBwdParams& p, hipStream_t stream) {
  if (!p.io_bf16) launch_io<false, true>(p, stream);
  else if (p.dy_f32) launch_io<true, true>(p, stream);
  else launch_io<true, false>(p, stream);
  return hipGetLastError();
}

}  // namespace ssm
