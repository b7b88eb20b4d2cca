// Backward of the causal depthwise convolution (+ bias, + SiLU) for gfx950:
//   a_t = bias + sum_k w_k x_{t-W+1+k},  g_t = dy_t silu'(a_t)
//   dx_t = sum_k w_k g_{t+W-1-k},  dw_k = sum g_t x_{t-W+1+k},  dbias = sum g_t
// with a recomputed.  Bound by HBM: x and dy are read once, dx is written once.
// A wave walks the steps of one stretch for 64 * V channels: x and g slide
// through registers, so a step costs one load of x and one of dy (asked for U
// steps ahead) and stores the dx of W - 1 steps before.  A stretch starts W - 1
// steps early in x and runs W - 1 steps over in x and dy, whose g only reach dx:
// that is 2 (W - 1) rows of x and W - 1 of dy read twice, from the L2.
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

template <bool BF16, int V>
struct Vals {
  uint32_t w[BF16 ? (V + 1) / 2 : V];
};

template <bool BF16, int V>
__device__ __forceinline__ Vals<BF16, V> load_vals(__amdgpu_buffer_rsrc_t r, uint32_t off) {
  Vals<BF16, V> o;
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

template <bool BF16, int V>
__device__ __forceinline__ float val(const Vals<BF16, V>& r, int v) {
  if constexpr (!BF16) return __uint_as_float(r.w[v]);
  else if constexpr (V == 1) return __uint_as_float(r.w[0] << 16);
  else return __uint_as_float((v & 1) ? (r.w[v >> 1] & 0xFFFF0000u) : (r.w[v >> 1] << 16));
}

template <int V>
__device__ __forceinline__ void store_vals(__amdgpu_buffer_rsrc_t r, uint32_t off, const float (&o)[V], bool f32) {
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

// `own` steps of a wave; workgroup (channel block, part of a row's steps, row).
template <bool BF16, bool DYF, int V, int W>
__global__ __launch_bounds__(64 * NW) void conv_bwd_kernel(ConvBwdParams p, unsigned nchb, unsigned nparts, int own) {
  constexpr int E = BF16 ? 2 : 4, DE = DYF ? 4 : 2;
  const int XE = p.dx_f32 ? 4 : 2;
  __shared__ float lds[NW][W + 1][64 * V];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), lane = threadIdx.x % 64;
  const unsigned blk = blockIdx.x;
  const int64_t c0 = (int64_t)(blk % nchb) * (64 * V);
  const int64_t pt = (blk / nchb) % nparts, b = blk / (nchb * nparts);
  const int64_t d0 = c0 + lane * V;
  const bool on = d0 < p.D;  // V divides D where it is 4
  const int64_t t0 = (pt * NW + wave) * own;
  const int64_t t1 = t0 + own < p.L ? t0 + own : p.L;
  float wk[V][W], bv[V], dw[V][W], db[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
#pragma unroll
    for (int k = 0; k < W; ++k) {
      wk[v][k] = on ? p.w[(d0 + v) * p.ws_d + k * p.ws_k] : 0.f;
      dw[v][k] = 0.f;
    }
    bv[v] = on && p.bias ? p.bias[(d0 + v) * p.bs_d] : 0.f;
    db[v] = 0.f;
  }
  if (t0 < p.L) {  // uniform in the wave
    // x from row tb on, the rows in front of step 0 read zeros; dy from row t0 on
    const int64_t tb = t0 > W - 1 ? t0 - (W - 1) : 0;
    const int skip = (int)(W - 1 - (t0 - tb));
    const int64_t tend = t1 + W - 1 < p.L ? t1 + W - 1 : p.L;
    const __amdgpu_buffer_rsrc_t rx = rsrc((const char*)p.x + (b * p.xs_b + tb * p.xs_t + c0) * E,
                                           row_range(tend - tb, p.xs_t, p.D - c0, E));
    const __amdgpu_buffer_rsrc_t rd = rsrc((const char*)p.dy + (b * p.dys_b + t0 * p.dys_t + c0) * DE,
                                           row_range(tend - t0, p.dys_t, p.D - c0, DE));
    const __amdgpu_buffer_rsrc_t ro = rsrc((char*)p.dx + (b * p.dxs_b + t0 * p.dxs_t + c0) * XE,
                                           row_range(t1 - t0, p.dxs_t, p.D - c0, XE));
    const uint32_t lx = on ? (uint32_t)(lane * V * E) : kFar, ld = on ? (uint32_t)(lane * V * DE) : kFar,
                   lo = on ? (uint32_t)(lane * V * XE) : kFar;
    const uint32_t row_x = (uint32_t)(p.xs_t * E), row_d = (uint32_t)(p.dys_t * DE), row_o = (uint32_t)(p.dxs_t * XE);
    const int nrows = (int)(tend - t0);    // steps with a dy, from t0 on
    const int nx = (int)(tend - tb);
    // row i of the stretch's x (from step t0 - (W - 1) on); past the end: zeros, whatever the strides
    auto x_at = [&](int i) {
      return load_vals<BF16, V>(rx, i >= skip && i - skip < nx ? lx + (uint32_t)(i - skip) * row_x : kFar);
    };
    auto d_at = [&](int i) { return load_vals<!DYF, V>(rd, i < nrows ? ld + (uint32_t)i * row_d : kFar); };
    Vals<BF16, V> xn[U];
    Vals<!DYF, V> dn[U];
    float xh[V][W - 1 + U], gh[V][W - 1 + U];
    {
      Vals<BF16, V> h[W > 1 ? W - 1 : 1];
#pragma unroll
      for (int i = 0; i < W - 1; ++i) h[i] = x_at(i);
#pragma unroll
      for (int i = 0; i < U; ++i) {
        xn[i] = x_at(W - 1 + i);
        dn[i] = d_at(i);
      }
#pragma unroll
      for (int i = 0; i < W - 1; ++i)
#pragma unroll
        for (int v = 0; v < V; ++v) {
          xh[v][i] = val<BF16, V>(h[i], v);
          gh[v][i] = 0.f;
        }
    }
    const int steps = (int)(t1 - t0) + W - 1;
    for (int s0 = 0; s0 < steps; s0 += U) {
      float dy[V][U];
#pragma unroll
      for (int i = 0; i < U; ++i)
#pragma unroll
        for (int v = 0; v < V; ++v) {
          xh[v][W - 1 + i] = val<BF16, V>(xn[i], v);
          dy[v][i] = val<!DYF, V>(dn[i], v);
        }
#pragma unroll
      for (int i = 0; i < U; ++i) {
        xn[i] = x_at(W - 1 + s0 + U + i);
        dn[i] = d_at(s0 + U + i);
      }
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const bool mine = s0 + i < (int)(t1 - t0);
        float out[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
          float g = dy[v][i];
          if (p.silu) {
            float a = bv[v];
#pragma unroll
            for (int k = 0; k < W; ++k) a = __builtin_fmaf(wk[v][k], xh[v][i + k], a);
            const float s = sigmoid(a);
            g *= s * __builtin_fmaf(a, 1.f - s, 1.f);
          }
          gh[v][W - 1 + i] = g;
          float o = 0.f;
#pragma unroll
          for (int k = 0; k < W; ++k) o = __builtin_fmaf(wk[v][k], gh[v][W - 1 + i - k], o);
          out[v] = o;
          const float gm = mine ? g : 0.f;
#pragma unroll
          for (int k = 0; k < W; ++k) dw[v][k] = __builtin_fmaf(gm, xh[v][i + k], dw[v][k]);
          db[v] += gm;
        }
        // the dx of W - 1 steps before; in front of the stretch and past it: another wave's
        const int row = s0 + i - (W - 1);
        store_vals<V>(ro, row >= 0 && row < (int)(t1 - t0) ? lo + (uint32_t)row * row_o : kFar, out, p.dx_f32);
      }
#pragma unroll
      for (int i = 0; i < W - 1; ++i)
#pragma unroll
        for (int v = 0; v < V; ++v) {
          xh[v][i] = xh[v][U + i];
          gh[v][i] = gh[v][U + i];
        }
    }
  }
#pragma unroll
  for (int v = 0; v < V; ++v) {
#pragma unroll
    for (int k = 0; k < W; ++k) lds[wave][k][lane * V + v] = dw[v][k];
    lds[wave][W][lane * V + v] = db[v];
  }
  __syncthreads();
  float* const part = p.part + (b * nparts + pt) * (W + 1) * p.D;
  for (int i = threadIdx.x; i < (W + 1) * 64 * V; i += 64 * NW) {
    const int k = i / (64 * V), c = i % (64 * V);
    if (c0 + c < p.D) part[k * p.D + c0 + c] = (lds[0][k][c] + lds[1][k][c]) + (lds[2][k][c] + lds[3][k][c]);
  }
}

// dweight[d][k], dbias[d] = the parts' sums, in a fixed order.  A workgroup
// takes 32 of the (W + 1) D columns; 32 threads share a column's parts.
__global__ __launch_bounds__(1024) void conv_bwd_sum_kernel(const float* part, int64_t parts, int64_t D, int64_t W,
                                                            float* dweight, float* dbias) {
  __shared__ float lds[32][33];
  const int lane = threadIdx.x % 32, run = threadIdx.x / 32;
  const int64_t c = (int64_t)blockIdx.x * 32 + lane, cols = (W + 1) * D;
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
  const int own = (int)conv_bwd_steps(p.batch, p.L, p.D) / NW;
  const unsigned nchb = (unsigned)((p.D + 64 * V - 1) / (64 * V));
  const int64_t parts = conv_bwd_parts(p.batch, p.L, p.D);
  const unsigned nparts = (unsigned)(parts / p.batch);
  hipLaunchKernelGGL((conv_bwd_kernel<BF16, DYF, V, W>), dim3((unsigned)(nchb * parts)), dim3(64 * NW), 0, stream, p,
                     nchb, nparts, own);
  hipLaunchKernelGGL(conv_bwd_sum_kernel, dim3((unsigned)(((W + 1) * p.D + 31) / 32)), dim3(1024), 0, stream, p.part,
                     parts, p.D, p.W, p.dweight, p.dbias);
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
  const bool vec = p.D % 4 == 0 && al(p.x, 4 * e) && al(p.dy, 4 * de) && al(p.dx, 4 * xe) && p.xs_b % 4 == 0 &&
                   p.xs_t % 4 == 0 && p.dys_b % 4 == 0 && p.dys_t % 4 == 0 && p.dxs_b % 4 == 0 && p.dxs_t % 4 == 0;
  if (vec) launch_v<BF16, DYF, 4>(p, stream);
  else launch_v<BF16, DYF, 1>(p, stream);
}

}  // namespace

int64_t conv_bwd_steps(int64_t batch, int64_t seqlen, int64_t dim) {
  (void)batch; (void)seqlen; (void)dim;
  return NW * 36;
}

hipError_t launch_conv_bwd(const ConvBwdParams& p, hipStream_t stream) {
  if (!p.io_bf16) launch_io<false, true>(p, stream);
  else if (p.dy_f32) launch_io<true, true>(p, stream);
  else launch_io<true, false>(p, stream);
  return hipGetLastError();
}

}  // namespace ssm
