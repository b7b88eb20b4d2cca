// A few rows times a matrix of 4-bit weights with group scales, for gfx950:
//   y[m,n] = sum_k x[m,k] (q[n,k] - zero) scale[n, k/group] + bias[n]
//
// Bound by reading the weights (half a byte each), and for small matrices by
// latency.  The products run on the bf16 matrix cores (16 x 16 x 32) even for
// one row: a weight costs one VALU operation to bring into bf16 and none to
// multiply.  A nibble q placed in the four top mantissa bits of a bf16 16.0 is
// 16 + q exactly, so a dword of eight weights becomes four dwords of bf16
// pairs with one shift and one and-or each; (16 + zero) times the group's sum
// of x, which the matrix cores compute too (a product with ones), is taken
// off before the group's scale.  16 is the smallest power that holds a nibble
// in the mantissa, and so the smallest cancellation.
//
// Roles: A = x (16 rows), B = weights (16 columns of outputs), so that a lane
// holds one output column and needs one scale per group.  A lane loads 16
// bytes, 32 consecutive weights of one output; a 4 x 4 transposition of dwords
// over the four lane groups (v_permlane16_swap, v_permlane32_swap) turns the
// four lane groups' 32 into the k order of four 32-wide products, each inside
// one scale group.  The pairs come out as weights (i, i + 4); x is put into
// the same order with v_perm.
//
// A workgroup of 8 waves owns 16 or 32 outputs and splits k in steps of 128;
// the waves' sums are added in order through LDS.
#include <hip/hip_runtime.h>

#include "ssm_internal.h"

namespace ssm {
namespace {

constexpr int W = 8;        // waves per workgroup
constexpr int NT = W * 64;
constexpr int KS = 128;     // k per step of a wave

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));

constexpr uint32_t kRsrcWord3 = 0x00020000u;
constexpr uint32_t kMaxRange = 0x7FFFFF00u;  // the host keeps every range below
constexpr uint32_t kFar = 0x7FFFFFF0u;       // past every range: loads give 0

__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc(const void* p, int64_t bytes) {
  const uint32_t range = bytes < (int64_t)kMaxRange ? (uint32_t)bytes : kMaxRange;
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), (short)0, (int)range, (int)kRsrcWord3);
}

__device__ __forceinline__ u32x4_t load16(__amdgpu_buffer_rsrc_t r, uint32_t off) {
  return __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(r, (int)off, 0, 0));
}

// dword j of lane group g <-> dword g of lane group j
__device__ __forceinline__ void transpose4(u32x4_t& d) {
  auto a = __builtin_amdgcn_permlane16_swap(d[0], d[1], false, false);
  auto b = __builtin_amdgcn_permlane16_swap(d[2], d[3], false, false);
  auto c = __builtin_amdgcn_permlane32_swap(a[0], b[0], false, false);
  auto e = __builtin_amdgcn_permlane32_swap(a[1], b[1], false, false);
  d[0] = c[0];
  d[2] = c[1];
  d[1] = e[0];
  d[3] = e[1];
}

// 16 + q of eight nibbles as bf16, in the order 0,4,1,5,2,6,3,7
__device__ __forceinline__ bf16x8_t widen(uint32_t w) {
  constexpr uint32_t mask = 0x00780078u, base = 0x41804180u;
  const u32x4_t o = {((w << 3) & mask) | base, ((w >> 1) & mask) | base, ((w >> 5) & mask) | base,
                     ((w >> 9) & mask) | base};
  return __builtin_bit_cast(bf16x8_t, o);
}

// eight values of x into the same order
__device__ __forceinline__ bf16x8_t reorder(u32x4_t x) {
  constexpr uint32_t lo = 0x05040100u, hi = 0x07060302u;  // low halves, high halves of (second, first)
  const u32x4_t o = {__builtin_amdgcn_perm(x[2], x[0], lo), __builtin_amdgcn_perm(x[2], x[0], hi),
                     __builtin_amdgcn_perm(x[3], x[1], lo), __builtin_amdgcn_perm(x[3], x[1], hi)};
  return __builtin_bit_cast(bf16x8_t, o);
}

// MT tiles of 16 rows, NL tiles of 16 outputs, GS = group / 32.
template <int MT, int NL, int GS>
__global__ __launch_bounds__(NT) void w4_kernel(W4Params p) {
  __shared__ float lds[W][MT * NL * 4][64];
  const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
  const int col = lane % 16, kg = lane / 16;
  const int64_t n0 = (int64_t)blockIdx.x * (16 * NL);
  const int64_t half = p.ins / 2, groups = p.ins / p.group;
  const int64_t nrows = p.outs - n0 < 16 * NL ? p.outs - n0 : 16 * NL;
  const __amdgpu_buffer_rsrc_t rw = rsrc(p.weight + n0 * half, nrows * half);
  const __amdgpu_buffer_rsrc_t rx = rsrc(p.x, ((p.rows - 1) * p.xs_m + p.ins) * 2);
  const int ins = (int)p.ins, steps = (ins + KS - 1) / KS;
  f32x4_t acc[MT][NL];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int n = 0; n < NL; ++n) acc[m][n] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  const bf16x8_t ones = __builtin_bit_cast(bf16x8_t, u32x4_t{0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u});

  u32x4_t wq[NL];
  auto fetch = [&](int s) {
#pragma unroll
    for (int n = 0; n < NL; ++n) {
      const int k = s * KS + kg * 32;
      const bool in = k < ins && n0 + n * 16 + col < p.outs;
      wq[n] = load16(rw, in ? (uint32_t)(n * 16 + col) * (uint32_t)half + (uint32_t)(k / 2) : kFar);
    }
  };
  if (wave < steps) fetch(wave);
  for (int s = wave; s < steps; s += W) {
    const int k0 = s * KS;
    bf16x8_t xa[MT][4];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int k = k0 + 32 * j + 8 * kg;
        const bool in = k < ins && m * 16 + col < p.rows;
        xa[m][j] = reorder(load16(rx, in ? (uint32_t)(m * 16 + col) * (uint32_t)(p.xs_m * 2) + (uint32_t)(k * 2) : kFar));
      }
    float sc[NL][4 / GS], zc[NL][4 / GS];
#pragma unroll
    for (int n = 0; n < NL; ++n)
#pragma unroll
      for (int g = 0; g < 4 / GS; ++g) {
        const int64_t gi = (k0 + 32 * GS * g) / p.group;
        const bool in = gi < groups && n0 + n * 16 + col < p.outs;
        const int64_t at = (n0 + n * 16 + col) * groups + gi;
        sc[n][g] = !in ? 0.f
                   : p.scale_f32 ? ((const float*)p.scale)[at]
                                 : __uint_as_float((uint32_t)((const uint16_t*)p.scale)[at] << 16);
        zc[n][g] = in && p.zero ? 16.f + (float)p.zero[at] : 24.f;
      }
    u32x4_t d[NL];
#pragma unroll
    for (int n = 0; n < NL; ++n) {
      d[n] = wq[n];
      transpose4(d[n]);
    }
    if (s + W < steps) fetch(s + W);
#pragma unroll
    for (int g = 0; g < 4 / GS; ++g) {
      f32x4_t sx[MT], ga[MT][NL];
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        sx[m] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int n = 0; n < NL; ++n) ga[m][n] = f32x4_t{0.f, 0.f, 0.f, 0.f};
      }
#pragma unroll
      for (int jj = 0; jj < GS; ++jj) {
        const int j = g * GS + jj;
#pragma unroll
        for (int m = 0; m < MT; ++m) sx[m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xa[m][j], ones, sx[m], 0, 0, 0);
#pragma unroll
        for (int n = 0; n < NL; ++n) {
          const bf16x8_t wb = widen(d[n][j]);
#pragma unroll
          for (int m = 0; m < MT; ++m)
            ga[m][n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xa[m][j], wb, ga[m][n], 0, 0, 0);
        }
      }
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int n = 0; n < NL; ++n)
#pragma unroll
          for (int r = 0; r < 4; ++r)
            acc[m][n][r] = __builtin_fmaf(sc[n][g], __builtin_fmaf(-zc[n][g], sx[m][r], ga[m][n][r]), acc[m][n][r]);
    }
  }
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int n = 0; n < NL; ++n)
#pragma unroll
      for (int r = 0; r < 4; ++r) lds[wave][(m * NL + n) * 4 + r][lane] = acc[m][n][r];
  __syncthreads();
  for (int i = threadIdx.x; i < MT * NL * 4 * 64; i += NT) {
    const int l = i % 64, q = i / 64;
    float sum = 0.f;
#pragma unroll
    for (int w = 0; w < W; ++w) sum += lds[w][q][l];
    const int64_t m = (q / (NL * 4)) * 16 + (l / 16) * 4 + q % 4;
    const int64_t n = n0 + (q / 4 % NL) * 16 + l % 16;
    if (m < p.rows && n < p.outs) {
      if (p.bias) sum += p.bias[n * p.bs_n];
      if (p.y_f32) ((float*)p.y)[m * p.ys_m + n] = sum;
      else ((__bf16*)p.y)[m * p.ys_m + n] = (__bf16)sum;
    }
  }
}

template <int MT, int NL>
void launch_g(const W4Params& p, hipStream_t stream) {
  const dim3 grid((unsigned)((p.outs + 16 * NL - 1) / (16 * NL)));
  if (p.group == 32) hipLaunchKernelGGL((w4_kernel<MT, NL, 1>), grid, dim3(NT), 0, stream, p);
  else if (p.group == 64) hipLaunchKernelGGL((w4_kernel<MT, NL, 2>), grid, dim3(NT), 0, stream, p);
  else hipLaunchKernelGGL((w4_kernel<MT, NL, 4>), grid, dim3(NT), 0, stream, p);
}

template <int MT>
void launch_n(const W4Params& p, hipStream_t stream) {
  // 32 outputs a workgroup share the rows of x and their order; 16 when that
  // would leave compute units without a workgroup
  if (p.outs >= 32 * 256) launch_g<MT, 2>(p, stream);
  else launch_g<MT, 1>(p, stream);
}

}  // namespace

hipError_t launch_w4_matvec(const W4Params& p, hipStream_t stream) {
  if (p.rows <= 16) launch_n<1>(p, stream);
  else if (p.rows <= 32) launch_n<2>(p, stream);
  else launch_n<4>(p, stream);
  return hipGetLastError();
}

}  // namespace ssm
