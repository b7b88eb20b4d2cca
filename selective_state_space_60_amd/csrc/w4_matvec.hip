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
// holds one output column and needs one scale per group.  An operand's layout
// puts neighbouring lanes in different rows; loaded so, every lane is a memory
// access of its own (at 16 x 5120 -> 2560 the loads alone took 11 us).  Loads
// are therefore made in row order, 64 bytes of a row of weights by four lanes
// and 256 bytes of a row of x by sixteen, and change lanes through LDS, in a
// part that belongs to the wave.  16-byte units of a row are stored at places
// XORed with the row, which spreads both directions over all banks.
// A lane then has 16 bytes, 32 consecutive weights, of one output; a 4 x 4
// transposition of dwords over the four lane groups (v_permlane16_swap,
// v_permlane32_swap) turns the four lane groups' 32 into the k order of four
// 32-wide products, each inside one scale group.  The pairs come out as
// weights (i, i + 4); x is put into the same order with v_perm before it is
// stored.
//
// A workgroup owns 16 or 32 outputs of 16 rows; its eight waves take every
// eighth step of 128 of k each, on their own: once a step's operands are in LDS
// the next step's loads are issued into the same registers, ahead of the
// products.  The waves' sums are added in order through LDS.  More rows are more
// workgroups, which read the weights again from L2: all rows in one workgroup
// (64 x 2560 -> 10240: 25.7 us against 16.8) leave a compute unit two of them
// and its neighbour one.
//
// Times here and below are of calls in a captured graph, replayed over matrices
// that together exceed the last-level cache: 1 x 2560 -> 10240 6.5 us, 16 x 5120
// -> 2560 6.1 (a launch is 2.3), 4 x 5120 -> 20480 16.4 (3.3 TB/s of weights), 64 x
// 2560 -> 10240 16.9 (the weights widened again for each 16 rows).  A lane's step is some 110
// VALU operations for 64 weights, 64 of them bringing weights into bf16.  Two
// steps of loads in flight are no better (16 x 5120 -> 2560: 6.6), for their registers.
#include <hip/hip_runtime.h>

#include "layer_internal.h"
#include "w4_loads.h"

namespace ssm {
namespace {

using namespace w4;

constexpr int NT = W * 64;

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));

constexpr uint32_t kRsrcWord3 = 0x00020000u;
constexpr uint32_t kMaxRange = 0x7FFFFF00u;  // the host keeps every range below

__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc(const void* p, int64_t bytes) {
  const uint32_t range = bytes < (int64_t)kMaxRange ? (uint32_t)bytes : kMaxRange;
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), (short)0, (int)range, (int)kRsrcWord3);
}

__device__ __forceinline__ u32x4_t load16(__amdgpu_buffer_rsrc_t r, uint32_t off, int step) {
  return __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(r, (int)off, step, 0));
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
__device__ __forceinline__ bf16x8_t widen(uint32_t w, uint32_t mask, uint32_t base) {
  const u32x4_t o = {((w << 3) & mask) | base, ((w >> 1) & mask) | base, ((w >> 5) & mask) | base,
                     ((w >> 9) & mask) | base};
  return __builtin_bit_cast(bf16x8_t, o);
}

// eight values of x into the same order
__device__ __forceinline__ u32x4_t reorder(u32x4_t x) {
  constexpr uint32_t lo = 0x05040100u, hi = 0x07060302u;  // low halves, high halves of (second, first)
  return u32x4_t{__builtin_amdgcn_perm(x[2], x[0], lo), __builtin_amdgcn_perm(x[2], x[0], hi),
                 __builtin_amdgcn_perm(x[3], x[1], lo), __builtin_amdgcn_perm(x[3], x[1], hi)};
}

// Orders a wave's LDS accesses of different lanes (no instruction).
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// XR loads of four rows of x (4 where a tile of 16 may be full), NL tiles of 16
// outputs, GS = group / 32, SF32: fp32 scales.  Without zero points their
// buffer is empty and gives zeros.
template <int XR, int NL, int GS, bool SF32>
__global__ __launch_bounds__(NT, 4) void w4_kernel(W4Params p, unsigned xtiles) {
  constexpr int NG = 4 / GS;                      // scale groups of a step
  constexpr int SN = scale_loads(NL, NG);         // loads of a step's scales
  constexpr int es = SF32 ? 4 : 2;
  struct Stage {
    u32x4_t w[NL][64], x[XR * 64];
    float2 sc[SN * 64];                           // (scale, -(16 + zero))
  };
  __shared__ union {
    Stage st[W];
    float sum[W][NL * 4][64];
  } sh;
  const int lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  const int col = lane % 16, kg = lane / 16;
  // A tile behind the last output has no rows and no steps: its loads are out of
  // range by the lane offset, at scalar offset 0 (a test up here would be a wait
  // for the first arguments ahead of the others).
  const int m0 = (int)blockIdx.y * 16;
  const int64_t n0 = ((int64_t)blockIdx.z * xtiles + blockIdx.x) * (16 * NL);
  const int nrows = tile_rows(p.outs, n0, 16 * NL);
  const int ins = (int)p.ins, half = ins / 2, groups = ins / (32 * GS), rows = (int)p.rows;
  const int steps = tile_steps(ins, nrows);
  const __amdgpu_buffer_rsrc_t rw = rsrc(p.weight + n0 * half, (int64_t)nrows * half);
  const __amdgpu_buffer_rsrc_t rs = rsrc((const char*)p.scale + n0 * groups * es, (int64_t)nrows * groups * es);
  const __amdgpu_buffer_rsrc_t rz = rsrc(p.zero ? p.zero + n0 * groups : nullptr, p.zero ? (int64_t)nrows * groups : 0);
  const __amdgpu_buffer_rsrc_t rx = rsrc(p.x, ((p.rows - 1) * p.xs_m + p.ins) * 2);
  const float zbase = p.zero ? -16.f : -24.f;
  Stage& st = sh.st[wave];
  // Row order of the loads: weights row lane / 4, unit lane % 4; x row lane /
  // 16 (+ 4 i), unit lane % 16.  The lane's offsets within a step; rows that
  // do not exist are out of range.
  const int wrow = lane / 4, wunit = (lane % 4) ^ (wrow / 4);
  uint32_t woff[NL], xoff[XR], soff[SN];
#pragma unroll
  for (int n = 0; n < NL; ++n) woff[n] = weight_offset(n * 16 + wrow, wunit, nrows, half);
#pragma unroll
  for (int i = 0; i < XR; ++i) xoff[i] = x_offset(m0 + 4 * i + kg, col, rows, p.xs_m);
#pragma unroll
  for (int i = 0; i < SN; ++i) soff[i] = scale_entry(lane + i * 64, NG, nrows, groups);
  const uint32_t xend = x_end(steps, col, ins), send = scale_end(steps, lane, NG, groups);
  // operand order of the reads
  const int wread = col * 4 + (kg ^ (col / 4));
  const int xrow = col % (XR * 4);
  f32x4_t acc[NL];
#pragma unroll
  for (int n = 0; n < NL; ++n) acc[n] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  // held in registers: with two literals the and and the or stay two instructions
  uint32_t mask = 0x00780078u, base = 0x41804180u;
  asm volatile("" : "+s"(mask), "+v"(base));
  const bf16x8_t ones = __builtin_bit_cast(bf16x8_t, u32x4_t{0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u});

  // A step's loads.  Behind the last step they are made too, out of range:
  // where paths with and without a load meet, the compiler waits for all.
  struct Loads {
    u32x4_t w[NL], x[XR];
    uint32_t sc[SN], z[SN];
  };
  auto load = [&](Loads& l, int s) {
    const Step q = step_at(s, steps, xend, send);
#pragma unroll
    for (int n = 0; n < NL; ++n) l.w[n] = load16(rw, woff[n] | q.w, weight_step(q));
#pragma unroll
    for (int i = 0; i < SN; ++i) {
      const uint32_t e = soff[i] | q.s;
      if constexpr (SF32) l.sc[i] = __builtin_amdgcn_raw_buffer_load_b32(rs, (int)(e * 4), scale_step(q, NG) * 4, 0);
      else l.sc[i] = __builtin_amdgcn_raw_buffer_load_b16(rs, (int)(e * 2), scale_step(q, NG) * 2, 0);
      l.z[i] = __builtin_amdgcn_raw_buffer_load_b8(rz, (int)e, p.zero ? scale_step(q, NG) : 0, 0);
    }
#pragma unroll
    for (int i = 0; i < XR; ++i) l.x[i] = load16(rx, xoff[i] | q.x, x_step(q));
  };
  auto step = [&](Loads& l, int s) {
    wave_sync();
#pragma unroll
    for (int n = 0; n < NL; ++n) st.w[n][lane] = l.w[n];
#pragma unroll
    for (int i = 0; i < SN; ++i)
      st.sc[lane + i * 64] = make_float2(__uint_as_float(SF32 ? l.sc[i] : l.sc[i] << 16), zbase - (float)l.z[i]);
#pragma unroll
    for (int i = 0; i < XR; ++i) {
      const int row = 4 * i + kg;
      st.x[row * 16 + (col ^ row)] = reorder(l.x[i]);
    }
    load(l, s + W);
    wave_sync();
    u32x4_t d[NL];
#pragma unroll
    for (int n = 0; n < NL; ++n) {
      d[n] = st.w[n][wread];
      transpose4(d[n]);
    }
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      f32x4_t sx = {0.f, 0.f, 0.f, 0.f}, ga[NL];
#pragma unroll
      for (int n = 0; n < NL; ++n) ga[n] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int jj = 0; jj < GS; ++jj) {
        const int j = g * GS + jj;
        const bf16x8_t xa = __builtin_bit_cast(bf16x8_t, st.x[xrow * 16 + ((4 * j + kg) ^ xrow)]);
        sx = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xa, ones, sx, 0, 0, 0);
#pragma unroll
        for (int n = 0; n < NL; ++n)
          ga[n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xa, widen(d[n][j], mask, base), ga[n], 0, 0, 0);
      }
#pragma unroll
      for (int n = 0; n < NL; ++n) {
        const float2 f = st.sc[(n * 16 + col) * NG + g];
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[n][r] = __builtin_fmaf(f.x, __builtin_fmaf(f.y, sx[r], ga[n][r]), acc[n][r]);
      }
    }
  };
  Loads l;
  load(l, wave);
  for (int s = wave; s < steps; s += W) step(l, s);
  __syncthreads();  // the stages are done with
#pragma unroll
  for (int n = 0; n < NL; ++n)
#pragma unroll
    for (int r = 0; r < 4; ++r) sh.sum[wave][n * 4 + r][lane] = acc[n][r];
  __syncthreads();
  for (int i = threadIdx.x; i < NL * 4 * 64; i += NT) {
    const int l = i % 64, q = i / 64;
    const int64_t m = m0 + (l / 16) * 4 + q % 4;
    const int64_t n = n0 + (q / 4) * 16 + l % 16;
    if (m >= p.rows || n >= p.outs) continue;
    float sum = p.bias ? p.bias[n * p.bs_n] : 0.f;
#pragma unroll
    for (int w = 0; w < W; ++w) sum += sh.sum[w][q][l];
    if (p.y_f32) ((float*)p.y)[m * p.ys_m + n] = sum;
    else ((__bf16*)p.y)[m * p.ys_m + n] = (__bf16)sum;
  }
}

template <int XR, int NL, int GS>
void launch_s(const W4Params& p, hipStream_t stream) {
  const Grid g = grid_of(p.rows, p.outs, 16 * NL);
  const dim3 grid(g.x, g.y, g.z);
  if (p.scale_f32) hipLaunchKernelGGL((w4_kernel<XR, NL, GS, true>), grid, dim3(NT), 0, stream, p, g.x);
  else hipLaunchKernelGGL((w4_kernel<XR, NL, GS, false>), grid, dim3(NT), 0, stream, p, g.x);
}

template <int XR, int NL>
void launch_g(const W4Params& p, hipStream_t stream) {
  if (p.group == 32) launch_s<XR, NL, 1>(p, stream);
  else if (p.group == 64) launch_s<XR, NL, 2>(p, stream);
  else launch_s<XR, NL, 4>(p, stream);
}

template <int XR>
void launch_n(const W4Params& p, hipStream_t stream) {
  // 32 outputs a workgroup share x's way through LDS, once there are more than
  // three tiles of 16 a compute unit (16 against 32: 1 x 2560 -> 14336 7.6 us
  // against 7.2, 64 x 2560 -> 10240 21.8 against 16.8; but 1 x 2560 -> 10240
  // 6.5 against 6.8, 16 x 5120 -> 2560 6.0 against 7.8).
  const int64_t tiles = (p.rows + 15) / 16 * ((p.outs + 15) / 16);
  if (tiles > 3 * 256) launch_g<XR, 2>(p, stream);
  else launch_g<XR, 1>(p, stream);
}

}  // namespace

hipError_t launch_w4_matvec(const W4Params& p, hipStream_t stream) {
  // one load of x a lane and step instead of four (1 x 2560 -> 10240: 6.5 us against 8.4)
  if (p.rows <= 4) launch_n<1>(p, stream);
  else launch_n<4>(p, stream);
  return hipGetLastError();
}

}  // namespace ssm
