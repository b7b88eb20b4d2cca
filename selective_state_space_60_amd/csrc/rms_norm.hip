// Root-mean-square norm of rows, with the residual's addition in front and an
// optional e4m3 output with scales, and its backward, for gfx950.
//
//   row = x + residual (rounded to the type it is stored in)
//   y   = weight row rstd,  rstd = rsqrt(mean(row^2) + eps)
//
// Times here and below are of calls in a captured graph, replayed over sets of
// inputs that together exceed the last-level cache; a backward is its kernel
// and its sums.
//
// Bound by HBM: a row is read once, kept in registers across the reduction
// and written once (16384 x 2560, bf16 in, fp32 residual in and out, bf16 out:
// 94 us, 5.3 TB/s; a large copy runs at 4.7).  A workgroup of four or eight waves
// owns a row, or a wave each of four narrow rows (no barrier).  A lane holds
// groups of 8 consecutive columns: 16-byte loads of bf16, and an e4m3 group of
// 32, 64 or 128 columns is 4, 8 or 16 neighbouring lanes, whose largest value is
// found with DPP.  Few rows take one pass of latencies (1 x 2560 2.8 us, of which a
// launch is 2.3; 333 x 5120 with a bf16 residual to e4m3 6.8, without it 5.3,
// without it to bf16 4.5).
#include <hip/hip_runtime.h>

#include <algorithm>

#include "column_sums.h"
#include "layer_internal.h"

namespace ssm {
namespace {

constexpr int NT = 256;
constexpr int V = 8;  // consecutive columns per lane
constexpr int kRowShift = 22;  // workgroups of a grid's x: fewer than 2^32 threads
constexpr float kE4M3Max = 448.f;
constexpr float kMinScale = 1.17549435e-38f;  // 2^-126: a group of zeros divides by a normal number

typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef float f32x2_t __attribute__((ext_vector_type(2)));
typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));

__device__ __forceinline__ uint32_t pack2(float a, float b) {
  const f32x2_t v = {a, b};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2_t));
}

// Batch row and step of row r (fewer than 2^24 rows).
__device__ __forceinline__ void split_row(int64_t r, int64_t batch, int64_t L, int64_t& b, int64_t& t) {
  b = batch == 1 ? 0 : (uint32_t)r / (uint32_t)L;
  t = r - b * L;
}

__device__ __forceinline__ float bf16_at(const void* p, int64_t i) {
  return __uint_as_float((uint32_t)((const uint16_t*)p)[i] << 16);
}

// Columns [col, col + 8) of a row, of which the first n exist (n may be <= 0
// or > 8); the others are 0.  Rows need only their element's alignment: wide
// global accesses may be unaligned here.
__device__ __forceinline__ void load8(const void* row, int type, int col, int n, float (&o)[V]) {
  if (type == kNormBF16) {
    if (n >= V) {
      u32x4_t w;
      __builtin_memcpy(&w, (const uint16_t*)row + col, 16);
#pragma unroll
      for (int i = 0; i < V; ++i) o[i] = __uint_as_float((i & 1) ? (w[i / 2] & 0xFFFF0000u) : (w[i / 2] << 16));
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) o[i] = i < n ? bf16_at(row, col + i) : 0.f;
    }
  } else {
    if (n >= V) {
      u32x4_t w[2];
      __builtin_memcpy(w, (const float*)row + col, 32);
#pragma unroll
      for (int i = 0; i < V; ++i) o[i] = __uint_as_float(w[i / 4][i % 4]);
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) o[i] = i < n ? ((const float*)row)[col + i] : 0.f;
    }
  }
}

// The same of bf16 as loaded, and brought to fp32.
__device__ __forceinline__ u32x4_t load8_raw(const void* row, int col, int n) {
  u32x4_t w = {0, 0, 0, 0};
  if (n >= V) {
    __builtin_memcpy(&w, (const uint16_t*)row + col, 16);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (i < n) w[i / 2] |= (uint32_t)((const uint16_t*)row)[col + i] << (16 * (i & 1));
  }
  return w;
}

__device__ __forceinline__ void widen8(u32x4_t w, float (&o)[V]) {
#pragma unroll
  for (int i = 0; i < V; ++i) o[i] = __uint_as_float((i & 1) ? (w[i / 2] & 0xFFFF0000u) : (w[i / 2] << 16));
}

__device__ __forceinline__ void store8(void* row, int type, int col, int n, const float (&o)[V]) {
  if (type == kNormBF16) {
    if (n >= V) {
      u32x4_t w;
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = pack2(o[2 * i], o[2 * i + 1]);
      __builtin_memcpy((uint16_t*)row + col, &w, 16);
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (i < n) ((__bf16*)row)[col + i] = (__bf16)o[i];
    }
  } else {
    if (n >= V) {
      u32x4_t w[2];
#pragma unroll
      for (int i = 0; i < V; ++i) w[i / 4][i % 4] = __float_as_uint(o[i]);
      __builtin_memcpy((float*)row + col, w, 32);
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (i < n) ((float*)row)[col + i] = o[i];
    }
  }
}

// Eight values, already divided by their scale, to e4m3 (nearest even).
__device__ __forceinline__ void store8_e4m3(void* row, int col, int n, const float (&o)[V]) {
  u32x2_t w = {0, 0};
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    w[i] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(o[4 * i], o[4 * i + 1], 0, false);
    w[i] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(o[4 * i + 2], o[4 * i + 3], (int)w[i], true);
  }
  if (n >= V) {
    __builtin_memcpy((uint8_t*)row + col, &w, 8);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (i < n) ((uint8_t*)row)[col + i] = (uint8_t)(w[i / 4] >> (8 * (i % 4)));
  }
}

// 1 / sqrt(v), correctly rounded steps: the hardware's estimate takes a
// subnormal mean (tiny rows, eps 0) for zero.  Once a row.
__device__ __forceinline__ float inv_root(float v) { return 1.f / __builtin_sqrtf(v); }

template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
  return __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), CTRL, 0xF, 0xF, true));
}

// The total in every lane of the wave.
__device__ __forceinline__ float wave_sum(float v) {
  v += dpp<0xB1>(v);   // quad_perm [1,0,3,2]
  v += dpp<0x4E>(v);   // quad_perm [2,3,0,1]
  v += dpp<0x141>(v);  // row_half_mirror
  v += dpp<0x140>(v);  // row_mirror
  v += __shfl_xor(v, 16);
  v += __shfl_xor(v, 32);
  return v;
}

// The total of a row's waves.
template <int N>
__device__ __forceinline__ float waves_sum(const float (&v)[N]) {
  if constexpr (N == 8) return ((v[0] + v[1]) + (v[2] + v[3])) + ((v[4] + v[5]) + (v[6] + v[7]));
  else return (v[0] + v[1]) + (v[2] + v[3]);
}

// The largest over aligned groups of `lanes` (4, 8, 16 or 64), in every lane.
__device__ __forceinline__ float group_max(float v, int lanes) {
  v = fmaxf(v, dpp<0xB1>(v));
  v = fmaxf(v, dpp<0x4E>(v));
  if (lanes >= 8) v = fmaxf(v, dpp<0x141>(v));
  if (lanes >= 16) v = fmaxf(v, dpp<0x140>(v));
  if (lanes >= 64) {
    v = fmaxf(v, __shfl_xor(v, 16));
    v = fmaxf(v, __shfl_xor(v, 32));
  }
  return v;
}

// TPR threads per row (64: a wave, or the workgroup's 256 or 512), CH groups of
// 8 columns per thread: dim <= TPR * 8 * CH.
template <int TPR, int CH>
__global__ __launch_bounds__(TPR > NT ? TPR : NT) void norm_fwd_kernel(NormParams p, int64_t rows) {
  constexpr int WPR = TPR / 64;  // waves per row
  constexpr int RPB = TPR > NT ? 1 : NT / TPR;
  const int D = (int)p.D;
  __shared__ float lds[2][WPR];
  const int lane = threadIdx.x % TPR, wave = threadIdx.x / 64;
  const int64_t r = ((int64_t)blockIdx.y << kRowShift | blockIdx.x) * RPB + threadIdx.x / TPR;
  if (r >= rows) return;  // whole waves; otherwise the whole workgroup
  int64_t b, t;
  split_row(r, p.batch, p.L, b, t);
  const int xe = p.x_type == kNormF32 ? 4 : 2, re = p.r_type == kNormF32 ? 4 : 2, oe = p.ro_type == kNormF32 ? 4 : 2;
  const void* x = (const char*)p.x + (b * p.xs_b + t * p.xs_t) * xe;
  float f[CH][V], w[CH][V];
  float ss = 0.f;
#pragma unroll
  for (int k = 0; k < CH; ++k) {
    const int col = (k * TPR + lane) * V;
    load8(x, p.x_type, col, D - col, f[k]);
  }
  // the weights come along with the row: asked for behind the reduction they
  // would be a second wait
#pragma unroll
  for (int k = 0; k < CH; ++k) load8(p.weight, kNormF32, (k * TPR + lane) * V, D - (k * TPR + lane) * V, w[k]);
  if (p.residual) {
    const void* res = (const char*)p.residual + (b * p.rs_b + t * p.rs_t) * re;
    void* out = (char*)p.residual_out + (b * p.ros_b + t * p.ros_t) * oe;
    float g[CH][V];
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      const int col = (k * TPR + lane) * V;
      load8(res, p.r_type, col, D - col, g[k]);
    }
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      const int col = (k * TPR + lane) * V;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        f[k][i] += g[k][i];
        if (p.ro_type == kNormBF16) f[k][i] = (float)(__bf16)f[k][i];
      }
      store8(out, p.ro_type, col, D - col, f[k]);
    }
  }
#pragma unroll
  for (int k = 0; k < CH; ++k)
#pragma unroll
    for (int i = 0; i < V; ++i) ss = __builtin_fmaf(f[k][i], f[k][i], ss);
  ss = wave_sum(ss);
  if constexpr (WPR > 1) {
    if (threadIdx.x % 64 == 0) lds[0][wave] = ss;
    __syncthreads();
    ss = waves_sum<WPR>(lds[0]);
  }
  const float rstd = inv_root(ss / (float)D + p.eps);
  float amax = 0.f;
#pragma unroll
  for (int k = 0; k < CH; ++k) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      f[k][i] = f[k][i] * rstd * w[k][i];
      amax = fmaxf(amax, fabsf(f[k][i]));
    }
  }
  void* y = (char*)p.y + (b * p.ys_b + t * p.ys_t) * (p.y_type == kNormF32 ? 4 : p.y_type == kNormBF16 ? 2 : 1);
  if (p.y_type != kNormE4M3) {
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      const int col = (k * TPR + lane) * V;
      store8(y, p.y_type, col, D - col, f[k]);
    }
    return;
  }
  if (p.group == 0) {
    amax = group_max(amax, 64);
    if constexpr (WPR > 1) {
      if (threadIdx.x % 64 == 0) lds[1][wave] = amax;
      __syncthreads();
      amax = lds[1][0];
#pragma unroll
      for (int i = 1; i < WPR; ++i) amax = fmaxf(amax, lds[1][i]);
    }
  }
  const int shift = p.group == 32 ? 5 : p.group == 64 ? 6 : 7;  // of a group
  const int64_t ng = p.group ? (D + (1 << shift) - 1) >> shift : 1;
#pragma unroll
  for (int k = 0; k < CH; ++k) {
    const int col = (k * TPR + lane) * V;
    float m = amax;
    if (p.group) {
      m = 0.f;
#pragma unroll
      for (int i = 0; i < V; ++i) m = fmaxf(m, fabsf(f[k][i]));
      m = group_max(m, (1 << shift) / V);
    }
    const float scale = fmaxf(m / kE4M3Max, kMinScale);
    const float inv = 1.f / scale;
#pragma unroll
    for (int i = 0; i < V; ++i) f[k][i] *= inv;
    store8_e4m3(y, col, D - col, f[k]);
    if (p.group ? col < D && (col & ((1 << shift) - 1)) == 0 : col == 0)
      p.scale[r * ng + (p.group ? col >> shift : 0)] = scale;
  }
}

// ------------------------------------------------------------------ backward
// Workgroups walk the rows with a stride and keep dweight's sums of their rows
// in registers; the four waves' sums are added in order through LDS.  AHEAD, for
// bf16 rows and gradients: the next row's, 8 registers for 8 columns, are asked
// for before this row's sums (16384 x 768 36.9 -> 32.0 us, 16384 x 2560 111 -> 86,
// 4096 x 16384 145 -> 102).  fp32 rows, as an fp32 residual stream has them, take
// no part in it (16384 x 768 36.4 us, 16384 x 2560 107, 4.7 TB/s).  Not where they would cost a wave a SIMD (256 threads
// with three column groups: 173 us at 16384 x 5120 against 203; 512 with two: 106
// at 8192 x 8192 either way).
template <int TPR, int CH>
constexpr bool kAhead = !(TPR == 256 && CH == 3) && !(TPR == 512 && CH == 2);

template <int TPR, int CH, bool AHEAD>
__global__ __launch_bounds__(TPR > NT ? TPR : NT, AHEAD && TPR == 256 && CH == 2 ? 4 : 1) void norm_bwd_kernel(
    NormBwdParams p, int64_t rows) {
  constexpr int RPB = TPR > NT ? 1 : NT / TPR, WPR = TPR / 64;
  const int D = (int)p.D;
  __shared__ float lds[2][2][WPR];
  const int lane = threadIdx.x % TPR, wave = threadIdx.x / 64, sub = threadIdx.x / TPR;
  const int de = p.dy_type == kNormF32 ? 4 : 2, re = p.row_type == kNormF32 ? 4 : 2;
  const int se = p.dres_type == kNormF32 ? 4 : 2, xe = p.dx_type == kNormF32 ? 4 : 2;
  float acc[CH][V];
#pragma unroll
  for (int k = 0; k < CH; ++k)
#pragma unroll
    for (int i = 0; i < V; ++i) acc[k][i] = 0.f;
  int buf = 0;
  u32x4_t nf[AHEAD ? CH : 1], ng[AHEAD ? CH : 1];
  auto load_next = [&](int64_t r) {
    int64_t b, t;
    split_row(r, p.batch, p.L, b, t);
    const void* dy = (const char*)p.dy + (b * p.dys_b + t * p.dys_t) * 2;
    const void* row = (const char*)p.row + (b * p.rs_b + t * p.rs_t) * 2;
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      const int col = (k * TPR + lane) * V;
      nf[k] = load8_raw(row, col, D - col);
      ng[k] = load8_raw(dy, col, D - col);
    }
  };
  const int64_t step = (int64_t)gridDim.x * RPB;
  int64_t r = (int64_t)blockIdx.x * RPB + sub;
  if (AHEAD && r < rows) load_next(r);
  // with a workgroup a row every thread runs the same number of rounds
  for (; r < rows; r += step, buf ^= 1) {
    int64_t b, t;
    split_row(r, p.batch, p.L, b, t);
    const void* dy = (const char*)p.dy + (b * p.dys_b + t * p.dys_t) * de;
    const void* row = (const char*)p.row + (b * p.rs_b + t * p.rs_t) * re;
    float f[CH][V], g[CH][V];
    if constexpr (AHEAD) {
#pragma unroll
      for (int k = 0; k < CH; ++k) {
        widen8(nf[k], f[k]);
        widen8(ng[k], g[k]);
      }
    } else {
#pragma unroll
      for (int k = 0; k < CH; ++k) {
        const int col = (k * TPR + lane) * V;
        load8(row, p.row_type, col, D - col, f[k]);
      }
#pragma unroll
      for (int k = 0; k < CH; ++k) {
        const int col = (k * TPR + lane) * V;
        load8(dy, p.dy_type, col, D - col, g[k]);
      }
    }
    // dres comes along with the row, and so do the weights: asked for behind
    // the reduction they would be a second wait (a wide row has too many to hold)
    constexpr bool kEarly = CH <= 2;
    const void* dres = (const char*)p.dres + (b * p.drs_b + t * p.drs_t) * se;
    float o[CH][V];
    auto load_dres = [&](int k) {
      const int col = (k * TPR + lane) * V;
      if (p.dres) {
        load8(dres, p.dres_type, col, D - col, o[k]);
      } else {
#pragma unroll
        for (int i = 0; i < V; ++i) o[k][i] = 0.f;
      }
    };
    if constexpr (kEarly) {
#pragma unroll
      for (int k = 0; k < CH; ++k) load_dres(k);
    }
    if constexpr (AHEAD) load_next(r + step < rows ? r + step : r);
    float ss = 0.f, s1 = 0.f;
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      const int col = (k * TPR + lane) * V;
      float w[V];
      load8(p.weight, kNormF32, col, D - col, w);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        ss = __builtin_fmaf(f[k][i], f[k][i], ss);
        s1 = __builtin_fmaf(g[k][i] * w[i], f[k][i], s1);
      }
    }
    ss = wave_sum(ss);
    s1 = wave_sum(s1);
    if constexpr (TPR > 64) {  // two buffers: a wave may be a round ahead of the others' reads
      if (threadIdx.x % 64 == 0) {
        lds[buf][0][wave] = ss;
        lds[buf][1][wave] = s1;
      }
      __syncthreads();
      ss = waves_sum<WPR>(lds[buf][0]);
      s1 = waves_sum<WPR>(lds[buf][1]);
    }
    const float rstd = inv_root(ss / (float)D + p.eps);
    const float coef = s1 * rstd / (float)D * rstd;  // mean(weight dy hat) rstd
    void* dx = (char*)p.dx + (b * p.dxs_b + t * p.dxs_t) * xe;
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      const int col = (k * TPR + lane) * V;
      float w[V];
      load8(p.weight, kNormF32, col, D - col, w);
      if constexpr (!kEarly) load_dres(k);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float hat = f[k][i] * rstd;
        acc[k][i] = __builtin_fmaf(g[k][i], hat, acc[k][i]);
        o[k][i] += __builtin_fmaf(rstd, g[k][i] * w[i], -hat * coef);
      }
      store8(dx, p.dx_type, col, D - col, o[k]);
    }
  }
  float* part = p.part + (int64_t)blockIdx.x * p.D;
  if constexpr (RPB > 1) {
    __shared__ float sums[TPR * V * CH];
    for (int w = 0; w < RPB; ++w) {
      if (wave == w) {
#pragma unroll
        for (int k = 0; k < CH; ++k)
#pragma unroll
          for (int i = 0; i < V; ++i) {
            float* s = &sums[(k * TPR + lane) * V + i];
            *s = w == 0 ? acc[k][i] : *s + acc[k][i];
          }
      }
      __syncthreads();
    }
    for (int64_t c = threadIdx.x; c < p.D; c += NT) part[c] = sums[c];
  } else {
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      const int col = (k * TPR + lane) * V;
      store8(part, kNormF32, col, D - col, acc[k]);
    }
  }
}

// Threads of a row.  A wave for narrow rows, once they are enough to fill the
// card; otherwise a workgroup of 256 or, for wide rows, 512.  Measured with the
// residual's addition, a wave against 256: 16384 x 768 33 us against 42, 2048 x
// 256 3.7 against 5.1; but 1024 x 768 4.5 against 4.3, 256 x 2560 5.4 against
// 3.9.  512 against 256: 1 x 2560 2.8 us against 3.3, 1024 x 4096 13.7 against
// 14.0, 4096 x 4096 38.4 against 40.9, 8192 x 8192 to e4m3 46.5 against 52.5; but
// 8192 x 4096 without a residual 23.9 against 21.9.
bool wave_rows(int64_t rows, int64_t dim) { return dim <= 1024 && rows >= 2048; }

int fwd_threads(int64_t rows, int64_t dim, bool residual) {
  if (wave_rows(rows, dim)) return 64;
  return dim > 4096 || (dim > 2048 && (rows <= 1024 || residual)) ? 512 : 256;
}

// Backward: 512 against 256: 333 x 5120 13.4 us against 15.4, 8192 x 8192 106
// against 122 (256 threads would hold four column groups each, at three waves a
// SIMD); but 16384 x 2560 118 against 107.
int bwd_threads(int64_t rows, int64_t dim) {
  if (wave_rows(rows, dim)) return 64;
  return dim > 3 * NT * V || (dim > 2048 && rows <= 1024) ? 512 : 256;
}

template <int TPR, int CH>
void launch_fwd(const NormParams& p, int64_t rows, hipStream_t stream) {
  constexpr int RPB = TPR > NT ? 1 : NT / TPR;
  const int64_t blocks = (rows + RPB - 1) / RPB, x = std::min<int64_t>(blocks, 1 << kRowShift);
  hipLaunchKernelGGL((norm_fwd_kernel<TPR, CH>), dim3((unsigned)x, (unsigned)((blocks + x - 1) / x)), dim3(RPB * TPR),
                     0, stream, p, rows);
}

template <int TPR, int CH>
void launch_bwd(const NormBwdParams& p, int64_t rows, hipStream_t stream) {
  if constexpr (kAhead<TPR, CH>)
    if (p.row_type == kNormBF16 && p.dy_type == kNormBF16) {
      hipLaunchKernelGGL((norm_bwd_kernel<TPR, CH, true>), dim3((unsigned)p.parts), dim3(TPR > NT ? TPR : NT), 0,
                         stream, p, rows);
      return;
    }
  hipLaunchKernelGGL((norm_bwd_kernel<TPR, CH, false>), dim3((unsigned)p.parts), dim3(TPR > NT ? TPR : NT), 0, stream,
                     p, rows);
}

}  // namespace

// As many workgroups as are resident at once: with more, a second, short round
// follows (16384 x 5120: 167 us at 1024 workgroups, 228 us at 1280).  A compute
// unit holds four workgroups of 256 threads or of 512 with one column group each,
// two of 512 with more.  Two rows each at least, as each workgroup's sums are
// written and read once (1001 x 1777: 14.0 us, with one row each 15.8).
int norm_bwd_parts(int64_t rows, int64_t dim) {
  const int threads = bwd_threads(rows, dim);
  const int64_t blocks = threads == 64 ? (rows + 3) / 4 : rows;
  const int64_t cap = 256 * (threads <= 256 || dim <= 512 * V ? 4 : dim <= 2 * 512 * V ? 2 : 1);
  return (int)std::min({blocks, cap, std::max<int64_t>(256, (blocks + 1) / 2)});
}

hipError_t launch_rms_norm(const NormParams& p, hipStream_t stream) {
  const int64_t rows = p.batch * p.L;
  const int threads = fwd_threads(rows, p.D, p.residual != nullptr);
  const int64_t ch = (p.D + threads * V - 1) / (threads * V);
  if (threads == 64) {
    if (ch <= 1) launch_fwd<64, 1>(p, rows, stream);
    else launch_fwd<64, 2>(p, rows, stream);
  } else if (threads == 256) {
    if (ch <= 1) launch_fwd<256, 1>(p, rows, stream);
    else launch_fwd<256, 2>(p, rows, stream);
  } else {
    if (ch <= 1) launch_fwd<512, 1>(p, rows, stream);
    else if (ch <= 2) launch_fwd<512, 2>(p, rows, stream);
    else launch_fwd<512, 4>(p, rows, stream);
  }
  return hipGetLastError();
}

hipError_t launch_rms_norm_bwd(const NormBwdParams& p, hipStream_t stream) {
  const int64_t rows = p.batch * p.L;
  const int threads = bwd_threads(rows, p.D);
  const int64_t ch = (p.D + threads * V - 1) / (threads * V);
  if (threads == 64) {
    if (ch <= 1) launch_bwd<64, 1>(p, rows, stream);
    else launch_bwd<64, 2>(p, rows, stream);
  } else if (threads == 256) {
    if (ch <= 1) launch_bwd<256, 1>(p, rows, stream);
    else if (ch <= 2) launch_bwd<256, 2>(p, rows, stream);
    else launch_bwd<256, 3>(p, rows, stream);
  } else {
    if (ch <= 1) launch_bwd<512, 1>(p, rows, stream);
    else if (ch <= 2) launch_bwd<512, 2>(p, rows, stream);
    else launch_bwd<512, 4>(p, rows, stream);
  }
  launch_column_sums(p.part, p.parts, p.D, p.D, p.dweight, nullptr, nullptr, stream);
  return hipGetLastError();
}

}  // namespace ssm
