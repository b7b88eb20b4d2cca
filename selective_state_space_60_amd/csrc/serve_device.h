// Device code shared by the kernels over packed sequences.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "packed_pieces.h"
#include "serve_internal.h"

namespace ssm {
namespace dev {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr uint32_t kRsrcWord3 = 0x00020000u;  // raw (unformatted) buffer access
constexpr uint32_t kFar = 0x40000000u;        // an offset past every range: reads return 0, writes are dropped

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// A buffer of `range` bytes at p; accesses at or past the range read 0 and write nothing.
static __device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc(const void* p, uint32_t range) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), (short)0, (int)range, (int)kRsrcWord3);
}

// Bytes that `rows` rows of a buffer cover from its first element on (`width`
// elements in the last row), kept below kFar; 0 rows: none.
static __device__ __forceinline__ uint32_t row_range(int64_t rows, int64_t stride, int64_t width, int e) {
  if (rows <= 0) return 0;
  const int64_t n = ((rows - 1) * stride + width) * e;
  return (uint32_t)(n < (int64_t)kFar ? n : kFar - 1);
}

template <bool BF16>
static __device__ __forceinline__ float raw2f(uint32_t v) {
  if constexpr (BF16) return __uint_as_float(v << 16);
  else return __uint_as_float(v);
}

template <bool BF16>
static __device__ __forceinline__ float load1(__amdgpu_buffer_rsrc_t r, uint32_t off) {
  if constexpr (BF16) return raw2f<true>((uint32_t)__builtin_amdgcn_raw_buffer_load_b16(r, (int)off, 0, 0));
  else return raw2f<false>(__builtin_amdgcn_raw_buffer_load_b32(r, (int)off, 0, 0));
}

// v in bf16 (nearest even) or fp32.
static __device__ __forceinline__ void store1(__amdgpu_buffer_rsrc_t r, uint32_t off, float v, bool f32) {
  if (f32) __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(v), r, (int)off, 0, 0);
  else __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(uint16_t, (__bf16)v), r, (int)off, 0, 0);
}

// Two floats to a bf16 pair (a in the low half), nearest even.
typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef float f32x2_t __attribute__((ext_vector_type(2)));
static __device__ __forceinline__ uint32_t pack2(float a, float b) {
  const f32x2_t v = {a, b};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2_t));
}

static __device__ __forceinline__ float sigmoid(float v) {
  return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-v * kLog2e));
}

// softplus(v) = max(v, 0) + log1p(e^-|v|), log1p(w) = log(u) w / (u - 1) with
// u = 1 + w (u - 1 is exact).
static __device__ __forceinline__ float softplus(float v) {
  const float w = __builtin_amdgcn_exp2f(-fabsf(v) * kLog2e);
  const float u = 1.f + w;
  const float lp = u == 1.f ? w : (__builtin_amdgcn_logf(u) * kLn2) * (w * __builtin_amdgcn_rcpf(u - 1.f));
  return fmaxf(v, 0.f) + lp;
}

// Rows of sequence s, in scalar registers.
static __device__ __forceinline__ packed::Run sequence_of(const PackedSeqs& q, int s) {
  if (!q.starts) return {s, s + 1};
  return packed::sequence(q.starts[s], q.starts[s + 1], q.tokens);
}

// The sequence that holds row `at`, in scalar registers; -1: none.  Every lane
// of the wave must be here.
static __device__ __forceinline__ int find_sequence(const PackedSeqs& q, int at) {
  const int lane = (int)__lane_id();
  return packed::last_start(q.seqs, [&](int lo, int stride, int n) {
    const int v = q.starts[lo + (lane < n ? lane : 0) * stride];
    return (int)__popcll(__ballot(lane < n && v <= at));
  });
}

// The slot that a sequence starts from and the one it ends in, or -1.
struct Slots {
  int64_t from, to;
};

// Both asked for at once and without a branch: a list that is not there is read
// from `any`, some memory of at least four bytes, and not used.
static __device__ __forceinline__ Slots slots_of(const PackedSeqs& q, int s, const void* any) {
  const int32_t* const ps = q.src ? q.src + s : (const int32_t*)any;
  const int32_t* const pd = q.dst ? q.dst + s : (const int32_t*)any;
  const int vs = *ps, vd = *pd;
  const int from = q.src ? vs : s, to = q.dst ? vd : from;
  return {from >= 0 && from < q.slots ? from : -1, to >= 0 && to < q.slots ? to : -1};
}

// The W taps of a thread's V channels from d0 on.  A dense (D, W) block is read by
// 16-byte words (V 4) or 8-byte words (V 2): one by one they are V W loads with
// every lane on another line.
template <int V, int W>
static __device__ __forceinline__ void load_taps(const float* w, int64_t d0, int64_t ws_d, int64_t ws_k,
                                                 float (&o)[V][W]) {
  if (V > 1 && ws_k == 1 && ws_d == W && ((uintptr_t)w & 15) == 0) {  // uniform
    const float* const at = w + d0 * W;
    float f[V * W];
    if constexpr (V == 4) {
#pragma unroll
      for (int i = 0; i < W; ++i) {
        const float4 v = ((const float4*)at)[i];
        f[4 * i] = v.x; f[4 * i + 1] = v.y; f[4 * i + 2] = v.z; f[4 * i + 3] = v.w;
      }
    } else if constexpr (V == 2) {
#pragma unroll
      for (int i = 0; i < W; ++i) {
        const float2 v = ((const float2*)at)[i];
        f[2 * i] = v.x; f[2 * i + 1] = v.y;
      }
    }
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int k = 0; k < W; ++k) o[v][k] = f[v * W + k];
    return;
  }
#pragma unroll
  for (int v = 0; v < V; ++v)
#pragma unroll
    for (int k = 0; k < W; ++k) o[v][k] = w[(d0 + v) * ws_d + k * ws_k];
}

// The kernel's first argument read anew: what only a late part needs is loaded
// there, not held in (or spilled from) scalar registers until then.
template <class P>
static __device__ __forceinline__ const P& args_anew() {
  auto at = (uint64_t)__builtin_amdgcn_kernarg_segment_ptr();
  asm volatile("" : "+s"(at));
  return *(const P*)(const __attribute__((address_space(4))) P*)at;
}

}  // namespace dev
}  // namespace ssm
