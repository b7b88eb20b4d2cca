// Sums of per-workgroup partial rows, in a fixed order (deterministic).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace ssm {

// N parts of a column from part k on, a load each 32 parts, all asked for at
// once; behind the last part the first is read again and counts as zero.
template <int N>
static __device__ __forceinline__ float column_run(const float* src, int64_t k, int64_t parts, int64_t stride,
                                                   float sum) {
  float v[N];
  const float* at = src + k * stride;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    v[i] = *(k + 32 * i < parts ? at : src);
    at += 32 * stride;
  }
#pragma unroll
  for (int i = 0; i < N; ++i) sum += k + 32 * i < parts ? v[i] : 0.f;
  return sum;
}

// out_y[c] = sum over k < parts of part[k * stride + y * D + c], for the up to
// three outputs y that are not null.  A workgroup takes 32 columns; 32 threads
// share a column's parts, and the 32 runs are added in order.  Latency is all
// there is, so a thread has 16 loads under way (with eight, and the rest one by
// one, 501 parts of 1777 columns cost 1.7 us more).
static __global__ __launch_bounds__(1024) void column_sums_kernel(const float* part, int64_t parts, int64_t stride,
                                                                  int64_t D, float* out0, float* out1, float* out2) {
  __shared__ float lds[32][33];
  const int lane = threadIdx.x % 32, run = threadIdx.x / 32;
  const int64_t c = (int64_t)blockIdx.x * 32 + lane;
  float* const out = blockIdx.y == 0 ? out0 : blockIdx.y == 1 ? out1 : out2;
  if (!out) return;  // block-uniform
  float sum = 0.f;
  if (c < D) {
    const float* src = part + blockIdx.y * D + c;
    if (parts <= 32 * 4) sum = column_run<4>(src, run, parts, stride, sum);
    else
      for (int64_t k = run; k < parts; k += 32 * 16) sum = column_run<16>(src, k, parts, stride, sum);
  }
  lds[run][lane] = sum;
  __syncthreads();
  if (run == 0 && c < D) {
#pragma unroll
    for (int k = 1; k < 32; ++k) sum += lds[k][lane];
    out[c] = sum;
  }
}

static inline void launch_column_sums(const float* part, int64_t parts, int64_t stride, int64_t D, float* out0,
                                      float* out1, float* out2, hipStream_t stream) {
  hipLaunchKernelGGL(column_sums_kernel, dim3((unsigned)((D + 31) / 32), out1 || out2 ? 3 : 1), dim3(1024), 0, stream,
                     part, parts, stride, D, out0, out1, out2);
}

}  // namespace ssm
