// Moves between the slots of a pool, in place and all at once, for gfx950:
// pool[dst[i]] <- what pool[src[i]] held before.  Bound by HBM: a slot that
// changes is read and written once (the states of 64 x 4 beams of 5120 x 16 fp32, of
// which half are other beams' copies: 15.3 us for 84 MB, 5.5 TB/s, part of it from the
// last-level cache; forks of a window: 2.2 us, a launch).
//
// A workgroup owns a slice of every slot's row and all moves of it: it loads
// every source's part into registers, waits for all of its threads, and then
// stores.  A thread loads its moves one behind the other, each as its source's number
// is there (up to 16 of them; many workgroups hide that where rows are wide).  Slices do
// not meet, so no order between workgroups is needed, and any
// permutation, fork or chain comes out right.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "serve_device.h"

namespace ssm {
namespace {

constexpr int NT = 1024;

// L threads of T bytes each are a slice; a thread has R of the moves.
template <class T, int L, int R>
__global__ __launch_bounds__(NT) void move_kernel(MoveParams p) {
  const int64_t at = ((int64_t)blockIdx.x * L + threadIdx.x % L) * (int64_t)sizeof(T);
  const bool in = at < p.row_bytes;
  T v[R];
  int to[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int i = r * (NT / L) + (int)threadIdx.x / L;
    to[r] = -1;
    v[r] = T{};
    if (i < p.moves && in) {
      const int src = p.src[i], dst = p.dst ? p.dst[i] : i;
      if (src < p.slots && dst >= 0 && dst < p.slots && src != dst) {
        to[r] = dst;
        if (src >= 0) v[r] = *(const T*)((const char*)p.pool + (int64_t)src * p.slot_bytes + at);
      }
    }
  }
  __syncthreads();
#pragma unroll
  for (int r = 0; r < R; ++r)
    if (to[r] >= 0) *(T*)((char*)p.pool + (int64_t)to[r] * p.slot_bytes + at) = v[r];
}

// Rows of more slices than one launch may have workgroups take several: no slice meets another.
template <class T, int L, int R>
void launch_r(MoveParams p, hipStream_t stream) {
  constexpr int64_t slice = L * (int64_t)sizeof(T);
  while (p.row_bytes > 0) {
    const int64_t n = std::min((p.row_bytes + slice - 1) / slice, kLaunchBlocks1024);
    hipLaunchKernelGGL((move_kernel<T, L, R>), dim3((unsigned)n), dim3(NT), 0, stream, p);
    p.pool = (char*)p.pool + n * slice;
    p.row_bytes -= n * slice;
  }
}

template <class T>
void launch_t(const MoveParams& p, hipStream_t stream) {
  if (p.moves <= 16) launch_r<T, 64, 1>(p, stream);
  else if (p.moves <= 64) launch_r<T, 16, 1>(p, stream);
  else if (p.moves <= 256) launch_r<T, 16, 4>(p, stream);
  else if (p.moves <= 1024) launch_r<T, 16, 16>(p, stream);
  else launch_r<T, 8, 16>(p, stream);
}

}  // namespace

hipError_t launch_state_move(const MoveParams& p, hipStream_t stream) {
  const uintptr_t all = (uintptr_t)p.pool | (uintptr_t)p.row_bytes | (uintptr_t)p.slot_bytes;
  if (all % 16 == 0) launch_t<uint4>(p, stream);
  else if (all % 4 == 0) launch_t<uint32_t>(p, stream);
  else launch_t<uint16_t>(p, stream);
  return hipGetLastError();
}

}  // namespace ssm
