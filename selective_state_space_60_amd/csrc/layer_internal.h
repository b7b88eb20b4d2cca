// Internal declarations of the recurrent layer's operators, shared by the host
// dispatch (layer_abi.cpp) and their kernels.  Not part of the public ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace ssm {

// --------------------------------------------------- gated linear recurrence
struct GatedParams {
  const void* x;       // (batch, L, D), innermost stride 1; likewise gate_a, gate_x, z, y
  const void* gate_a;
  const void* gate_x;
  const void* z;       // or null
  void* y;             // null: only the checkpoints are wanted
  const float* A;      // (D)
  const float* bias_a; // (D) or null
  const float* bias_x; // (D) or null
  const float* h0;     // (batch, D) or null
  float* h_last;       // (batch, D) or null
  const int32_t* lens; // (batch) or null
  float* ckpt;         // (batch, ceil(L/64), D): the state before every 64th step, or null
  int64_t batch, L, D;
  int64_t xs_b, xs_t, gas_b, gas_t, gxs_b, gxs_t, zs_b, zs_t, ys_b, ys_t;  // element strides
  int64_t As_d, bas_d, bxs_d;
  int io_bf16;  // x, gate_a, gate_x, z are bf16 (1) or fp32 (0)
  int y_f32;    // y stored as fp32 (1) or in the io type (0)
  void* chain;  // words of the segments (gated_chain_bytes), 256-byte aligned; unused for one segment
  int polls;    // bound of a workgroup's wait for its predecessor; 0: none waits
};

// Tiling (also used by the host planner): a workgroup owns 32 lanes x (1 or 2)
// channels over a segment of 8 chunks.
constexpr int kGatedFwdChunks = 8;
constexpr int kGatedBwdChunks = 8;
constexpr int kGatedFwdSteps = 16;  // steps per chunk, forward
constexpr int kGatedBwdSteps = 8;   // steps per chunk, backward
constexpr int kGatedCkptSteps = 64;
constexpr int kGatedSpanSteps = 128;  // rows a kernel addresses from one base, at most
constexpr int kGatedPolls = 1 << 16;  // tens of milliseconds; a wait is microseconds

// Bytes of the words of nseg segments: a pair and a state per channel.
inline int64_t gated_chain_bytes(int64_t batch, int64_t dim, int64_t nseg) {
  return nseg > 1 ? (nseg * batch * dim * 12 + 255) / 256 * 256 : 0;
}

hipError_t launch_gated_scan(const GatedParams& p, hipStream_t stream);

struct GatedBwdParams {
  GatedParams f;       // the forward's inputs; f.ckpt: the checkpoints
  const void* dy;
  const float* dh_last;  // (batch, D) or null
  void* dx;
  void* dgate_a;
  void* dgate_x;
  void* dz;            // or null
  float* dA;           // (D)
  float* dbias_a;      // (D) or null
  float* dbias_x;      // (D) or null
  float* dh0;          // (batch, D) or null
  int64_t dys_b, dys_t, dxs_b, dxs_t, dgas_b, dgas_t, dgxs_b, dgxs_t, dzs_b, dzs_t;
  int g_f32;           // dy, dx, dgate_a, dgate_x, dz are fp32 (1) or in the io type (0)
  float* part;         // (segments * batch, 3, D): sums of dA, dbias_a, dbias_x over one segment of one row
};

hipError_t launch_gated_scan_bwd(const GatedBwdParams& p, hipStream_t stream);

struct GatedUpdateParams {
  const void* x;
  const void* gate_a;
  const void* gate_x;
  const void* z;       // or null
  void* y;
  const float* A;
  const float* bias_a; // or null
  const float* bias_x; // or null
  const float* state;  // (batch, D)
  float* state_out;    // (batch, D), may be state
  int64_t batch, D;
  int64_t xs_b, gas_b, gxs_b, zs_b, ys_b, As_d, bas_d, bxs_d;
  int io_bf16, y_f32;
};

hipError_t launch_gated_state_update(const GatedUpdateParams& p, hipStream_t stream);

// --------------------------------------------------------------------- norm
enum NormType : int { kNormF32 = 0, kNormBF16 = 1, kNormE4M3 = 2 };

struct NormParams {
  const void* x;
  const void* residual;  // or null
  const float* weight;
  void* y;
  void* residual_out;    // null without residual
  float* scale;          // (rows, groups) or null
  int64_t batch, L, D, group;
  int64_t xs_b, xs_t, rs_b, rs_t, ros_b, ros_t, ys_b, ys_t;
  float eps;
  int x_type, r_type, ro_type, y_type;  // NormType
};

hipError_t launch_rms_norm(const NormParams& p, hipStream_t stream);

struct NormBwdParams {
  const void* dy;
  const void* row;
  const float* weight;
  const void* dres;  // or null
  void* dx;
  float* dweight;
  float* part;       // (parts, D): sums of dweight over one workgroup's rows
  int parts;         // workgroups
  int64_t batch, L, D;
  int64_t dys_b, dys_t, rs_b, rs_t, drs_b, drs_t, dxs_b, dxs_t;
  float eps;
  int dy_type, row_type, dres_type, dx_type;  // NormType, F32 or BF16
};

// Workgroups of the norm's backward for this many rows of this width.
int norm_bwd_parts(int64_t rows, int64_t dim);

hipError_t launch_rms_norm_bwd(const NormBwdParams& p, hipStream_t stream);

// ------------------------------------------------------------ 4-bit weights
struct W4Params {
  const void* x;          // (rows, ins) bf16
  const uint8_t* weight;  // (outs, ins / 2)
  const void* scale;      // (outs, ins / group) fp32 or bf16
  const uint8_t* zero;    // (outs, ins / group) or null
  const float* bias;      // (outs) or null
  void* y;                // (rows, outs)
  int64_t rows, ins, outs, group;
  int64_t xs_m, ys_m, bs_n;
  int scale_f32, y_f32;
};

hipError_t launch_w4_matvec(const W4Params& p, hipStream_t stream);

}  // namespace ssm
