// Internal declarations of the operators over packed sequences and pools of
// states, of the convolution's backward, of the beam selection and of the slot
// moves, shared by the host dispatch (serve_abi.cpp) and their kernels.  Not
// part of the public ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace ssm {

// Workgroups of 1024 threads that one launch is given at most (it holds fewer than 2^32 threads).
constexpr int64_t kLaunchBlocks1024 = (int64_t)1 << 21;

// Where packed sequences lie, start and end.
struct PackedSeqs {
  const int32_t* starts;  // (seqs + 1), or null: one row each
  const int32_t* src;     // (seqs), or null: slot s
  const int32_t* dst;     // (seqs), or null: src
  int tokens, seqs;
  int64_t slots;          // 0: no pool
};

// ------------------------------------------------------------- packed conv
struct ConvPackedParams {
  PackedSeqs q;
  const void* x;      // (tokens, D), innermost stride 1
  const float* w;     // (D, W)
  const float* bias;  // (D) or null
  void* y;            // (tokens, D), innermost stride 1
  void* windows;      // (slots, W - 1, D), innermost stride 1, or null
  int64_t D, W;
  int64_t xs_t, ys_t, ws_d, ws_k, bs_d;  // element strides; ys_t >= D
  int64_t wins_s, wins_t;                // of the windows: slot, row
  int io_bf16, y_f32, silu;
};

constexpr int kConvPackedStep = 32;  // rows of a piece

hipError_t launch_conv_packed(const ConvPackedParams& p, hipStream_t stream);

// ----------------------------------------------------------- conv backward
struct ConvBwdParams {
  const void* dy;      // (batch, L, D), innermost stride 1; likewise x, dx
  const void* x;
  const float* w;      // (D, W)
  const float* bias;   // (D) or null
  void* dx;
  float* dweight;      // (D, W) contiguous
  float* dbias;        // (D) or null
  float* part;         // (parts, W + 1, D): sums of one workgroup's steps
  int64_t batch, L, D, W;
  int64_t dys_b, dys_t, xs_b, xs_t, dxs_b, dxs_t, ws_d, ws_k, bs_d;
  int io_bf16, dy_f32, dx_f32, silu;
};

constexpr int64_t kConvBwdSteps = 4 * 32;  // of a workgroup
inline int64_t conv_bwd_parts(int64_t batch, int64_t seqlen) {
  return batch * ((seqlen + kConvBwdSteps - 1) / kConvBwdSteps);
}

hipError_t launch_conv_bwd(const ConvBwdParams& p, hipStream_t stream);

// ------------------------------------------------------------- packed scan
struct ScanPackedParams {
  PackedSeqs q;
  const void* x;      // (tokens, D), innermost stride 1; likewise delta, z, y
  const void* delta;
  const void* z;      // or null
  void* y;
  const void* B;      // (tokens, N)
  const void* C;
  const float* A;     // (D, N)
  const float* Dskip; // (D) or null
  const float* dbias; // (D) or null
  float* states;      // (slots, D, N), or null
  int64_t D, N;
  int64_t xs_t, ds_t, zs_t, ys_t, Bs_t, Bs_n, Cs_t, Cs_n, As_d, As_n, Ds_d, dbs_d;  // element strides
  int64_t sts_s;      // from slot to slot
  int io_bf16, y_f32, euler, dsoftplus;
  int step;           // rows of a piece (a multiple of 16)
  int lines;          // grid lines behind row 0; 0: no sequence is cut
  // words of the grid lines, for the sequences that cross them
  float* H;           // (lines, D, N): state at the line, from zeros at the line before (or the sequence's start)
  float* E;           // (lines, D, N): state at the end of a sequence that ends behind the line, from zeros there
  int* order;         // (lines + seqs): the pieces, the longest first, or null: in their order
  float* dsum;        // (lines, D): log2(e) times the sum of delta over the piece that ends at the line
  float* esum;        // (lines, D): the same over the piece from the line to its sequence's end
};

constexpr int kScanOrdered = 256;  // pieces that are put in order, at most

// The plan of a packed scan: rows of a piece, grid lines and workspace bytes.
struct ScanPackedPlan {
  int64_t step, lines, ws_H, ws_E, ws_S, ws_order, ws_total;
};
ScanPackedPlan plan_scan_packed(int64_t tokens, int64_t seqs, int64_t dim, int64_t dstate, bool single);

hipError_t launch_scan_packed(const ScanPackedParams& p, hipStream_t stream);

// ---------------------------------------------------------- beam selection
struct BeamParams {
  const void* logits;   // (batch, beams, V), innermost stride 1
  const float* scores;  // (batch, beams)
  float* out_scores;    // (batch, k)
  int32_t* tokens;
  int32_t* parents;
  int64_t batch, beams, V;
  int k;
  int64_t ls_b, ls_n, ss_b, ss_n;
  int f32;              // logits are fp32 (1) or bf16 (0)
  int values, parts;    // values of a thread, pieces of a row
  float2* stat;         // (batch, beams, parts): largest logit, sum of exp(logit - largest)
  uint64_t* cand;       // (batch, beams, parts, k): the best of a piece in falling order; 0: none
};

// Values of a thread, and pieces that a row of logits is cut into.
struct BeamPieces {
  int values;
  int64_t parts;
};
BeamPieces beam_pieces(int64_t rows, int64_t vocab);

hipError_t launch_beam_select(const BeamParams& p, hipStream_t stream);

// -------------------------------------------------------------- slot moves
struct MoveParams {
  void* pool;
  const int32_t* src;
  const int32_t* dst;   // or null: move i goes to slot i
  int64_t slots, row_bytes, slot_bytes;  // bytes of a row, and from slot to slot
  int moves;
};

hipError_t launch_state_move(const MoveParams& p, hipStream_t stream);

}  // namespace ssm
