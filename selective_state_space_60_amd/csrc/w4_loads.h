// Where the 4-bit product's loads go: the lane's offsets, each step's scalar
// offset, the tiles of the grid.  Plain arithmetic (constexpr functions run on
// the device as well), so that the host can walk every load of a launch.
//
// A buffer load's range check takes the scalar offset off the range, so that
// offset never passes the range: what does not exist is sent out of range by
// the lane offset alone, at a scalar offset that stays inside (0 where there
// is no step).
#pragma once

#include <stdint.h>

namespace ssm {
namespace w4 {

constexpr int W = 8;                    // waves
constexpr int KS = 128;                 // k of a step: one 16-byte load of weights per lane and tile
constexpr uint32_t kFar = 0x7FFFFFF0u;  // lane offset past every range: loads give 0

// Outputs of the tile at n0 that exist.
constexpr int tile_rows(int64_t outs, int64_t n0, int width) {
  return outs <= n0 ? 0 : outs - n0 < width ? (int)(outs - n0) : width;
}

constexpr int tile_steps(int ins, int nrows) { return nrows ? (ins + KS - 1) / KS : 0; }

// Loads of a step's scales per lane, for NL tiles of 16 outputs with NG groups each.
constexpr int scale_loads(int NL, int NG) { return (16 * NL * NG + 63) / 64; }

// The lane's offsets within a step: 16 bytes of a row of weights, 16 bytes of a
// row of x, an entry (not yet times its size) of the scales and zero points.
constexpr uint32_t weight_offset(int row, int unit, int nrows, int half) {
  return row < nrows ? (uint32_t)row * (uint32_t)half + (uint32_t)unit * 16 : kFar;
}

constexpr uint32_t x_offset(int row, int unit, int rows, int64_t stride) {
  return row < rows ? (uint32_t)row * (uint32_t)(stride * 2) + (uint32_t)unit * 16 : kFar;
}

constexpr uint32_t scale_entry(int e, int NG, int nrows, int groups) {
  return e / NG < nrows ? (uint32_t)(e / NG * groups + e % NG) : kFar / 4;
}

// The last step may end early: its x and scales are zeros there (weights of
// the next row, which are finite, meet x of zero).
constexpr uint32_t x_end(int steps, int unit, int ins) { return (steps - 1) * KS + unit * 8 < ins ? 0 : kFar; }

constexpr uint32_t scale_end(int steps, int lane, int NG, int groups) {
  return (steps - 1) * NG + lane % NG < groups ? 0 : kFar / 4;
}

// Step s of a wave, which may lie behind the last: what is or-ed onto the
// lane's offsets of weights, x and scales, and the step that the scalar
// offsets are taken from.
struct Step {
  int at;
  uint32_t w, x, s;
};

constexpr Step step_at(int s, int steps, uint32_t xend, uint32_t send) {
  const bool past = s >= steps;
  const uint32_t far = past ? kFar : 0;
  return Step{past ? 0 : s, far, s == steps - 1 ? xend : far, s == steps - 1 ? send : far / 4};
}

// Scalar offsets: bytes of weights and x, entries of scales and zero points.
constexpr int weight_step(const Step& q) { return q.at * (KS / 2); }
constexpr int x_step(const Step& q) { return q.at * (KS * 2); }
constexpr int scale_step(const Step& q, int NG) { return q.at * NG; }

// x tiles of outputs, then the same with the next 16 rows (y), then the next
// tiles (z, at most 65535): with eight, a tile's weights are read again on the
// same XCD.  The last z may have tiles behind the last output.
struct Grid {
  unsigned x, y, z;
};

constexpr Grid grid_of(int64_t rows, int64_t outs, int width) {
  const unsigned mtiles = (unsigned)((rows + 15) / 16), ntiles = (unsigned)((outs + width - 1) / width);
  const unsigned x = mtiles == 1 ? ntiles : 8 * (ntiles / (8 * 65535) + 1);
  return Grid{x, mtiles, (ntiles + x - 1) / x};
}

}  // namespace w4
}  // namespace ssm
