// How packed sequences are cut into pieces of work.  Plain arithmetic
// (constexpr functions run on the device as well), so that the host can walk
// every piece of a launch.
//
// The rows are cut by a grid of `step` rows.  A sequence of at most `step` rows
// is one piece.  A longer one's first piece runs to the next grid line behind its
// start, and every grid line inside it starts another.  So the host, which does
// not know the lengths, launches one piece for each sequence and one for each grid
// line, whatever the sequences are.
#pragma once

#include <stdint.h>

namespace ssm {
namespace packed {

struct Run {
  int begin, end;  // rows [begin, end); empty where end <= begin
};

// Rows of sequence s, inside [0, tokens] whatever `starts` holds.
constexpr Run sequence(int start, int next, int tokens) {
  const int b = start < 0 ? 0 : (start < tokens ? start : tokens);
  return {b, next < b ? b : (next < tokens ? next : tokens)};
}

// The first piece of a sequence.
constexpr Run first_piece(Run seq, int step) {
  if (seq.end - seq.begin <= step) return seq;
  const int line = (seq.begin / step + 1) * step;
  return {seq.begin, seq.end < line ? seq.end : line};
}

// The piece from the grid line `at` on, for a sequence that is cut there (longer
// than a step, begin < at < end), else empty.
constexpr Run later_piece(Run seq, int at, int step) {
  if (at <= seq.begin || at >= seq.end || seq.end - seq.begin <= step) return {at, at};
  return {at, seq.end < at + step ? seq.end : at + step};
}

// Pieces for `seqs` sequences over `tokens` rows: the sequences' first, then
// one for each grid line behind row 0.
constexpr int64_t pieces(int64_t tokens, int64_t seqs, int64_t step) { return seqs + (tokens - 1) / step; }

// The last s with starts[s] <= at, or -1.  count(lo, stride, n) says how many
// of the n <= 64 values starts[lo], starts[lo + stride], .. are <= at: a wave
// looks at 64 at once.
template <class Count>
constexpr int last_start(int seqs, Count count) {
  int lo = 0, len = seqs;
  for (;;) {
    const int stride = (len + 63) / 64, n = (len + stride - 1) / stride;
    const int c = count(lo, stride, n);
    if (c == 0) return -1;
    lo += (c - 1) * stride;
    if (stride == 1) return lo;
    len = len - (c - 1) * stride < stride ? len - (c - 1) * stride : stride;
  }
}

}  // namespace packed
}  // namespace ssm
