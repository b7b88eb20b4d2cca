"""The pieces that packed sequences are cut into, walked on the host with the
functions that the kernels use: every row of every sequence is in exactly one
piece, no other row is in any, and whatever the starts hold no piece leaves the
rows."""
import os
import random
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "selective_state_space_60_amd",
                    "csrc")

WALK = r"""
#include <cstdio>
#include <cstdlib>
#include <vector>
#include "packed_pieces.h"
using namespace ssm::packed;

int main(int argc, char** a) {
  const int tokens = atoi(a[1]), step = atoi(a[2]), width = atoi(a[3]), ordered = atoi(a[4]);
  std::vector<int> starts;
  for (int i = 5; i < argc; ++i) starts.push_back(atoi(a[i]));
  const int seqs = (int)starts.size() - 1;
  std::vector<int> seen(tokens, 0), owner(tokens, -1);
  auto take = [&](Run r, int s) {
    for (int t = r.begin; t < r.end; ++t) {
      if (t < 0 || t >= tokens) { std::printf("row %d\n", t); std::exit(1); }
      ++seen[t];
      owner[t] = s;
    }
  };
  for (int64_t piece = 0; piece < pieces(tokens, seqs, step); ++piece) {
    if (piece < seqs) {
      const int s = (int)piece;
      const Run q = sequence(starts[s], starts[s + 1], tokens), r = first_piece(q, step);
      if (r.end - r.begin > step) { std::printf("long\n"); return 1; }
      take(r, s);
      // as the convolution: a first piece that is shorter than the window takes the next as well
      if (width && r.end < q.end && r.end - q.begin < width - 1) take(later_piece(q, r.end, step), s);
    } else {
      const int at = (int)(piece - seqs + 1) * step;
      const int s = last_start(seqs, [&](int lo, int stride, int n) {
        int c = 0;
        for (int i = 0; i < n; ++i) {
          if (lo + i * stride < 0 || lo + i * stride >= seqs || n > 64) { std::printf("probe\n"); std::exit(1); }
          c += starts[lo + i * stride] <= at;
        }
        return c;
      });
      if (s < -1 || s >= seqs) { std::printf("sequence %d\n", s); return 1; }
      if (s < 0) continue;
      const Run q = sequence(starts[s], starts[s + 1], tokens);
      if (width && at - q.begin < width - 1) continue;
      const Run r = later_piece(q, at, step);
      if (r.end - r.begin > step) { std::printf("long\n"); return 1; }
      take(r, s);
    }
  }
  if (!ordered) return 0;
  for (int t = 0; t < tokens; ++t) {
    int want = -1;
    for (int s = 0; s < seqs; ++s)
      if (starts[s] <= t && t < starts[s + 1]) want = s;
    if (owner[t] != want || seen[t] != (want >= 0)) { std::printf("row %d: %d times, %d\n", t, seen[t], owner[t]); return 1; }
  }
  return 0;
}
"""


@pytest.fixture(scope="module")
def walk(tmp_path_factory):
    d = tmp_path_factory.mktemp("pieces")
    src, exe = d / "walk.cpp", d / "walk"
    src.write_text(WALK)
    subprocess.run(["g++", "-O1", "-std=c++17", "-Wall", "-Werror", "-fsanitize=address,undefined", "-I", CSRC, str(src),
                    "-o", str(exe)], check=True)
    return str(exe)


def go(walk, tokens, step, width, starts, ordered=True):
    r = subprocess.run([walk, str(tokens), str(step), str(width), str(int(ordered))] + [str(s) for s in starts],
                       stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    assert r.returncode == 0, (tokens, step, width, starts, r.stdout)


@pytest.mark.parametrize("step,width", [(32, 0), (32, 2), (32, 4), (32, 8), (16, 0), (256, 0)])
def test_every_row_once(walk, step, width):
    rng = random.Random(step + width)
    for n in (1, 2, 5, 64, 65, 130, 300):
        lens = [rng.choice([0, 0, 1, 1, 2, 3, 7, step - 1, step, step + 1, rng.randrange(4 * step)]) for _ in range(n)]
        first = rng.choice([0, 0, 3])
        starts = [first]
        for v in lens:
            starts.append(starts[-1] + v)
        go(walk, starts[-1] + rng.choice([1, 2, 40]), step, width, starts)
        go(walk, max(1, starts[-1]), step, width, starts)


def test_wide_search(walk):
    """More than 64 x 64 sequences."""
    starts = list(range(0, 5000)) + [9000]
    go(walk, 9000, 256, 0, starts)


def test_starts_that_break_the_rules(walk):
    rng = random.Random(1)
    for _ in range(60):
        n = rng.choice([1, 3, 70, 140])
        starts = [rng.choice([-2 ** 31, -1, 0, 5, 99, 100, 101, 2 ** 31 - 1, rng.randrange(200)]) for _ in range(n + 1)]
        go(walk, 100, rng.choice([16, 32]), rng.choice([0, 4]), starts, ordered=False)
