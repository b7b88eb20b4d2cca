"""Every buffer load of the 4-bit product's launches, walked on the host with
the functions that the kernel takes its offsets from: the scalar offset stays
inside the buffer's range (the range check takes it off the range), what exists
is read where it lies, and everything else is out of range by the lane offset
alone, the tiles behind the last output included."""
import itertools
import os
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "selective_state_space_60_amd",
                    "csrc")

WALK = r"""
#include <cstdio>
#include <cstdlib>
#include "w4_loads.h"
using namespace ssm::w4;

static long seen = 0, surplus = 0;

// bytes [off + scalar, off + scalar + size) of a buffer of `range` bytes; `real`: the load is of something
static void load(const char* what, uint32_t off, int scalar, int size, int64_t range, bool real, int64_t want) {
  ++seen;
  const bool bad_scalar = scalar < 0 || scalar > range;
  const bool in = !bad_scalar && (int64_t)off + size <= range - scalar;   // as the hardware takes it
  const bool out = !bad_scalar && (int64_t)off >= range - scalar;
  if (bad_scalar || (real ? !in || (int64_t)off + scalar != want : !in && !out)) {
    std::printf("%s: offset %u scalar %d size %d range %lld real %d\n", what, off, scalar, size, (long long)range, real);
    std::exit(1);
  }
}

int main(int, char** a) {
  const int rows = atoi(a[1]), ins = atoi(a[2]), outs = atoi(a[3]), GS = atoi(a[4]), NL = atoi(a[5]), XR = atoi(a[6]);
  const int pad = atoi(a[7]);
  const int NG = 4 / GS, half = ins / 2, groups = ins / (32 * GS), es = 2;
  const int64_t xs = ins + pad;
  const Grid g = grid_of(rows, outs, 16 * NL);
  long tiles = 0;
  for (unsigned z = 0; z < g.z; ++z)
    for (unsigned y = 0; y < g.y; ++y)
      for (unsigned x = 0; x < g.x; ++x) {
        const int64_t n0 = ((int64_t)z * g.x + x) * (16 * NL);
        const int nrows = tile_rows(outs, n0, 16 * NL), steps = tile_steps(ins, nrows);
        if (y == 0 && nrows) ++tiles;
        surplus += nrows == 0;
        const int64_t rw = (int64_t)nrows * half, rs = (int64_t)nrows * groups * es, rx = ((rows - 1) * xs + ins) * 2;
        for (int wave = 0; wave < W; ++wave)
          for (int s = wave; s == wave || s - W < steps; s += W)   // the first loads, and each round's next
            for (int lane = 0; lane < 64; ++lane) {
              const int col = lane % 16, kg = lane / 16, wrow = lane / 4, unit = (lane % 4) ^ (wrow / 4);
              const uint32_t xend = x_end(steps, col, ins), send = scale_end(steps, lane, NG, groups);
              const Step q = step_at(s, steps, xend, send);
              const bool live = s < steps;
              for (int n = 0; n < NL; ++n) {
                const int r = n * 16 + wrow, k = s * (KS / 2) + unit * 16;
                load("weights", weight_offset(r, unit, nrows, half) | q.w, weight_step(q), 16, rw,
                     live && r < nrows && k < half, (int64_t)r * half + k);
              }
              for (int i = 0; i < scale_loads(NL, NG); ++i) {
                const int e = lane + i * 64, r = e / NG, k = s * NG + e % NG;
                const uint32_t at = scale_entry(e, NG, nrows, groups) | q.s;
                const bool real = live && r < nrows && k < groups;
                load("scales", at * es, scale_step(q, NG) * es, es, rs, real, ((int64_t)r * groups + k) * es);
                load("zeros", at, scale_step(q, NG), 1, rs / es, real, (int64_t)r * groups + k);
                if (!real && (int64_t)at + scale_step(q, NG) < rs / es) { std::printf("a scale too many\n"); return 1; }
              }
              for (int i = 0; i < XR; ++i) {
                const int r = (int)y * 16 + 4 * i + kg, k = s * KS + col * 8;
                const uint32_t at = x_offset(r, col, rows, xs) | q.x;
                const bool real = live && r < rows && k < ins;
                load("x", at, x_step(q), 16, rx, real, (r * xs + k) * 2);
                if (!real && (int64_t)at + x_step(q) < rx) { std::printf("x too many\n"); return 1; }
              }
            }
      }
  if (tiles * 16 * NL < outs) { std::printf("tiles missing\n"); return 1; }
  std::printf("%ld loads, %ld tiles behind the last\n", seen, surplus);
  return 0;
}
"""


@pytest.fixture(scope="module")
def walk(tmp_path_factory):
    d = tmp_path_factory.mktemp("w4")
    (d / "walk.cpp").write_text(WALK)
    subprocess.run(["g++", "-O2", "-std=c++17", "-Wall", "-Werror", "-I", CSRC, str(d / "walk.cpp"), "-o",
                    str(d / "walk")], check=True)
    return str(d / "walk")


SIZES = [(1, 128, 16), (1, 32, 1), (1, 1152, 33), (3, 2080, 50), (4, 1024, 300), (5, 96, 40), (16, 1280, 17),
         (17, 1280, 100), (33, 384, 80), (64, 640, 15), (64, 1184, 129), (40, 256, 8200), (33, 160, 1)]


@pytest.mark.parametrize("rows,ins,outs", SIZES)
def test_every_load(walk, rows, ins, outs):
    behind = 0
    for gs, nl, pad in itertools.product((1, 2, 4), (1, 2), (0, 24)):
        if ins % (32 * gs):
            continue
        xr = 1 if rows <= 4 else 4
        r = subprocess.run([walk] + [str(v) for v in (rows, ins, outs, gs, nl, xr, pad)], capture_output=True, text=True)
        assert r.returncode == 0, (rows, ins, outs, gs, nl, pad, r.stdout)
        behind += int(r.stdout.split()[2])
    tiles = (outs + 15) // 16
    assert (behind > 0) == (rows > 16 and (tiles % 8 != 0 or (outs + 31) // 32 % 8 != 0))
