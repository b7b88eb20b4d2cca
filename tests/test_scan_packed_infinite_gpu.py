"""Infinite states in the packed scan: what they reach is not finite up to the sequence's end, in y as in the slot, and
nothing else is touched."""
import math

import pytest
import torch

import _serve_ref as ref
from _gpu import banner
from _layer_ref import check
from test_scan_packed_gpu import TYPES, make, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("euler", [False, True])
@pytest.mark.parametrize("y_dtype", [None, torch.float32])
@pytest.mark.parametrize("shift", [-3.0, 2.0])
def test_infinite_slot(dtype, euler, y_dtype, shift):
    """A sequence over many grid lines that starts from a slot with infinite states, next to one that does not.  With
    steps around 2 all other states are forgotten within one tile behind a line."""
    banner("infinite slot %s euler %s shift %g" % (dtype, euler, shift))
    T, D, N = 1717, 40, 16
    starts, src, dst = [0, 5, T], [0, 1], [2, 3]
    v = make(200, T, D, N, 4, TYPES[dtype], shift=shift)
    bad = {k: t if t is None else t.clone() for k, t in v.items()}
    bad["states"][1, 5, 3] = math.inf
    bad["states"][1, 17] = -math.inf
    out, pool = run(bad, starts, src, dst, euler=euler, y_dtype=y_dtype)
    out, pool = out.float().cpu(), pool.cpu()
    assert not bool(out[5:, [5, 17]].isfinite().any())
    assert not math.isfinite(float(pool[3, 5, 3])) and not bool(pool[3, 17].isfinite().any())
    # all else is as without them, to the arithmetic's bound
    rest = torch.tensor([d for d in range(D) if d not in (5, 17)])
    y, h, mag, mh = ref.scan(v["x"][5:], v["delta"][5:], v["A"], v["B"][5:], v["C"][5:], v["D"], v["z"][5:], euler, True,
                             v["delta_bias"], v["states"][1])
    rel = ref.rel_scan(T - 5, 0.003 if shift == -3.0 else 0.4, 1.0, 4.0)
    got = out[5:, rest].to(TYPES[dtype] if y_dtype is None else y_dtype)
    check(got, y[:, rest], mag[:, rest], rel, "y")
    check(pool[3, rest], h[rest], mh[rest], rel, "states")
    keep = [n for n in range(N) if n != 3]
    check(pool[3, 5, keep], h[5, keep], mh[5, keep], rel, "the channel's other states")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_overflow_in_an_earlier_piece(dtype):
    """One state grows past the largest fp32 far in front of the end, beside states that decay."""
    T, D, N = 2000, 16, 4
    A = -torch.arange(1.0, N + 1).repeat(D, 1)
    A[3, 1] = 0.125
    v = make(201, T, D, N, 1, TYPES[dtype], z=False, A=A)
    v["delta"] = torch.ones(T, D).to(TYPES[dtype])
    v["C"] = (1 + v["C"].float().abs()).to(TYPES[dtype])
    out, pool = run(v, [0, T], [-1], [0], softplus=False)
    y, h, mag, _ = ref.scan(v["x"], v["delta"], v["A"], v["B"], v["C"], v["D"], None, False, False)
    top = torch.finfo(torch.float32).max
    over = int((y[:, 3].abs() < 64 * top).nonzero().max()) + 1   # behind it |h| > 4 top, since |C| < 16
    assert 600 < over < 900 and float(v["C"].float().abs().max()) < 16
    out = out.float().cpu()
    assert not bool(out[over:, 3].isfinite().any()) and not bool(pool[0, 3, 1].isfinite())
    rest = torch.tensor([d for d in range(D) if d != 3])
    assert bool(out[:, rest].isfinite().all()) and bool(pool[0, rest].isfinite().all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("euler", [False, True])
@pytest.mark.parametrize("N", [4, 16, 40])
def test_infinite_state_in_a_slot_keeps_its_sign(dtype, euler, N):
    """No step's decay is zero (exp(-72) at least), so the slot ends as infinite as it began, also where the product of
    a piece's decays is below the smallest fp32."""
    banner("infinite slot's end %s euler %s N %d" % (dtype, euler, N))
    T, D = 1717, 20
    v = make(202, T, D, N, 4, TYPES[dtype], shift=2.0, A=-(1 + torch.arange(N) * 15 / N).repeat(D, 1))
    sign = torch.randint(0, 2, (D, N), generator=torch.Generator().manual_seed(1)) * 2 - 1.0
    v["states"][1] = sign * math.inf
    _, pool = run(v, [0, 5, T], [0, 1], [2, 3], euler=euler)
    assert torch.equal(pool[3].cpu(), v["states"][1])
