"""States that later inputs cancel: y of a sequence in pieces holds the slot's state to its type's precision, also where
that was a small part of the state for a while."""
import pytest
import torch

import selective_state_space_60_amd as ssm
import _serve_ref as ref
from _gpu import banner
from _layer_ref import check

pytestmark = pytest.mark.gpu
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def run(v, T, **kw):
    i32 = lambda t: torch.tensor(t, dtype=torch.int32).cuda()  # noqa: E731
    g = {k: t.cuda() for k, t in v.items()}
    y = ssm.selective_scan_packed(g["x"], g["delta"], g["A"], g["B"], g["C"], g["states"], starts=i32([0, T]),
                                  src=i32([0]), dst=i32([1]), **kw)
    torch.cuda.synchronize()
    return y.cpu(), g["states"].cpu()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("euler", [False, True])
@pytest.mark.parametrize("big", [2.0 ** 17, 2.0 ** 21, 2.0 ** 22])
def test_whole_numbers(dtype, euler, big):
    """Nothing decays (A = 0) and every sum is a whole number below 2^24, so fp32 y is exact: the state of the slot, the
    inputs, and what is left of them once they cancel."""
    T, D, N = 1500, 20, 4
    banner("whole numbers %s euler %s" % (dtype, euler))
    dt = TYPES[dtype]
    x = torch.zeros(T, D)
    x[1::64], x[45::64] = big, -big       # inside one piece, or over a line
    v = {"x": x.to(dt), "delta": torch.ones(T, D).to(dt), "A": torch.zeros(D, N), "B": torch.ones(T, N).to(dt),
         "C": torch.tensor([1.0, 0, 0, 0]).expand(T, N).contiguous().to(dt),
         "states": torch.ones(2, D, N)}
    y, pool = run(v, T, euler=euler, y_dtype=torch.float32)
    h = v["states"][0, :, 0] + x.double().cumsum(0)
    assert torch.equal(y.double(), h)
    assert torch.equal(pool[1].double(), h[-1, :, None].expand(D, N))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_bound_of_a_bf16_y(dtype):
    """A bf16 y may lack 2^-16 of the sum of its absolute terms, an fp32 y 2^-24: large inputs, cancelled a tile later
    by one that is made for it, over a state that decays."""
    T, D, N = 1500, 16, 4
    g = torch.Generator().manual_seed(5)
    dt = TYPES[dtype]
    A = -(0.5 + torch.rand(D, N, generator=g) / 4)
    x = 0.01 * torch.randn(T, D, generator=g)
    step = 2.0 ** -5
    for t in range(3, T - 40, 41):
        x[t:t + 8] += 1e6
        x[t + 24] -= 8e6 * 0.6            # leaves about as much of them as decays in 20 steps
    v = {"x": x.to(dt), "delta": torch.full((T, D), step).to(dt), "A": A, "B": torch.ones(T, N).to(dt),
         "C": torch.randn(T, N, generator=g).to(dt), "states": torch.randn(2, D, N, generator=g)}
    yr, h, mag, mh = ref.scan(v["x"], v["delta"], v["A"], v["B"], v["C"], euler=True, h0=v["states"][0])
    rel = ref.rel_scan(T, step, 0.5)
    for kw in ({}, {"y_dtype": torch.float32}):
        y, pool = run(v, T, euler=True, **kw)
        check(y, yr, mag, rel + (2.0 ** -24 if y.dtype == torch.float32 else 2.0 ** -16), "y")
        check(pool[1], h, mh, rel, "state")
