"""Steps that a selective model all but ignores (delta of zero or next to it, x not small) beside large steps of the
same channel, packed and as single tokens: what they add, and what is kept over them, is good to its own terms."""
import pytest
import torch

import selective_state_space_60_amd as ssm
import _serve_ref as ref
from _gpu import banner
from _layer_ref import check

pytestmark = pytest.mark.gpu
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
U = ref.U


def make(seed, starts, D, N, slots, dt):
    """One step of 0.5 in every sequence and channel, at any place; the others 0 or 1e-7 to 1e-5, with x around 100."""
    T = starts[-1]
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    delta = torch.tensor([0.0, 1e-7, 1e-6, 1e-5])[torch.randint(0, 4, (T, D), generator=g)]
    for a, b in zip(starts, starts[1:]):
        delta[a + torch.randint(0, b - a, (D,), generator=g), torch.arange(D)] = 0.5
    return {"x": (100 * n(T, D)).to(dt), "delta": delta.to(dt), "B": n(T, N).to(dt), "C": n(T, N).to(dt),
            "A": -torch.arange(1.0, N + 1).repeat(D, 1),
            "states": n(slots, D, N) * 10 ** (-6 * torch.rand(slots, D, N, generator=g))}


def run(v, starts, src, dst):
    i32 = lambda t: None if t is None else torch.tensor(t, dtype=torch.int32).cuda()  # noqa: E731
    g = {k: t.cuda() for k, t in v.items()}
    y = ssm.selective_scan_packed(g["x"], g["delta"], g["A"], g["B"], g["C"], g["states"], starts=i32(starts),
                                  src=i32(src), dst=i32(dst), y_dtype=torch.float32)
    torch.cuda.synchronize()
    return y, g["states"]


def terms(v, rows, h0):
    """y, final h and the sums of their absolute terms, fp64."""
    x, dt, A, B, C = (v[k].double() for k in ("x", "delta", "A", "B", "C"))
    h, m, ys, ms = h0.double(), h0.double().abs(), [], []
    for t in rows:
        u = dt[t, :, None] * A
        add = torch.expm1(u) / A * B[t] * x[t, :, None]
        h, m = torch.exp(u) * h + add, torch.exp(u) * m + add.abs()
        ys.append((C[t] * h).sum(1))
        ms.append((C[t].abs() * m).sum(1))
    return torch.stack(ys), h, torch.stack(ms), m


# A term is within 24 U of itself (an exp2 and a difference or a polynomial of five coefficients, four products), or
# for sequences of bf16 within 2^-11.  A step multiplies the state by a decay within (|u| + 2) U and adds within U / 2;
# |u| sums up to 8 for the one large step, and states that are chained over grid lines add as much again.  The readout
# adds N / 2 U; y of a sequence in pieces may lack 2^-20 of its terms.

@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D,N", [(24, 16), (16, 5), (33, 32), (5, 64)])
def test_ignored_steps(dtype, D, N):
    banner("ignored steps D %d N %d %s" % (D, N, dtype))
    starts = [0, 16, 29, 45, 64, 96, 98]
    S = len(starts) - 1
    v = make(D * N, starts, D, N, 2 * S, TYPES[dtype])
    if N > 16:
        v["A"] = -(1 + torch.arange(N) * 15 / (N - 1)).repeat(D, 1)
    y, pool = run(v, starts, list(range(S)), list(range(S, 2 * S)))
    for s in range(S):
        rows = range(starts[s], starts[s + 1])
        yr, h, my, mh = terms(v, rows, v["states"][s])
        rel = (2.0 ** -11 if dtype == "bf16" else 0) + (24 + 3 * len(rows) + 16) * U
        check(pool[S + s], h, mh, rel, "state %d" % s)
        check(y[starts[s]:starts[s + 1]], yr, my, rel + N / 2 * U + 2.0 ** -20, "y %d" % s)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D,N", [(24, 16), (16, 5), (5, 64)])
def test_ignored_single_tokens(dtype, D, N):
    T = 70
    v = make(D + N, list(range(0, T + 1, 2)), D, N, T, TYPES[dtype])
    if N > 16:
        v["A"] = -(1 + torch.arange(N) * 15 / (N - 1)).repeat(D, 1)
    y, pool = run(v, None, None, None)
    for s in range(T):
        yr, h, my, mh = terms(v, [s], v["states"][s])
        rel = (24 + 3 + 8) * U
        check(pool[s], h, mh, rel, "state %d" % s)
        check(y[s:s + 1], yr, my, rel + N / 2 * U, "y %d" % s)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("L", [16, 11])
def test_no_step_keeps_the_bits(dtype, L):
    """Behind one large step only steps of zero: with x or without, the state is the same to the bit."""
    D, N = 20, 16
    v = make(L, [0, L], D, N, 2, TYPES[dtype])
    v["delta"][0], v["delta"][1:] = 0.5, 0
    v["states"][1] = v["states"][0]
    twice = {k: t if k in ("A", "states") else torch.cat([t, t]) for k, t in v.items()}
    twice["x"] = twice["x"].clone()
    twice["x"][L + 1:] = 0
    _, pool = run(twice, [0, L, 2 * L], [0, 1], [0, 1])
    assert torch.equal(pool[0], pool[1])
