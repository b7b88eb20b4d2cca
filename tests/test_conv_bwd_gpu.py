"""The convolution's backward, against the fp64 formula, against differences of
the forward, and as a step of a training graph."""
import pytest
import torch

import selective_state_space_60_amd as ssm
import _serve_ref as ref
from _gpu import banner
from _layer_ref import check

pytestmark = pytest.mark.gpu
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def make(seed, b, L, D, W, dt, dyt=None):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    return n(b, L, D).to(dyt or dt), n(b, L, D).to(dt), n(D, W) / W ** 0.5, 0.1 * n(D)


def compare(got, dy, x, w, b, silu):
    r = ref.conv_bwd(dy, x, w, b, silu)
    B, L, _ = x.shape
    W = w.shape[1]
    check(got["dx"], r["dx"], r["mag_dx"], ref.rel_conv_bwd(W, r["amax"]), "dx")
    rel = ref.rel_conv_sum(W, r["amax"], L, B)
    check(got["dweight"], r["dweight"], r["mag_dweight"], rel, "dweight")
    if b is not None:
        check(got["dbias"], r["dbias"], r["mag_dbias"], rel, "dbias")
    else:
        assert "dbias" not in got


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("b,L,D,W", [(1, 1, 1, 4), (2, 3, 5, 4), (1, 300, 64, 4), (3, 515, 41, 4), (2, 64, 260, 2),
                                     (1, 77, 129, 8), (2, 130, 64, 8), (1, 1000, 12, 5), (1, 9, 36, 7), (2, 65, 20, 1),
                                     (1, 33, 8, 3), (1, 40, 6, 6)])
def test_gradients(dtype, b, L, D, W):
    banner("conv bwd %s" % ((b, L, D, W, dtype),))
    dy, x, w, bias = make(L + D, b, L, D, W, TYPES[dtype])
    for silu, bb in ((True, bias), (False, None)):
        got = ssm.causal_conv1d_bwd(dy.cuda(), x.cuda(), w.cuda(), bias=None if bb is None else bb.cuda(), silu=silu)
        torch.cuda.synchronize()
        assert got["dx"].dtype == dy.dtype
        compare(got, dy, x, w, bb, silu)


def test_types_and_strides():
    """fp32 dy to bf16 x, gradient in the other type, slices of projections in and out, permuted weights."""
    b, L, D, W = 2, 150, 40, 4
    dy, x, w, bias = make(1, b, L, D, W, torch.bfloat16, torch.float32)
    wide = torch.zeros(b, L, 3 * D + 2, dtype=torch.bfloat16)
    wide[..., D + 1:2 * D + 1] = x
    gw = w.t().contiguous().cuda().t()
    out = torch.full((b, L, 2 * D), 9.0, dtype=torch.bfloat16, device="cuda")
    got = ssm.causal_conv1d_bwd(dy.cuda(), wide.cuda()[..., D + 1:2 * D + 1], gw, bias=bias.cuda(), silu=True,
                                dx=out[..., :D])
    torch.cuda.synchronize()
    compare(got, dy, x, w, bias, True)
    assert got["dx"].data_ptr() == out.data_ptr() and bool((out[..., D:] == 9).all())
    got = ssm.causal_conv1d_bwd(dy.cuda(), x.cuda(), w.cuda(), silu=True, grad_dtype=torch.bfloat16)
    compare(got, dy, x, w, None, True)


def test_against_differences():
    """The gradients against central differences of the forward kernel in fp32 (silu's third derivative is below 1,
    so a step of 2^-6 is off by 2^-12 / 6 of the terms, and the forward's rounding by 2^-24 2^7 of them)."""
    b, L, D, W = 1, 40, 8, 4
    dy, x, w, bias = make(5, b, L, D, W, torch.float32)
    got = ssm.causal_conv1d_bwd(dy.cuda(), x.cuda(), w.cuda(), bias=bias.cuda(), silu=True)
    f = lambda x, w, bias: float((ssm.causal_conv1d(x.cuda(), w.cuda(), bias.cuda(), silu=True).cpu().double() *  # noqa
                                  dy.double()).sum())
    h = 2.0 ** -6
    g = torch.Generator().manual_seed(6)
    for name, t, grad in (("x", x, got["dx"]), ("w", w, got["dweight"]), ("bias", bias, got["dbias"])):
        dirn = torch.randint(0, 2, t.shape, generator=g).float() * 2 - 1
        args = {"x": x, "w": w, "bias": bias}
        up, dn = dict(args), dict(args)
        up[name], dn[name] = t + h * dirn, t - h * dirn
        diff = (f(**up) - f(**dn)) / (2 * h)
        want = float((grad.cpu().double() * dirn.double()).sum())
        # a direction of ones moves an a by at most sum |w| (or sum |x|, or 1) times the step
        move = {"x": float(w.abs().sum(1).max()), "w": 4 * float(x.abs().max()), "bias": 1.0}[name]
        scale = float(dy.double().abs().sum())
        tol = scale * (h * h / 6 * move ** 3 + 2.0 ** -17 * (1 + move))
        assert abs(diff - want) <= tol, (name, diff, want, tol)


def test_deterministic_and_graph():
    """Equal bits from call to call, and from a captured graph replayed between eager work."""
    dy, x, w, bias = (t.cuda() for t in make(7, 2, 700, 96, 4, torch.bfloat16))
    first = ssm.causal_conv1d_bwd(dy, x, w, bias=bias, silu=True)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        ssm.causal_conv1d_bwd(dy, x, w, bias=bias, silu=True)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = ssm.causal_conv1d_bwd(dy, x, w, bias=bias, silu=True)
    for k in range(3):
        for v in held.values():
            v.zero_()
        graph.replay()
        eager = ssm.causal_conv1d_bwd(dy, x, w, bias=bias, silu=True)
        torch.cuda.synchronize()
        for name in first:
            assert torch.equal(held[name], first[name]) and torch.equal(eager[name], first[name]), (k, name)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_expanded_gradient_and_neighbours(dtype):
    """dy of a plain sum (one row for all), and a batch element of NaN next to others: their dx stays theirs."""
    g = torch.Generator().manual_seed(31)
    b, L, D, W = 3, 70, 48, 4
    x = torch.randn(b, L, D, generator=g).to(dtype)
    w, bias = torch.randn(D, W, generator=g), torch.randn(D, generator=g)
    row = torch.randn(D, generator=g).to(dtype)
    got = ssm.causal_conv1d_bwd(row.cuda().expand(b, L, D), x.cuda(), w.cuda(), bias.cuda(), silu=True)
    want = ssm.causal_conv1d_bwd(row.expand(b, L, D).contiguous().cuda(), x.cuda(), w.cuda(), bias.cuda(), silu=True)
    for k in want:
        assert torch.equal(got[k], want[k]), k
    x[1] = float("nan")
    bad = ssm.causal_conv1d_bwd(row.cuda().expand(b, L, D), x.cuda(), w.cuda(), bias.cuda(), silu=True)
    assert torch.equal(bad["dx"][0], want["dx"][0]) and torch.equal(bad["dx"][2], want["dx"][2])
