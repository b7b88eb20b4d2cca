"""The gated recurrence with A > 0, whose decays exp(A r) pass 1: nothing enters
the state (s = 0), and products of many decays pass the largest fp32 while the
states themselves need not."""
import pytest

import _layer_ref as ref
from _gpu import banner

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a GPU", allow_module_level=True)

import selective_state_space_60_amd as ssm  # noqa: E402
from test_gated_gpu import backward, by_abi, forward, make, up  # noqa: E402


@pytest.mark.parametrize("io,b", [("f32", 1), ("bf16", 1), ("bf16", 70), ("f32", 200)])
def test_a_zero_state_stays_zero(io, b):
    """A up to 6 over 400 steps: decays multiply up to exp(6 x 400).  A state of
    zero is zero all the way, and a gradient that reaches only the first steps
    is theirs."""
    banner("gated growth %s %d" % (io, b))
    L, A = 400, torch.tensor([0.5, 2.0, 6.0, -0.3]).repeat(16)
    t = make(b, L, 64, io, z=False, h0=True, seed=b, A=A)
    t["h0"][:, :] = 0
    t["dh_last"][:, :] = 0
    t["dy"][:, 4:] = 0
    c = up(t)
    ckpt = ssm.gated_scan_ckpt(b, L, 64)
    y, h = forward(c, want_hlast=True, ckpt=ckpt)
    grow = (A > 0).cuda()
    assert not bool(y[..., grow].any()) and not bool(h[:, grow].any()) and not bool(ckpt[..., grow].any())
    assert bool(torch.isfinite(y).all()) and bool(y[..., ~grow].any())
    want = ref.gated(t["x"], t["ga"], t["gx"], A, t["ba"], t["bx"], h0=t["h0"], dy=t["dy"], dh_last=t["dh_last"])
    for g in (backward(c, ckpt=ckpt), backward(c)):
        for k, v in g.items():
            assert bool(torch.isfinite(v).all()), k
        for k in ("dx", "dA"):
            assert not bool(g[k][..., grow].any()), k
        # four steps of growth: |u| <= 6, each step off by (10 |u| + 2) x 2^-23
        ref.check(g["dh0"], want["dh0"], want["mag_dh0"], (64 + 4 * 62) * 2.0 ** -23, "dh0")


def test_growth_of_a_state():
    """A state that grows over 400 steps, within fp32: A r of a step at most 0.2."""
    banner("gated growth of a state")
    L, A = 400, torch.full((40,), 0.2)
    t = make(2, L, 40, "f32", z=False, seed=5, A=A, lens=[400, 170])
    c = up(t)
    y, h = forward(c, want_hlast=True)
    want = ref.gated(t["x"], t["ga"], t["gx"], A, t["ba"], t["bx"], h0=t["h0"], lens=t["lens"])
    rel = (64 + L * (10 * 0.2 + 2)) * 2.0 ** -23
    ref.check(y, want["y"], want["mag_y"], rel, "y")
    ref.check(h, want["h_last"], want["mag_h_last"], rel, "h_last")


def test_no_wait_gives_the_same_bits():
    """The entering state computed by every workgroup itself, where products overflow."""
    banner("gated growth, no wait")
    t = make(1, 700, 33, "f32", z=False, h0=True, bias=False, seed=8, A=torch.full((33,), 4.0))
    t["h0"][:, ::2] = 0
    t["dy"][:, 20:] = 0
    t["dh_last"][:, :] = 0
    c = up(t)
    y, h = forward(c, want_hlast=True)
    grads = backward(c)
    assert not bool(y[..., ::2].any())
    sizes = {"batch": 1, "seqlen": 700, "dim": 33}
    ins = {"x": c["x"], "gate_a": c["ga"], "gate_x": c["gx"], "A": c["A"], "h0": c["h0"]}
    # states that overflow may be NaN; a NaN that is passed on has bits of its own
    same = lambda p, q: torch.equal(torch.isnan(p), torch.isnan(q)) and \
        torch.equal(torch.nan_to_num(p), torch.nan_to_num(q))  # noqa: E731
    y2, h2 = torch.full_like(y, 3.0), torch.full_like(h, 3.0)
    by_abi("ssm_gated_scan_fwd", ssm.GatedDesc, ssm.GatedPtrs, ssm.SSM_HAS_H0 | ssm.SSM_WANT_HLAST | ssm.SSM_NO_WAIT,
           sizes, dict(ins, y=y2, h_last=h2))
    assert same(y, y2) and same(h, h2)
    out = {k: torch.full_like(v, 3.0) for k, v in grads.items()}
    by_abi("ssm_gated_scan_bwd", ssm.GatedBwdDesc, ssm.GatedBwdPtrs,
           ssm.SSM_HAS_H0 | ssm.SSM_HAS_DHLAST | ssm.SSM_NO_WAIT, sizes,
           dict(ins, dy=c["dy"], dh_last=c["dh_last"], **out))
    assert all(same(out[k], grads[k]) for k in grads)
