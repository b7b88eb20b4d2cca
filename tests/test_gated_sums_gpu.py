"""The gated scan backward's sums over batch and time, held to the roundings
that its order of adding has."""
import pytest

import _layer_ref as ref
from _gpu import banner

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a GPU", allow_module_level=True)

import selective_state_space_60_amd as ssm  # noqa: E402
from test_gated_gpu import backward, forward, make, up  # noqa: E402


def rel_sum(b, L):
    """Half a step for every addition that a term passes: eight steps in a lane,
    eight chunks of a segment, a run of every 32nd of the b ceil(L / 64)
    segments, 32 runs."""
    parts = b * -(-L // 64)
    return (8 + 8 + -(-parts // 32) + 32) * ref.U32


@pytest.mark.parametrize("io,size", [("f32", (2, 5000, 40)), ("f32", (1, 20000, 33)), ("f32", (70, 257, 66)),
                                     ("bf16", (131, 150, 64))], ids=lambda v: v if isinstance(v, str) else
                         "x".join(map(str, v)))
def test_sums(io, size):
    """The sums of the gradients that the call itself returns in fp32: dbias_a
    and dbias_x are sums of dgate_a and dgate_x, so what the elements' own
    rounding adds is not in the way."""
    banner("gated sums %s %s" % (io, size))
    b, L, D = size
    t = make(b, L, D, io, seed=L)
    c = up(t)
    c["dy"] = c["dy"].float()
    g = backward(c)
    for name in ("gate_a", "gate_x"):
        each = g["d" + name].double().cpu()
        assert g["d" + name].dtype == torch.float32
        want, mag = each.sum((0, 1)), each.abs().sum((0, 1))
        ref.check(g["dbias_" + name[-1]], want, mag, rel_sum(b, L), "dbias_" + name[-1])


def test_sums_from_checkpoints_and_without_lengths_agree():
    """Rows that a length cuts add exactly nothing."""
    banner("gated sums, lengths")
    t = make(3, 500, 64, "f32", seed=2)
    c = up(t)
    c["lens"] = torch.tensor([500, 130, 0], dtype=torch.int32, device="cuda")
    ckpt = ssm.gated_scan_ckpt(3, 500, 64)
    forward(c, ckpt=ckpt)
    g, g2 = backward(c, ckpt=ckpt), backward(c)
    assert all(torch.equal(g[k], g2[k]) for k in g)
    for name in ("gate_a", "gate_x"):
        each = g["d" + name].double().cpu()
        assert not bool(each[1, 130:].any()) and not bool(each[2].any())
        ref.check(g["dbias_" + name[-1]], each.sum((0, 1)), each.abs().sum((0, 1)), rel_sum(3, 500), name)
