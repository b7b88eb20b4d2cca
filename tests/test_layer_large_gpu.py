"""The recurrent layer's operators where element offsets pass 32 bits: the last
rows of a long tensor against the same rows on their own."""
import pytest

import _layer_ref as ref
from _gpu import banner

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a GPU", allow_module_level=True)

import selective_state_space_60_amd as ssm  # noqa: E402


def test_long_scan():
    """1 x 900001 x 2560 bf16 (2.3e9 elements a stream, strided through one
    projection of 6.9e9): the last steps, forward and backward, equal a scan of
    the tail alone.  With A <= -2 and an open gate a step keeps at most e^-1.4
    of the state, so nothing of what lies 2000 steps back is left."""
    banner("long scan")
    L, D, tail = 900001, 2560, 4000
    p = torch.empty(1, L, 3 * D, dtype=torch.bfloat16, device="cuda").normal_()
    x, ga, gx = p.split(D, -1)
    A, b = torch.full((D,), -2.0, device="cuda"), torch.full((D,), 6.0, device="cuda")
    y, h = ssm.gated_scan_fwd(x, ga, gx, A, b, None, want_hlast=True)
    cut = [t[:, -tail:] for t in (x, ga, gx)]
    y2, h2 = ssm.gated_scan_fwd(*cut, A, b, None, want_hlast=True)
    torch.cuda.synchronize()
    # the same values fall into other chunks, so sums associate differently: a few fp32 roundings, then bf16's own
    assert float((h - h2).abs().max()) <= 64 * ref.U32 * float(h2.abs().max())
    a, c = y[:, -2000:].float(), y2[:, -2000:].float()
    assert float((a - c).abs().max()) <= 2.0 ** -7 * float(c.abs().max())
    assert float((a != c).float().mean()) < 0.01
    g = ssm.gated_scan_bwd(y, x, ga, gx, A, b, None)
    g2 = ssm.gated_scan_bwd(y[:, -tail:], *cut, A, b, None)
    torch.cuda.synchronize()
    for k in ("dx", "dgate_a", "dgate_x"):
        a, c = g[k][:, -2000:].float(), g2[k][:, -2000:].float()
        assert float((a - c).abs().max()) <= 2.0 ** -7 * float(c.abs().max()), k
        assert float((a != c).float().mean()) < 0.01, k


def test_long_norm():
    """900001 x 2560: the last rows' norm and gradients equal those of the rows alone."""
    banner("long norm")
    R, D = 900001, 2560
    x = torch.empty(R, D, dtype=torch.bfloat16, device="cuda").normal_()
    w = torch.rand(D, device="cuda")
    y, res, _ = ssm.rms_norm(x, w, residual=x)
    y2, res2, _ = ssm.rms_norm(x[-3:], w, residual=x[-3:])
    assert torch.equal(y[-3:], y2) and torch.equal(res[-3:], res2)
    g = ssm.rms_norm_bwd(y, res, w, dres=x)["dx"][-3:]
    assert torch.equal(g, ssm.rms_norm_bwd(y2, res2, w, dres=x[-3:])["dx"])


def test_many_rows_of_a_norm():
    """2^22 + 3 rows of a workgroup each: more than a grid's first dimension holds."""
    banner("2^22 + 3 rows")
    R, D = (1 << 22) + 3, 1032
    x = torch.empty(R, D, dtype=torch.bfloat16, device="cuda").normal_()
    w = torch.rand(D, device="cuda")
    y = ssm.rms_norm(x, w)[0]
    for cut in (slice(0, 5), slice(R - 7, R)):
        assert torch.equal(y[cut], ssm.rms_norm(x[cut], w)[0])


def test_large_weights():
    """2^20 + 5 outputs of 5120: 2.7e9 bytes of weights."""
    banner("large 4-bit matrix")
    outs, ins = (1 << 20) + 5, 5120
    q = torch.randint(0, 256, (outs, ins // 2), dtype=torch.uint8, device="cuda")
    s = torch.rand(outs, ins // 128, device="cuda").bfloat16()
    x = torch.randn(2, ins, device="cuda").bfloat16()
    y = ssm.w4_matvec(x, q, s)
    y2 = ssm.w4_matvec(x, q[-37:].clone(), s[-37:].clone())
    assert torch.equal(y[:, -37:], y2)
