"""A training step of the gated layer on a padded batch whose padding holds
anything: what lies behind a row's length reaches no weight's gradient."""
import pytest

from _gpu import banner

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a GPU", allow_module_level=True)

from selective_state_space_60_amd import block  # noqa: E402
from test_layer_gpu import weights  # noqa: E402


@pytest.mark.parametrize("eps", [1e-5, 0.0])
@pytest.mark.parametrize("fill", [float("nan"), float("inf"), 1e30, 0.0])
def test_padding_reaches_no_gradient(fill, eps):
    banner("padding %s eps %s" % (fill, eps))
    b, L, M, E = 3, 150, 128, 192
    lens = [150, 33, 0]
    g = torch.Generator().manual_seed(3)
    w, _ = weights(M, E)
    w.eps = eps
    u, residual = torch.randn(b, L, M, generator=g).bfloat16(), torch.randn(b, L, M, generator=g)
    dout, dres = torch.randn(b, L, M, generator=g).bfloat16(), torch.randn(b, L, M, generator=g)
    h0, n = torch.randn(b, E, generator=g).cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda")

    def step():
        out, row, state, saved = block.gated_layer_fwd(u.cuda(), residual.cuda(), w, h0=h0, lens=n, train=True)
        return out, row, state, block.gated_layer_bwd(dout.cuda(), dres.cuda(), w, saved)

    want = step()
    for v in (u, residual, dout):
        for r, k in enumerate(lens):
            v[r, k:] = fill
    got = step()
    assert torch.equal(got[2], want[2])
    for r, k in enumerate(lens):
        assert torch.equal(got[0][r, :k], want[0][r, :k]) and torch.equal(got[1][r, :k], want[1][r, :k])
        assert torch.equal(got[3]["du"][r, :k], want[3]["du"][r, :k]) and not bool(got[0][r, k:].any())
        assert torch.equal(got[3]["du"][r, k:].cpu(), dres[r, k:])
    for k in want[3]:
        if k != "du":
            assert torch.equal(got[3][k], want[3][k]) and bool(torch.isfinite(got[3][k]).all()), k
