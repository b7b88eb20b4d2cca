"""One-step views with a large time stride, which addresses nothing."""
import pytest

from _gpu import banner

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a GPU", allow_module_level=True)

import selective_state_space_60_amd as ssm  # noqa: E402
from test_gated_gpu import backward, forward, make, up  # noqa: E402


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("b", [3, 300])
def test_large_time_stride(io, b):
    banner("one step, large stride %s %d" % (io, b))
    D = 64
    c = up(make(b, 1, D, io, seed=4, pack=False))
    want, h = forward(c, want_hlast=True)
    grads = backward(c)
    for stride in (1 << 33, 3):
        far = lambda v: torch.as_strided(v, (b, 1, D), (D, stride, 1))  # noqa: E731
        f = {k: far(v) if v.dim() == 3 else v for k, v in c.items() if v is not None}
        f["lens"] = None
        y, h2 = forward(f, want_hlast=True, y=far(torch.empty_like(want)))
        out = {k: far(torch.empty_like(grads[k])) for k in ("dx", "dgate_a", "dgate_x", "dz")}
        got = backward(f, out=out)
        assert torch.equal(y, want) and torch.equal(h, h2)
        assert all(torch.equal(got[k], grads[k]) for k in grads)
