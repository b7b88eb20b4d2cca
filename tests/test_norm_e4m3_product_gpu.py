"""The norm's e4m3 output as an 8-bit projection takes it: values times scales,
multiplied with a weight matrix, against the fp64 norm's product."""
import pytest

import _layer_ref as ref
from _gpu import banner

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a GPU", allow_module_level=True)

import selective_state_space_60_amd as ssm  # noqa: E402


@pytest.mark.parametrize("group", [0, 32, 128])
@pytest.mark.parametrize("rows,dim,outs", [(1, 256, 40), (37, 1000, 24), (2050, 520, 8)])
def test_product(rows, dim, outs, group):
    """A value is off by 2^-4 of itself at most, or by half of e4m3's smallest
    step (2^-10) times the scale; the fp32 norm adds dim / 512 + 24 half steps and
    the fp64 product nothing."""
    banner("e4m3 product %dx%d -> %d group %d" % (rows, dim, outs, group))
    g = torch.Generator().manual_seed(rows + dim)
    x, residual = torch.randn(rows, dim, generator=g).bfloat16(), 3 * torch.randn(rows, dim, generator=g)
    weight, w = 1 + 0.2 * torch.randn(dim, generator=g), torch.randn(dim, outs, generator=g).double()
    y, row, scale = ssm.rms_norm(x.cuda(), weight.cuda(), residual=residual.cuda(), y_dtype=torch.float8_e4m3fn,
                                 group=group)
    each = group or dim
    s = scale.double().cpu().repeat_interleave(each, 1)[:, :dim]
    got = torch.mm(y.float().double().cpu() * s, w)
    want = ref.norm(ref.norm_row(x, residual), weight, 1e-5)
    off = torch.maximum(want.abs() * 2.0 ** -4, s * 2.0 ** -10) * (1 + 2.0 ** -9) + \
        (dim / 512 + 24) * ref.U32 * want.abs()
    assert bool(((got - torch.mm(want, w)).abs() <= torch.mm(off, w.abs())).all())
    # rounding errors of either sign: the product is far closer than its bound
    assert float((got - torch.mm(want, w)).norm() / torch.mm(want, w).norm()) < 2.0 ** -4
