"""The 4-bit product past 768 tiles, where a workgroup takes 32 outputs, with
more steps of k than waves (a wave's second round of loads), ragged tiles and
every form of scales: against the dense fp64 product."""
import pytest

import _layer_ref as ref
from _gpu import banner

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a GPU", allow_module_level=True)

import selective_state_space_60_amd as ssm  # noqa: E402
from test_w4_gpu import BF16, F32, check, make  # noqa: E402


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("size", [(1, 1152, 12305), (4, 2080, 12320), (4, 2304, 12310), (16, 1280, 12301),
                                  (40, 1280, 8200), (64, 2176, 3100), (33, 1056, 4129)],
                         ids=lambda s: "x".join(map(str, s)))
def test_two_tiles_a_workgroup(size, group):
    rows, ins, outs = size
    if ins % group:
        pytest.skip("the group does not divide the columns")
    assert -(-rows // 16) * -(-outs // 16) > 768 and ins > 8 * 128
    banner("w4 wide %s group %d" % (size, group))
    for k, (zero, bias, sdt, ydt) in enumerate([(False, False, BF16, BF16), (True, True, F32, F32),
                                                (True, False, BF16, F32)]):
        t = make(rows, ins, outs, group, zero, bias, seed=k + ins, scale_dtype=sdt)
        c = [None if v is None else v.cuda() for v in t]
        y = ssm.w4_matvec(c[0], c[1], c[2], zero=c[3], bias=c[4], y_dtype=ydt)
        check(y, *t, group)
        few = ssm.w4_matvec(c[0], c[1][-50:].clone(), c[2][-50:].clone(), zero=None if c[3] is None else c[3][-50:].clone(),
                            bias=None if c[4] is None else c[4][-50:], y_dtype=ydt)
        assert torch.equal(few, y[:, -50:])   # one tile a workgroup: the same bits


@pytest.mark.parametrize("rows", [17, 33, 64])
@pytest.mark.parametrize("outs", [1, 15, 16, 100, 129, 272])
def test_rows_above_sixteen(rows, outs):
    """Tiles of outputs short of a multiple of eight: rows and outputs behind the
    last are left as they were."""
    banner("w4 rows %d outs %d" % (rows, outs))
    t = make(rows, 1280, outs, 64, True, True, seed=rows + outs)
    c = [v.cuda() for v in t]
    buf = torch.full((rows + 2, outs + 9), 3.0, device="cuda")
    y = ssm.w4_matvec(c[0], c[1], c[2], zero=c[3], bias=c[4], y=buf[1:rows + 1, 4:outs + 4])
    check(y, *t, 64)
    keep = torch.ones_like(buf, dtype=torch.bool)
    keep[1:rows + 1, 4:outs + 4] = False
    assert bool((buf[keep] == 3).all())
