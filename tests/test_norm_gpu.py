"""GPU parity of the RMS norm (ssm_rms_norm_fwd / _bwd) against its fp64
definition, at widths around a lane's 8 columns, a wave's 512, a workgroup's
2048 and the largest, and at row counts on both sides of the split between a
wave and a workgroup per row."""
import pytest

import _layer_ref as ref
from _gpu import banner

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a GPU", allow_module_level=True)

import selective_state_space_60_amd as ssm  # noqa: E402

F32, BF16, E4M3 = torch.float32, torch.bfloat16, torch.float8_e4m3fn
EPS = 1e-5


def rel(dim):
    """Sum of squares: dim / 256 adds in a lane at most and 10 across lanes,
    halved by the root; rsqrt one ulp, two products, the division."""
    return (dim / 512 + 16) * ref.U32


def make(rows, dim, dt, residual=None, seed=0):
    g = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    x = rnd(rows, dim).to(dt)
    r = None if residual is None else (3 * rnd(rows, dim)).to(residual)
    return x, r, 1 + 0.2 * rnd(dim), rnd(rows, dim).to(dt), None if r is None else rnd(rows, dim).to(residual)


SIZES = [(1, 1), (3, 7), (2, 8), (5, 9), (4, 511), (3, 512), (2, 513), (7, 2047), (2, 2048), (3, 2056), (2, 4097),
         (1, 8200), (2, 16384), (1030, 40), (1025, 520), (1500, 1025), (1024, 1536), (1024, 2049), (1026, 2560),
         (1024, 2570), (1024, 4096), (2047, 264), (2048, 7), (2050, 512), (2049, 513), (2051, 1024), (2048, 1025)]
PAIRS = [(F32, None), (F32, F32), (BF16, None), (BF16, BF16), (BF16, F32)]


@pytest.mark.parametrize("dt,res", PAIRS, ids=lambda v: str(v).replace("torch.", ""))
@pytest.mark.parametrize("size", SIZES, ids=lambda s: "%dx%d" % s)
def test_forward_backward(size, dt, res):
    rows, dim = size
    banner("norm %s %s %s" % (size, dt, res))
    x, r, w, dy, dres = make(rows, dim, dt, res, seed=rows + dim)
    up = lambda t: None if t is None else t.cuda()  # noqa: E731
    y, ro, scale = ssm.rms_norm(up(x), up(w), eps=EPS, residual=up(r))
    assert scale is None and (ro is None) == (r is None)
    row = ref.norm_row(x, r)
    if r is not None:
        assert torch.equal(ro.cpu(), row)
    want = ref.norm(row, w, EPS)
    ref.check(y, want, want.abs(), rel(dim), "y")
    got = ssm.rms_norm_bwd(up(dy), up(row), up(w), eps=EPS, dres=up(dres))
    dx, dw, mx, mw = ref.norm_bwd(dy, row, w, EPS, dres)
    # the mean of dim products adds a second sum of the same length
    ref.check(got["dx"], dx, mx, 3 * rel(dim), "dx")
    ref.check(got["dweight"], dw, mw, rel(dim) + (rows / 64 + 128) * ref.U32, "dweight")


@pytest.mark.parametrize("dt,res", [(BF16, None), (BF16, F32), (F32, None)], ids=lambda v: str(v).replace("torch.", ""))
@pytest.mark.parametrize("size", [(1025, 2049), (1025, 4096), (1025, 4097), (1030, 6144), (1030, 6145), (1100, 8192),
                                  (1025, 8193), (5, 2049), (1, 4096)], ids=lambda s: "%dx%d" % s)
def test_workgroup_sizes(size, dt, res):
    """Both sides of the split between workgroups of 256 and 512 threads a row."""
    test_forward_backward(size, dt, res)


@pytest.mark.parametrize("group", [0, 32, 64, 128])
@pytest.mark.parametrize("size", [(3, 5), (2, 32), (4, 100), (3, 128), (2, 1000), (3, 2049), (2, 5120), (1, 16384),
                                  (1100, 72), (1030, 1537), (2050, 72), (2049, 1000)], ids=lambda s: "%dx%d" % s)
def test_e4m3(size, group):
    """Scales are the group's largest |y| / 448; values the nearest e4m3 of
    y / scale (half a step: 2^-4 of the value, 2^-10 below the normals)."""
    rows, dim = size
    banner("norm e4m3 %s group %d" % (size, group))
    x, r, w, _, _ = make(rows, dim, BF16, F32, seed=dim)
    x[0] = 0
    r[0] = 0                                   # a row of zeros
    if dim > 64:
        w[:32] = 0                             # a group of zeros in every row
    y, ro, scale = ssm.rms_norm(x.cuda(), w.cuda(), eps=EPS, residual=r.cuda(), y_dtype=E4M3, group=group)
    g = group or dim
    ng = -(-dim // g)
    assert y.dtype == E4M3 and scale.shape == (rows, ng)
    want = ref.norm(ref.norm_row(x, r), w, EPS)
    pad = torch.nn.functional.pad(want, (0, ng * g - dim)).view(rows, ng, g)
    amax = pad.abs().amax(-1)
    s64 = (amax / 448).clamp_min(2.0 ** -126)
    s = scale.double().cpu()
    assert bool(((s - s64).abs() <= (rel(dim) + 2 * ref.U32) * s64).all())
    v = (pad / s[..., None]).view(rows, ng * g)[:, :dim]
    q = y.cpu().float().double()
    slack = (rel(dim) + 8 * ref.U32) * v.abs()
    bound = torch.maximum(v.abs() * 2.0 ** -4, torch.full_like(v, 2.0 ** -10)) * (1 + 2.0 ** -10) + slack
    assert bool(((q - v).abs() <= bound).all())
    assert not bool(y[0].float().any()) and bool((scale[0] == 2.0 ** -126).all())
    assert bool((y.float().abs().amax(-1)[1:] == 448).all())


def test_output_types_and_3d():
    """bf16 rows with fp32 y; a bf16 sum of fp32 residuals; (batch, L, dim)
    slices; y and the sum inside sentinel-filled buffers."""
    b, L, dim = 2, 5, 50
    g = torch.Generator().manual_seed(4)
    base = torch.randn(b, L, 2 * dim, generator=g).to(BF16)
    resb = torch.randn(b, 2 * L, dim, generator=g)
    w = torch.rand(dim, generator=g)
    bc, rc = base.cuda(), resb.cuda()
    ybuf = torch.full((b, L, dim + 7), 9.0, device="cuda")
    obuf = torch.full((b, L + 1, dim), 9.0, device="cuda", dtype=BF16)
    y, ro, _ = ssm.rms_norm(bc[..., dim:], w.cuda(), eps=EPS, residual=rc[:, ::2], residual_out=obuf[:, :L],
                            y=ybuf[..., 3:3 + dim])
    row = ref.norm_row(base[..., dim:], resb[:, ::2], BF16)
    assert torch.equal(ro.cpu(), row) and bool((obuf[:, L] == 9).all())
    want = ref.norm(row, w, EPS)
    ref.check(y, want, want.abs(), rel(dim), "y")
    assert bool((ybuf[..., :3] == 9).all()) and bool((ybuf[..., 3 + dim:] == 9).all())
    got = ssm.rms_norm_bwd(bc[..., :dim], ro, w.cuda(), eps=EPS, grad_dtype=F32)
    dx, dw, mx, mw = ref.norm_bwd(base[..., :dim], row, w, EPS)
    assert got["dx"].dtype == F32
    ref.check(got["dx"], dx, mx, 3 * rel(dim), "dx")
    ref.check(got["dweight"], dw, mw, rel(dim) + 128 * ref.U32, "dweight")


def test_residual_in_place():
    x, r, w, _, _ = make(9, 300, BF16, F32, seed=6)
    res = r.cuda()
    y, ro, _ = ssm.rms_norm(x.cuda(), w.cuda(), residual=res, residual_out=res)
    assert ro is res and torch.equal(res.cpu(), ref.norm_row(x, r))
    want = ref.norm(ref.norm_row(x, r), w, EPS)
    ref.check(y, want, want.abs(), rel(300), "y")


def test_nan_and_infinities():
    """A NaN makes its row NaN, an infinity makes it zeros with NaN at its own
    place (0 x inf), other rows stay; the e4m3 output keeps the NaN."""
    x = torch.randn(4, 40)
    x[1, 3] = float("nan")
    x[2, 5] = float("inf")
    w = torch.ones(40)
    y = ssm.rms_norm(x.cuda(), w.cuda())[0].cpu()
    assert torch.isnan(y[1]).all() and torch.isnan(y[2, 5]) and not y[2, torch.arange(40) != 5].any()
    assert torch.isfinite(y[[0, 3]]).all()
    q = ssm.rms_norm(x.cuda(), w.cuda(), y_dtype=E4M3)[0].float().cpu()
    assert torch.isnan(q[1]).all() and torch.isnan(q[2, 5]) and torch.isfinite(q[[0, 3]]).all()


def test_gradients_against_differences():
    dim = 24
    x, r, w, dy, dres = make(3, dim, F32, F32, seed=8)
    row = ref.norm_row(x, r)
    got = ssm.rms_norm_bwd(dy.cuda(), row.cuda(), w.cuda(), eps=EPS, dres=dres.cuda())
    gen = torch.Generator().manual_seed(2)
    d, dw = torch.randn(3, dim, generator=gen).double(), torch.randn(dim, generator=gen).double()

    def loss(rr, ww):
        return float((ref.norm(rr, ww, EPS) * dy.double()).sum() + (rr * dres.double()).sum())

    e = 1e-5
    for key, vec, hi, lo in (("dx", d, loss(row.double() + e * d, w), loss(row.double() - e * d, w)),
                             ("dweight", dw, loss(row.double(), w.double() + e * dw), loss(row.double(), w.double() - e * dw))):
        terms = got[key].double().cpu() * vec
        assert abs((hi - lo) / (2 * e) - float(terms.sum())) <= 1e-5 * float(terms.abs().sum()), key


@pytest.mark.parametrize("res", [None, BF16, F32], ids=lambda v: str(v).replace("torch.", ""))
@pytest.mark.parametrize("size", [(9000, 40), (8200, 769), (2000, 1500), (3000, 2050), (1500, 4096), (700, 8193),
                                  (300, 16384), (1, 1024), (257, 9000)], ids=lambda s: "%dx%d" % s)
def test_backward_of_several_rows_a_workgroup(size, res):
    """bf16 gradients with odd strides: the loads of the row that comes next
    reach no further than the last."""
    rows, dim = size
    banner("norm backward %s %s" % (size, res))
    x, r, w, dy, dres = make(rows, dim, BF16, res, seed=rows + dim)
    row = ref.norm_row(x, r)
    wide = torch.full((rows, dim + 3), float("nan"), dtype=BF16, device="cuda")
    wide[:, 1:dim + 1] = dy.cuda()
    got = ssm.rms_norm_bwd(wide[:, 1:dim + 1], row.cuda(), w.cuda(), eps=EPS,
                           dres=None if dres is None else dres.cuda())
    dx, dw, mx, mw = ref.norm_bwd(dy, row, w, EPS, dres)
    ref.check(got["dx"], dx, mx, 3 * rel(dim), "dx")
    ref.check(got["dweight"], dw, mw, rel(dim) + (rows / 64 + 128) * ref.U32, "dweight")


@pytest.mark.parametrize("group", [0, 128])
def test_e4m3_workgroup_sizes(group):
    for size in ((1025, 2049), (1030, 6145), (3, 8200)):
        test_e4m3(size, group)
