"""GPU parity of ssm_w4_matvec (rows times 4-bit weights with group scales)
against the dense fp64 product, at k around a step's 128 and the eight waves'
1024, outputs around a tile's 16, and rows around the tiles of 16."""
import pytest

import _layer_ref as ref
from _gpu import banner

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a GPU", allow_module_level=True)

import selective_state_space_60_amd as ssm  # noqa: E402

F32, BF16 = torch.float32, torch.bfloat16


def make(rows, ins, outs, group, zero, bias, seed=0, scale_dtype=BF16):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, ins, generator=g).to(BF16)
    w = torch.randint(0, 256, (outs, ins // 2), generator=g, dtype=torch.uint8)
    s = ((0.1 + torch.rand(outs, ins // group, generator=g)) / ins ** 0.5).to(scale_dtype)
    z = torch.randint(0, 16, (outs, ins // group), generator=g, dtype=torch.uint8) if zero else None
    b = torch.randn(outs, generator=g) if bias else None
    return x, w, s, z, b


def check(y, x, w, s, z, b, group):
    ins = x.shape[1]
    want = x.double() @ ref.w4_dense(w, group, s, z).t()
    # the sums run over 16 + q and take off (16 + zero) sum(x): both enter the magnitude
    s64 = s.double().repeat_interleave(group, 1)
    z64 = 8.0 if z is None else z.double().repeat_interleave(group, 1)
    q = ref.w4_dense(w, group, torch.ones_like(s)) + 8.0
    mag = x.double().abs() @ ((q + 32.0 + z64) * s64).t()
    if b is not None:
        want, mag = want + b.double(), mag + b.double().abs()
    # 128 products of a group in fp32 (rounded at every add at worst), then the
    # groups of a wave's steps, eight waves and the bias
    ref.check(y, want, mag, (128 + ins / 256 + 16) * ref.U32, "y")


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("size", [(1, 128, 16), (1, 1024, 33), (2, 1152, 17), (15, 896, 1), (16, 2048, 48),
                                  (17, 1280, 100), (33, 384, 80), (64, 640, 15), (3, 128, 8197), (40, 256, 8200)],
                         ids=lambda s: "x".join(map(str, s)))
def test_sizes(size, group):
    rows, ins, outs = size
    banner("w4 %s group %d" % (size, group))
    for k, (zero, bias, sdt, ydt) in enumerate([(False, False, BF16, BF16), (True, True, F32, F32)]):
        t = make(rows, ins, outs, group, zero, bias, seed=k + ins, scale_dtype=sdt)
        c = [None if v is None else v.cuda() for v in t]
        y = ssm.w4_matvec(c[0], c[1], c[2], zero=c[3], bias=c[4], y_dtype=ydt)
        assert y.dtype == ydt
        check(y, *t, group)


@pytest.mark.parametrize("ins,group", [(32, 32), (96, 32), (64, 64), (192, 64), (160, 32), (1120, 32)])
def test_short_k(ins, group):
    """k that ends inside a step of 128."""
    banner("w4 k %d group %d" % (ins, group))
    t = make(5, ins, 40, group, True, False, seed=ins)
    c = [None if v is None else v.cuda() for v in t]
    check(ssm.w4_matvec(c[0], c[1], c[2], zero=c[3], y_dtype=F32), *t, group)


def test_exact_small_integers():
    """Whole numbers come out exactly: every nibble in every place of a dword,
    one hot x at a time (a wrong order of weights cannot cancel)."""
    ins, outs = 128, 16
    q = (torch.arange(outs)[:, None] * 5 + torch.arange(ins)[None] * 7) % 16
    w = (q[:, 0::2] | (q[:, 1::2] << 4)).to(torch.uint8).cuda()
    s = torch.ones(outs, 1, dtype=BF16, device="cuda")
    for k0 in range(0, ins, 64):
        x = torch.zeros(64, ins, dtype=BF16)
        x[torch.arange(64), torch.arange(64) + k0] = 1
        y = ssm.w4_matvec(x.cuda(), w, s, y_dtype=F32).cpu()
        assert torch.equal(y, (q[:, k0:k0 + 64].t() - 8).float())


def test_strides_and_neighbours():
    """x and y as slices; the rest of y's buffer stays."""
    t = make(7, 256, 50, 64, False, True, seed=3)
    wide = torch.zeros(7, 512, dtype=BF16, device="cuda")
    wide[:, 64:320] = t[0].cuda()
    buf = torch.full((9, 61), 5.0, device="cuda")
    y = ssm.w4_matvec(wide[:, 64:320], t[1].cuda(), t[2].cuda(), bias=t[4].cuda(), y=buf[1:8, 4:54])
    check(y, *t, 64)
    keep = torch.ones_like(buf, dtype=torch.bool)
    keep[1:8, 4:54] = False
    assert bool((buf[keep] == 5).all())


def test_nonfinite_rows():
    """A row of x with an infinity or a NaN gives a row of NaN; other rows stay."""
    t = list(make(4, 256, 32, 128, False, False, seed=5))
    t[0][1, 200] = float("inf")
    t[0][2, 3] = float("nan")
    y = ssm.w4_matvec(t[0].cuda(), t[1].cuda(), t[2].cuda()).cpu()
    assert torch.isnan(y[1:3]).all() and torch.isfinite(y[[0, 3]]).all()


def test_quantize():
    """w4_quantize: half a step off at most, and the product of its weights."""
    g = torch.Generator().manual_seed(1)
    w = torch.randn(40, 256, generator=g)
    w[3, :64] = 0
    packed, s = ssm.w4_quantize(w, group=64, scale_dtype=F32)
    dense = ref.w4_dense(packed, 64, s)
    step = s.double().repeat_interleave(64, 1)
    assert bool(((dense - w.double()).abs() <= 0.5 * step * (1 + 2.0 ** -20)).all()) and not dense[3, :64].any()
    x = torch.randn(3, 256, generator=g).to(BF16)
    y = ssm.w4_matvec(x.cuda(), packed.cuda(), s.cuda(), y_dtype=F32)
    check(y, x, packed, s, None, None, 64)


def test_large_rows():
    """|x| just below 2^112: no group's sum overflows, zero points of 255 included."""
    banner("w4 large x")
    x, w, s, _, _ = make(2, 512, 40, 128, False, False, seed=9, scale_dtype=F32)
    x = (torch.sign(x.float()) * 2.0 ** 111 * 1.9).to(BF16)
    x[0] = x[0].abs()
    z = torch.full((40, 4), 255, dtype=torch.uint8)
    for zero in (None, z):
        y = ssm.w4_matvec(x.cuda(), w.cuda(), s.cuda(), zero=None if zero is None else zero.cuda(), y_dtype=F32)
        check(y, x, w, s, zero, None, 128)
