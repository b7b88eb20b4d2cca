"""Plain fp64 definitions (CPU, torch) of the recurrent layer's operators and
the bounds their outputs are held to.  They share no code with the kernels.

Bounds.  A stored value is off by half a step of its type at most, relative to
the value: bf16 2^-8, e4m3 2^-4 (torch.finfo(t).eps / 2).  What the fp32
arithmetic before the store adds is bounded per operator below, relative to a
magnitude that the reference computes (the sum of absolute terms), so that
cancellation is accounted for and not guessed.
"""
import torch

U32 = 2.0 ** -24  # half a step of fp32, relative
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: U32}


def sig(v):
    return torch.sigmoid(v)


def gates(x, ga, gx, A, ba=None, bx=None):
    """r, i, a, s of every step, fp64."""
    r = sig(ga.double() + (0 if ba is None else ba.double()))
    i = sig(gx.double() + (0 if bx is None else bx.double()))
    u = A.double() * r
    return r, i, torch.exp(u), torch.sqrt((-torch.expm1(2 * u)).clamp_min(0))


def gated(x, ga, gx, A, ba=None, bx=None, z=None, h0=None, lens=None, dy=None, dh_last=None):
    """Forward (and, with dy, backward) of the gated recurrence, step by step.
    Returns a dict of fp64 tensors; "mag_*" hold the sums of absolute terms."""
    b, L, D = x.shape
    x64 = x.double()
    r, i, a, s = gates(x, ga, gx, A, ba, bx)
    v = s * i * torch.nan_to_num(x64)
    n = torch.full((b,), L) if lens is None else lens.long().clamp(0, L)
    live = (torch.arange(L)[None] < n[:, None])[..., None]
    r, i, a, s, v = (torch.where(live, t, torch.zeros(())) for t in (r, i, a, s, v))
    a = torch.where(live, a, torch.ones((), dtype=torch.float64))
    x64 = torch.where(live, x64, torch.zeros((), dtype=torch.float64))
    h = torch.zeros(b, D, dtype=torch.float64) if h0 is None else h0.double()
    m = h.abs()
    first = h
    hs, ms = [], []
    for t in range(L):
        h = a[:, t] * h + v[:, t]
        m = a[:, t] * m + v[:, t].abs()
        hs.append(h)
        ms.append(m)
    hs, ms = torch.stack(hs, 1), torch.stack(ms, 1)
    z64 = None if z is None else torch.where(live, z.double(), torch.zeros((), dtype=torch.float64))
    sz = None if z is None else z64 * sig(z64)
    y = hs if z is None else hs * sz
    out = {"y": torch.where(live, y, torch.zeros((), dtype=torch.float64)), "h_last": h, "mag_h": ms,
           "mag_y": ms if z is None else ms * sz.abs(), "mag_h_last": m, "live": live, "h": hs}
    if dy is None:
        return out
    dy64 = torch.where(live, dy.double(), torch.zeros((), dtype=torch.float64))
    g = dy64 if z is None else dy64 * sz
    prev = torch.cat([first[:, None], hs[:, :-1]], 1)
    mprev = torch.cat([first.abs()[:, None], ms[:, :-1]], 1)
    inv = torch.where(s > 0, 1 / s, torch.zeros(()))
    c = torch.zeros(b, D, dtype=torch.float64) if dh_last is None else dh_last.double()
    mc = c.abs()
    dx, da, dg, dA, mx, ma, mg, mA = ([None] * L for _ in range(8))
    A64 = A.double()
    for t in reversed(range(L)):
        lam, ml = g[:, t] + c, g[:, t].abs() + mc
        c, mc = a[:, t] * lam, a[:, t] * ml
        w = i[:, t] * x64[:, t] * a[:, t] ** 2 * inv[:, t]
        du = lam * (a[:, t] * prev[:, t] - w)
        mu = ml * (a[:, t] * mprev[:, t] + w.abs())
        k = live[:, t].double()
        dx[t], mx[t] = k * lam * s[:, t] * i[:, t], ml * s[:, t] * i[:, t]
        # 1 - r and 1 - i lose their relative accuracy at open gates: the magnitudes leave them out
        da[t], ma[t] = k * du * A64 * r[:, t] * (1 - r[:, t]), mu * A64.abs() * r[:, t]
        q = s[:, t] * x64[:, t] * i[:, t] * (1 - i[:, t])
        dg[t], mg[t] = k * lam * q, ml * (s[:, t] * x64[:, t] * i[:, t]).abs()
        dA[t], mA[t] = k * du * r[:, t], mu * r[:, t]
    st = lambda v: torch.stack(v, 1)  # noqa: E731
    out.update(dx=st(dx), dgate_a=st(da), dgate_x=st(dg), dA=st(dA).sum((0, 1)), dbias_a=st(da).sum((0, 1)),
               dbias_x=st(dg).sum((0, 1)), dh0=c, mag_dx=st(mx), mag_dgate_a=st(ma), mag_dgate_x=st(mg),
               mag_dA=st(mA).sum((0, 1)), mag_dbias_a=st(ma).sum((0, 1)), mag_dbias_x=st(mg).sum((0, 1)), mag_dh0=mc)
    if z is not None:
        d = sig(z64) * (1 + z64 * (1 - sig(z64)))
        out["dz"] = dy64 * hs * d
        # silu'(z) = sig(z) (1 + z (1 - sig(z))) has the terms 1 and z (1 - sig(z)), which cancel where z is near
        # -1.278 (its zero): an error of 2^-23 of a term is no small part of their sum there, so the magnitude
        # adds the terms' absolute values as everywhere else
        out["mag_dz"] = (dy64 * ms * sig(z64) * (1 + z64.abs() * (1 - sig(z64)))).abs()
    return out


# The recurrence's arithmetic, relative to the sum of absolute terms.  With
# |gate + bias| <= 8 and |A| <= 1 (u = A r): exp2 and the reciprocal are good
# to one ulp (2^-23) each and the rounded argument adds |g| 2^-24, so r and i
# are within 10 x 2^-23; a within (10 |u| + 1) x 2^-23; s, half the error of
# 1 - a^2, within 25 x 2^-23 (the worst case sits at |u| = 0.17, where
# 1 - a^2 = 0.29 loses two bits).  An input term is within 40 x 2^-23.  A step multiplies
# the state by a (and, folded over chunks, by products of a): (10 |u| + 2) x
# 2^-23 a step, over a memory of at most N = min(L, 1 / |u|) steps.
def rel_state(L, A, r_min=0.05):
    """Bound of h (and lam) relative to the sum of absolute terms."""
    u = float(A.abs().min()) * r_min
    n = L if u == 0 else min(L, 1 / u)
    return (64 + 2 * n) * 2.0 ** -23


def rel_grad(L, A, **kw):
    """A gradient holds a state, an adjoint and about five more factors."""
    return 2 * rel_state(L, A, **kw) + 72 * 2.0 ** -23


def rel_sum(L, batch):
    """Adding up fp32 terms: a lane adds L / 16 of them at most, then 16 chunks, then the rows."""
    return (L / 16 + batch + 64) * U32


def norm_row(x, residual=None, out_dtype=None):
    """What is normalised: x, or the fp32 sum x + residual, rounded to out_dtype."""
    if residual is None:
        return x
    return (x.float() + residual.float()).to(out_dtype or residual.dtype)


def norm(row, weight, eps):
    row = row.double()
    return weight.double() * row / torch.sqrt((row * row).mean(-1, keepdim=True) + eps)


def norm_bwd(dy, row, weight, eps, dres=None):
    """(dx, dweight, sum of absolute terms of dx, of dweight)."""
    dy, row, w = dy.double(), row.double(), weight.double()
    rstd = 1 / torch.sqrt((row * row).mean(-1, keepdim=True) + eps)
    hat = row * rstd
    mean = (w * dy * hat).mean(-1, keepdim=True)
    mmean = (w * dy * hat).abs().mean(-1, keepdim=True)
    d = torch.zeros(()) if dres is None else dres.double()
    dx = rstd * (w * dy - hat * mean) + d
    mag = rstd * ((w * dy).abs() + hat.abs() * mmean) + d.abs()
    lead = tuple(range(dy.dim() - 1))
    return dx, (dy * hat).sum(lead), mag, (dy * hat).abs().sum(lead)


def w4_dense(weight, group, scale, zero=None):
    """The (outs, ins) fp64 matrix that 4-bit weights stand for."""
    outs, half = weight.shape
    q = torch.empty(outs, 2 * half, dtype=torch.float64)
    q[:, 0::2] = (weight & 15).double()
    q[:, 1::2] = (weight >> 4).double()
    z = 8.0 if zero is None else zero.double().repeat_interleave(group, 1)
    return (q - z) * scale.double().repeat_interleave(group, 1)


def check(got, want, mag, rel, what, floor=0.0):
    """|got - want| <= half(type) |want| + rel mag + floor, everywhere; got may
    not be finite where want is not."""
    assert got.shape == want.shape, (what, got.shape, want.shape)
    g, w = got.double().cpu(), want.cpu()
    bound = HALF.get(got.dtype, U32) * w.abs() + rel * mag.cpu() + floor
    bad = ~((g - w).abs() <= bound)
    worst = float(((g - w).abs() / bound.clamp_min(1e-300)).max()) if g.numel() else 0.0
    print("%s: worst error %.3g of its bound" % (what, worst), flush=True)
    assert not bool(bad.any()), "%s: %d of %d outside, worst %.3g of the bound" % (what, int(bad.sum()), g.numel(),
                                                                                    worst)
