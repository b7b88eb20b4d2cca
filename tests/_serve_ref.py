"""Plain fp64 definitions (CPU, torch) of the operators over packed sequences and
pools of states, of the convolution's backward and of the beam selection, and
the bounds their outputs are held to.  They share no code with the kernels.

Each reference returns the sum of the absolute terms ("mag") next to a value;
the fp32 arithmetic of an operator is bounded relative to that, so that
cancellation is accounted for.  The stored value's own rounding (half a step of
its type) is added by _layer_ref.check.

Elementary errors, in units of U = 2^-23 (one ulp of fp32): exp2, log2 and the
reciprocal are good to one ulp; an argument rounded to fp32 moves e^v by |v| / 2
ulp, so sigmoid(v) is within (|v| + 4) U and silu(v) within (|v| + 5) U.
softplus(v) is within 8 U of itself for the values here (|v| <= 16: the log's
argument and the quotient w / (u - 1) add a few ulp)."""
import torch

U = 2.0 ** -23


def conv(x, weight, bias=None, silu=False, before=None):
    """One sequence: x (L, D), before (W - 1, D) or None.  (y, mag, largest |a|)."""
    L, D = x.shape
    W = weight.shape[1]
    w = weight.double()
    line = torch.cat([torch.zeros(W - 1, D, dtype=torch.float64) if before is None else before.double(), x.double()])
    a = torch.zeros(L, D, dtype=torch.float64) if bias is None else bias.double().expand(L, D).clone()
    mag = a.abs()
    for k in range(W):
        a = a + w[:, k] * line[k:k + L]
        mag = mag + (w[:, k] * line[k:k + L]).abs()
    return (a * torch.sigmoid(a) if silu else a), mag, line[L:] if W > 1 else line[:0]


def rel_conv(W, mag):
    """W + 1 roundings of the sum (|silu'| < 1.1), then silu (|silu(a)| <= |a| <= mag)."""
    return (0.55 * (W + 1) + float(mag.max()) + 5) * U


def conv_bwd(dy, x, weight, bias=None, silu=False):
    """Gradients and mags: dict of dx, dweight, dbias, mag_*, amax."""
    b, L, D = x.shape
    W = weight.shape[1]
    w, x64, dy64 = weight.double(), x.double(), dy.double()
    padded = torch.cat([torch.zeros(b, W - 1, D, dtype=torch.float64), x64], 1)
    a = torch.zeros_like(x64) if bias is None else bias.double().expand_as(x64).clone()
    ma = a.abs()
    for k in range(W):
        a = a + w[:, k] * padded[:, k:k + L]
        ma = ma + (w[:, k] * padded[:, k:k + L]).abs()
    if silu:
        s = torch.sigmoid(a)
        g, mg = dy64 * (s * (1 + a * (1 - s))), dy64.abs() * (1 + ma)
    else:
        g, mg = dy64, dy64.abs()
    late = lambda t: torch.cat([t, torch.zeros(b, W - 1, D, dtype=torch.float64)], 1)  # noqa: E731
    gl, ml = late(g), late(mg)
    dx, mx = torch.zeros_like(x64), torch.zeros_like(x64)
    dw, mw = torch.zeros(D, W, dtype=torch.float64), torch.zeros(D, W, dtype=torch.float64)
    for k in range(W):
        dx += w[:, k] * gl[:, W - 1 - k:W - 1 - k + L]
        mx += w[:, k].abs() * ml[:, W - 1 - k:W - 1 - k + L]
        dw[:, k] = (g * padded[:, k:k + L]).sum((0, 1))
        mw[:, k] = (mg * padded[:, k:k + L].abs()).sum((0, 1))
    return {"dx": dx, "dweight": dw, "dbias": g.sum((0, 1)), "mag_dx": mx, "mag_dweight": mw,
            "mag_dbias": mg.sum((0, 1)), "amax": float(ma.max())}


def rel_conv_bwd(W, amax):
    """g = dy silu'(a) is within (amax + 8 + W) U of dy (1 + sum of |terms| of a): silu' = s (1 + a (1 - s)) has the
    terms' errors (|a| + 4) U s and its slope (< 0.51) the W + 1 roundings of a.  W more for the sum over k."""
    return (amax + 8 + 2 * W) * U


def rel_conv_sum(W, amax, L, batch):
    """A lane adds up to 64 steps, then come 4 waves and the parts: at most batch L / 64 of them in runs of 1 / 32."""
    return rel_conv_bwd(W, amax) + 0.5 * (64 + 4 + batch * L / (64 * 32) + 64) * U


def scan(x, delta, A, B, C, D=None, z=None, euler=False, softplus=False, bias=None, h0=None):
    """One sequence: x, delta, z (L, D), B, C (L, N); h0 (D, N) or None.  (y, h, mag_y, mag_h): the mags hold the
    sum of absolute terms and, for the form that multiplies the update out, of |B x / A|."""
    L, Dm = x.shape
    N = A.shape[1]
    A64 = A.double()
    dt = delta.double()
    if softplus:
        dt = dt + (0 if bias is None else bias.double())
        dt = torch.logaddexp(dt, torch.zeros_like(dt))
    h = torch.zeros(Dm, N, dtype=torch.float64) if h0 is None else h0.double().clone()
    m = h.abs()
    ys, ms = [], []
    x64, B64, C64 = x.double(), B.double(), C.double()
    inv = torch.where(A64 != 0, 1 / A64, torch.zeros(()))
    for t in range(L):
        u = dt[t, :, None] * A64
        gain = dt[t, :, None].expand_as(u) if euler else torch.where(A64 != 0, torch.expm1(u) * inv,
                                                                     dt[t, :, None].expand_as(u))
        v = B64[t] * x64[t, :, None]
        h = torch.exp(u) * h + gain * v
        m = torch.exp(u) * m + (gain * v).abs() + (0 if euler else (v * inv).abs() / 16)
        ys.append((C64[t] * h).sum(1))
        ms.append((C64[t].abs() * m).sum(1))
    y = torch.stack(ys) if L else torch.zeros(0, Dm, dtype=torch.float64)
    mag = torch.stack(ms) if L else y
    if D is not None:
        y, mag = y + D.double() * x64, mag + (D.double() * x64).abs()
    if z is not None:
        s = z.double() * torch.sigmoid(z.double())
        y, mag = y * s, mag * s.abs()
    return y, h, mag, m


def rel_scan(L, dt_min, a_min, zmax=0.0):
    """A step multiplies the state by a decay within (|u| + 2) U and adds a term within 24 U (the step size 8, its
    product with A and exp or the polynomial 10, the products 3); delta's own error moves a decay by 8 |u| U, summed
    over the exponent that a term has seen, of which 16 is all that counts (e^-16 is below 2^-23).  A state
    remembers min(L, 1 / |u|) steps.  The multiplied-out form adds 4 roundings of |B x / A|, which the mags hold with
    the weight 1/16: 64 U.  The readout and the gate add 24 U and (|z| + 5) U."""
    n = min(L, 1 / max(dt_min * a_min, 1e-30))
    return (64 + 8 * 16 + 24 + 24 + 5 + zmax + 3 * n) * U


def packed(starts, src, dst, slots, tokens):
    """(begin, end, source slot or None, end slot or None) of every sequence."""
    out = []
    seqs = tokens if starts is None else len(starts) - 1
    for s in range(seqs):
        b, e = (s, s + 1) if starts is None else (starts[s], starts[s + 1])
        f = s if src is None else src[s]
        t = f if dst is None else dst[s]
        out.append((b, e, f if 0 <= f < slots else None, t if 0 <= t < slots else None))
    return out


def beam(logits, scores):
    """(batch, beams vocab) fp64 scores of all continuations; -inf throughout for beams that offer nothing."""
    l64, s64 = logits.double(), scores.double()
    off = s64 - torch.logsumexp(l64, -1)
    out = off[..., None] + l64
    live = torch.isfinite(off)[..., None]
    out = torch.where(live, out, torch.full((), float("-inf"), dtype=torch.float64))
    return out.flatten(1)
