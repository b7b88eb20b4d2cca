"""The selective scan of packed sequences over a pool of states, against the fp64
definition sequence by sequence."""
import pytest
import torch

import selective_state_space_60_amd as ssm
import _serve_ref as ref
from _gpu import banner
from _layer_ref import check

pytestmark = pytest.mark.gpu
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def make(seed, T, D, N, slots, dt, z=True, A=None, shift=-3.0):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    v = {"x": n(T, D).to(dt), "delta": n(T, D).clamp(-2.5, 2.5).to(dt), "B": n(T, N).to(dt), "C": n(T, N).to(dt),
         "D": 1 + 0.1 * n(D), "delta_bias": shift + 0.1 * n(D).clamp(-2, 2), "states": n(slots, D, N)}
    v["z"] = n(T, D).clamp(-4, 4).to(dt) if z else None
    v["A"] = -torch.arange(1.0, N + 1).repeat(D, 1) if A is None else A
    return v


def run(v, starts, src, dst, y=None, softplus=True, euler=False, **kw):
    i32 = lambda t: None if t is None else torch.tensor(t, dtype=torch.int32).cuda()  # noqa: E731
    g = {k: None if t is None else t.cuda() for k, t in v.items()}
    out = ssm.selective_scan_packed(g["x"], g["delta"], g["A"], g["B"], g["C"], g["states"], starts=i32(starts),
                                    src=i32(src), dst=i32(dst), D=g["D"], z=g["z"], euler=euler, y=y,
                                    delta_softplus=softplus, delta_bias=g["delta_bias"] if softplus else None, **kw)
    torch.cuda.synchronize()
    return out, g["states"]


def compare(out, pool, v, starts, src, dst, softplus=True, euler=False, dt_min=None, a_min=1.0):
    dt_min = 0.003 if dt_min is None else dt_min   # softplus(-2.5 - 3.2) = 0.0034
    kept = [None] * v["states"].shape[0]
    for begin, end, f, t in ref.packed(starts, src, dst, v["states"].shape[0], v["x"].shape[0]):
        row = slice(begin, end)
        y, h, mag, mh = ref.scan(v["x"][row], v["delta"][row], v["A"], v["B"][row], v["C"][row], v["D"],
                                 None if v["z"] is None else v["z"][row], euler, softplus,
                                 v["delta_bias"] if softplus else None, None if f is None else v["states"][f])
        rel = ref.rel_scan(end - begin, dt_min, a_min, 4.0)
        if end > begin:
            check(out[row], y, mag, rel, "rows %d:%d" % (begin, end))
        if t is not None:
            kept[t] = (h, mh, rel)
    for s, k in enumerate(kept):
        if k is None:
            assert torch.equal(pool[s].cpu(), v["states"][s]), "slot %d changed" % s
        else:
            check(pool[s], k[0], k[1], k[2], "slot %d" % s)


STARTS = [0, 1, 2, 2, 17, 33, 49, 305, 306, 322, 940, 956, 972]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D,N", [(16, 16), (64, 16), (70, 16), (33, 4), (20, 1), (24, 8), (17, 13), (8, 32), (5, 64),
                                 (18, 50), (3, 2), (130, 7)])
def test_ragged(dtype, D, N):
    banner("packed scan D %d N %d %s" % (D, N, dtype))
    S = len(STARTS) - 1
    v = make(D * N, STARTS[-1], D, N, 2 * S, TYPES[dtype])
    src = [(5 * s) % S if s % 3 else -1 for s in range(S)]
    src[4], src[5] = 99, src[7]
    dst = [S + s for s in range(S)]
    dst[10] = -1
    out, pool = run(v, STARTS, src, dst)
    compare(out, pool, v, STARTS, src, dst)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_in_place_and_forms(dtype):
    """src is dst; without z; the simplified discretisation; delta as given; A = 0, of one sign and both; tiny and
    large steps."""
    S, D, N = len(STARTS) - 1, 20, 16
    g = torch.Generator().manual_seed(1)
    mixed = -torch.rand(D, N, generator=g) * 4 - 0.25
    mixed[::3, 2] = 0.0
    for k, kw in enumerate(({}, {"euler": True}, {"A": mixed}, {"shift": -9.0}, {"shift": 2.0},
                            {"A": mixed, "shift": -9.0})):
        kw = dict(kw)
        euler = kw.pop("euler", False)
        v = make(10 + k, STARTS[-1], D, N, S, TYPES[dtype], z=k % 2 == 0, **kw)
        out, pool = run(v, STARTS, None, None, euler=euler)
        # with A = 0 a state remembers everything
        lo = {-9.0: 1e-5, 2.0: 0.4}.get(kw.get("shift"), 0.003)
        compare(out, pool, v, STARTS, None, None, euler=euler, dt_min=lo, a_min=0.0 if "A" in kw else 1.0)
    v = make(30, STARTS[-1], D, N, S, TYPES[dtype])
    v["delta"] = (v["delta"].float().abs() * 0.1 + 0.01).to(TYPES[dtype])
    out, pool = run(v, STARTS, None, None, softplus=False)
    compare(out, pool, v, STARTS, None, None, softplus=False)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shift", [-3.0, -7.0])
def test_long(dtype, shift):
    """Sequences over many grid lines: what is walked again from the true state, where states decay fast and where
    they hardly do, starts and ends at and next to lines."""
    D, N = 19, 16
    starts = [0, 255, 256, 700, 3000, 3008, 5120]
    v = make(40, starts[-1], D, N, 8, TYPES[dtype], shift=shift)
    src, dst = [0, -1, 1, 2, 2, 3], [0, 1, 4, 5, 6, 3]
    src[2] = 7
    out, pool = run(v, starts, src, dst)
    compare(out, pool, v, starts, src, dst, dt_min=0.003 if shift == -3.0 else 5e-5)


def test_small_steps_keep_their_accuracy():
    """Steps of 1e-6: (exp(delta A) - 1) / A has lost nothing, in either type."""
    for dtype in ("bf16", "f32"):
        v = make(60, 64, 16, 16, 2, TYPES[dtype], z=False)
        v["delta"] = torch.full((64, 16), 2.0 ** -20).to(TYPES[dtype])
        v["D"], v["states"] = torch.zeros(16), torch.zeros(2, 16, 16)
        out, pool = run(v, [0, 64], [-1], [1], softplus=False)
        _, h, _, _ = ref.scan(v["x"], v["delta"], v["A"], v["B"], v["C"])
        gain = (v["B"].double()[:, None, :] * v["x"].double()[:, :, None]).abs().sum(0) * 2.0 ** -20
        check(pool[1], h, gain, 96 * ref.U, dtype)   # 64 additions and a term's own error


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_wide_ranges_of_decay(dtype):
    """Channels and states whose decays are orders of magnitude apart, side by side in a wave: each keeps its accuracy.
    A term is good to 2^-14 (fp32) or 2^-11 (bf16) at the channel's largest step, and every step is the same here; 120
    additions and decays add 240 roundings."""
    T, D, N = 120, 32, 16
    g = torch.Generator().manual_seed(61)
    v = make(62, T, D, N, 2, TYPES[dtype], z=False, A=-(10 ** (torch.rand(D, N, generator=g) * 6 - 4)))
    step = 10 ** (torch.rand(D, generator=g) * 4 - 4)
    v["delta"] = step.expand(T, D).to(TYPES[dtype])
    v["D"], v["states"] = torch.zeros(D), torch.zeros(2, D, N)
    out, pool = run(v, [0, T], [-1], [1], softplus=False)
    _, h, _, _ = ref.scan(v["x"], v["delta"], v["A"], v["B"], v["C"])
    u = v["delta"][0].double()[:, None] * v["A"].double()
    mag = torch.zeros(D, N, dtype=torch.float64)
    for t in range(T):
        mag = torch.exp(u) * mag + (torch.expm1(u) / v["A"].double() * v["B"][t].double() *
                                    v["x"][t].double()[:, None]).abs()
    check(pool[1], h, mag, (2.0 ** -11 if dtype == "bf16" else 2.0 ** -14) + 240 * ref.U, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("S,D,N", [(1, 16, 16), (64, 80, 16), (3, 33, 4), (7, 130, 1), (5, 20, 64), (9, 17, 13),
                                   (2, 64, 32), (4, 8, 8)])
def test_single_tokens(dtype, S, D, N):
    banner("packed step S %d D %d N %d" % (S, D, N))
    v = make(S * D, S, D, N, 2 * S + 1, TYPES[dtype], z=S % 2 == 0)
    src = [2 * S - s for s in range(S)]
    src[0] = -5
    for s, d in ((None, None), (src, None), (src, [s if s != 1 else 9999 for s in range(S)])):
        out, pool = run(v, None, s, d)
        compare(out, pool, v, None, s, d)


def test_zero_decay_step():
    v = make(70, 3, 12, 16, 3, torch.float32, A=torch.zeros(12, 16))
    out, pool = run(v, None, None, None)
    compare(out, pool, v, None, None, None, a_min=0.0)


def test_parts_are_the_whole():
    """A prompt in parts, then tokens one by one, against the scan of the whole batch entry point."""
    D, N, T = 48, 16, 700
    v = make(80, T, D, N, 3, torch.float32)
    g = {k: None if t is None else t.cuda() for k, t in v.items()}
    want, h = ssm.selective_scan_fwd(g["x"][None], g["delta"][None], g["A"], g["B"][None], g["C"][None], D=g["D"],
                                     z=g["z"][None], want_hlast=True, delta_softplus=True, delta_bias=g["delta_bias"])
    i = lambda t: torch.tensor(t, dtype=torch.int32).cuda()  # noqa: E731
    parts, at = [], 0
    for n in (1, 300, 2, 1, 1, 350, 44, 1):
        row = slice(at, at + n)
        parts.append(ssm.selective_scan_packed(g["x"][row], g["delta"][row], g["A"], g["B"][row], g["C"][row],
                                               g["states"], starts=None if n == 1 else i([0, n]),
                                               src=i([-1 if at == 0 else 2]), dst=i([2]), D=g["D"], z=g["z"][row],
                                               delta_softplus=True, delta_bias=g["delta_bias"]))
        at += n
    assert at == T
    y, hr, mag, mh = ref.scan(v["x"], v["delta"], v["A"], v["B"], v["C"], v["D"], v["z"], False, True, v["delta_bias"])
    rel = ref.rel_scan(T, 0.003, 1.0, 4.0)
    check(torch.cat(parts), y, mag, rel, "parts")
    check(g["states"][2], hr, mh, rel, "state")
    check(want[0], y, mag, 4 * rel, "batch entry point")
    check(h[0], hr, mh, 4 * rel, "its state")


def test_rows_outside_stay_and_padding_poison():
    """NaN and infinity in rows of no sequence, and right behind a sequence's end, reach nothing."""
    D, N = 20, 16
    v = make(90, 120, D, N, 3, torch.bfloat16)
    for k in ("x", "delta", "B", "C", "z"):
        v[k] = v[k].clone()
        v[k][:3], v[k][101:] = float("nan"), float("inf")
    y = torch.full((120, D), 7.0, dtype=torch.bfloat16, device="cuda")
    starts, src, dst = [3, 60, 101], [-1, 0], [1, 2]
    out, pool = run(v, starts, src, dst, y=y)
    compare(out, pool, v, starts, src, dst)
    assert bool((y[:3] == 7).all()) and bool((y[101:] == 7).all())
    # a sequence of NaN between others
    v = make(91, 120, D, N, 3, torch.float32)
    v["B"], v["x"] = v["B"].clone(), v["x"].clone()
    v["B"][40:60], v["x"][40:60] = float("nan"), float("inf")
    starts = [0, 40, 60, 120]
    out, pool = run(v, starts, None, None)
    clean = {k: None if t is None else t.clone() for k, t in v.items()}
    clean["B"][40:60], clean["x"][40:60] = 0, 0
    o2, p2 = run(clean, starts, None, None)
    assert torch.equal(out[:40], o2[:40]) and torch.equal(out[60:], o2[60:])
    assert torch.equal(pool[0], p2[0]) and torch.equal(pool[2], p2[2]) and bool(pool[1].isnan().all())


def test_starts_out_of_order_stay_inside():
    D, N = 16, 16
    v = make(95, 64, D, N, 4, torch.float32)
    buf = torch.full((96, D), 3.0, device="cuda")
    run(v, [40, 10, -5, 2 ** 30, 64], [0, 1, 2, 3], None, y=buf[16:80])
    assert bool((buf[:16] == 3).all()) and bool((buf[80:] == 3).all())


def test_strides_and_types():
    """Streams as columns of projections, B and C columns of one, A shared by the channels, a pool of several layers,
    fp32 output of bf16 input; without a pool."""
    T, D, N, S = 90, 24, 16, 3
    v = make(100, T, D, N, S, torch.bfloat16)
    proj = torch.cat([v["x"], v["z"], v["delta"]], 1).cuda()
    bc = torch.cat([torch.zeros(T, 3).to(torch.bfloat16), v["B"], v["C"]], 1).cuda()
    pool = torch.zeros(S, 4, D, N)
    pool[:, 2] = v["states"]
    gp = pool.cuda()
    A = v["A"][0].cuda().expand(D, N)
    starts = [0, 30, 31, 90]
    args = (proj[:, :D], proj[:, 2 * D:], A, bc[:, 3:3 + N], bc[:, 3 + N:])
    kw = dict(starts=torch.tensor(starts, dtype=torch.int32).cuda(), D=v["D"].cuda(), z=proj[:, D:2 * D],
              delta_softplus=True, delta_bias=v["delta_bias"].cuda(), y_dtype=torch.float32)
    out = ssm.selective_scan_packed(*args, gp[:, 2], **kw)
    torch.cuda.synchronize()
    assert out.dtype == torch.float32
    compare(out, gp[:, 2], v, starts, None, None)
    for k in (0, 1, 3):
        assert bool((gp[:, k] == 0).all())
    out = ssm.selective_scan_packed(*args, **kw)
    v["states"] = v["states"] * 0
    compare(out, v["states"].cuda(), v, starts, [-1] * 3, [-1] * 3)


def test_many_sequences():
    """More sequences than a wave looks at in one go, over several lines."""
    D, N = 16, 16
    g = torch.Generator().manual_seed(3)
    n = torch.randint(0, 4, (150,), generator=g)
    n[70], n[149] = 900, 600
    starts = [0] + n.cumsum(0).tolist()
    v = make(110, starts[-1], D, N, 150, torch.float32, z=False)
    out, pool = run(v, starts, None, None)
    compare(out, pool, v, starts, None, None)


def test_far_rows_and_slots():
    banner("packed scan far rows")
    D, N, T, st, slot = 8, 16, 600, 4_000_000, 1_200_000_000
    v = make(120, T, D, N, 3, torch.bfloat16)
    big = torch.empty(T * st, dtype=torch.bfloat16, device="cuda").as_strided((T, D), (st, 1))
    big.copy_(v["x"])
    pool = torch.empty(2 * slot + D * N, device="cuda").as_strided((3, D, N), (slot, N, 1))
    pool.copy_(v["states"])
    g = {k: None if t is None else t.cuda() for k, t in v.items()}
    i = lambda t: torch.tensor(t, dtype=torch.int32).cuda()  # noqa: E731
    starts, src, dst = [0, 290, 600], [0, 2], [1, 2]
    out = ssm.selective_scan_packed(big, g["delta"], g["A"], g["B"], g["C"], pool, starts=i(starts), src=i(src),
                                    dst=i(dst), D=g["D"], z=g["z"], delta_softplus=True, delta_bias=g["delta_bias"])
    torch.cuda.synchronize()
    compare(out, pool, v, starts, src, dst)
    v2 = {k: (t if k in ("A", "D", "delta_bias", "states") or t is None else t[:2]) for k, t in v.items()}
    pool.copy_(v["states"])
    out = ssm.selective_scan_packed(big[:2], g["delta"][:2], g["A"], g["B"][:2], g["C"][:2], pool, src=i([2, 0]),
                                    dst=i([1, 0]), D=g["D"], z=g["z"][:2], delta_softplus=True,
                                    delta_bias=g["delta_bias"])
    compare(out, pool, v2, None, [2, 0], [1, 0])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_more_pieces_than_run_at_once(dtype):
    """Sequences of very different lengths over many channels: the pieces are taken longest first.  Channels do not
    meet, so a few of them show all."""
    T, D, N = 16400, 1040, 16
    banner("ordered pieces %s" % dtype)
    g = torch.Generator().manual_seed(81)
    starts = [0] + sorted(torch.randint(0, T + 1, (69,), generator=g).tolist()) + [T]
    seqs = len(starts) - 1
    v = make(82, T, D, N, seqs, TYPES[dtype])
    v["states"] = torch.randn(seqs, D, N, generator=g)
    src = [s if s % 3 else -1 for s in range(seqs)]
    out, pool = run(v, starts, src, list(range(seqs)))
    keep = torch.tensor(list(range(0, D, 97)) + [15, 16, 63, 64, D - 17, D - 16, D - 1])
    cut = {k: None if t is None else t[keep] if k in ("A", "D", "delta_bias") else
           t[:, keep] if k in ("x", "delta", "z", "states") else t for k, t in v.items()}
    compare(out.cpu()[:, keep], pool.cpu()[:, keep], cut, starts, src, list(range(seqs)))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N", [16, 5, 1])
@pytest.mark.parametrize("euler", [False, True])
def test_many_single_tokens(dtype, N, euler):
    """Enough of them that a wave takes two, and one too many for that."""
    S, D = 65, 1100
    banner("single tokens %d x %d x %d %s" % (S, D, N, dtype))
    v = make(83, S, D, N, S + 3, TYPES[dtype])
    src = [-1 if s == 64 else (s * 7) % S + 2 for s in range(S)]
    dst = [(s * 7) % S + 2 if s % 9 else -1 for s in range(S)]
    out, pool = run(v, None, src, dst, euler=euler)
    compare(out, pool, v, None, src, dst, euler=euler)


def test_no_steps_and_a_hair_of_decay():
    """A channel whose |A| is next to nothing and whose steps are zero keeps its state, next to channels that decay."""
    T, D, N = 40, 16, 4
    v = make(84, T, D, N, 1, torch.float32, z=False)
    v["A"] = torch.full((D, N), -40.0)
    v["A"][3] = -torch.tensor([1e-38, 1e-39, 2.0 ** -126, 1.0])
    v["x"] = v["x"] + 9
    v["delta"] = torch.full((T, D), 0.5)
    v["delta"][:, 3] = 0
    v["D"] = torch.zeros(D)
    out, pool = run(v, [0, T], None, None, softplus=False)
    assert torch.equal(pool[0, 3].cpu(), v["states"][0, 3])
    compare(out, pool, v, [0, T], [0], [0], softplus=False, dt_min=0.5, a_min=1.0)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_smallest(dtype):
    """One token, one channel, one state: as a sequence and as a token."""
    for starts in ([0, 1], None):
        for src in (None, [-1]):
            v = make(85, 1, 1, 1, 1, TYPES[dtype])
            out, pool = run(v, starts, src, [0])
            compare(out, pool, v, starts, src, [0])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("single", [False, True])
def test_neighbours_do_not_meet(dtype, single):
    """NaN and infinities in other sequences and other slots reach nothing."""
    D, N = 40, 16
    starts = None if single else STARTS
    S = 33 if single else len(STARTS) - 1
    at = list(range(S + 1)) if single else STARTS
    v = make(86, at[-1], D, N, 2 * S, TYPES[dtype])
    src, dst = [s if s % 4 < 2 else -1 for s in range(S)], [S + s for s in range(S)]
    clean, clean_pool = run(v, starts, src, dst)
    for bad in (0, 1):
        p = dict(v)
        for k in ("x", "delta", "z", "B", "C", "states"):
            p[k] = v[k].clone()
        for s in range(S):
            if s % 2 == bad:
                for k in ("x", "z", "B", "C"):
                    p[k][at[s]:at[s + 1]] = float("inf") if s % 3 else float("nan")
                p["delta"][at[s]:at[s + 1]] = float("nan") if s % 3 else 30.0
                p["states"][s] = float("nan")
        out, pool = run(p, starts, src, dst)
        for s in range(S):
            if s % 2 != bad:
                assert torch.equal(out[at[s]:at[s + 1]], clean[at[s]:at[s + 1]]), s
                assert torch.equal(pool[S + s], clean_pool[S + s]), s


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N", [3, 8, 16, 32, 64])
@pytest.mark.parametrize("euler", [False, True])
def test_chained_states_of_every_width(dtype, N, euler):
    """Sequences over many grid lines that are walked again from their true states, with B and C by rows and by columns,
    where states hardly decay."""
    T, D = 1400, 18
    banner("chained N %d euler %s %s" % (N, euler, dtype))
    starts = [0, 5, 905, 940, 1400]
    v = make(87 + N, T, D, N, 6, TYPES[dtype], shift=-6.0, A=-(0.1 + torch.arange(N) / 8).repeat(D, 1))
    src, dst = [5, 0, -1, 1], [0, 2, 3, 4]
    src[1] = 1
    out, pool = run(v, starts, src, dst, euler=euler)
    compare(out, pool, v, starts, src, dst, euler=euler, dt_min=1e-4, a_min=0.1)
    by_column = dict(v)
    for k in ("B", "C"):
        by_column[k] = v[k].t().contiguous().cuda().t()
    out2, pool2 = run(by_column, starts, src, dst, euler=euler)
    assert torch.equal(out2, out) and torch.equal(pool2, pool)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_growth_from_nothing(dtype):
    """States that grow (A > 0) and are zero for many pieces, over which the product of the growths passes the largest
    fp32; then a few steps with inputs.  And a small state that grows by more than that over one piece."""
    T, D, N = 400, 16, 8
    v = make(88, T, D, N, 2, TYPES[dtype], z=False, A=torch.full((D, N), 8.0))
    v["x"][:395] = 0
    v["delta"] = torch.ones(T, D).to(TYPES[dtype])
    v["D"] = torch.zeros(D)
    out, pool = run(v, [0, T], [-1], [1], softplus=False)
    compare(out, pool, v, [0, T], [-1], [1], softplus=False, dt_min=1.0, a_min=8.0)
    A = torch.zeros(D, N)
    v = make(89, 64, D, N, 2, torch.float32, z=False, A=A)
    v["A"][:] = 6.0
    v["x"][:] = 0
    v["delta"] = torch.ones(64, D)
    v["delta"][16:] = 0
    v["D"], v["states"] = torch.zeros(D), torch.full((2, D, N), 1e-30)
    out, pool = run(v, [0, 64], [0], [1], softplus=False)
    # 16 steps, each factor within (6 + 2) ulp, their exponents' sums exact
    want = 1e-30 * torch.exp(torch.tensor(96.0, dtype=torch.float64))
    assert float((pool[1].double().cpu() / want - 1).abs().max()) <= 16 * 8 * ref.U
