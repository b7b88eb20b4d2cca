"""Beam search's selection against fp64 scores of all continuations, and the moves
of a pool's slots against indexing a copy of it."""
import math

import pytest
import torch

import selective_state_space_60_amd as ssm
import _serve_ref as ref
from _gpu import banner

pytestmark = pytest.mark.gpu
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}

# The normaliser: a lane adds up to 64 exponentials and six more levels, each exponential within 17 ulp for arguments
# down to -32 (what lies below adds nothing): (35 + 17) 2^-23 of it, so of the score in absolute terms.
SLACK = 52 * 2.0 ** -23


def compare(got, logits, scores, k):
    """Scores by rank; every chosen continuation has its rank's score; all differ; ties by index."""
    gs, gt, gp = (t.cpu() for t in got)
    V = logits.shape[-1]
    allscores = ref.beam(logits, scores)
    want = torch.sort(allscores, dim=-1, descending=True, stable=True)
    index = gp.long() * V + gt.long()
    assert bool(((gt >= 0) & (gt < V) & (gp >= 0) & (gp < logits.shape[1])).all())
    for b in range(logits.shape[0]):
        assert len(set(index[b].tolist())) == k
        ws, mine = want.values[b, :k], allscores[b][index[b]]
        fin = torch.isfinite(ws)
        assert torch.equal(torch.isneginf(gs[b]), ~fin) and torch.equal(torch.isneginf(mine), ~fin)
        assert bool(((gs[b].double() - ws)[fin].abs() <= SLACK + ws[fin].abs() * 2.0 ** -24).all())
        assert bool(((mine - ws)[fin].abs() <= 2 * SLACK).all())
        # where the order is not within the arithmetic's reach it has to be the reference's
        clear = torch.ones(k, dtype=torch.bool)
        near = want.values[b, :k + 1] if want.values.shape[1] > k else want.values[b]
        for i in range(k):
            for j in (i - 1, i + 1):
                if 0 <= j < len(near) and bool(fin[i]):
                    same_beam = want.indices[b, i] // V == want.indices[b, j] // V
                    if not same_beam and float((near[i] - near[j]).abs()) <= 2 * SLACK:
                        clear[i] = False
        assert torch.equal(index[b][clear], want.indices[b, :k][clear]), b
    return clear


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("batch,beams,V,k", [(1, 1, 1, 1), (2, 3, 7, 5), (1, 1, 1000, 1), (3, 4, 1025, 8), (2, 2, 65, 64),
                                             (1, 16, 4097, 32), (5, 1, 9000, 64), (64, 5, 2100, 10), (2, 4, 50281, 8),
                                             (1, 3, 131, 64), (300, 16, 1030, 3), (40, 8, 20000, 6)])
def test_random(dtype, batch, beams, V, k):
    banner("beam %s" % ((batch, beams, V, k, dtype),))
    g = torch.Generator().manual_seed(V + k)
    logits = (3 * torch.randn(batch, beams, V, generator=g)).to(TYPES[dtype])
    scores = -10 * torch.rand(batch, beams, generator=g)
    compare(ssm.beam_select(logits.cuda(), scores.cuda(), k), logits, scores, k)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_ties(dtype):
    """Equal logits, equal beams, both zeros: the lower index first, exactly."""
    for V in (40, 3000, 5000):
        k = 20
        flat = torch.zeros(2, 3, V)
        flat[1, :, 1::2] = -0.0
        got = ssm.beam_select(flat.to(TYPES[dtype]).cuda(), torch.zeros(2, 3).cuda(), k)
        assert torch.equal(got[1].cpu(), torch.arange(k, dtype=torch.int32).expand(2, k))
        assert bool((got[2] == 0).all())
        steps = (torch.arange(V) % 11).float().expand(1, 4, V).to(TYPES[dtype])
        got = ssm.beam_select(steps.cuda(), torch.zeros(1, 4).cuda(), k)
        at = sorted(((n, v) for n in range(4) for v in range(V)), key=lambda c: (-(c[1] % 11), c))[:k]
        assert got[2].cpu()[0].tolist() == [n for n, _ in at] and got[1].cpu()[0].tolist() == [v for _, v in at]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("order", [1, -1])
def test_sorted_rows(dtype, order):
    """Rising and falling rows: one lane holds all of the best."""
    V, k = 6000, 33
    row = torch.arange(V).float() if dtype == "f32" else (torch.arange(V) // 24).float()
    logits = (row if order == 1 else row.flip(0)).expand(1, 2, V).to(TYPES[dtype])
    scores = torch.tensor([[0.0, -0.5]])
    compare(ssm.beam_select(logits.cuda(), scores.cuda(), k), logits, scores, k)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_banned_and_broken(dtype):
    """Rows with few or no tokens left, beams not in use, NaN and infinities: their place, and nothing else's."""
    inf, nan = math.inf, math.nan
    g = torch.Generator().manual_seed(4)
    V, k = 5000, 12
    logits = torch.randn(7, 4, V, generator=g).to(TYPES[dtype])
    scores = -torch.rand(7, 4, generator=g)
    logits[0, 1] = -inf                              # all banned
    logits[1, :, :] = -inf                           # one token left in each beam
    for n in range(4):
        logits[1, n, 1234 * n + 7] = 0.5
    scores[2, 1:] = -inf                             # the first step: one beam in use
    logits[3, 2, 4321] = nan
    logits[4, 0, 17] = inf
    logits[5] = -inf                                 # nothing at all
    scores[6] = torch.tensor([nan, inf, -inf, -1.0])
    got = ssm.beam_select(logits.cuda(), scores.cuda(), k)
    compare(got, logits, scores, k)
    gs, gt, gp = (t.cpu() for t in got)
    assert gp[1, :4].sort().values.tolist() == [0, 1, 2, 3] and bool(torch.isneginf(gs[1, 4:]).all())
    assert gt[1, 4:].tolist() == [0, 1, 2, 3, 4, 5, 6, 8] and bool((gp[1, 4:] == 0).all())
    assert gt[5].tolist() == list(range(k)) and bool((gp[5] == 0).all())
    assert bool((gp[2] == 0).all()) and bool((gp[6] == 3).all())
    assert 2 not in gp[3].tolist() and 0 not in gp[4].tolist()


def test_strided_logits_and_scores():
    g = torch.Generator().manual_seed(6)
    wide = torch.randn(3, 5, 2003, generator=g).to(torch.bfloat16)
    scores = torch.randn(5, 3, generator=g)
    got = ssm.beam_select(wide.cuda()[:, 1:4, 1:1900], scores.cuda().t()[:, 1:4], 9)
    compare(got, wide[:, 1:4, 1:1900], scores.t()[:, 1:4], 9)


def test_large_values():
    """Logits whose exponentials overflow, and scores far apart."""
    logits = (torch.randn(2, 3, 3000, generator=torch.Generator().manual_seed(7)) * 1e4)
    scores = torch.tensor([[0.0, -1e6, -3e4], [-5.0, -5.0, -5.0]])
    got = [t.cpu() for t in ssm.beam_select(logits.cuda(), scores.cuda(), 6)]
    want = torch.sort(ref.beam(logits, scores), dim=-1, descending=True, stable=True)
    assert torch.equal((got[2].long() * 3000 + got[1].long()), want.indices[:, :6])


# --------------------------------------------------------------------- moves

def moved(pool, src, dst):
    out = pool.clone()
    for i, s in enumerate(src):
        d = i if dst is None else dst[i]
        if s < pool.shape[0] and 0 <= d < pool.shape[0]:
            out[d] = 0 if s < 0 else pool[s]
    return out


def do(pool, src, dst):
    i32 = lambda v: None if v is None else torch.tensor(v, dtype=torch.int32).cuda()  # noqa: E731
    g = pool.cuda()
    assert ssm.state_move(g, i32(src), i32(dst)) is g
    torch.cuda.synchronize()
    return g.cpu()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("slots,row", [(1, 1), (5, 3), (16, 1024), (17, 515), (70, 96), (300, 40), (1100, 36),
                                       (2048, 9), (4, 40000)])
def test_permutations_forks_and_clears(dtype, slots, row):
    banner("move slots %d row %d %s" % (slots, row, dtype))
    g = torch.Generator().manual_seed(slots + row)
    pool = torch.randn(slots, row, generator=g).to(TYPES[dtype])
    perm = torch.randperm(slots, generator=g).tolist()
    assert torch.equal(do(pool, perm, None), moved(pool, perm, None))
    rot = [(s + 1) % slots for s in range(slots)]
    assert torch.equal(do(pool, rot, None), moved(pool, rot, None))
    parents = torch.randint(-1, slots + 1, (slots,), generator=g).tolist()   # forks, clears, a source outside
    assert torch.equal(do(pool, parents, None), moved(pool, parents, None))
    dst = torch.randperm(slots, generator=g).tolist()
    dst[0] = -1
    if slots > 2:
        dst[1] = slots
    assert torch.equal(do(pool, parents, dst), moved(pool, parents, dst))
    few = [slots - 1, 0]
    assert torch.equal(do(pool, few, [0, slots - 1]), moved(pool, few, [0, slots - 1]))


def test_move_strided_pool():
    """One layer's states in a pool of several: the others stay."""
    pool = torch.randn(6, 3, 10, 16, generator=torch.Generator().manual_seed(1)).cuda()
    before = pool.clone()
    ssm.state_move(pool[:, 1], torch.tensor([5, 4, 3, 2, 1, 0], dtype=torch.int32).cuda())
    assert torch.equal(pool[:, 1], before[:, 1].flip(0))
    assert torch.equal(pool[:, 0], before[:, 0]) and torch.equal(pool[:, 2], before[:, 2])


def test_move_far_slots():
    banner("move far slots")
    slot = 1_200_000_000
    pool = torch.empty(2 * slot + 64, device="cuda").as_strided((3, 64), (slot, 1))
    pool.copy_(torch.arange(3.0)[:, None].expand(3, 64))
    ssm.state_move(pool, torch.tensor([2, 0, 1], dtype=torch.int32).cuda())
    assert pool.cpu()[:, 0].tolist() == [2, 0, 1] and bool((pool[:, 63] == pool[:, 0]).all())


def test_move_same_destination():
    """Two moves to one slot: one of them wins in each element; the rest is as it should be."""
    pool = torch.arange(4.0)[:, None].expand(4, 200).contiguous()
    out = do(pool, [1, 2, 0], [3, 3, 0])
    assert bool(((out[3] == 1) | (out[3] == 2)).all()) and torch.equal(out[:3], pool[:3])
