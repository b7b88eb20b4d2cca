"""The recurrent layer's operators together, as they are used: a training step
of a pre-norm layer, prefill and decode, HIP graphs, streams."""
import pytest

import _layer_ref as ref
from _gpu import banner

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a GPU", allow_module_level=True)

import selective_state_space_60_amd as ssm  # noqa: E402
from selective_state_space_60_amd import block  # noqa: E402

# Every value between two operators is rounded to bf16 (2^-8 at most, 2^-9.5 in
# the mean square of a uniform remainder); a layer's output passes five such
# roundings (row's norm, projection, state output, output, and the weights'
# own) that enter independently, each at most a few times amplified.
BF16_LAYER = 2e-2


def rel(got, want):
    g, w = got.detach().double().cpu(), want.detach().double().cpu()
    assert bool(torch.isfinite(g).all())
    return float((g - w).norm() / w.norm())


def weights(M, E, seed=0, group=None, dense4=False):
    """Layer weights on the GPU and the same in fp64 on the CPU.  dense4: the
    bf16 projections hold what the 4-bit weights stand for."""
    g = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    h = {"norm": 1 + 0.1 * rnd(M), "w_in": (rnd(4 * E, M) / M ** 0.5).bfloat16(),
         "w_out": (rnd(M, E) / E ** 0.5).bfloat16(), "A": -torch.exp(-4 * torch.rand(E, generator=g)),
         "bias_a": 0.5 * rnd(E), "bias_x": 0.5 * rnd(E)}
    w = block.GatedLayerWeights(*[h[k].cuda() for k in ("norm", "w_in", "w_out", "A", "bias_a", "bias_x")],
                                group=group)
    h = {k: v.double() for k, v in h.items()}
    if dense4:
        for k, q in (("w_in", w.q_in), ("w_out", w.q_out)):
            h[k] = ref.w4_dense(q[0].cpu(), group, q[1].cpu())
        w.w_in_t, w.w_out_t = (h[k].t().contiguous().bfloat16().cuda() for k in ("w_in", "w_out"))
    return w, h


def layer64(u, residual, h, h0, lens=None):
    """The layer in fp64 (differentiable): output, residual, final state."""
    row = u + residual
    y = h["norm"] * row * torch.rsqrt((row * row).mean(-1, keepdim=True) + 1e-5)
    x, ga, gx, z = (y @ h["w_in"].t()).chunk(4, -1)
    r, i = torch.sigmoid(ga + h["bias_a"]), torch.sigmoid(gx + h["bias_x"])
    e = h["A"] * r
    a, v = torch.exp(e), torch.sqrt(-torch.expm1(2 * e)) * i * x
    n = torch.full((u.shape[0],), u.shape[1]) if lens is None else lens
    s, ys = h0, []
    for t in range(u.shape[1]):
        live = (t < n)[:, None]
        s = torch.where(live, a[:, t] * s + v[:, t], s)
        ys.append(torch.where(live, s * torch.nn.functional.silu(z[:, t]), torch.zeros_like(s)))
    return torch.stack(ys, 1) @ h["w_out"].t(), row, s


def test_training_step():
    """Forward and backward of a layer on a padded batch, every gradient
    against autograd in fp64."""
    banner("layer training step")
    b, L, M, E = 3, 150, 128, 192
    g = torch.Generator().manual_seed(1)
    w, h = weights(M, E)
    u, residual = torch.randn(b, L, M, generator=g).bfloat16(), torch.randn(b, L, M, generator=g)
    h0, lens = torch.randn(b, E, generator=g), torch.tensor([150, 33, 128])
    dout, dres = torch.randn(b, L, M, generator=g).bfloat16(), torch.randn(b, L, M, generator=g)
    dstate = torch.randn(b, E, generator=g)
    out, row, state, saved = block.gated_layer_fwd(u.cuda(), residual.cuda(), w, h0=h0.cuda(),
                                                   lens=lens.int().cuda(), train=True)
    got = block.gated_layer_bwd(dout.cuda(), dres.cuda(), w, saved, dstate=dstate.cuda())
    leaf = {k: v.clone().requires_grad_() for k, v in h.items()}
    u64, h64 = u.double().requires_grad_(), h0.double().requires_grad_()
    o, r, s = layer64(u64, residual.double(), leaf, h64, lens)
    loss = (o * dout.double()).sum() + (r * dres.double()).sum() + (s * dstate.double()).sum()
    loss.backward()
    want = {"du": u64.grad, "dh0": h64.grad, "dnorm": leaf["norm"].grad, "dA": leaf["A"].grad,
            "dbias_a": leaf["bias_a"].grad, "dbias_x": leaf["bias_x"].grad, "dw_in_t": leaf["w_in"].grad.t(),
            "dw_out_t": leaf["w_out"].grad.t()}
    errors = {"out": rel(out, o), "row": rel(row, r), "state": rel(state, s)}
    errors.update({k: rel(got[k], v) for k, v in want.items()})
    print(errors, flush=True)
    assert all(v <= BF16_LAYER for v in errors.values()), errors


@pytest.mark.parametrize("batch", [1, 5, 33])
def test_prefill_then_decode(batch):
    """Prefill of a prompt with the 4-bit weights' values, then steps with the
    4-bit weights themselves, against one fp64 pass over all tokens."""
    banner("layer decode batch %d" % batch)
    L, new, M, E = 40, 6, 256, 128
    g = torch.Generator().manual_seed(batch)
    w, h = weights(M, E, seed=2, group=64, dense4=True)
    u, residual = torch.randn(batch, L + new, M, generator=g).bfloat16(), torch.randn(batch, L + new, M, generator=g)
    o64, r64, s64 = layer64(u.double(), residual.double(), h, torch.zeros(batch, E, dtype=torch.float64))
    uc, rc = u.cuda(), residual.cuda()
    out, row, state = block.gated_layer_fwd(uc[:, :L], rc[:, :L], w)
    outs, rows = [out], [row]
    for t in range(L, L + new):
        o, r = block.gated_layer_step(uc[:, t], rc[:, t], w, state)
        outs.append(o[:, None])
        rows.append(r[:, None])
    errors = {"out": rel(torch.cat(outs, 1)[:, L:], o64[:, L:]), "prefill": rel(outs[0], o64[:, :L]),
              "row": rel(torch.cat(rows, 1), r64), "state": rel(state, s64)}
    print(errors, flush=True)
    assert all(v <= BF16_LAYER for v in errors.values()), errors


def test_mamba_layer():
    """The Mamba block behind the norm: the same bits as norm, then block."""
    import synth
    spec = synth.block_spec(synth.BLOCK2_8B, batch=1, seqlen=64, d_model=64, d_inner=128, dstate=16, dt_rank=4)
    w = block.BlockWeights(synth.block_inputs(spec, 0), 16, 4)
    g = torch.Generator().manual_seed(3)
    u = torch.randn(1, 64, 64, generator=g).bfloat16().cuda()
    residual, norm = torch.randn(1, 64, 64, generator=g).cuda(), torch.rand(64, generator=g).cuda()
    out, row = block.mamba_layer_fwd(u, residual, w, norm)
    y, row2, _ = ssm.rms_norm(u, norm, residual=residual)
    assert torch.equal(row, row2) and torch.equal(out, block.mamba_block_fwd(y, w))


def scan_inputs(b, L, D, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    return {"x": r(b, L, D), "gate_a": r(b, L, D), "gate_x": r(b, L, D), "A": -torch.rand(D, generator=g, device="cuda"),
            "bias_a": r(D), "bias_x": r(D), "z": r(b, L, D), "h0": r(b, D)}


def train_scan(t, dy, stream=None):
    ckpt = ssm.gated_scan_ckpt(*t["x"].shape)
    y, h = ssm.gated_scan_fwd(**t, want_hlast=True, ckpt=ckpt, stream=stream)
    return [y, h] + list(ssm.gated_scan_bwd(dy, **t, ckpt=ckpt, stream=stream).values())


def test_scan_in_a_graph():
    """Forward and backward of many segments (fill, wait, sums) captured once
    and replayed on new inputs, with eager work between the replays."""
    banner("graph scan")
    t, dy = scan_inputs(2, 1500, 70, 1), torch.randn(2, 1500, 70, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        train_scan(t, dy)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = train_scan(t, dy)
    for k in range(4):
        new = scan_inputs(2, 1500, 70, 10 + k)
        for name in t:
            t[name].copy_(new[name])
        dy.copy_(torch.randn(2, 1500, 70, device="cuda"))
        want = [v.clone() for v in train_scan(t, dy)]
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want)), k
        torch.randn(1000, 1000, device="cuda").sum().item()  # eager work, another allocation


def test_decode_in_a_graph():
    """A captured decode step replayed: state and residual move on as they do
    eagerly."""
    banner("graph decode")
    w, _ = weights(128, 128, seed=4, group=128)
    u, residual = torch.randn(3, 128, device="cuda").bfloat16(), torch.randn(3, 128, device="cuda")
    state = torch.zeros(3, 128, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        block.gated_layer_step(u, residual, w, state)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, row = block.gated_layer_step(u, residual, w, state)
    state.zero_()
    eager = torch.zeros(3, 128, device="cuda")
    for k in range(5):
        u.copy_(torch.randn(3, 128, device="cuda"))
        o, r = block.gated_layer_step(u, residual, w, eager)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, o) and torch.equal(row, r) and torch.equal(state, eager), k


def test_streams():
    """The current stream of a context, a given stream, and two scans at once
    on two streams, each with a workspace of its own: the same bits."""
    banner("streams")
    t, dy = scan_inputs(1, 6000, 64, 5), torch.randn(1, 6000, 64, device="cuda")
    t2, dy2 = scan_inputs(1, 5000, 64, 6), torch.randn(1, 5000, 64, device="cuda")
    want, want2 = train_scan(t, dy), train_scan(t2, dy2)
    torch.cuda.synchronize()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(3):
        with torch.cuda.stream(a):
            got = train_scan(t, dy)
        got2 = train_scan(t2, dy2, stream=b)
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got, want))
        assert all(torch.equal(p, q) for p, q in zip(got2, want2))
    x, w = torch.randn(50, 96, device="cuda"), torch.rand(96, device="cuda")
    y = ssm.rms_norm(x, w)[0]
    torch.cuda.synchronize()
    y2 = ssm.rms_norm(x, w, stream=a)[0]
    a.synchronize()
    assert torch.equal(y, y2)


def test_permuted_rows_on_a_stream():
    """Rows laid out (L, batch, dim): the outputs' layout, and with it what a
    repeated call is looked up by, is the same on a given stream and without."""
    banner("permuted rows, streams")
    side = torch.cuda.Stream()
    flip = lambda v: v.transpose(0, 1).contiguous().transpose(0, 1)  # noqa: E731
    t, dy = scan_inputs(3, 200, 48, 7), torch.randn(3, 200, 48, device="cuda")
    x, w = torch.randn(3, 50, 96, device="cuda"), torch.rand(96, device="cuda")
    want, y = train_scan(t, dy), ssm.rms_norm(x, w)[0]
    bwd = ssm.rms_norm_bwd(x, x, w)
    t = {k: flip(v) if v.dim() == 3 else v for k, v in t.items()}
    dy, x = flip(dy), flip(x)
    torch.cuda.synchronize()
    for stream in (None, side, None):
        got = train_scan(t, dy, stream=stream)
        y2, again = ssm.rms_norm(x, w, stream=stream)[0], ssm.rms_norm_bwd(x, x, w, stream=stream)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), stream
        assert torch.equal(y2, y) and torch.equal(again["dx"], bwd["dx"])
    t = {k: v[:, 0] if v.dim() == 3 else v for k, v in t.items() if k != "h0"}
    state = torch.zeros(3, 48, device="cuda")
    one = [ssm.gated_state_update(state.clone(), **t, stream=s) for s in (None, side, None)]
    torch.cuda.synchronize()
    assert torch.equal(one[0], one[1]) and torch.equal(one[0], one[2])


def test_lazy_copy_of_a_state():
    """A state that shares its memory with another tensor until it is written
    is written alone."""
    banner("lazy copy")
    t = {k: v[:, 0] if v.dim() == 3 else v for k, v in scan_inputs(2, 1, 64, 8).items() if k != "h0"}
    first = torch.randn(2, 64, device="cuda")
    state, keep = torch._lazy_clone(first), first.clone()
    ssm.gated_state_update(state, **t)
    torch.cuda.synchronize()
    assert torch.equal(first, keep) and not torch.equal(state, keep)


def test_wrappers_check_their_arguments():
    x = torch.zeros(2, 4, 8, device="cuda")
    v = torch.zeros(8, device="cuda")
    for call in (lambda: ssm.gated_scan_fwd(x, x, x, v.cpu()), lambda: ssm.rms_norm(x, v, residual=x[:1]),
                 lambda: ssm.rms_norm(x, v, residual_out=x), lambda: ssm.rms_norm_bwd(x, x[0], v),
                 lambda: ssm.w4_matvec(x[0].bfloat16(), x[0], v)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: ssm.gated_scan_fwd(x, x, x.bfloat16(), v), lambda: ssm.rms_norm(x, v.double()),
                 lambda: ssm.gated_state_update(x[0], x[0], x[0], x[0], v, y=x[0]),
                 lambda: ssm.gated_scan_bwd(x.double(), x, x, x, v)):
        with pytest.raises(ssm.SSMError):
            call()
    big = torch.zeros(65, 32, device="cuda", dtype=torch.bfloat16)
    with pytest.raises(ssm.SSMError):  # more rows than the product takes
        ssm.w4_matvec(big, torch.zeros(4, 16, dtype=torch.uint8, device="cuda"), torch.ones(4, 1, device="cuda"))
