"""The operators that serve a selective state space model over a pool of
states, and the backward pass of its short convolution, as cases to be timed:

* the causal convolution over packed sequences, each started from and kept in
  a window of a pool (prompts of any length, or single tokens),
* its backward over a padded batch, as a training step runs it,
* the selective scan over packed sequences with a pool of states (prompts, or
  single tokens),
* the selection of a beam search over beams and vocabulary,
* the moves of a pool's slots: forking, copying, reordering, freeing.

``own`` False computes them in plain torch operations, True through the
package's entry points."""
import math

import torch

own = False


def listed():
    return [
        # prompts of a serving batch at the 2.8B-shaped layer's width: 16384 tokens in 24 sequences of a few to
        # thousands of tokens, half of them continued from a window that an earlier part left in the pool
        {"name": "conv_prompts", "kind": "conv", "tokens": 16384, "seqs": 24, "dim": 5120, "width": 4, "dtype": "bf16",
         "single": False},
        # one token of each of 64 sequences at that width: the decode step's convolution
        {"name": "conv_tokens", "kind": "conv", "tokens": 64, "seqs": 64, "dim": 5120, "width": 4, "dtype": "bf16",
         "single": True},
        # the convolution's backward in a training step of the 130M-shaped layer (8 x 2048 tokens, 1536 channels)
        {"name": "conv_train_130m", "kind": "conv_bwd", "batch": 8, "seqlen": 2048, "dim": 1536, "width": 4,
         "dtype": "bf16"},
        # the same in fp32 at odd sizes
        {"name": "conv_train_odd", "kind": "conv_bwd", "batch": 3, "seqlen": 515, "dim": 641, "width": 4,
         "dtype": "f32"},
        # the scan of the same serving batch of prompts: 16384 tokens in 24 sequences
        {"name": "scan_prompts", "kind": "scan", "tokens": 16384, "seqs": 24, "dim": 5120, "dstate": 16,
         "dtype": "bf16", "z": True, "single": False},
        # a small mixed batch in fp32 at the 130M-shaped width: a few longer prompts among short ones and single
        # tokens
        {"name": "scan_mixed", "kind": "scan", "tokens": 1111, "seqs": 37, "dim": 1536, "dstate": 16, "dtype": "f32",
         "z": False, "single": False},
        # one token of each of 64 sequences at 5120 channels: the decode step's state update in a pool
        {"name": "step_64", "kind": "scan", "tokens": 64, "seqs": 64, "dim": 5120, "dstate": 16, "dtype": "bf16",
         "z": True, "single": True},
        # one token of one sequence: nothing but latency
        {"name": "step_1", "kind": "scan", "tokens": 1, "seqs": 1, "dim": 1536, "dstate": 16, "dtype": "f32",
         "z": False, "single": True},
        # one step of a beam search for 64 requests with 4 beams each over an odd vocabulary, twice the beams kept
        {"name": "beam_batch", "kind": "beam", "batch": 64, "beams": 4, "vocab": 50281, "k": 8, "dtype": "bf16"},
        # one request with 5 beams, fp32 logits: latency
        {"name": "beam_one", "kind": "beam", "batch": 1, "beams": 5, "vocab": 32000, "k": 5, "dtype": "f32"},
        # the states of 64 requests with 4 beams each after a selection: in every request two beams go on as copies
        {"name": "move_beams", "kind": "move", "groups": 64, "beams": 4, "forks": 2, "row": 5120 * 16, "dtype": "f32"},
        # forks of one request's convolution windows (3 rows of 1537 channels)
        {"name": "move_windows", "kind": "move", "groups": 1, "beams": 6, "forks": 5, "row": 3 * 1537,
         "dtype": "bf16"},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["conv", "conv_bwd", "scan", "scan", "beam", "move"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if kind in ("conv", "scan"):
        single = rng.random() < 0.4
        dim = _log_int(rng, 16, 5120)
        if single:
            seqs = _log_int(rng, 1, 256)
            tokens = seqs
        else:
            tokens = _log_int(rng, 2, min(16384, 16384 * 5120 // (2 * dim)))
            seqs = _log_int(rng, 1, min(64, tokens))
        case = {"kind": kind, "tokens": tokens, "seqs": seqs, "dim": dim, "dtype": dtype, "single": single}
        if kind == "conv":
            case["width"] = rng.choice([2, 3, 4, 4, 4, 5, 8])
        else:
            case["dstate"] = rng.choice([4, 8, 13, 16, 16, 16])
            case["z"] = rng.random() < 0.5
        return case
    if kind == "conv_bwd":
        dim = _log_int(rng, 16, 5120)
        batch = _log_int(rng, 1, 8)
        seqlen = _log_int(rng, 1, max(1, min(4096, 8 * 2048 * 1536 // (dim * batch))))
        return {"kind": kind, "batch": batch, "seqlen": seqlen, "dim": dim, "width": rng.choice([2, 3, 4, 4, 5, 8]),
                "dtype": dtype}
    if kind == "beam":
        beams = _log_int(rng, 1, 16)
        vocab = _log_int(rng, 64, 131072)
        batch = _log_int(rng, 1, max(1, min(64, 64 * 4 * 50281 // (beams * vocab))))
        return {"kind": kind, "batch": batch, "beams": beams, "vocab": vocab, "k": rng.choice([beams, 2 * beams]),
                "dtype": dtype}
    beams = rng.randint(2, 12)
    row = _log_int(rng, 3, 5120 * 16)
    groups = _log_int(rng, 1, max(1, min(64, 64 * 4 * 5120 * 16 // (beams * row))))
    return {"kind": kind, "groups": groups, "beams": beams, "forks": rng.randint(1, beams - 1), "row": row,
            "dtype": dtype}


_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def _lengths(gen, tokens, seqs):
    """Lengths of `seqs` sequences, at least one token each, `tokens` in all, spread over their logarithm."""
    if seqs == tokens:
        return [1] * seqs
    share = torch.exp(7.0 * torch.rand(seqs, generator=gen, dtype=torch.float64))
    cuts = (share.cumsum(0) / share.sum() * (tokens - seqs)).round().long().tolist()
    return [b - a + 1 for a, b in zip([0] + cuts[:-1], cuts)]


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    host = torch.Generator()
    host.manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda")

    st = {"case": case}
    kind = case["kind"]
    dt = _TYPES[case["dtype"]]
    if kind in ("conv", "scan"):
        T, S, D = case["tokens"], case["seqs"], case["dim"]
        st["lengths"] = _lengths(host, T, S)
        st["starts"] = None
        if not case["single"]:
            st["starts"] = torch.tensor([0] + st["lengths"], device="cuda").cumsum(0).to(torch.int32)
        # the pool holds twice as many slots as sequences run: a sequence reads one and keeps its end in another
        slots = torch.randperm(2 * S, generator=host).to(torch.int32)
        src, dst = slots[:S].clone(), slots[S:].clone()
        if not case["single"]:
            src[torch.rand(S, generator=host) < 0.5] = -1  # starts from zeros
        st["src"], st["dst"] = src.cuda(), dst.cuda()
        if kind == "conv":
            W = case["width"]
            # x is the first half of the input projection's output, z the other
            st["x"] = normal(T, 2 * D).to(dt)[:, :D]
            st["weight"] = normal(D, W) / math.sqrt(W)
            st["bias"] = 0.1 * normal(D)
            st["windows"] = normal(2 * S, W - 1, D).to(dt)
            return st
        N = case["dstate"]
        st["x"] = torch.nn.functional.silu(normal(T, D)).to(dt)
        st["delta"] = normal(T, D).to(dt)  # before its bias and the softplus
        st["delta_bias"] = -3.0 + 0.1 * normal(D)
        st["z"] = normal(T, 2 * D).to(dt)[:, D:] if case["z"] else None
        bc = normal(T, 2 * N).to(dt)
        st["B"], st["C"] = bc[:, :N], bc[:, N:]
        st["A"] = -torch.arange(1, N + 1, device="cuda", dtype=torch.float32).repeat(D, 1)
        st["D"] = 1.0 + 0.1 * normal(D)
        st["states"] = 0.3 * normal(2 * S, D, N)
        return st
    if kind == "conv_bwd":
        b, L, D, W = case["batch"], case["seqlen"], case["dim"], case["width"]
        st["x"] = normal(b, L, 2 * D).to(dt)[..., :D]
        st["dy"] = normal(b, L, D).to(dt)
        st["weight"] = normal(D, W) / math.sqrt(W)
        st["bias"] = 0.1 * normal(D)
        return st
    if kind == "beam":
        b, n, V = case["batch"], case["beams"], case["vocab"]
        logits = 3.0 * normal(b, n, V)
        # tokens that the program bans: one in sixteen
        logits = torch.where(torch.rand((b, n, V), generator=gen, device="cuda") < 1 / 16,
                             torch.full((), -math.inf, device="cuda"), logits)
        st["logits"] = logits.to(dt)
        st["scores"] = -20.0 * torch.rand((b, n), generator=gen, device="cuda")
        return st
    G, n, f = case["groups"], case["beams"], case["forks"]
    st["pool"] = normal(G * n, case["row"]).to(dt)
    # in every group the first slots of a random order survive, the others become copies of survivors
    order = torch.rand((G, n), generator=host).argsort(1)
    src = torch.arange(n).repeat(G, 1)
    pick = torch.randint(0, n - f, (G, f), generator=host)
    src.scatter_(1, order[:, n - f:], order.gather(1, pick))
    st["src"] = (src + n * torch.arange(G)[:, None]).reshape(-1).to(torch.int32).cuda()
    return st


def work(case):
    kind = case["kind"]
    e = 2 if case["dtype"] == "bf16" else 4
    if kind == "conv":
        T, S, D, W = case["tokens"], case["seqs"], case["dim"], case["width"]
        return {"bytes": e * D * (2 * T + 2 * (W - 1) * S) + 4 * D * (W + 1), "flops": T * D * (2 * W + 5)}
    if kind == "conv_bwd":
        n = case["batch"] * case["seqlen"] * case["dim"]
        return {"bytes": 3 * e * n + 8 * case["dim"] * (case["width"] + 1), "flops": n * (6 * case["width"] + 12)}
    if kind == "scan":
        T, S, D, N = case["tokens"], case["seqs"], case["dim"], case["dstate"]
        z = 1 if case["z"] else 0
        return {"bytes": e * T * (D * (3 + z) + 2 * N) + 8 * S * D * N + 4 * D * (N + 2),
                "flops": T * D * (9 * N + 10 + 6 * z)}
    if kind == "beam":
        n = case["batch"] * case["beams"] * case["vocab"]
        return {"bytes": e * n + 4 * case["batch"] * (case["beams"] + 3 * case["k"]), "flops": 4 * n}
    moved = case["groups"] * case["forks"] * case["row"]
    return {"bytes": 2 * e * moved + 4 * case["groups"] * case["beams"], "flops": 0}


# --------------------------------------------------------------- plain forms

def _behind(lengths, W, src):
    """For every token and tap the row of [tokens | windows in order of the sequences | zeros] that it reads, and for
    every sequence the rows that its window ends as.  src < 0: zeros before the sequence."""
    S, T = len(lengths), sum(lengths)
    n = torch.tensor(lengths, device="cuda")
    begin = n.cumsum(0) - n
    seq = torch.repeat_interleave(torch.arange(S, device="cuda"), n, output_size=T)

    def rows(first, s):
        """The W - 1 or W rows from `first` (counted within sequence s) on."""
        window = T + s * (W - 1) + W - 1 + first
        window = torch.where(src[s] < 0, T + S * (W - 1), window)
        return torch.where(first >= 0, begin[s] + first, window)

    taps = torch.arange(W, device="cuda")
    at = (torch.arange(T, device="cuda") - begin[seq])[:, None] - (W - 1) + taps
    ends = n[:, None] - (W - 1) + taps[:W - 1]
    each = torch.arange(S, device="cuda")
    return rows(at, seq[:, None].expand(T, W)), rows(ends, each[:, None].expand(S, W - 1))


def _plain_conv(st):
    W, D = st["case"]["width"], st["case"]["dim"]
    x, src, dst = st["x"], st["src"].long(), st["dst"].long()
    taps, ends = _behind(st["lengths"], W, src)
    before = st["windows"][src.clamp_min(0)].reshape(-1, D)
    rows = torch.cat([x, before, torch.zeros(1, D, dtype=x.dtype, device="cuda")])
    acc = st["bias"].expand(x.shape[0], D)
    for k in range(W):
        acc = acc + st["weight"][:, k] * rows[taps[:, k]].float()
    y = (acc * torch.sigmoid(acc)).to(x.dtype)
    st["windows"][dst] = rows[ends]
    return {"y": y, "windows": st["windows"]}


def _plain_conv_bwd(st):
    W, L = st["case"]["width"], st["case"]["seqlen"]
    x, dy = st["x"].float(), st["dy"].float()
    padded = torch.nn.functional.pad(x, (0, 0, W - 1, 0))
    acc = st["bias"].expand_as(x)
    for k in range(W):
        acc = acc + st["weight"][:, k] * padded[:, k:k + L]
    s = torch.sigmoid(acc)
    g = dy * (s * (1.0 + acc * (1.0 - s)))
    later = torch.nn.functional.pad(g, (0, 0, 0, W - 1))
    dx = torch.zeros_like(x)
    dweight = []
    for k in range(W):
        dx = dx + st["weight"][:, k] * later[:, W - 1 - k:W - 1 - k + L]
        dweight.append((g * padded[:, k:k + L]).sum((0, 1)))
    return {"dx": dx.to(st["x"].dtype), "dweight": torch.stack(dweight, 1), "dbias": g.sum((0, 1))}


def _plain_scan(st):
    """Sequences side by side, the longest first; 32 steps are discretised at a time."""
    T, S, D, N = (st["case"][k] for k in ("tokens", "seqs", "dim", "dstate"))
    lengths, src, dst = st["lengths"], st["src"].long(), st["dst"].long()
    order = sorted(range(S), key=lambda s: -lengths[s])
    n = [lengths[s] for s in order]
    count = torch.tensor(lengths, device="cuda")
    begin = (count.cumsum(0) - count)[order]
    src, dst = src[order], dst[order]
    A, y = st["A"], torch.empty(T, D, device="cuda")
    h = torch.where((src < 0)[:, None, None], torch.zeros((), device="cuda"), st["states"][src.clamp_min(0)])
    for t0 in range(0, n[0], 32):
        live = sum(1 for v in n if v > t0)
        steps = min(32, n[0] - t0)
        t = t0 + torch.arange(steps, device="cuda")
        inside = t[None, :] < torch.tensor(n[:live], device="cuda")[:, None]
        row = torch.where(inside, begin[:live, None] + t, 0)
        u = st["delta"][row].float() + st["delta_bias"]
        dt = torch.clamp_min(u, 0.0) + torch.log1p(torch.exp(-u.abs()))
        dt = torch.where(inside[..., None], dt, 0.0)
        x, B, C = st["x"][row].float(), st["B"][row].float(), st["C"][row].float()
        decay = dt[..., None] * A
        fed = torch.expm1(decay) / A * B[:, :, None, :] * x[..., None]
        decay = torch.exp(decay)
        hs, now = [], h[:live]
        for k in range(steps):
            now = torch.addcmul(fed[:, k], decay[:, k], now)
            hs.append(now)
        h[:live] = now
        out = (torch.stack(hs, 1) * C[:, :, None, :]).sum(-1) + st["D"] * x
        if st["z"] is not None:
            z = st["z"][row].float()
            out = out * (z * torch.sigmoid(z))
        y[row[inside]] = out[inside]
    st["states"][dst] = h
    return {"y": y.to(st["x"].dtype), "states": st["states"]}


def _plain_beam(st):
    """Scores in 64 bits: candidates of different beams may lie next to each other."""
    b, n, V = st["logits"].shape
    logits = st["logits"].double()
    top = logits.amax(-1, keepdim=True)
    lse = top + torch.log(torch.exp(logits - top).sum(-1, keepdim=True))
    score = (st["scores"].double()[..., None] - lse + logits).view(b, n * V)
    value, at = torch.sort(score, dim=-1, descending=True, stable=True)
    k = st["case"]["k"]
    value, at = value[:, :k], at[:, :k]
    return {"scores": value.float(), "tokens": (at % V).to(torch.int32),
            "parents": torch.div(at, V, rounding_mode="floor").to(torch.int32)}


def _plain_move(st):
    src = st["src"].long()
    st["pool"].copy_(st["pool"][src])
    return {"pool": st["pool"]}


# ------------------------------------------------------------ the framework's

def _own(st):
    import selective_state_space_60_amd as ssm

    case = st["case"]
    kind = case["kind"]
    if kind == "conv":
        y = ssm.causal_conv1d_packed(st["x"], st["weight"], st["windows"], starts=st["starts"], src=st["src"],
                                     dst=st["dst"], bias=st["bias"], silu=True)
        return {"y": y, "windows": st["windows"]}
    if kind == "conv_bwd":
        return ssm.causal_conv1d_bwd(st["dy"], st["x"], st["weight"], bias=st["bias"], silu=True)
    if kind == "scan":
        y = ssm.selective_scan_packed(st["x"], st["delta"], st["A"], st["B"], st["C"], st["states"],
                                      starts=st["starts"], src=st["src"], dst=st["dst"], D=st["D"], z=st["z"],
                                      delta_softplus=True, delta_bias=st["delta_bias"])
        return {"y": y, "states": st["states"]}
    if kind == "beam":
        scores, tokens, parents = ssm.beam_select(st["logits"], st["scores"], case["k"])
        return {"scores": scores, "tokens": tokens, "parents": parents}
    return {"pool": ssm.state_move(st["pool"], st["src"])}


def run(st):
    if own:
        return _own(st)
    return {"conv": _plain_conv, "conv_bwd": _plain_conv_bwd, "scan": _plain_scan, "beam": _plain_beam,
            "move": _plain_move}[st["case"]["kind"]](st)


# --------------------------------------------------------------- in 64 bits

def _silu64(v):
    return v / (1.0 + torch.exp(-v))


def _exact_conv(st):
    """One sequence after the other, in front of each its window."""
    W, D = st["case"]["width"], st["case"]["dim"]
    src, dst = st["src"].tolist(), st["dst"].tolist()
    w, bias, windows = st["weight"].double(), st["bias"].double(), st["windows"].double()
    ys, kept, at = [], windows.clone(), 0
    for s, n in enumerate(st["lengths"]):
        before = windows[src[s]] if src[s] >= 0 else torch.zeros(W - 1, D, dtype=torch.float64, device="cuda")
        line = torch.cat([before, st["x"][at:at + n].double()])
        at += n
        ys.append(_silu64(sum(line[k:k + n] * w[:, k] for k in range(W)) + bias))
        kept[dst[s]] = line[n:]
    return {"y": torch.cat(ys), "windows": kept}


def _exact_conv_bwd(st):
    x, w, b = (st[k].double().requires_grad_(True) for k in ("x", "weight", "bias"))
    L, W = x.shape[1], w.shape[1]
    acc = b
    for k in range(W):  # tap k reads the step W - 1 - k back
        back = W - 1 - k
        if back < L:
            acc = acc + torch.cat([torch.zeros_like(x[:, :back]), x[:, :L - back]], 1) * w[:, k]
    dx, dw, db = torch.autograd.grad((_silu64(acc.expand_as(x)) * st["dy"].double()).sum(), [x, w, b])
    return {"dx": dx, "dweight": dw, "dbias": db}


def _exact_scan(st):
    D = st["case"]["dim"]
    src, dst = st["src"].tolist(), st["dst"].tolist()
    A, states = st["A"].double(), st["states"].double()
    kept, ys, at = states.clone(), [], 0
    for s, n in enumerate(st["lengths"]):
        h = states[src[s]] if src[s] >= 0 else torch.zeros_like(states[0])
        for t0 in range(at, at + n, 128):
            part = slice(t0, min(t0 + 128, at + n))
            raw = st["delta"][part].double() + st["delta_bias"].double()
            delta = torch.logaddexp(raw, torch.zeros_like(raw))
            x, B, C = st["x"][part].double(), st["B"][part].double(), st["C"][part].double()
            u = torch.einsum("td,dn->tdn", delta, A)
            gain = torch.expm1(u) / A
            decays = torch.exp(u).unbind(0)
            feds = (gain * (x[:, :, None] * B[:, None, :])).unbind(0)
            path = []
            for a, f in zip(decays, feds):
                h = torch.addcmul(f, a, h)
                path.append(h)
            y = (torch.stack(path) * C[:, None, :]).sum(2) + st["D"].double() * x
            if st["z"] is not None:
                y = y * _silu64(st["z"][part].double())
            ys.append(y)
        at += n
        kept[dst[s]] = h
    return {"y": torch.cat(ys).view(-1, D), "states": kept}


def _exact_beam(st):
    """The best by one maximum after the other, the lowest index among equals."""
    logits = st["logits"].double()
    b, n, V = logits.shape
    flat = (logits - torch.logsumexp(logits, -1, keepdim=True) + st["scores"].double()[..., None]).reshape(b, n * V)
    index = torch.arange(n * V, device="cuda").expand(b, n * V)
    scores, at = [], []
    for _ in range(st["case"]["k"]):
        best = flat.max(1, keepdim=True).values
        where = torch.where(flat == best, index, n * V).min(1, keepdim=True).values
        scores.append(best)
        at.append(where)
        flat = flat.scatter(1, where, -math.inf)
    at = torch.cat(at, 1)
    return {"scores": torch.cat(scores, 1), "tokens": (at % V).to(torch.int32), "parents": (at // V).to(torch.int32)}


def exact(case, seed):
    st = prepare(case, seed)
    kind = case["kind"]
    if kind == "move":
        return {"pool": torch.stack([st["pool"][s] for s in st["src"].tolist()]).double()}
    return {"conv": _exact_conv, "conv_bwd": _exact_conv_bwd, "scan": _exact_scan, "beam": _exact_beam}[kind](st)
