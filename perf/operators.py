"""The operators of a pre-norm gated recurrent layer, as cases to be timed:

* the gated linear recurrence over a sequence (forward, and forward with
  backward as a training step runs them) and its one-token form,
* the root-mean-square norm with the residual's addition, with a bf16 / fp32
  output (and its backward) or an e4m3 output with scales,
* the product of a few rows with a matrix of 4-bit weights, as a decode step
  uses for its projections.

``own`` False computes them in plain torch operations, True through the
package's entry points."""
import math

import torch

own = False

EPS = 1e-5
E4M3_MAX = 448.0
# a scale never goes below this, so that a row of zeros divides by a normal number
E4M3_MIN_SCALE = 2.0 ** -126


def listed():
    return [
        # prefill or training forward of the 2.8B-shaped layer (batch 4 x 4096 tokens, 5120 channels): the four
        # streams are slices of one projection's output
        {"name": "scan_2_8b", "kind": "scan", "batch": 4, "seqlen": 4096, "dim": 5120, "dtype": "bf16", "z": True,
         "h0": False, "lens": False},
        # one long fp32 sequence: 1536 channels cannot fill the card, so time has to be split
        {"name": "scan_long", "kind": "scan", "batch": 1, "seqlen": 131072, "dim": 1536, "dtype": "f32", "z": False,
         "h0": True, "lens": False},
        # a training step's recurrence at the 130M-shaped layer (8 x 2048 x 1536)
        {"name": "train_130m", "kind": "train", "batch": 8, "seqlen": 2048, "dim": 1536, "dtype": "bf16", "z": True,
         "h0": False, "lens": False},
        # a small padded batch of odd sizes in fp32, started from a state, with the state's gradient
        {"name": "train_ragged", "kind": "train", "batch": 3, "seqlen": 515, "dim": 641, "dtype": "f32", "z": False,
         "h0": True, "lens": True},
        # one token for each of 64 sequences at 5120 channels
        {"name": "step_64", "kind": "step", "batch": 64, "dim": 5120, "dtype": "bf16", "z": True},
        # one token of one sequence: nothing but latency
        {"name": "step_1", "kind": "step", "batch": 1, "dim": 1536, "dtype": "f32", "z": False},
        # the layer's norm at 4 x 4096 tokens of 2560, residual stream in fp32
        {"name": "norm_2_8b", "kind": "norm", "rows": 16384, "dim": 2560, "dtype": "bf16", "residual": "f32",
         "out": "io", "group": 0},
        # a ragged batch of tokens, output in e4m3 with a scale for each 128 columns, for an 8-bit projection
        {"name": "norm_e4m3", "kind": "norm", "rows": 333, "dim": 5120, "dtype": "bf16", "residual": "bf16",
         "out": "e4m3", "group": 128},
        # a training step's norm at the 130M-shaped layer (8 x 2048 tokens of 768)
        {"name": "norm_train_130m", "kind": "norm_train", "rows": 16384, "dim": 768, "dtype": "bf16",
         "residual": "f32"},
        # odd sizes, fp32
        {"name": "norm_train_odd", "kind": "norm_train", "rows": 1001, "dim": 1777, "dtype": "f32",
         "residual": "f32"},
        # the decode step's input projection for one token (2560 -> 2 x 5120)
        {"name": "w4_one", "kind": "w4", "rows": 1, "ins": 2560, "outs": 10240, "group": 128, "zero": False,
         "bias": False, "out": "bf16"},
        # the output projection for a batch of 16 tokens, with zero points
        {"name": "w4_batch", "kind": "w4", "rows": 16, "ins": 5120, "outs": 2560, "group": 64, "zero": True,
         "bias": True, "out": "bf16"},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["scan", "scan", "train", "train", "step", "norm", "norm", "norm_train", "w4", "w4"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if kind in ("scan", "train"):
        most = 4 * 4096 * 5120 // 4 if kind == "scan" else 8 * 2048 * 1536 // 2
        dim = _log_int(rng, 16, 5120)
        batch = _log_int(rng, 1, 8)
        seqlen = _log_int(rng, 1, min(32768 if kind == "scan" else 4096, most // (dim * batch)))
        return {"kind": kind, "batch": batch, "seqlen": seqlen, "dim": dim, "dtype": dtype,
                "z": rng.random() < 0.5, "h0": rng.random() < 0.5, "lens": rng.random() < 0.5}
    if kind == "step":
        return {"kind": kind, "batch": _log_int(rng, 1, 256), "dim": _log_int(rng, 16, 8192), "dtype": dtype,
                "z": rng.random() < 0.5}
    if kind in ("norm", "norm_train"):
        dim = _log_int(rng, 8, 8192)
        rows = _log_int(rng, 1, min(16384, 4 * 4096 * 2560 // dim))
        case = {"kind": kind, "rows": rows, "dim": dim, "dtype": dtype,
                "residual": rng.choice(["none", dtype, "f32"])}
        if kind == "norm":
            case["out"] = rng.choice(["io", "e4m3"])
            case["group"] = rng.choice([0, 32, 64, 128]) if case["out"] == "e4m3" else 0
        return case
    group = rng.choice([32, 64, 128])
    return {"kind": kind, "rows": _log_int(rng, 1, 64), "ins": group * _log_int(rng, 1, 8192 // group),
            "outs": _log_int(rng, 16, 16384), "group": group, "zero": rng.random() < 0.5,
            "bias": rng.random() < 0.5, "out": rng.choice(["bf16", "f32"])}


_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda")

    def uniform(lo, hi, *shape):
        return lo + (hi - lo) * torch.rand(shape, generator=gen, device="cuda")

    st = {"case": case}
    kind = case["kind"]
    if kind in ("scan", "train", "step"):
        dt = _TYPES[case["dtype"]]
        D, n = case["dim"], 4 if case["z"] else 3
        lead = (case["batch"],) if kind == "step" else (case["batch"], case["seqlen"])
        # one projection's output: x | recurrence gate | input gate | z
        proj = normal(*lead, n * D).to(dt)
        st["x"], st["gate_a"], st["gate_x"] = proj[..., :D], proj[..., D:2 * D], proj[..., 2 * D:3 * D]
        st["z"] = proj[..., 3 * D:] if case["z"] else None
        # decays exp(A) from 0.43 to 0.992 at an open gate, spread over their logarithm
        st["A"] = -torch.exp(uniform(math.log(0.008), math.log(0.84), D))
        st["bias_a"], st["bias_x"] = 0.5 * normal(D), 0.5 * normal(D)
        if kind == "step":
            st["state"] = normal(case["batch"], D)
            st["state_out"] = torch.empty_like(st["state"])
            return st
        st["h0"] = normal(case["batch"], D) if case["h0"] else None
        st["lens"] = None
        if case["lens"]:
            st["lens"] = torch.randint(0, case["seqlen"] + 1, (case["batch"],), generator=gen, device="cuda",
                                       dtype=torch.int32)
        if kind == "train":
            st["dy"] = normal(*lead, D).to(dt)
        return st
    if kind in ("norm", "norm_train"):
        dt = _TYPES[case["dtype"]]
        R, D = case["rows"], case["dim"]
        st["x"] = normal(R, D).to(dt)
        st["residual"] = None
        if case["residual"] != "none":
            st["residual"] = (3.0 * normal(R, D)).to(_TYPES[case["residual"]])
        st["weight"] = 1.0 + 0.1 * normal(D)
        if kind == "norm_train":
            st["dy"] = normal(R, D).to(dt)
            # the gradient that reaches the residual stream from above
            st["dres"] = None if st["residual"] is None else normal(R, D).to(st["residual"].dtype)
        return st
    M, K, N, g = case["rows"], case["ins"], case["outs"], case["group"]
    st["x"] = normal(M, K).to(torch.bfloat16)
    st["wq"] = torch.randint(0, 256, (N, K // 2), generator=gen, device="cuda", dtype=torch.uint8)
    st["scale"] = (uniform(0.1, 0.3, N, K // g) / math.sqrt(K)).to(torch.bfloat16)
    st["zero"] = None
    if case["zero"]:
        st["zero"] = torch.randint(4, 12, (N, K // g), generator=gen, device="cuda", dtype=torch.uint8)
    st["bias"] = 0.1 * normal(N) if case["bias"] else None
    return st


def work(case):
    kind = case["kind"]
    if kind in ("scan", "train", "step"):
        e = 2 if case["dtype"] == "bf16" else 4
        n = case["batch"] * case["dim"] * (1 if kind == "step" else case["seqlen"])
        z = 1 if case["z"] else 0
        states = 8 * case["batch"] * case["dim"]
        if kind == "train":
            # forward: x, two gates, z in, y out; backward: those and dy in, their gradients out
            return {"bytes": n * e * ((4 + z) + (4 + z) + (3 + z)) + states + 24 * case["dim"], "flops": 70 * n}
        return {"bytes": n * e * (4 + z) + states + 12 * case["dim"], "flops": 25 * n}
    if kind in ("norm", "norm_train"):
        e = 2 if case["dtype"] == "bf16" else 4
        re = {"none": 0, "bf16": 2, "f32": 4}[case["residual"]]
        n = case["rows"] * case["dim"]
        if kind == "norm":
            oe = 1 if case["out"] == "e4m3" else e
            groups = -(-case["dim"] // case["group"]) if case["group"] else 1
            return {"bytes": n * (e + 2 * re + oe) + 4 * case["dim"] +
                    (4 * case["rows"] * groups if case["out"] == "e4m3" else 0), "flops": 6 * n}
        # forward, then dy, the saved row and the residual's gradient in, dx out
        return {"bytes": n * ((2 * e + 2 * re) + (e + (re or e) + re + e)) + 12 * case["dim"], "flops": 20 * n}
    M, K, N, g = case["rows"], case["ins"], case["outs"], case["group"]
    return {"bytes": N * K // 2 + N * (K // g) * (3 if case["zero"] else 2) + 2 * M * K + (4 * N if case["bias"] else 0) +
            M * N * (2 if case["out"] == "bf16" else 4), "flops": 2 * M * N * K}


# --------------------------------------------------------------- plain forms

def _gates(st):
    """Decay, input scale and gates of every step, in 32 bits: (r, i, a, s), a = exp(A r), s = sqrt(1 - a^2)."""
    r = torch.sigmoid(st["gate_a"].float() + st["bias_a"])
    i = torch.sigmoid(st["gate_x"].float() + st["bias_x"])
    u = st["A"] * r
    return r, i, torch.exp(u), torch.sqrt(-torch.expm1(2.0 * u))


def _scan(a, v):
    """h_t = a_t h_{t-1} + v_t along dimension 1, by doubling spans."""
    h, p, step = v, a, 1
    while step < a.shape[1]:
        h = torch.cat([h[:, :step], h[:, step:] + p[:, step:] * h[:, :-step]], 1)
        p = torch.cat([p[:, :step], p[:, step:] * p[:, :-step]], 1)
        step *= 2
    return h


def _plain_recurrence(st, train):
    x = st["x"].float()
    batch, L, D = x.shape
    r, i, a, s = _gates(st)
    v = s * i * x
    live = None
    if st["lens"] is not None:
        live = (torch.arange(L, device="cuda") < st["lens"].clamp(0, L)[:, None])[:, :, None]
        a, v = torch.where(live, a, 1.0), torch.where(live, v, 0.0)
    h0 = st["h0"] if st["h0"] is not None else torch.zeros(batch, D, device="cuda")
    first = torch.cat([(a[:, :1] * h0[:, None]) + v[:, :1], v[:, 1:]], 1)
    h = _scan(a, first)
    if st["z"] is not None:
        z = st["z"].float()
        sz = torch.sigmoid(z)
        y = h * (z * sz)
    else:
        y = h
    if live is not None:
        y = torch.where(live, y, 0.0)
    out = {"y": y.to(st["x"].dtype), "h_last": h[:, -1].clone()}
    if not train:
        return out
    dy = st["dy"].float()
    if live is not None:
        dy = torch.where(live, dy, 0.0)
    g = dy
    if st["z"] is not None:
        g = dy * (z * sz)
        dz = dy * h * (sz * (1.0 + z * (1.0 - sz)))
        out["dz"] = dz.to(st["x"].dtype)
    # lam_t = g_t + a_{t+1} lam_{t+1}: the same scan, backwards in time
    later = torch.cat([torch.ones_like(a[:, :1]), a.flip(1)[:, :-1]], 1)
    lam = _scan(later, g.flip(1)).flip(1)
    before = torch.cat([h0[:, None], h[:, :-1]], 1)
    e = torch.exp(st["A"] * r)
    du = lam * (e * before - i * x * (e * e / s))
    dr = du * st["A"] * r * (1.0 - r)
    di = lam * s * x * i * (1.0 - i)
    dx = lam * s * i
    dA = du * r
    if live is not None:
        dr, di, dx, dA = (torch.where(live, t, 0.0) for t in (dr, di, dx, dA))
    dt = st["x"].dtype
    out.update(dx=dx.to(dt), dgate_a=dr.to(dt), dgate_x=di.to(dt), dA=dA.sum((0, 1)), dbias_a=dr.sum((0, 1)),
               dbias_x=di.sum((0, 1)))
    if st["h0"] is not None:
        out["dh0"] = a[:, 0] * lam[:, 0]
    return out


def _plain_step(st):
    r, i, a, s = _gates(st)
    h = a * st["state"] + s * i * st["x"].float()
    y = h
    if st["z"] is not None:
        z = st["z"].float()
        y = h * (z * torch.sigmoid(z))
    return {"y": y.to(st["x"].dtype), "state": h}


def _plain_norm(st):
    case = st["case"]
    row = st["x"]
    out = {}
    if st["residual"] is not None:
        row = (st["x"].float() + st["residual"].float()).to(st["residual"].dtype)
        out["residual"] = row
    f = row.float()
    y = f * torch.rsqrt(f.square().mean(-1, keepdim=True) + EPS) * st["weight"]
    if case.get("out") != "e4m3":
        out["y"] = y.to(st["x"].dtype)
        return out
    R, D = y.shape
    group = case["group"] or D
    groups = -(-D // group)
    wide = torch.zeros(R, groups * group, device="cuda")
    wide[:, :D] = y
    wide = wide.view(R, groups, group)
    scale = (wide.abs().amax(-1) / E4M3_MAX).clamp_min(E4M3_MIN_SCALE)
    out["y"] = (wide / scale[..., None]).view(R, groups * group)[:, :D].to(torch.float8_e4m3fn)
    out["scale"] = scale
    return out


def _plain_norm_train(st):
    out = _plain_norm(st)
    row = out.get("residual", st["x"]).float()
    rstd = torch.rsqrt(row.square().mean(-1, keepdim=True) + EPS)
    hat = row * rstd
    dy = st["dy"].float()
    g = dy * st["weight"]
    dx = rstd * (g - hat * (g * hat).mean(-1, keepdim=True))
    if st["dres"] is not None:
        dx = dx + st["dres"].float()
    out["dx"] = dx.to(st["x"].dtype)
    out["dweight"] = (dy * hat).sum(0)
    return out


def _plain_w4(st):
    case = st["case"]
    N, G = st["scale"].shape
    q = torch.stack([st["wq"] & 15, st["wq"] >> 4], -1).float().view(N, G, case["group"])
    zero = st["zero"].float()[..., None] if st["zero"] is not None else 8.0
    w = ((q - zero) * st["scale"].float()[..., None]).view(N, -1)
    y = st["x"].float() @ w.t()
    if st["bias"] is not None:
        y = y + st["bias"]
    return {"y": y.to(_TYPES[case["out"]])}


# ------------------------------------------------------------ the framework's

def _own(st):
    import selective_state_space_60_amd as ssm

    case = st["case"]
    kind = case["kind"]
    if kind == "step":
        y = ssm.gated_state_update(st["state"], st["x"], st["gate_a"], st["gate_x"], st["A"], st["bias_a"],
                                   st["bias_x"], z=st["z"], state_out=st["state_out"])
        return {"y": y, "state": st["state_out"]}
    if kind in ("scan", "train"):
        ckpt = ssm.gated_scan_ckpt(case["batch"], case["seqlen"], case["dim"], st["x"].device) \
            if kind == "train" else None
        y, h_last = ssm.gated_scan_fwd(st["x"], st["gate_a"], st["gate_x"], st["A"], st["bias_a"], st["bias_x"],
                                       z=st["z"], h0=st["h0"], lens=st["lens"], want_hlast=True, ckpt=ckpt)
        out = {"y": y, "h_last": h_last}
        if kind == "train":
            out.update(ssm.gated_scan_bwd(st["dy"], st["x"], st["gate_a"], st["gate_x"], st["A"], st["bias_a"],
                                          st["bias_x"], z=st["z"], h0=st["h0"], lens=st["lens"], ckpt=ckpt))
        return out
    if kind in ("norm", "norm_train"):
        e4m3 = case.get("out") == "e4m3"
        y, residual, scale = ssm.rms_norm(st["x"], st["weight"], eps=EPS, residual=st["residual"],
                                          y_dtype=torch.float8_e4m3fn if e4m3 else None,
                                          group=case.get("group", 0))
        out = {"y": y}
        if residual is not None:
            out["residual"] = residual
        if e4m3:
            out["scale"] = scale
        if kind == "norm_train":
            row = st["x"] if residual is None else residual
            out.update(ssm.rms_norm_bwd(st["dy"], row, st["weight"], eps=EPS, dres=st["dres"],
                                        grad_dtype=st["x"].dtype))
        return out
    return {"y": ssm.w4_matvec(st["x"], st["wq"], st["scale"], zero=st["zero"], bias=st["bias"],
                               y_dtype=_TYPES[case["out"]])}


def run(st):
    if own:
        return _own(st)
    kind = st["case"]["kind"]
    if kind == "step":
        return _plain_step(st)
    if kind in ("scan", "train"):
        return _plain_recurrence(st, kind == "train")
    if kind == "norm":
        return _plain_norm(st)
    if kind == "norm_train":
        return _plain_norm_train(st)
    return _plain_w4(st)


# --------------------------------------------------------------- in 64 bits

def _exact_recurrence(st, train):
    leaf = {k: st[k].double().requires_grad_(train) for k in ("x", "gate_a", "gate_x", "A", "bias_a", "bias_x")}
    for k in ("z", "h0"):
        leaf[k] = None if st[k] is None else st[k].double().requires_grad_(train)
    batch, L, D = leaf["x"].shape
    decay = torch.exp(leaf["A"] / (1.0 + torch.exp(-leaf["gate_a"] - leaf["bias_a"])))
    fed = torch.sqrt((1.0 - decay) * (1.0 + decay)) * leaf["x"] / (1.0 + torch.exp(-leaf["gate_x"] - leaf["bias_x"]))
    h = leaf["h0"] if leaf["h0"] is not None else torch.zeros(batch, D, dtype=torch.float64, device="cuda")
    alive = torch.ones(batch, L, 1, dtype=torch.bool, device="cuda")
    if st["lens"] is not None:
        alive = (torch.arange(L, device="cuda")[None, :] < st["lens"][:, None].clamp(0, L))[..., None]
    decays, feds, alives, hs = decay.unbind(1), fed.unbind(1), alive.unbind(1), []
    for t in range(L):
        h = torch.where(alives[t], torch.addcmul(feds[t], decays[t], h), h)
        hs.append(h)
    y = torch.stack(hs, 1)
    if leaf["z"] is not None:
        y = y * leaf["z"] / (1.0 + torch.exp(-leaf["z"]))
    y = torch.where(alive, y, torch.zeros((), dtype=torch.float64, device="cuda"))
    out = {"y": y.detach(), "h_last": h.detach()}
    if train:
        names = [k for k in leaf if leaf[k] is not None]
        grads = torch.autograd.grad((y * st["dy"].double()).sum(), [leaf[k] for k in names], allow_unused=True)
        for k, g in zip(names, grads):
            out["d" + k] = torch.zeros_like(leaf[k]) if g is None else g
    return out


def exact(case, seed):
    st = prepare(case, seed)
    kind = case["kind"]
    if kind in ("scan", "train"):
        return _exact_recurrence(st, kind == "train")
    if kind == "step":
        decay = torch.exp(st["A"].double() / (1.0 + torch.exp(-st["gate_a"].double() - st["bias_a"].double())))
        i = 1.0 / (1.0 + torch.exp(-st["gate_x"].double() - st["bias_x"].double()))
        h = decay * st["state"].double() + torch.sqrt((1.0 - decay) * (1.0 + decay)) * i * st["x"].double()
        y = h if st["z"] is None else h * st["z"].double() / (1.0 + torch.exp(-st["z"].double()))
        return {"y": y, "state": h}
    if kind in ("norm", "norm_train"):
        out = {}
        x = st["x"].double()
        if st["residual"] is not None:
            out["residual"] = x + st["residual"].double()
            # what is normalised is the residual as stored (32 bits hold the sum of two 16-bit values or of a
            # 16- and a 32-bit one rounded once)
            x = out["residual"].to(st["residual"].dtype).double()
        x = x.detach().requires_grad_(kind == "norm_train")
        w = st["weight"].double().requires_grad_(kind == "norm_train")
        y = w * x / torch.sqrt((x * x).sum(-1, keepdim=True) / x.shape[-1] + EPS)
        out["y"] = y.detach()
        if case.get("out") == "e4m3":
            group = case["group"] or y.shape[1]
            parts = y.split(group, 1)
            scales = [p.abs().max(1).values.clamp_min(E4M3_MAX * E4M3_MIN_SCALE) / E4M3_MAX for p in parts]
            out["y"] = torch.cat([p / s[:, None] for p, s in zip(parts, scales)], 1)
            out["scale"] = torch.stack(scales, 1)
        if kind == "norm_train":
            dx, out["dweight"] = torch.autograd.grad((y * st["dy"].double()).sum(), [x, w])
            out["dx"] = dx if st["dres"] is None else dx + st["dres"].double()
        return out
    N, K = case["outs"], case["ins"]
    q = torch.empty(N, K, dtype=torch.float64, device="cuda")
    q[:, 0::2] = (st["wq"] % 16).double()
    q[:, 1::2] = torch.div(st["wq"], 16, rounding_mode="floor").double()
    spread = lambda t: t.double().repeat_interleave(case["group"], 1)  # noqa: E731
    w = (q - (8.0 if st["zero"] is None else spread(st["zero"]))) * spread(st["scale"])
    y = torch.mm(st["x"].double(), w.t().contiguous())
    return {"y": y if st["bias"] is None else y + st["bias"].double()}
