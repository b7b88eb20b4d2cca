"""One Mamba block forward on MI355X: the projections are hipBLASLt GEMMs
(through torch.mm on contiguous bf16 operands); the causal conv + SiLU and the
selective scan (with the softplus step size, D skip and SiLU(z) gate fused)
are this library's kernels (``causal_conv1d``, ``selective_scan_fwd``).

Order of the block ("Mamba 논문 리뷰", tildalice.io, Mamba 블록 아키텍처 and the
SelectiveSSM listing): in_proj to x and z; Conv1D + SiLU on x; x_proj to
B | C | dt; dt_proj (with bias, softplus applied in the scan); the selective
scan; y * SiLU(z); out_proj.

``mamba_block_bwd`` is its backward.  ``mamba_block_packed`` runs the block over
packed sequences that live in a pool of windows and states: prompts of different
lengths, parts of prompts, or (without starts) one token each of many sequences;
``beam_advance`` is a beam search's step over such a pool.

``mamba_layer_fwd`` puts the block behind an RMS norm on a residual stream.
``gated_layer_fwd`` / ``gated_layer_bwd`` are the same kind of layer around the
gated linear recurrence, and ``gated_layer_step`` is its decode step, whose
projections take 4-bit weights.
"""
from __future__ import annotations

import torch

from . import (beam_select, causal_conv1d, causal_conv1d_bwd, causal_conv1d_packed, gated_scan_bwd, gated_scan_ckpt,
               gated_scan_fwd, gated_state_update, rms_norm, rms_norm_bwd, scan_ckpt, selective_scan_bwd,
               selective_scan_fwd, selective_scan_packed, state_move, w4_matvec, w4_quantize)
from .serve import MOVE_MAX_MOVES


class BlockWeights:
    """Device weights of one block.  Projection weights are stored transposed
    ((in, out), contiguous) so each projection is one plain GEMM."""

    def __init__(self, host: dict, dstate: int, dt_rank: int, device="cuda"):
        bf = lambda a: torch.from_numpy(a.view("int16")).view(torch.bfloat16) if a.dtype.name == "uint16" \
            else torch.from_numpy(a)
        t = lambda k: bf(host[k]).to(device).t().contiguous()
        f = lambda k: torch.from_numpy(host[k]).to(device).contiguous()
        self.W_in_t, self.W_x_t, self.W_dt_t, self.W_out_t = t("W_in"), t("W_x"), t("W_dt"), t("W_out")
        self.conv_w, self.conv_b, self.b_dt, self.A, self.D = f("conv_w"), f("conv_b"), f("b_dt"), f("A"), f("D")
        self.N, self.R = dstate, dt_rank
        self.E = self.W_in_t.shape[1] // 2
        self.M = self.W_in_t.shape[0]


def mamba_block_fwd(u: torch.Tensor, w: BlockWeights, mark=None, train=False):
    """u: (batch, L, d_model) bf16 -> (batch, L, d_model) bf16.  `mark`, if
    given, is called after each stage (for timing).  With train: (output, what
    mamba_block_bwd takes)."""
    batch, L, M = u.shape
    E, N, R = w.E, w.N, w.R
    T = batch * L
    xz = torch.mm(u.reshape(T, M), w.W_in_t).view(batch, L, 2 * E)       # in_proj
    if mark: mark("in_proj")
    x, z = xz[..., :E], xz[..., E:]
    xc = causal_conv1d(x, w.conv_w, w.conv_b, silu=True)                 # conv + SiLU
    if mark: mark("conv")
    xd = torch.mm(xc.view(T, E), w.W_x_t)                               # x_proj: B | C | dt | padding
    delta = torch.mm(xd[:, 2 * N:2 * N + R], w.W_dt_t).view(batch, L, E)  # dt_proj (bias in the scan)
    if mark: mark("x_proj+dt_proj")
    xd = xd.view(batch, L, -1)
    ckpt = scan_ckpt(batch, L, E, N, u.device) if train else None
    y, _ = selective_scan_fwd(xc, delta, w.A, xd[..., :N], xd[..., N:2 * N], D=w.D, z=z,
                              delta_softplus=True, delta_bias=w.b_dt, ckpt=ckpt)
    if mark: mark("scan")
    out = torch.mm(y.view(T, E), w.W_out_t).view(batch, L, M)           # out_proj
    if mark: mark("out_proj")
    if train:
        return out, {"u": u, "xz": xz, "xc": xc, "xd": xd, "delta": delta, "y": y, "ckpt": ckpt}
    return out


def mamba_block_bwd(dout: torch.Tensor, w: BlockWeights, saved: dict) -> dict:
    """Gradients of mamba_block_fwd(..., train=True): dout (batch, L, d_model)
    bf16 reaches its output.  Returns du (bf16) and the weights' gradients, the
    projections' dW_in_t, dW_x_t, dW_dt_t, dW_out_t in bf16 as the GEMMs hold the
    weights, dconv_w, dconv_b, db_dt, dA, dD in fp32."""
    u, xz, xc, xd, delta = (saved[k] for k in ("u", "xz", "xc", "xd", "delta"))
    batch, L, M = u.shape
    E, N, R, T = w.E, w.N, w.R, batch * L
    across = lambda t: t.t().contiguous()  # noqa: E731
    x, z = xz[..., :E], xz[..., E:]
    dout2 = dout.reshape(T, M)
    dy = torch.mm(dout2, across(w.W_out_t)).view(batch, L, E)
    g = selective_scan_bwd(dy, xc, delta, w.A, xd[..., :N], xd[..., N:2 * N], D=w.D, z=z, delta_softplus=True,
                           delta_bias=w.b_dt, ckpt=saved["ckpt"])
    ddelta = g["ddelta"].view(T, E)
    dxd = torch.zeros_like(xd).view(T, -1)                              # B | C | dt | padding
    dxd[:, :N], dxd[:, N:2 * N] = g["dB"].view(T, N), g["dC"].view(T, N)
    dxd[:, 2 * N:2 * N + R] = torch.mm(ddelta, across(w.W_dt_t))
    dxc = g["dx"].view(T, E) + torch.mm(dxd, across(w.W_x_t))
    dxz = torch.empty_like(xz)
    c = causal_conv1d_bwd(dxc.view(batch, L, E), x, w.conv_w, w.conv_b, silu=True, dx=dxz[..., :E])
    dxz[..., E:] = g["dz"]
    dxz2 = dxz.view(T, 2 * E)
    return {"du": torch.mm(dxz2, across(w.W_in_t)).view(batch, L, M),
            "dW_in_t": torch.mm(across(u.reshape(T, M)), dxz2), "dW_x_t": torch.mm(across(xc.view(T, E)), dxd),
            "dW_dt_t": torch.mm(across(xd.view(T, -1)[:, 2 * N:2 * N + R]), ddelta),
            "dW_out_t": torch.mm(across(saved["y"].view(T, E)), dout2), "dconv_w": c["dweight"], "dconv_b": c["dbias"],
            "db_dt": g["ddelta_bias"], "dA": g["dA"], "dD": g["dD"]}


def mamba_block_packed(u, w: BlockWeights, windows, states, starts=None, src=None, dst=None):
    """The block over packed sequences: u (tokens, d_model) bf16, sequence s rows
    starts[s] to starts[s + 1] (without starts each row is one token of a
    sequence).  windows (slots, width - 1, E) bf16 and states (slots, E, N) fp32
    are the pool that the sequences start from and end in (see
    causal_conv1d_packed), updated in place.  Returns (tokens, d_model) bf16; rows
    of no sequence hold anything."""
    E, N, R = w.E, w.N, w.R
    xz = torch.mm(u, w.W_in_t)
    seqs = dict(starts=starts, src=src, dst=dst)
    xc = causal_conv1d_packed(xz[:, :E], w.conv_w, windows, bias=w.conv_b, silu=True, **seqs)
    xd = torch.mm(xc, w.W_x_t)
    delta = torch.mm(xd[:, 2 * N:2 * N + R], w.W_dt_t)
    y = selective_scan_packed(xc, delta, w.A, xd[:, :N], xd[:, N:2 * N], states, D=w.D, z=xz[:, E:],
                              delta_softplus=True, delta_bias=w.b_dt, **seqs)
    return torch.mm(y, w.W_out_t)


def beam_advance(logits, scores, slots, pools):
    """A beam search's step: from logits (batch, beams, vocab) and scores (batch,
    beams) fp32 the `beams` best continuations of every batch element, and the
    pools' slots moved so that beam n's slot slots[b, n] (int32, each slot once) holds
    the state of the beam it continues.  pools: the windows and states of every
    layer.  The logits may have fewer beams (one, at the first step), not more.
    Returns (scores, tokens, parents), each (batch, beams)."""
    if slots.dim() != 2 or logits.dim() != 3 or logits.shape[0] != slots.shape[0] or logits.shape[1] > slots.shape[1]:
        raise ValueError("beam_advance: slots are (batch, beams), a slot for every beam of the logits (%s for %s)" %
                         (tuple(slots.shape), tuple(logits.shape)))
    scores, tokens, parents = beam_select(logits, scores, slots.shape[1])
    src, dst = slots.gather(1, parents.long()).view(-1), slots.reshape(-1)
    step = MOVE_MAX_MOVES // slots.shape[1] * slots.shape[1]  # whole batch elements: theirs are the only slots they read
    for pool in pools:
        for i in range(0, src.shape[0], step):
            state_move(pool, src[i:i + step], dst[i:i + step])
    return scores, tokens, parents


def mamba_layer_fwd(u: torch.Tensor, residual: torch.Tensor, w: BlockWeights, norm_weight: torch.Tensor,
                    eps: float = 1e-5):
    """Pre-norm layer: adds u (batch, L, d_model) bf16 to the residual stream
    (bf16 or fp32) and runs the block on its RMS norm.  Returns (block output,
    new residual)."""
    y, residual, _ = rms_norm(u, norm_weight, eps=eps, residual=residual)
    return mamba_block_fwd(y, w), residual


class GatedLayerWeights:
    """Device weights of one pre-norm gated recurrent layer: d_model M, width
    E.  norm (M,), A, bias_a, bias_x (E,) fp32; w_in (4 E, M) and w_out (M, E)
    bf16, the rows of w_in in the order x, recurrence gate, input gate, z.
    The GEMMs take the projections transposed, as BlockWeights keeps them; with
    `group` (32, 64 or 128, a divisor of M and E) they are also kept in 4 bits
    with a scale for each `group` columns, as the decode step takes them."""

    def __init__(self, norm, w_in, w_out, A, bias_a, bias_x, group=None, eps=1e-5):
        self.norm, self.A, self.bias_a, self.bias_x, self.eps = norm, A, bias_a, bias_x, eps
        self.E, self.M = w_out.shape[1], w_out.shape[0]
        self.w_in_t, self.w_out_t = w_in.t().contiguous(), w_out.t().contiguous()
        if group is not None:
            self.q_in, self.q_out = w4_quantize(w_in, group), w4_quantize(w_out, group)

    def split(self, proj):
        """x, recurrence gate, input gate, z: slices of a projection's output (or of its gradient)."""
        return proj.split(self.E, -1)


def _behind(lens, L):
    """(batch, L, 1): the steps behind each row's length."""
    return (torch.arange(L, device=lens.device) >= lens[:, None]).unsqueeze(-1)


def gated_layer_fwd(u, residual, w: GatedLayerWeights, h0=None, lens=None, train=False):
    """u: (batch, L, M) bf16; residual: (batch, L, M) bf16 or fp32; h0, lens as
    in gated_scan_fwd.  Returns (output (batch, L, M) bf16, new residual, final
    state (batch, E) fp32), and with train what gated_layer_bwd takes.

    Behind a row's length u and residual may hold anything: the output is zeros
    there, the new residual is their sum, and nothing reaches a gradient of a
    weight (products of the padding with zeros would, where it is infinite or
    NaN, so what the backward takes does not hold it)."""
    batch, L, M = u.shape
    y, residual, _ = rms_norm(u, w.norm, eps=w.eps, residual=residual)
    row = residual
    if train and lens is not None:
        behind = _behind(lens, L)
        y.masked_fill_(behind, 0)
        row = residual.masked_fill(behind, 1)  # a row of zeros has no norm with eps 0
    proj = torch.mm(y.reshape(batch * L, M), w.w_in_t).view(batch, L, 4 * w.E)
    x, ga, gx, z = w.split(proj)
    ckpt = gated_scan_ckpt(batch, L, w.E, u.device) if train else None
    h, state = gated_scan_fwd(x, ga, gx, w.A, w.bias_a, w.bias_x, z=z, h0=h0, lens=lens, want_hlast=True, ckpt=ckpt)
    out = torch.mm(h.reshape(batch * L, w.E), w.w_out_t).view(batch, L, M)
    if not train:
        return out, residual, state
    return out, residual, state, {"row": row, "y": y, "proj": proj, "h": h, "h0": h0, "lens": lens, "ckpt": ckpt}


def gated_layer_bwd(dout, dresidual, w: GatedLayerWeights, saved: dict, dstate=None) -> dict:
    """Gradients of gated_layer_fwd(..., train=True): dout (batch, L, M) bf16
    and dresidual (the residual's type) reach its outputs, dstate (batch, E)
    its final state.  Returns du (of the layer input and of the residual alike,
    the residual's type), dh0, and the weights' gradients dnorm, dA, dbias_a,
    dbias_x (fp32), dw_in_t, dw_out_t (bf16, as the GEMMs hold the weights).
    Behind a row's length dout may hold anything, and du is dresidual."""
    batch, L, M = dout.shape
    T = batch * L
    if saved["lens"] is not None:
        dout = dout.masked_fill(_behind(saved["lens"], L), 0)
    dout2 = dout.reshape(T, M)
    dh = torch.mm(dout2, w.w_out_t.t().contiguous()).view(batch, L, w.E)
    dw_out_t = torch.mm(saved["h"].reshape(T, w.E).t().contiguous(), dout2)
    x, ga, gx, z = w.split(saved["proj"])
    dproj = torch.empty_like(saved["proj"])
    parts = dict(zip(("dx", "dgate_a", "dgate_x", "dz"), w.split(dproj)))
    g = gated_scan_bwd(dh, x, ga, gx, w.A, w.bias_a, w.bias_x, z=z, h0=saved["h0"], lens=saved["lens"],
                       dh_last=dstate, ckpt=saved["ckpt"], out=parts)
    dproj2 = dproj.view(T, 4 * w.E)
    dy = torch.mm(dproj2, w.w_in_t.t().contiguous()).view(batch, L, M)
    dw_in_t = torch.mm(saved["y"].reshape(T, M).t().contiguous(), dproj2)
    n = rms_norm_bwd(dy, saved["row"], w.norm, eps=w.eps, dres=dresidual, grad_dtype=dresidual.dtype)
    return {"du": n["dx"], "dh0": g.get("dh0"), "dnorm": n["dweight"], "dA": g["dA"], "dbias_a": g["dbias_a"],
            "dbias_x": g["dbias_x"], "dw_in_t": dw_in_t, "dw_out_t": dw_out_t}


def gated_layer_step(u, residual, w: GatedLayerWeights, state):
    """One token of each of up to 64 sequences: u (batch, M) bf16, residual
    (batch, M), state (batch, E) fp32, advanced in place.  The projections are
    products with the 4-bit weights.  Returns (output (batch, M) bf16, new
    residual)."""
    y, residual, _ = rms_norm(u, w.norm, eps=w.eps, residual=residual)
    x, ga, gx, z = w.split(w4_matvec(y, *w.q_in))
    h = gated_state_update(state, x, ga, gx, w.A, w.bias_a, w.bias_x, z=z)
    return w4_matvec(h, *w.q_out), residual
