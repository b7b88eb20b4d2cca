"""One Mamba block forward on MI355X: the projections are hipBLASLt GEMMs
(through torch.mm on contiguous bf16 operands); the causal conv + SiLU and the
selective scan (with the softplus step size, D skip and SiLU(z) gate fused)
are this library's kernels (``causal_conv1d``, ``selective_scan_fwd``).

Order of the block ("Mamba 논문 리뷰", tildalice.io, Mamba 블록 아키텍처 and the
SelectiveSSM listing): in_proj to x and z; Conv1D + SiLU on x; x_proj to
B | C | dt; dt_proj (with bias, softplus applied in the scan); the selective
scan; y * SiLU(z); out_proj.

``mamba_layer_fwd`` puts the block behind an RMS norm on a residual stream.
``gated_layer_fwd`` / ``gated_layer_bwd`` are the same kind of layer around the
gated linear recurrence, and ``gated_layer_step`` is its decode step, whose
projections take 4-bit weights.
"""
from __future__ import annotations

import torch

from . import (causal_conv1d, gated_scan_bwd, gated_scan_ckpt, gated_scan_fwd, gated_state_update, rms_norm,
               rms_norm_bwd, selective_scan_fwd, w4_matvec, w4_quantize)


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


def mamba_block_fwd(u: torch.Tensor, w: BlockWeights, mark=None) -> torch.Tensor:
    """u: (batch, L, d_model) bf16 -> (batch, L, d_model) bf16.  `mark`, if
    given, is called after each stage (for timing)."""
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
    y, _ = selective_scan_fwd(xc, delta, w.A, xd[..., :N], xd[..., N:2 * N], D=w.D, z=z,
                              delta_softplus=True, delta_bias=w.b_dt)
    if mark: mark("scan")
    out = torch.mm(y.view(T, E), w.W_out_t).view(batch, L, M)           # out_proj
    if mark: mark("out_proj")
    return out


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
