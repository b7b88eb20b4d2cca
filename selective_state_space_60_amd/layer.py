"""Binding of the operators of a pre-norm gated recurrent layer: the gated
linear recurrence (``gated_scan_fwd``, ``gated_scan_bwd``,
``gated_state_update``), the RMS norm (``rms_norm``, ``rms_norm_bwd``) and the
product with 4-bit weights (``w4_matvec``).  Argument marshalling only, as in
the package; definitions stand in include/ssm.h.

``stream`` is where a call runs (default: the current stream of its tensors'
device).  What the call allocates belongs to that stream; the tensors that are
passed in are the caller's to keep until the stream is past the call.

The descriptor of a call (shapes, strides, types, flags) and the workspace
size it asks for are kept by exactly these values, so that a call that repeats
a shape costs a lookup; pointers and values are never kept.
"""
from __future__ import annotations

import ctypes
import importlib.util
import os

import torch

from . import (_GATED_BWD_T, _GATED_T, _GATED_UPD_T, _NORM_BWD_T, _NORM_T, _W4_T, SSM_HAS_BIAS, SSM_HAS_BIAS_A,
               SSM_HAS_BIAS_X, SSM_HAS_CKPT, SSM_HAS_DHLAST, SSM_HAS_H0, SSM_HAS_LENS, SSM_HAS_RESIDUAL,
               SSM_HAS_STATE_OUT, SSM_HAS_Z, SSM_HAS_ZERO, SSM_WANT_CKPT, SSM_WANT_HLAST, GatedBwdDesc, GatedDesc,
               GatedUpdateDesc, NormBwdDesc, NormDesc, W4Desc, _check, lib, tensor_desc)

GATED_CKPT_STEPS = 64  # SSM_GATED_CKPT_STEPS
NORM_MAX_DIM = 16384   # SSM_NORM_MAX_DIM
W4_MAX_ROWS = 64       # SSM_W4_MAX_ROWS

_MAX_PLANS = 1024
_plans: dict = {}

# The current stream's handle without building a Stream object (a microsecond of a decode step's call).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda index: torch.cuda.current_stream(index).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


MARSHAL_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "_marshal.so")


def _bind():
    """Put the native module's functions (csrc/marshal.cpp) in the place of the four below."""
    global _sig, _run, _new_like, _new
    if not os.path.exists(MARSHAL_PATH):
        raise ImportError("_marshal.so is not built (run __graft_entry__.build()): " + MARSHAL_PATH)
    spec = importlib.util.spec_from_file_location(__package__ + "._marshal", MARSHAL_PATH)
    native = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(native)
    _sig, _run, _new_like, _new = native.signature, native.launch, native.like, native.empty


def _sig(tensors):
    """What a descriptor depends on: type, device, sizes and strides of each tensor."""
    _bind()
    return _sig(tensors)


def _run(*args):
    """The status of an entry point called on a tuple of tensors, with a workspace of its own."""
    _bind()
    return _run(*args)


def _new_like(t, dtype):
    """Memory like t's, of a dtype or (None) its own."""
    _bind()
    return _new_like(t, dtype)


def _new(t, shape, dtype):
    """Contiguous memory on t's device."""
    _bind()
    return _new(t, shape, dtype)


class _Plan:
    """An entry point with a descriptor of fixed shapes, and the workspace size it asks for."""
    __slots__ = ("entry", "fn", "desc", "address", "index", "written", "nbytes")

    def __init__(self, entry, Desc, names, sizes, flags, tensors, written, size_entry=None):
        index = tensors[0].get_device()
        if index < 0:
            raise ValueError("%s: tensors must be on a GPU" % entry)
        for t in tensors:
            if t is not None and t.get_device() != index:
                raise ValueError("%s: all tensors must be on one GPU" % entry)
        d = Desc()
        for name, v in sizes:
            setattr(d, name, v)
        d.flags = flags
        for name, t in zip(names, tensors):
            setattr(d, name, tensor_desc(t))
        # the pointer structs of these entry points hold one pointer per tensor, in the order of `names`
        self.entry, self.index, self.desc, self.address = entry, index, d, ctypes.addressof(d)
        self.fn = ctypes.cast(getattr(lib(), entry), ctypes.c_void_p).value
        self.written = sum(1 << i for i, name in enumerate(names) if name in written)
        self.nbytes = -1  # an entry point without a workspace
        if size_entry is not None:
            n = ctypes.c_size_t()
            _check(getattr(lib(), size_entry)(self.address, ctypes.byref(n)), size_entry)
            self.nbytes = n.value


def _keep(key, plan):
    if len(_plans) >= _MAX_PLANS:
        _plans.clear()
    _plans[key] = plan
    return plan


def _launch(plan, tensors, stream):
    """Run the plan on these tensors, on `stream` (default: the current stream of their device)."""
    if stream is not None and stream.device.index != plan.index:
        raise ValueError("%s: the stream is on another device than the tensors" % plan.entry)
    if plan.index != _current_device():
        with torch.cuda.device(plan.index):
            return _launch(plan, tensors, stream)
    if stream is None:
        status = _run(plan.fn, plan.address, tensors, plan.written, plan.nbytes, _raw_stream(plan.index))
    else:
        with torch.cuda.stream(stream):  # the workspace belongs to its pool
            status = _run(plan.fn, plan.address, tensors, plan.written, plan.nbytes, stream.cuda_stream)
    if status:
        _check(status, plan.entry)


def _empty(stream, t, shape, dtype):
    """Memory on t's device for a call on `stream`: it belongs to that stream's
    pool, so that freeing it early is safe there."""
    if stream is None:
        return _new(t, shape, dtype)
    with torch.cuda.stream(stream):
        return _new(t, shape, dtype)


def _like(stream, t, dtype=None):
    """Memory of t's shape, dense (contiguous unless t is a dense permutation).
    Its strides follow from t's alone: a plan's key does not hold them."""
    if stream is None:
        return _new_like(t, dtype)
    with torch.cuda.stream(stream):
        return _new_like(t, dtype)


# -------------------------------------------------- gated linear recurrence

def gated_scan_ckpt(batch: int, seqlen: int, dim: int, device="cuda"):
    """An uninitialised checkpoint buffer for gated_scan_fwd(ckpt=...) and
    gated_scan_bwd(ckpt=...): the state before every 64th step."""
    return torch.empty((batch, (seqlen + GATED_CKPT_STEPS - 1) // GATED_CKPT_STEPS, dim), dtype=torch.float32,
                       device=device)


def _gated_flags(bias_a, bias_x, z):
    return ((SSM_HAS_BIAS_A if bias_a is not None else 0) | (SSM_HAS_BIAS_X if bias_x is not None else 0) |
            (SSM_HAS_Z if z is not None else 0))


def gated_scan_fwd(x, gate_a, gate_x, A, bias_a=None, bias_x=None, z=None, h0=None, lens=None, want_hlast=False,
                   y_dtype=None, y=None, ckpt=None, stream=None):
    """y = gated linear recurrence of x (see include/ssm.h).  Returns (y,
    h_last or None).

    x, gate_a, gate_x, z: (batch, L, dim), all fp32 or all bf16, unit innermost
    stride; A, bias_a, bias_x: (dim,) fp32; h0: (batch, dim) fp32; lens:
    (batch,) int32 on the GPU, the steps of each row that count (later y are
    zeros, h_last is the state after the last that counts).  ckpt: optional
    gated_scan_ckpt(...) buffer, filled for gated_scan_bwd(ckpt=...)."""
    key = ("gated_scan_fwd", want_hlast, y_dtype, _sig((x, gate_a, gate_x, A, bias_a, bias_x, z, h0, lens, y, ckpt)))
    plan = _plans.get(key)
    if y is None:
        y = _like(stream, x, y_dtype)
    h_last = None
    if want_hlast:
        h_last = _empty(stream, x, (x.shape[0], x.shape[2]), torch.float32)
    tensors = (x, gate_a, gate_x, A, bias_a, bias_x, z, y, h0, h_last, lens, ckpt)
    if plan is None:
        batch, L, dim = x.shape
        flags = (_gated_flags(bias_a, bias_x, z) | (SSM_HAS_H0 if h0 is not None else 0) |
                 (SSM_WANT_HLAST if want_hlast else 0) | (SSM_HAS_LENS if lens is not None else 0) |
                 (SSM_WANT_CKPT if ckpt is not None else 0))
        plan = _keep(key, _Plan("ssm_gated_scan_fwd", GatedDesc, _GATED_T,
                                (("batch", batch), ("seqlen", L), ("dim", dim)), flags, tensors,
                                ("y", "h_last", "ckpt"), "ssm_gated_scan_workspace_size"))
    _launch(plan, tensors, stream)
    return y, h_last


_GATED_OUT = ("dx", "dgate_a", "dgate_x", "dz")


def gated_scan_bwd(dy, x, gate_a, gate_x, A, bias_a=None, bias_x=None, z=None, h0=None, lens=None, dh_last=None,
                   ckpt=None, out=None, stream=None) -> dict:
    """Gradients of sum(dy * y) + sum(dh_last * h_last) for y, h_last =
    gated_scan_fwd(x, gate_a, gate_x, A, bias_a, bias_x, z, h0, lens) (see
    include/ssm.h).  ckpt: the forward's checkpoints of the same inputs;
    without them they are recomputed.  out: optional dict with memory for any
    of dx, dgate_a, dgate_x, dz (slices of one projection's gradient, say).

    Returns a dict: dx, dgate_a, dgate_x, dz (if z), all of dy's dtype (x's or
    fp32), and fp32 dA, dbias_a, dbias_x (dim,; if given) and dh0 (if h0)."""
    ins = (x, gate_a, gate_x, A, bias_a, bias_x, z, h0, lens, ckpt, dy, dh_last)
    given = (None,) * 4
    if out:
        given = tuple([out.get(k) for k in _GATED_OUT])
        if not out.keys() <= set(_GATED_OUT):
            raise ValueError("gated_scan_bwd: out takes " + ", ".join(_GATED_OUT))
        if z is None and given[3] is not None:
            raise ValueError("gated_scan_bwd: out holds dz, but there is no z")
    key = ("gated_scan_bwd", _sig(ins), _sig(given) if out else None)
    plan = _plans.get(key)
    dx, dga, dgx, dz = [_like(stream, dy) if t is None else t for t in given[:3]] + [given[3]]
    if z is not None and dz is None:
        dz = _like(stream, dy)
    out = {"dx": dx, "dgate_a": dga, "dgate_x": dgx, "dz": dz, "dA": _like(stream, A),
           "dbias_a": None if bias_a is None else _like(stream, bias_a),
           "dbias_x": None if bias_x is None else _like(stream, bias_x),
           "dh0": None if h0 is None else _like(stream, h0)}
    tensors = ins + tuple(out.values())
    if plan is None:
        batch, L, dim = x.shape
        flags = (_gated_flags(bias_a, bias_x, z) | (SSM_HAS_H0 if h0 is not None else 0) |
                 (SSM_HAS_LENS if lens is not None else 0) | (SSM_HAS_CKPT if ckpt is not None else 0) |
                 (SSM_HAS_DHLAST if dh_last is not None else 0))
        plan = _keep(key, _Plan("ssm_gated_scan_bwd", GatedBwdDesc, _GATED_BWD_T,
                                (("batch", batch), ("seqlen", L), ("dim", dim)), flags, tensors, tuple(out),
                                "ssm_gated_scan_bwd_workspace_size"))
    _launch(plan, tensors, stream)
    return {k: v for k, v in out.items() if v is not None}


def gated_state_update(state, x, gate_a, gate_x, A, bias_a=None, bias_x=None, z=None, state_out=None, y_dtype=None,
                       y=None, stream=None):
    """One decode step of the gated recurrence (see include/ssm.h): advances
    ``state`` (batch, dim) fp32 in place, or into ``state_out`` if given, and
    returns y (batch, dim).  x, gate_a, gate_x, z: (batch, dim)."""
    ins = (x, gate_a, gate_x, A, bias_a, bias_x, z)
    key = ("gated_state_update", y_dtype, _sig(ins + (y, state, state_out)))
    plan = _plans.get(key)
    if y is None:
        y = _like(stream, x, y_dtype)
    tensors = ins + (y, state, state_out)
    if plan is None:
        batch, dim = x.shape
        flags = _gated_flags(bias_a, bias_x, z) | (SSM_HAS_STATE_OUT if state_out is not None else 0)
        plan = _keep(key, _Plan("ssm_gated_state_update", GatedUpdateDesc, _GATED_UPD_T,
                                (("batch", batch), ("dim", dim)), flags, tensors,
                                ("y", "state" if state_out is None else "state_out")))
    _launch(plan, tensors, stream)
    return y


# ---------------------------------------------------------------------- norm

def _rows(t):
    """(batch, L, dim) view of a tensor of two or three dimensions."""
    return t if t is None or t.dim() == 3 else t.unsqueeze(0)


def rms_norm(x, weight, eps=1e-5, residual=None, residual_dtype=None, residual_out=None, y_dtype=None, group=0,
             y=None, stream=None):
    """RMS norm of the rows of x (+ residual) (see include/ssm.h).  Returns
    (y, residual_out or None, scale or None).

    x, residual: (batch, L, dim) or (rows, dim), unit innermost stride; weight
    (dim,) fp32.  residual_out (the sum) has residual_dtype, default
    residual's; it may be residual itself.  y_dtype: x's dtype (default),
    torch.float32, or torch.float8_e4m3fn, which comes with fp32 scales, one
    for each `group` columns (32, 64 or 128; 0: one a row): scale has x's
    leading shape and ceil(dim / group) columns."""
    key = ("rms_norm", eps, residual_dtype, y_dtype, group, _sig((x, weight, residual, residual_out, y)))
    plan = _plans.get(key)
    if plan is None:
        if x.dim() not in (2, 3) or (residual is not None and residual.shape != x.shape):
            raise ValueError("rms_norm: x and residual are (rows, dim) or (batch, L, dim), of one shape")
        if residual is None and residual_out is not None:
            raise ValueError("rms_norm: residual_out without residual")
    if y is None:
        y = _like(stream, x, y_dtype)
    if residual is not None and residual_out is None:
        residual_out = _like(stream, x, residual_dtype or residual.dtype)
    scale = None
    if y.dtype == torch.float8_e4m3fn:
        scale = _empty(stream, x, x.shape[:-1] + ((x.shape[-1] + group - 1) // group if group > 0 else 1,),
                       torch.float32)
    tensors = (x, residual, weight, y, residual_out, scale)
    if plan is None:
        x3 = _rows(x)
        plan = _keep(key, _Plan("ssm_rms_norm_fwd", NormDesc, _NORM_T,
                                (("batch", x3.shape[0]), ("seqlen", x3.shape[1]), ("dim", x3.shape[2]),
                                 ("group", group), ("eps", float(eps))),
                                SSM_HAS_RESIDUAL if residual is not None else 0,
                                (x3, _rows(residual), weight, _rows(y), _rows(residual_out), _rows(scale)),
                                ("y", "residual_out", "scale")))
    _launch(plan, tensors, stream)
    return y, residual_out, scale


def rms_norm_bwd(dy, row, weight, eps=1e-5, dres=None, grad_dtype=None, stream=None) -> dict:
    """Gradients of sum(dy * y) + sum(dres * residual_out) for y, residual_out
    = rms_norm(...) (see include/ssm.h).  row: what was normalised
    (residual_out, or x without a residual); dres: the gradient that reaches
    residual_out besides.

    Returns {"dx": grad_dtype, default dy's -- the gradient of x and of
    residual alike, "dweight": (dim,) fp32}."""
    key = ("rms_norm_bwd", eps, grad_dtype, _sig((dy, row, weight, dres)))
    plan = _plans.get(key)
    if plan is None and (row.dim() not in (2, 3) or dy.shape != row.shape or
                         (dres is not None and dres.shape != row.shape)):
        raise ValueError("rms_norm_bwd: dy, row and dres are (rows, dim) or (batch, L, dim), of one shape")
    dx = _like(stream, dy, grad_dtype)
    dweight = _like(stream, weight)
    tensors = (dy, row, weight, dres, dx, dweight)
    if plan is None:
        r3 = _rows(row)
        plan = _keep(key, _Plan("ssm_rms_norm_bwd", NormBwdDesc, _NORM_BWD_T,
                                (("batch", r3.shape[0]), ("seqlen", r3.shape[1]), ("dim", r3.shape[2]),
                                 ("eps", float(eps))), SSM_HAS_RESIDUAL if dres is not None else 0,
                                (_rows(dy), r3, weight, _rows(dres), _rows(dx), dweight), ("dx", "dweight"),
                                "ssm_rms_norm_bwd_workspace_size"))
    _launch(plan, tensors, stream)
    return {"dx": dx, "dweight": dweight}


# ------------------------------------------------------------ 4-bit weights

def w4_quantize(weight, group=128, scale_dtype=torch.bfloat16):
    """(packed, scale) of a weight matrix (outs, ins) for w4_matvec, symmetric
    about 8: scale = amax(|w|) / 7 of every group of a row (rounded to
    scale_dtype), q = round(w / scale) + 8 in 1..15; the even column of a pair
    is the low half of its byte.  Done once when weights are loaded, on the
    weight's own device."""
    outs, ins = weight.shape
    if group not in (32, 64, 128) or ins % group:
        raise ValueError("w4_quantize: group is 32, 64 or 128 and divides the columns")
    w = weight.detach().float().reshape(outs, ins // group, group)
    scale = (w.abs().amax(-1) / 7.0).to(scale_dtype)
    s = scale.float().unsqueeze(-1)
    q = torch.where(s > 0, torch.round(w / s), torch.zeros_like(w)).clamp(-7, 7).to(torch.int32) + 8
    q = q.reshape(outs, ins // 2, 2)
    return (q[..., 0] | (q[..., 1] << 4)).to(torch.uint8), scale


def w4_matvec(x, weight, scale, zero=None, bias=None, y_dtype=None, y=None, stream=None):
    """y = x W^T + bias with 4-bit weights (see include/ssm.h).  x: (rows,
    ins) bf16, rows <= 64; weight: (outs, ins / 2) uint8, two weights a byte;
    scale: (outs, ins / group) bf16 or fp32, group 32, 64 or 128; zero: (outs,
    ins / group) uint8 (default 8); bias: (outs,) fp32.  Returns y (rows,
    outs), bf16 by default."""
    key = ("w4_matvec", y_dtype, _sig((x, weight, scale, zero, bias, y)))
    plan = _plans.get(key)
    if y is None:
        y = _empty(stream, x, (x.shape[0], weight.shape[0]), y_dtype)
    tensors = (x, weight, scale, zero, bias, y)
    if plan is None:
        rows, ins = x.shape
        if scale.dim() != 2 or scale.shape[1] == 0 or ins % scale.shape[1]:
            raise ValueError("w4_matvec: scale is (outs, ins / group)")
        plan = _keep(key, _Plan("ssm_w4_matvec", W4Desc, _W4_T,
                                (("rows", rows), ("ins", ins), ("outs", weight.shape[0]),
                                 ("group", ins // scale.shape[1])),
                                (SSM_HAS_ZERO if zero is not None else 0) |
                                (SSM_HAS_BIAS if bias is not None else 0), tensors, ("y",)))
    _launch(plan, tensors, stream)
    return y
