"""Binding of the operators that serve a selective state space model over a
pool of states -- the convolution and the scan of packed sequences
(``causal_conv1d_packed``, ``selective_scan_packed``), beam search's selection
(``beam_select``) and the moves of a pool's slots (``state_move``) -- and of the
convolution's backward (``causal_conv1d_bwd``).  Argument marshalling only, as in
the package; definitions stand in include/ssm.h.

``stream`` and the kept descriptors are as in ``layer``."""
from __future__ import annotations

import torch

from . import (_BEAM_T, _CONV_BWD_T, _CONV_PACKED_T, _MOVE_T, _SCAN_PACKED_T, SSM_DISC_EULER, SSM_HAS_BIAS, SSM_HAS_D,
               SSM_HAS_DST, SSM_HAS_SRC, SSM_HAS_STARTS, SSM_HAS_STATES, SSM_HAS_Z, SSM_SILU, BeamDesc, ConvBwdDesc,
               ConvPackedDesc, MoveDesc, ScanPackedDesc, _delta_flags)
from . import layer as _l

BEAM_MAX_K = 64        # SSM_BEAM_MAX_K
MOVE_MAX_MOVES = 2048  # SSM_MOVE_MAX_MOVES


def _packed(what, x, pool, starts, src, dst):
    """(sequences, slots, flags) of packed sequences."""
    if pool is None and (src is not None or dst is not None):
        raise ValueError("%s: src and dst are slots of a pool, and there is none" % what)
    if starts is not None and (starts.dim() != 1 or starts.shape[0] < 2):
        raise ValueError("%s: starts is (sequences + 1,)" % what)
    flags = ((SSM_HAS_STARTS if starts is not None else 0) | (SSM_HAS_STATES if pool is not None else 0) |
             (SSM_HAS_SRC if src is not None else 0) | (SSM_HAS_DST if dst is not None else 0))
    return x.shape[0] if starts is None else starts.shape[0] - 1, 0 if pool is None else pool.shape[0], flags


def causal_conv1d_packed(x, weight, windows=None, starts=None, src=None, dst=None, bias=None, silu=False, y_dtype=None,
                         y=None, stream=None):
    """y = causal depthwise convolution (+ bias, + SiLU) of packed sequences
    (see include/ssm.h).  Returns y.

    x: (tokens, dim) fp32 or bf16, unit innermost stride; weight (dim, width),
    bias (dim,) fp32.  starts: (sequences + 1,) int32 on the GPU, sequence s is
    rows starts[s] to starts[s + 1]; without it each row is a sequence of one
    token.  windows: (slots, width - 1, dim) of x's type, the inputs in front of
    each sequence, updated in place: sequence s starts from slot src[s] (int32;
    default s; outside the pool: zeros) and its last width - 1 inputs are left in
    slot dst[s] (default src; outside the pool: not kept).  Rows of y that belong
    to no sequence are left as they are."""
    tensors = (x, weight, bias, y, windows, starts, src, dst)
    key = ("causal_conv1d_packed", silu, y_dtype, _l._sig(tensors))
    plan = _l._plans.get(key)
    if y is None:
        y = _l._empty(stream, x, tuple(x.shape), y_dtype)
    tensors = (x, weight, bias, y, windows, starts, src, dst)
    if plan is None:
        seqs, slots, flags = _packed("causal_conv1d_packed", x, windows, starts, src, dst)
        plan = _l._keep(key, _l._Plan("ssm_causal_conv1d_packed", ConvPackedDesc, _CONV_PACKED_T,
                                      (("tokens", x.shape[0]), ("seqs", seqs), ("dim", x.shape[1]),
                                       ("width", weight.shape[1]), ("slots", slots)),
                                      flags | (SSM_HAS_BIAS if bias is not None else 0) | (SSM_SILU if silu else 0),
                                      tensors, ("y", "windows")))
    _l._launch(plan, tensors, stream)
    return y


def causal_conv1d_bwd(dy, x, weight, bias=None, silu=False, grad_dtype=None, dx=None, stream=None) -> dict:
    """Gradients of sum(dy * y) for y = causal_conv1d(x, weight, bias, silu) (see
    include/ssm.h).  x: (batch, L, dim) fp32 or bf16; dy: the same shape, x's
    type or fp32.  dx: optional memory for that gradient (a slice of one
    projection's gradient, say).

    Returns a dict: dx (grad_dtype, default dy's dtype), dweight (dim, width) and,
    with a bias, dbias (dim,), both fp32."""
    key = ("causal_conv1d_bwd", silu, grad_dtype, _l._sig((dy, x, weight, bias, dx)))
    plan = _l._plans.get(key)
    if dx is None:
        dx = _l._empty(stream, x, tuple(x.shape), grad_dtype or dy.dtype)
    dweight = _l._empty(stream, x, tuple(weight.shape), torch.float32)
    dbias = None if bias is None else _l._empty(stream, x, tuple(bias.shape), torch.float32)
    tensors = (dy, x, weight, bias, dx, dweight, dbias)
    if plan is None:
        batch, L, dim = x.shape
        plan = _l._keep(key, _l._Plan("ssm_causal_conv1d_bwd", ConvBwdDesc, _CONV_BWD_T,
                                      (("batch", batch), ("seqlen", L), ("dim", dim), ("width", weight.shape[1])),
                                      (SSM_HAS_BIAS if bias is not None else 0) | (SSM_SILU if silu else 0), tensors,
                                      ("dx", "dweight", "dbias"), "ssm_causal_conv1d_bwd_workspace_size"))
    _l._launch(plan, tensors, stream)
    out = {"dx": dx, "dweight": dweight}
    if bias is not None:
        out["dbias"] = dbias
    return out


def selective_scan_packed(x, delta, A, B, C, states=None, starts=None, src=None, dst=None, D=None, z=None, euler=False,
                          y_dtype=None, y=None, stream=None, delta_softplus=False, delta_bias=None):
    """y = selective scan of packed sequences over a pool of states (see
    include/ssm.h).  Returns y.

    x, delta, z: (tokens, dim); B, C: (tokens, dstate), all fp32 or all bf16; A
    (dim, dstate), D, delta_bias (dim,) fp32.  states: (slots, dim, dstate) fp32,
    updated in place; starts, src and dst as in causal_conv1d_packed: without
    starts each row is one token of a sequence of its own (the decode step).
    Several sequences may start from one slot (a shared prefix); no slot that one
    sequence ends in may be another's."""
    tensors = (x, delta, A, B, C, D, z, y, delta_bias, states, starts, src, dst)
    key = ("selective_scan_packed", euler, delta_softplus, y_dtype, _l._sig(tensors))
    plan = _l._plans.get(key)
    if y is None:
        y = _l._empty(stream, x, tuple(x.shape), y_dtype)
    tensors = (x, delta, A, B, C, D, z, y, delta_bias, states, starts, src, dst)
    if plan is None:
        seqs, slots, flags = _packed("selective_scan_packed", x, states, starts, src, dst)
        plan = _l._keep(key, _l._Plan("ssm_selective_scan_packed", ScanPackedDesc, _SCAN_PACKED_T,
                                      (("tokens", x.shape[0]), ("seqs", seqs), ("dim", x.shape[1]),
                                       ("dstate", A.shape[1]), ("slots", slots)),
                                      flags | (SSM_HAS_Z if z is not None else 0) |
                                      (SSM_HAS_D if D is not None else 0) | (SSM_DISC_EULER if euler else 0) |
                                      _delta_flags(delta_softplus, delta_bias), tensors, ("y", "states"),
                                      "ssm_selective_scan_packed_workspace_size"))
    _l._launch(plan, tensors, stream)
    return y


def beam_select(logits, scores, k, stream=None):
    """One selection of a beam search (see include/ssm.h): the k best of every
    batch element's beams x vocab continuations by scores + log_softmax(logits),
    equal ones by their index.  logits: (batch, beams, vocab) fp32 or bf16, unit
    innermost stride; scores: (batch, beams) fp32.  Returns (scores fp32, tokens
    int32, parents int32), each (batch, k), the best first; parents are the beams
    that the tokens continue."""
    key = ("beam_select", k, _l._sig((logits, scores)))
    plan = _l._plans.get(key)
    if plan is None and (logits.dim() != 3 or not 0 < k <= BEAM_MAX_K):
        raise ValueError("beam_select: logits are (batch, beams, vocab), k is 1 to %d" % BEAM_MAX_K)
    shape = (logits.shape[0], k)
    out = (_l._empty(stream, logits, shape, torch.float32), _l._empty(stream, logits, shape, torch.int32),
           _l._empty(stream, logits, shape, torch.int32))
    tensors = (logits, scores) + out
    if plan is None:
        batch, beams, vocab = logits.shape
        plan = _l._keep(key, _l._Plan("ssm_beam_select", BeamDesc, _BEAM_T,
                                      (("batch", batch), ("beams", beams), ("vocab", vocab), ("k", k)), 0, tensors,
                                      ("out_scores", "tokens", "parents"), "ssm_beam_select_workspace_size"))
    _l._launch(plan, tensors, stream)
    return out


def state_move(pool, src, dst=None, stream=None):
    """pool[dst[i]] <- what pool[src[i]] held before the call, for all i at once
    (see include/ssm.h): forks, reorders, compacts slots; src < 0 clears one.
    pool: (slots, ...) fp32 or bf16 in place, a slot contiguous; src, dst:
    (moves,) int32 on the GPU, dst default 0, 1, ...  Returns pool."""
    key = ("state_move", _l._sig((pool, src, dst)))
    plan = _l._plans.get(key)
    tensors = (pool, src, dst)
    if plan is None:
        if pool.dim() < 2 or pool.shape[0] == 0:
            raise ValueError("state_move: pool is (slots, ...), at least one")
        row = pool.flatten(1) if pool[0].is_contiguous() else None
        if row is None or row.data_ptr() != pool.data_ptr():
            raise ValueError("state_move: a slot of the pool must be contiguous")
        plan = _l._keep(key, _l._Plan("ssm_state_move", MoveDesc, _MOVE_T,
                                      (("slots", pool.shape[0]), ("row", row.shape[1]), ("moves", src.shape[0])),
                                      SSM_HAS_DST if dst is not None else 0, (row, src, dst), ("pool",)))
    _l._launch(plan, tensors, stream)
    return pool
