"""Refusals of the recurrent layer's entry points (gated scan, norm, 4-bit
weights) on the host, before any HIP call, and what their Python wrappers
refuse (no compute runs here)."""
import ctypes

import pytest

ssm = pytest.importorskip("selective_state_space_60_amd")

torch = pytest.importorskip("torch")
if torch.cuda.is_available():  # pragma: no cover
    # the calls below pass fake device addresses and must be rejected on the
    # host; with a GPU visible a validation gap would launch on them
    pytest.skip("host-validation tests run without a GPU", allow_module_level=True)

S = ssm
CODE = {"f32": S.SSM_F32, "bf16": S.SSM_BF16, "f16": S.SSM_F16, "e4m3": S.SSM_E4M3, "i32": S.SSM_I32, "u8": S.SSM_U8}


def td(shape, dtype="f32", strides=None):
    d = S.TensorDesc()
    d.dtype, d.ndim = CODE[dtype], len(shape)
    acc = 1
    for i in reversed(range(len(shape))):
        d.shape[i], d.stride[i] = shape[i], acc if strides is None else strides[i]
        acc *= shape[i]
    return d


def fill(d, p, tensors):
    for i, (k, t) in enumerate(tensors.items()):
        setattr(d, k, t)
        setattr(p, k, (i + 1) << 36)


def gated(batch=2, L=100, D=8, io="bf16", flags=0):
    d, p = S.GatedDesc(), S.GatedPtrs()
    d.batch, d.seqlen, d.dim, d.flags = batch, L, D, flags
    fill(d, p, {"x": td((batch, L, D), io), "gate_a": td((batch, L, D), io), "gate_x": td((batch, L, D), io),
                "A": td((D,)), "bias_a": td((D,)), "bias_x": td((D,)), "z": td((batch, L, D), io),
                "y": td((batch, L, D), io), "h0": td((batch, D)), "h_last": td((batch, D)),
                "lens": td((batch,), "i32"), "ckpt": td((batch, (L + 63) // 64, D))})
    return d, p


GATED_ALL = (S.SSM_HAS_Z | S.SSM_HAS_H0 | S.SSM_WANT_HLAST | S.SSM_WANT_CKPT | S.SSM_HAS_BIAS_A | S.SSM_HAS_BIAS_X |
             S.SSM_HAS_LENS)


def set_(obj, name, i, v):
    getattr(obj, name).__setitem__(i, v)


@pytest.mark.parametrize("mutate,status", [
    (lambda d, p: setattr(p, "x", None), S.SSM_ERR_NULL),
    (lambda d, p: setattr(p, "gate_a", None), S.SSM_ERR_NULL),
    (lambda d, p: setattr(p, "bias_x", None), S.SSM_ERR_NULL),
    (lambda d, p: setattr(p, "z", None), S.SSM_ERR_NULL),
    (lambda d, p: setattr(p, "lens", None), S.SSM_ERR_NULL),
    (lambda d, p: setattr(p, "ckpt", None), S.SSM_ERR_NULL),
    (lambda d, p: setattr(d, "batch", 0), S.SSM_ERR_SHAPE),
    (lambda d, p: setattr(d, "seqlen", 0), S.SSM_ERR_SHAPE),
    (lambda d, p: setattr(d, "dim", -1), S.SSM_ERR_SHAPE),
    (lambda d, p: setattr(d, "flags", d.flags | S.SSM_HAS_D), S.SSM_ERR_UNSUPPORTED),
    (lambda d, p: setattr(d, "flags", d.flags | S.SSM_HAS_DHLAST), S.SSM_ERR_UNSUPPORTED),
    (lambda d, p: setattr(d, "batch", 1 << 41), S.SSM_ERR_UNSUPPORTED),
    (lambda d, p: setattr(d.x, "dtype", S.SSM_F16), S.SSM_ERR_UNSUPPORTED),
    (lambda d, p: setattr(d.x, "dtype", S.SSM_U8), S.SSM_ERR_DTYPE),
    (lambda d, p: setattr(d.gate_x, "dtype", S.SSM_F32), S.SSM_ERR_DTYPE),
    (lambda d, p: setattr(d.A, "dtype", S.SSM_BF16), S.SSM_ERR_DTYPE),
    (lambda d, p: setattr(d.lens, "dtype", S.SSM_F32), S.SSM_ERR_DTYPE),
    (lambda d, p: set_(d.gate_a, "shape", 2, 9), S.SSM_ERR_SHAPE),
    (lambda d, p: set_(d.ckpt, "shape", 1, 3), S.SSM_ERR_SHAPE),
    (lambda d, p: setattr(d.A, "ndim", 2), S.SSM_ERR_SHAPE),
    (lambda d, p: set_(d.x, "stride", 2, 2), S.SSM_ERR_STRIDE),
    (lambda d, p: set_(d.z, "stride", 1, -8), S.SSM_ERR_STRIDE),
    (lambda d, p: set_(d.y, "stride", 1, 4), S.SSM_ERR_STRIDE),
    (lambda d, p: set_(d.h0, "stride", 0, 16), S.SSM_ERR_STRIDE),
    (lambda d, p: set_(d.x, "stride", 1, 1 << 30), S.SSM_ERR_UNSUPPORTED),
    (lambda d, p: set_(d.y, "stride", 1, 1 << 22), S.SSM_ERR_UNSUPPORTED),
    (lambda d, p: set_(d.x, "stride", 0, 1 << 60), S.SSM_ERR_UNSUPPORTED),
    (lambda d, p: setattr(p, "x", (1 << 36) + 1), S.SSM_ERR_ALIGN),
    (lambda d, p: setattr(p, "h_last", (50 << 36) + 2), S.SSM_ERR_ALIGN),
    (lambda d, p: setattr(p, "y", p.x), S.SSM_ERR_ALIAS),
    (lambda d, p: setattr(p, "h_last", p.h0), S.SSM_ERR_ALIAS),
    (lambda d, p: setattr(p, "ckpt", p.y + 16), S.SSM_ERR_ALIAS),
    (lambda d, p: setattr(p, "y", p.lens), S.SSM_ERR_ALIAS),
])
def test_gated_scan(mutate, status):
    d, p = gated(flags=GATED_ALL)
    mutate(d, p)
    assert S.lib().ssm_gated_scan_fwd(ctypes.byref(d), ctypes.byref(p), None, 0, None) == status


def test_gated_scan_null_and_workspace():
    L = S.lib()
    n = ctypes.c_size_t()
    d, p = gated()
    assert L.ssm_gated_scan_fwd(None, ctypes.byref(p), None, 0, None) == S.SSM_ERR_NULL
    assert L.ssm_gated_scan_fwd(ctypes.byref(d), None, None, 0, None) == S.SSM_ERR_NULL
    assert L.ssm_gated_scan_workspace_size(ctypes.byref(d), None) == S.SSM_ERR_NULL
    assert L.ssm_gated_scan_workspace_size(ctypes.byref(d), ctypes.byref(n)) == S.SSM_OK and n.value == 0
    # few channels, many steps: the sequence is split and needs a workspace
    d, p = gated(batch=1, L=100000, D=64)
    assert L.ssm_gated_scan_workspace_size(ctypes.byref(d), ctypes.byref(n)) == S.SSM_OK and n.value > 0
    call = lambda ws, nb: L.ssm_gated_scan_fwd(ctypes.byref(d), ctypes.byref(p), ws, nb, None)  # noqa: E731
    assert call(None, 0) == S.SSM_ERR_WORKSPACE
    assert call(1 << 45, n.value - 1) == S.SSM_ERR_WORKSPACE
    assert call((1 << 45) + 8, n.value) == S.SSM_ERR_ALIGN
    assert call(p.x, n.value) == S.SSM_ERR_ALIAS


def gated_bwd(batch=2, L=100, D=8, io="bf16", g="bf16", flags=0):
    d, p = S.GatedBwdDesc(), S.GatedBwdPtrs()
    d.batch, d.seqlen, d.dim, d.flags = batch, L, D, flags
    bld = (batch, L, D)
    t = {k: td(bld, io) for k in ("x", "gate_a", "gate_x", "z")}
    t.update({k: td((D,)) for k in ("A", "bias_a", "bias_x", "dA", "dbias_a", "dbias_x")})
    t.update({k: td((batch, D)) for k in ("h0", "dh_last", "dh0")})
    t.update({k: td(bld, g) for k in ("dy", "dx", "dgate_a", "dgate_x", "dz")})
    t["lens"], t["ckpt"] = td((batch,), "i32"), td((batch, (L + 63) // 64, D))
    fill(d, p, t)
    return d, p


BWD_ALL = (S.SSM_HAS_Z | S.SSM_HAS_H0 | S.SSM_HAS_CKPT | S.SSM_HAS_BIAS_A | S.SSM_HAS_BIAS_X | S.SSM_HAS_LENS |
           S.SSM_HAS_DHLAST)


@pytest.mark.parametrize("mutate,status", [
    (lambda d, p: setattr(p, "dy", None), S.SSM_ERR_NULL),
    (lambda d, p: setattr(p, "dz", None), S.SSM_ERR_NULL),
    (lambda d, p: setattr(p, "ckpt", None), S.SSM_ERR_NULL),
    (lambda d, p: setattr(p, "dh_last", None), S.SSM_ERR_NULL),
    (lambda d, p: setattr(p, "dbias_a", None), S.SSM_ERR_NULL),
    (lambda d, p: setattr(p, "dh0", None), S.SSM_ERR_NULL),
    (lambda d, p: setattr(d, "flags", d.flags | S.SSM_WANT_CKPT), S.SSM_ERR_UNSUPPORTED),
    (lambda d, p: setattr(d, "flags", d.flags | S.SSM_WANT_HLAST), S.SSM_ERR_UNSUPPORTED),
    (lambda d, p: setattr(d.dx, "dtype", S.SSM_F32), S.SSM_ERR_DTYPE),   # not dy's type
    (lambda d, p: setattr(d.dy, "dtype", S.SSM_E4M3), S.SSM_ERR_DTYPE),
    (lambda d, p: setattr(d.dA, "dtype", S.SSM_BF16), S.SSM_ERR_DTYPE),
    (lambda d, p: set_(d.dgate_x, "shape", 1, 99), S.SSM_ERR_SHAPE),
    (lambda d, p: set_(d.dgate_a, "stride", 1, 0), S.SSM_ERR_STRIDE),
    (lambda d, p: set_(d.dA, "stride", 0, 2), S.SSM_ERR_STRIDE),
    (lambda d, p: set_(d.dz, "stride", 1, 1 << 24), S.SSM_ERR_UNSUPPORTED),
    (lambda d, p: setattr(p, "dx", p.x), S.SSM_ERR_ALIAS),
    (lambda d, p: setattr(p, "dbias_a", p.dA), S.SSM_ERR_ALIAS),
    (lambda d, p: setattr(p, "dh0", p.dh_last), S.SSM_ERR_ALIAS),
    (lambda d, p: setattr(p, "dx", p.ckpt), S.SSM_ERR_ALIAS),
    (lambda d, p: setattr(p, "dz", p.dz + 1), S.SSM_ERR_ALIGN),
    (lambda d, p: None, S.SSM_ERR_WORKSPACE),
])
def test_gated_bwd(mutate, status):
    d, p = gated_bwd(flags=BWD_ALL)
    mutate(d, p)
    assert S.lib().ssm_gated_scan_bwd(ctypes.byref(d), ctypes.byref(p), None, 0, None) == status


def test_gated_bwd_workspace():
    L, n, m = S.lib(), ctypes.c_size_t(), ctypes.c_size_t()
    d, p = gated_bwd()
    assert L.ssm_gated_scan_bwd_workspace_size(ctypes.byref(d), ctypes.byref(n)) == S.SSM_OK
    d.flags = S.SSM_HAS_CKPT
    assert L.ssm_gated_scan_bwd_workspace_size(ctypes.byref(d), ctypes.byref(m)) == S.SSM_OK and 0 < m.value < n.value
    call = lambda ws, nb: L.ssm_gated_scan_bwd(ctypes.byref(d), ctypes.byref(p), ws, nb, None)  # noqa: E731
    assert call(1 << 45, m.value - 1) == S.SSM_ERR_WORKSPACE
    assert call((1 << 45) + 64, m.value) == S.SSM_ERR_ALIGN
    assert call(p.dA, m.value) == S.SSM_ERR_ALIAS


def test_columns_of_one_buffer():
    """Gradients as columns of one matrix interleave without overlapping;
    columns that meet, or rows of another length, are refused."""
    L, D, wide = 100, 8, 32
    for shift, status in ((0, S.SSM_ERR_WORKSPACE), (1, S.SSM_ERR_ALIAS)):
        d, p = gated_bwd(L=L, D=D, flags=BWD_ALL)
        for k, name in enumerate(("dx", "dgate_a", "dgate_x", "dz")):
            setattr(d, name, td((2, L, D), "bf16", (L * wide, wide, 1)))
            setattr(p, name, (1 << 45) + 2 * (k * D - (shift if k == 2 else 0)))
        assert S.lib().ssm_gated_scan_bwd(ctypes.byref(d), ctypes.byref(p), None, 0, None) == status
    d, p = gated_bwd(L=L, D=D, flags=BWD_ALL)
    d.dx, p.dx = td((2, L, D), "bf16", (L * wide, wide, 1)), 1 << 45
    d.dz, p.dz = td((2, L, D), "bf16", (L * (wide + 4), wide + 4, 1)), (1 << 45) + 16
    assert S.lib().ssm_gated_scan_bwd(ctypes.byref(d), ctypes.byref(p), None, 0, None) == S.SSM_ERR_ALIAS
    # y into a free column block of the buffer that holds the inputs: only the workspace is missing
    for col, status in ((3, S.SSM_ERR_WORKSPACE), (2, S.SSM_ERR_ALIAS)):
        d, p = gated(L=300)
        for name, k in (("x", 0), ("gate_a", 1), ("gate_x", 2), ("y", col)):
            setattr(d, name, td((2, 300, 8), "bf16", (300 * wide, wide, 1)))
            setattr(p, name, (1 << 45) + 16 * k)
        assert S.lib().ssm_gated_scan_fwd(ctypes.byref(d), ctypes.byref(p), None, 0, None) == status


def gated_update(batch=3, D=8, io="bf16", flags=0):
    d, p = S.GatedUpdateDesc(), S.GatedUpdatePtrs()
    d.batch, d.dim, d.flags = batch, D, flags
    t = {k: td((batch, D), io) for k in ("x", "gate_a", "gate_x", "z", "y")}
    t.update({k: td((D,)) for k in ("A", "bias_a", "bias_x")})
    t.update({k: td((batch, D)) for k in ("state", "state_out")})
    fill(d, p, t)
    return d, p


@pytest.mark.parametrize("mutate,status", [
    (lambda d, p: setattr(p, "state", None), S.SSM_ERR_NULL),
    (lambda d, p: setattr(p, "state_out", None), S.SSM_ERR_NULL),
    (lambda d, p: setattr(p, "y", None), S.SSM_ERR_NULL),
    (lambda d, p: setattr(d, "dim", 0), S.SSM_ERR_SHAPE),
    (lambda d, p: setattr(d, "flags", d.flags | S.SSM_HAS_H0), S.SSM_ERR_UNSUPPORTED),
    (lambda d, p: setattr(d.x, "dtype", S.SSM_F16), S.SSM_ERR_UNSUPPORTED),
    (lambda d, p: setattr(d.state, "dtype", S.SSM_BF16), S.SSM_ERR_DTYPE),
    (lambda d, p: set_(d.state, "stride", 0, 9), S.SSM_ERR_STRIDE),
    (lambda d, p: set_(d.y, "stride", 0, 0), S.SSM_ERR_STRIDE),
    (lambda d, p: setattr(p, "state_out", p.state), S.SSM_ERR_ALIAS),
    (lambda d, p: setattr(p, "y", p.state), S.SSM_ERR_ALIAS),
    (lambda d, p: setattr(p, "state_out", p.A), S.SSM_ERR_ALIAS),
])
def test_gated_update(mutate, status):
    d, p = gated_update(flags=S.SSM_HAS_Z | S.SSM_HAS_BIAS_A | S.SSM_HAS_BIAS_X | S.SSM_HAS_STATE_OUT)
    mutate(d, p)
    assert S.lib().ssm_gated_state_update(ctypes.byref(d), ctypes.byref(p), None) == status


def norm(batch=2, L=5, D=40, io="bf16", y="bf16", group=0, flags=S.SSM_HAS_RESIDUAL):
    d, p = S.NormDesc(), S.NormPtrs()
    d.batch, d.seqlen, d.dim, d.group, d.eps, d.flags = batch, L, D, group, 1e-5, flags
    bld = (batch, L, D)
    fill(d, p, {"x": td(bld, io), "residual": td(bld), "weight": td((D,)), "y": td(bld, y), "residual_out": td(bld),
                "scale": td((batch, L, -(-D // group) if group else 1))})
    return d, p


@pytest.mark.parametrize("mutate,status", [
    (lambda d, p: setattr(p, "weight", None), S.SSM_ERR_NULL),
    (lambda d, p: setattr(p, "residual", None), S.SSM_ERR_NULL),
    (lambda d, p: setattr(p, "residual_out", None), S.SSM_ERR_NULL),
    (lambda d, p: setattr(p, "scale", None), S.SSM_ERR_NULL),
    (lambda d, p: setattr(d, "seqlen", 0), S.SSM_ERR_SHAPE),
    (lambda d, p: set_(d.scale, "shape", 2, 1), S.SSM_ERR_SHAPE),
    (lambda d, p: set_(d.weight, "shape", 0, 41), S.SSM_ERR_SHAPE),
    (lambda d, p: setattr(d, "dim", S.NORM_MAX_DIM + 1), S.SSM_ERR_UNSUPPORTED),
    (lambda d, p: setattr(d, "eps", -1.0), S.SSM_ERR_UNSUPPORTED),
    (lambda d, p: setattr(d, "eps", float("nan")), S.SSM_ERR_UNSUPPORTED),
    (lambda d, p: setattr(d, "group", 16), S.SSM_ERR_UNSUPPORTED),
    (lambda d, p: setattr(d, "group", -32), S.SSM_ERR_UNSUPPORTED),
    (lambda d, p: setattr(d.y, "dtype", S.SSM_BF16), S.SSM_ERR_UNSUPPORTED),  # a group without e4m3
    (lambda d, p: setattr(d, "flags", d.flags | S.SSM_HAS_Z), S.SSM_ERR_UNSUPPORTED),
    (lambda d, p: setattr(d.x, "dtype", S.SSM_F16), S.SSM_ERR_UNSUPPORTED),
    (lambda d, p: setattr(d.x, "dtype", S.SSM_E4M3), S.SSM_ERR_DTYPE),
    (lambda d, p: setattr(d.residual, "dtype", S.SSM_F16), S.SSM_ERR_DTYPE),
    (lambda d, p: setattr(d.weight, "dtype", S.SSM_BF16), S.SSM_ERR_DTYPE),
    (lambda d, p: set_(d.x, "stride", 2, 3), S.SSM_ERR_STRIDE),
    (lambda d, p: set_(d.y, "stride", 1, 39), S.SSM_ERR_STRIDE),
    (lambda d, p: setattr(p, "residual_out", p.residual + 4), S.SSM_ERR_ALIAS),
    (lambda d, p: setattr(p, "residual_out", p.x), S.SSM_ERR_ALIAS),
    (lambda d, p: setattr(p, "y", p.x), S.SSM_ERR_ALIAS),
    (lambda d, p: setattr(p, "y", p.residual_out + 8), S.SSM_ERR_ALIAS),
    (lambda d, p: setattr(p, "residual", p.residual + 2), S.SSM_ERR_ALIGN),
    # in place, but of another type
    (lambda d, p: (setattr(d.residual_out, "dtype", S.SSM_BF16), setattr(p, "residual_out", p.residual)),
     S.SSM_ERR_ALIAS),
])
def test_norm(mutate, status):
    d, p = norm(y="e4m3", group=32)
    mutate(d, p)
    assert S.lib().ssm_rms_norm_fwd(ctypes.byref(d), ctypes.byref(p), None) == status


def norm_bwd(batch=2, L=5, D=40, flags=S.SSM_HAS_RESIDUAL):
    d, p = S.NormBwdDesc(), S.NormBwdPtrs()
    d.batch, d.seqlen, d.dim, d.eps, d.flags = batch, L, D, 1e-5, flags
    bld = (batch, L, D)
    fill(d, p, {"dy": td(bld, "bf16"), "row": td(bld), "weight": td((D,)), "dres": td(bld), "dx": td(bld, "bf16"),
                "dweight": td((D,))})
    return d, p


@pytest.mark.parametrize("mutate,status", [
    (lambda d, p: setattr(p, "dres", None), S.SSM_ERR_NULL),
    (lambda d, p: setattr(p, "dweight", None), S.SSM_ERR_NULL),
    (lambda d, p: setattr(d, "batch", -1), S.SSM_ERR_SHAPE),
    (lambda d, p: setattr(d, "dim", S.NORM_MAX_DIM + 1), S.SSM_ERR_UNSUPPORTED),
    (lambda d, p: setattr(d, "flags", 1), S.SSM_ERR_UNSUPPORTED),
    (lambda d, p: setattr(d.row, "dtype", S.SSM_F16), S.SSM_ERR_UNSUPPORTED),
    (lambda d, p: setattr(d.dx, "dtype", S.SSM_E4M3), S.SSM_ERR_DTYPE),
    (lambda d, p: set_(d.dx, "stride", 1, 0), S.SSM_ERR_STRIDE),
    (lambda d, p: set_(d.dres, "shape", 2, 41), S.SSM_ERR_SHAPE),
    (lambda d, p: setattr(p, "dx", p.dy), S.SSM_ERR_ALIAS),
    (lambda d, p: setattr(p, "dweight", p.weight), S.SSM_ERR_ALIAS),
    (lambda d, p: None, S.SSM_ERR_WORKSPACE),
])
def test_norm_bwd(mutate, status):
    d, p = norm_bwd()
    mutate(d, p)
    assert S.lib().ssm_rms_norm_bwd(ctypes.byref(d), ctypes.byref(p), None, 0, None) == status
    n = ctypes.c_size_t()
    d, p = norm_bwd()
    assert S.lib().ssm_rms_norm_bwd_workspace_size(ctypes.byref(d), ctypes.byref(n)) == S.SSM_OK and n.value > 0


def w4(rows=3, ins=256, outs=20, group=64, flags=S.SSM_HAS_ZERO | S.SSM_HAS_BIAS):
    d, p = S.W4Desc(), S.W4Ptrs()
    d.rows, d.ins, d.outs, d.group, d.flags = rows, ins, outs, group, flags
    fill(d, p, {"x": td((rows, ins), "bf16"), "weight": td((outs, ins // 2), "u8"),
                "scale": td((outs, ins // group), "bf16"), "zero": td((outs, ins // group), "u8"), "bias": td((outs,)),
                "y": td((rows, outs), "bf16")})
    return d, p


@pytest.mark.parametrize("mutate,status", [
    (lambda d, p: setattr(p, "weight", None), S.SSM_ERR_NULL),
    (lambda d, p: setattr(p, "zero", None), S.SSM_ERR_NULL),
    (lambda d, p: setattr(p, "bias", None), S.SSM_ERR_NULL),
    (lambda d, p: setattr(d, "rows", 0), S.SSM_ERR_SHAPE),
    (lambda d, p: setattr(d, "ins", 250), S.SSM_ERR_SHAPE),
    (lambda d, p: setattr(d, "rows", S.W4_MAX_ROWS + 1), S.SSM_ERR_UNSUPPORTED),
    (lambda d, p: setattr(d, "group", 16), S.SSM_ERR_UNSUPPORTED),
    (lambda d, p: setattr(d, "group", 256), S.SSM_ERR_UNSUPPORTED),
    (lambda d, p: setattr(d, "outs", 1 << 45), S.SSM_ERR_UNSUPPORTED),
    (lambda d, p: setattr(d.x, "dtype", S.SSM_F32), S.SSM_ERR_DTYPE),
    (lambda d, p: setattr(d.weight, "dtype", S.SSM_I32), S.SSM_ERR_DTYPE),
    (lambda d, p: setattr(d.zero, "dtype", S.SSM_BF16), S.SSM_ERR_DTYPE),
    (lambda d, p: setattr(d.y, "dtype", S.SSM_E4M3), S.SSM_ERR_DTYPE),
    (lambda d, p: set_(d.scale, "shape", 1, 5), S.SSM_ERR_SHAPE),
    (lambda d, p: set_(d.weight, "stride", 0, 256), S.SSM_ERR_STRIDE),
    (lambda d, p: set_(d.x, "stride", 0, 260), S.SSM_ERR_ALIGN),
    (lambda d, p: set_(d.x, "stride", 0, 1 << 32), S.SSM_ERR_UNSUPPORTED),
    (lambda d, p: setattr(p, "x", p.x + 8), S.SSM_ERR_ALIGN),
    (lambda d, p: setattr(p, "weight", p.weight + 4), S.SSM_ERR_ALIGN),
    (lambda d, p: setattr(p, "y", p.x), S.SSM_ERR_ALIAS),
    (lambda d, p: setattr(p, "y", p.scale), S.SSM_ERR_ALIAS),
])
def test_w4(mutate, status):
    d, p = w4()
    mutate(d, p)
    assert S.lib().ssm_w4_matvec(ctypes.byref(d), ctypes.byref(p), None) == status


def test_wrappers_refuse_host_tensors():
    x = torch.zeros(2, 4, 8)
    v = torch.zeros(8)
    for call in (lambda: S.gated_scan_fwd(x, x, x, v), lambda: S.gated_scan_bwd(x, x, x, x, v),
                 lambda: S.gated_state_update(x[0], x[0], x[0], x[0], v), lambda: S.rms_norm(x, v),
                 lambda: S.rms_norm_bwd(x, x, v),
                 lambda: S.w4_matvec(torch.zeros(1, 32), torch.zeros(4, 16, dtype=torch.uint8), torch.zeros(4, 1))):
        with pytest.raises(ValueError, match="GPU"):
            call()


def test_a_stream_of_another_device_is_refused():
    from types import SimpleNamespace
    from selective_state_space_60_amd import layer
    with pytest.raises(ValueError, match="another device"):
        layer._launch(SimpleNamespace(index=0, entry="e"), (), SimpleNamespace(device=torch.device("cuda", 1)))


def test_backward_refuses_unknown_outputs():
    x, v = torch.zeros(2, 4, 8), torch.zeros(8)
    with pytest.raises(ValueError, match="dgate_a"):
        S.gated_scan_bwd(x, x, x, x, v, out={"dA": v})


def test_quantize_on_the_host():
    w = torch.tensor([[7.0, -7.0, 0.0, 1.0] * 8, [0.0] * 32])
    packed, scale = S.w4_quantize(w, group=32)
    assert packed.shape == (2, 16) and scale.tolist() == [[1.0], [0.0]]
    assert packed[0, :2].tolist() == [15 | (1 << 4), 8 | (9 << 4)] and set(packed[1].tolist()) == {8 | (8 << 4)}
    for bad in (lambda: S.w4_quantize(w, group=16), lambda: S.w4_quantize(w, group=64)):
        with pytest.raises(ValueError):
            bad()


def test_signatures():
    """What a call's descriptor is looked up by tells apart type, shape,
    strides and absence, and does not depend on address or values."""
    from selective_state_space_60_amd import layer

    def sig(*tensors):
        return layer._sig(tensors)

    a = torch.zeros(4, 6)
    assert sig(a) == sig(torch.ones(4, 6)) and sig(a, None) != sig(a) != sig(None, a)
    others = [torch.zeros(6, 4), torch.zeros(4, 6, dtype=torch.bfloat16), torch.zeros(4, 12)[:, ::2],
              torch.zeros(4, 12)[:, :6], torch.zeros(1, 4, 6), torch.zeros(1, 6).expand(4, 6)]
    assert len({sig(t) for t in others + [a]}) == len(others) + 1
    for bad in (3, [a]):
        with pytest.raises(TypeError):
            sig(bad)
    with pytest.raises(TypeError):
        layer._sig([a])
    with pytest.raises((TypeError, ValueError)):
        layer._run(0, 0, (a,), -1, 0)
    with pytest.raises(TypeError):
        layer._run(1, 2, 3)
    for call in (lambda: layer._new_like(None, None), lambda: layer._new_like(a, 3), lambda: layer._new(a, [2], None),
                 lambda: layer._new(a, ("2",), None)):
        with pytest.raises(TypeError):
            call()
    flip = torch.zeros(3, 4).t()
    assert layer._new_like(flip, torch.bfloat16).stride() == flip.stride()
    e = layer._new(a.requires_grad_(), (2, 5), None)
    assert e.shape == (2, 5) and e.dtype == a.dtype and not e.requires_grad
