"""What the layer's binding does with memory: operands that are only read stay
shared, what is written is written alone, and an allocation that fails says so."""
import pytest

from _gpu import banner

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a GPU", allow_module_level=True)

import selective_state_space_60_amd as ssm  # noqa: E402

BF16 = torch.bfloat16


def lazy(tensors):
    return {k: torch._lazy_clone(v) for k, v in tensors.items()}


def shared(tensors):
    torch.cuda.synchronize()
    return [k for k, v in tensors.items() if not torch._C._is_cow_tensor(v)]


def test_lazily_copied_operands_stay_shared():
    """A lazily copied input is read where it lies: no copy of a weight is made for reading it."""
    banner("lazy operands")
    r = lambda *s: torch.randn(s, device="cuda")  # noqa: E731
    base = {"x": r(2, 200, 64), "gate_a": r(2, 200, 64), "gate_x": r(2, 200, 64), "A": -r(64).abs(), "bias_a": r(64),
            "bias_x": r(64), "z": r(2, 200, 64), "h0": r(2, 64)}
    dy, ckpt = r(2, 200, 64), ssm.gated_scan_ckpt(2, 200, 64)
    want = ssm.gated_scan_fwd(**base, want_hlast=True, ckpt=ckpt)
    t = lazy(base)
    got = ssm.gated_scan_fwd(**t, want_hlast=True)
    assert shared(t) == [] and all(torch.equal(p, q) for p, q in zip(want, got))
    t = lazy(dict(base, dy=dy, ckpt=ckpt))
    ssm.gated_scan_bwd(**t)
    assert shared(t) == []
    t = lazy(dict({k: v[:, 0] if v.dim() == 3 else v for k, v in base.items() if k != "h0"}, state=base["h0"]))
    ssm.gated_state_update(**t, state_out=torch.empty_like(base["h0"]))
    assert shared(t) == []
    t = lazy({"x": base["x"], "weight": base["bias_a"], "residual": base["z"]})
    ssm.rms_norm(**t)
    assert shared(t) == []
    t = lazy({"dy": dy, "row": base["x"], "weight": base["bias_a"], "dres": base["z"]})
    ssm.rms_norm_bwd(**t)
    assert shared(t) == []
    packed, scale = ssm.w4_quantize(r(40, 64), 32)
    t = lazy({"x": r(2, 64).to(BF16), "weight": packed, "scale": scale, "bias": r(40)})
    ssm.w4_matvec(**t)
    assert shared(t) == []


def test_lazily_copied_outputs_are_written_alone():
    banner("lazy outputs")
    x, w = torch.randn(5, 64, device="cuda"), torch.rand(64, device="cuda")
    first = torch.randn(5, 64, device="cuda")
    res, keep = torch._lazy_clone(first), first.clone()
    y, out, _ = ssm.rms_norm(x, w, residual=res, residual_out=res)
    torch.cuda.synchronize()
    assert torch.equal(first, keep) and torch.equal(res, x + keep) and out is res
    buf = torch._lazy_clone(first)
    ssm.rms_norm(x, w, y=buf)
    torch.cuda.synchronize()
    assert torch.equal(first, keep) and torch.equal(buf, ssm.rms_norm(x, w)[0])


def test_out_of_memory_is_torchs_own_error():
    """An output that does not fit what the process may use: the error that a
    caller catches for torch's own allocations."""
    banner("out of memory")
    x = torch.zeros(1, 1024, device="cuda", dtype=BF16).expand(1 << 23, 1024)  # 16 GiB of y
    w = torch.ones(1024, device="cuda")
    torch.cuda.empty_cache()
    torch.cuda.set_per_process_memory_fraction(0.02)
    try:
        with pytest.raises(torch.OutOfMemoryError):
            ssm.rms_norm(x, w)
    finally:
        torch.cuda.set_per_process_memory_fraction(1.0)
    assert ssm.rms_norm(x[:3], w)[0].shape == (3, 1024)
