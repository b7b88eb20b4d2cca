"""The binding's native call (csrc/marshal.cpp) with an entry point of its own,
on host tensors."""
import ctypes

import pytest

pytest.importorskip("selective_state_space_60_amd")
torch = pytest.importorskip("torch")

from selective_state_space_60_amd import layer  # noqa: E402


def call(tensors, written, write=(), nbytes=-1):
    """layer._run on an entry point that notes its pointers and writes 5.0 through those of `write`."""
    seen = []

    def entry(desc, ptrs, *rest):
        seen.extend(ptrs[i] for i in range(len(tensors)))
        seen.append(rest)
        for i in write:
            ctypes.c_float.from_address(ptrs[i]).value = 5.0
        return 7

    args = [ctypes.c_void_p, ctypes.POINTER(ctypes.c_void_p)] + ([ctypes.c_void_p, ctypes.c_size_t]
                                                                 if nbytes >= 0 else []) + [ctypes.c_void_p]
    fn = ctypes.CFUNCTYPE(ctypes.c_int, *args)(entry)
    assert layer._run(ctypes.cast(fn, ctypes.c_void_p).value, 0, tensors, written, nbytes, 0) == 7
    return seen


def test_what_is_read_stays_shared():
    first = torch.zeros(3)
    x, y = torch._lazy_clone(first), torch._lazy_clone(first)
    seen = call((x, None, y), 4, write=(2,))
    assert torch._C._is_cow_tensor(x) and not torch._C._is_cow_tensor(y)
    assert seen[1] is None and seen[0] != seen[2] == y.data_ptr()
    assert first.tolist() == [0, 0, 0] and y.tolist() == [5, 0, 0]


@pytest.mark.parametrize("written", [1, 2])
def test_the_same_tensor_read_and_written(written):
    """In place under two names: both are the written memory."""
    first = torch.zeros(3)
    t = torch._lazy_clone(first)
    seen = call((t, t), written, write=(0,))
    assert seen[0] == seen[1] == t.data_ptr() and first.tolist() == [0, 0, 0] and t.tolist() == [5, 0, 0]


def test_workspace():
    a = torch.zeros(3)
    assert call((a,), 0, nbytes=0)[1][:2] == (None, 0)
    ws, n, stream = call((a,), 0, nbytes=100)[1]
    assert ws and n == 100 and stream is None


def test_written_outputs_of_every_entry_point(monkeypatch):
    """The masks that the wrappers pass name the outputs, and the state only where it is written."""
    masks = {}

    class Plan:
        def __init__(self, entry, Desc, names, sizes, flags, tensors, written, size_entry=None):
            assert len(names) == len(tensors) and set(written) <= set(names)
            masks.setdefault(entry, []).append(set(written))

    monkeypatch.setattr(layer, "_Plan", Plan)
    monkeypatch.setattr(layer, "_launch", lambda *a: None)
    monkeypatch.setattr(layer, "_plans", {})
    x, v, s = torch.zeros(2, 4, 32), torch.zeros(32), torch.zeros(2, 32)
    layer.gated_scan_fwd(x, x, x, v)
    layer.gated_scan_bwd(x, x, x, x, v)
    layer.gated_state_update(s, s, s, s, v)
    layer.gated_state_update(s, s, s, s, v, state_out=s)
    layer.rms_norm(x, v, residual=x)
    layer.rms_norm_bwd(x, x, v)
    layer.w4_matvec(s.bfloat16(), torch.zeros(4, 16, dtype=torch.uint8), torch.zeros(4, 1))
    grads = {"dx", "dgate_a", "dgate_x", "dz", "dA", "dbias_a", "dbias_x", "dh0"}
    assert masks == {"ssm_gated_scan_fwd": [{"y", "h_last", "ckpt"}], "ssm_gated_scan_bwd": [grads],
                     "ssm_gated_state_update": [{"y", "state"}, {"y", "state_out"}],
                     "ssm_rms_norm_fwd": [{"y", "residual_out", "scale"}], "ssm_rms_norm_bwd": [{"dx", "dweight"}],
                     "ssm_w4_matvec": [{"y"}]}
