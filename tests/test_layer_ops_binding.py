"""Host-side checks of the binding of the norm, the short convolution and the
selective scan, with stand-ins for torch and for tensors (no GPU)."""
import types

import pytest

import gated_delta_rule_104_b200._binding as b


class HalfWay:
    """A torch that lets another thread's whole call run at its k-th lookup."""

    def __init__(self, k, call):
        self._left, self._call, self._C = k, call, self

    def __getattr__(self, name):
        self._left -= 1
        if self._left == 0:
            self._call()
        return {"_cuda_getDevice": lambda: 3, "_cuda_getCurrentRawStream": lambda dev: 40 + dev}.get(name, name)


@pytest.mark.parametrize("k", range(1, 9))
def test_first_calls_of_two_threads(monkeypatch, k):
    """A thread that makes its first call while another one looks torch's queries up finds all of them or looks them up itself."""
    index = types.SimpleNamespace(dtype="int32", get_device=lambda: 3, shape=(4,), is_contiguous=lambda: True, data_ptr=lambda: 64)
    value = types.SimpleNamespace(dtype="float32", get_device=lambda: 3, shape=(4,), is_contiguous=lambda: True, data_ptr=lambda: 128)
    seen = []

    def call():
        seen.append((b._device(), b._raw_stream(None, 3), b._f32(value, "A", (4,), 3), b._index(index, "slot", 4, 3),
                     b._code_of(types.SimpleNamespace(dtype="bfloat16"))))

    half = HalfWay(k, call)
    for name in ("_found", "_codes", "_getdevice", "_getstream", "_i32"):
        if hasattr(b, name):
            monkeypatch.setattr(b, name, None)
    monkeypatch.setattr(b, "_torch", lambda: half)
    assert b._device() == 3
    call()
    assert set(seen) == {(3, 43, 128, 64, b.DL_BF16)}
