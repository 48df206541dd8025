"""Host-side checks of the binding of the norm, the short convolution and the
selective scan, with stand-ins for torch and for tensors (no GPU)."""
import math
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


def test_a_torch_without_its_own_queries(monkeypatch):
    """The public queries stand in for the ones that a torch need not have."""
    torch = types.SimpleNamespace(
        _C=types.SimpleNamespace(), float32=1, bfloat16=2, int8=3, float8_e4m3fn=4, int32=5,
        cuda=types.SimpleNamespace(current_device=lambda: 6, current_stream=lambda dev: types.SimpleNamespace(cuda_stream=70 + dev)))
    monkeypatch.setattr(b, "_found", None)
    monkeypatch.setattr(b, "_torch", lambda: torch)
    assert b._device() == 6 and b._raw_stream(None, 6) == 76


class Stand:
    """What the binding asks of a contiguous tensor on the current device, of any size."""

    is_cuda = True

    def __init__(self, shape, dtype, ptr):
        self.shape, self.dtype, self._ptr = tuple(shape), dtype, ptr

    def dim(self):
        return len(self.shape)

    def get_device(self):
        return 0

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return self._ptr

    def numel(self):
        return math.prod(self.shape)


OVER = 2 ** 32 + 64  # its lower 32 bits are a size that every call takes


def test_sizes_past_31_bits_are_refused(monkeypatch):
    """Sizes that do not fit the C ABI's int: a row of that width, that many tokens, channels, slots and sequences."""
    torch = pytest.importorskip("torch")
    f32, i8, i32 = torch.float32, torch.int8, torch.int32
    monkeypatch.setattr(b, "_found", ({f32: b.DL_F32, i8: b.DL_I8}, lambda: 0, lambda dev: 0, i32))
    place = iter(range(1, 1000))
    t = lambda *shape, dtype=f32: Stand(shape, dtype, (1 << 46) + (next(place) << 38))  # noqa: E731

    def conv(step, rows=8, channels=64, P=OVER - 60, n=2):
        x, w, state, y = t(rows, channels), t(channels, 4), t(P, 3, channels), t(rows, channels)
        if step:
            b.dl_conv_step(x, w, None, state, None, y)
        else:
            b.dl_conv_prompt(x, w, None, state, t(n + 1, dtype=i32), None, y)

    def scan(n):
        S, x, v = t(4, 1, 64, 64), t(8, 1, 64), t(8, 1, 64)
        b.dl_ssm_prompt(S, t(n + 1, dtype=i32), None, x, t(8, 1), t(1), v, v, t(8, 1, 64))

    calls = [lambda: b.dl_rms_norm(t(1, OVER), t(OVER), 1e-5, t(1, OVER)),
             lambda: b.dl_rows_from_8bit(t(1, OVER, dtype=i8), t(1), t(1, OVER)),
             lambda: conv(False, rows=OVER), lambda: conv(False, channels=OVER), lambda: conv(False), lambda: conv(True),
             lambda: conv(True, rows=OVER, P=OVER), lambda: conv(False, P=4, n=2 ** 32 + 2), lambda: scan(2 ** 32 + 2),
             lambda: b.dl_ssm_work_bytes(OVER, 1, 1, 64, 64)]
    for call in calls:
        with pytest.raises(ValueError, match="exceeds 2"):
            call()
