"""ctypes binding of libdeltalog.so (include/deltalog.h).

Argument marshalling only: every function here checks that the tensors are
CUDA, contiguous and of a supported dtype, reads their shapes, and passes raw
device pointers, sizes and the stream to the C ABI. All arithmetic runs in the
library's CUDA kernels. There is no fallback: a missing library raises.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

HERE = os.path.dirname(os.path.abspath(__file__))
# the library a process loads: libdeltalog.so, or the file DELTALOG_LIBRARY
# names (e.g. the index-guard debug build, libdeltalog_guard.so)
LIB_PATH = os.environ.get("DELTALOG_LIBRARY") or os.path.join(HERE, "libdeltalog.so")
GUARD_LIB_PATH = os.path.join(HERE, "libdeltalog_guard.so")

DL_OK, DL_ERR_INVALID_ARG, DL_ERR_UNSUPPORTED, DL_ERR_LOG_FULL, DL_ERR_CUDA = range(5)
DL_F32, DL_BF16, DL_I8, DL_E4M3 = 0, 1, 2, 3
DL_DECAY_HEAD, DL_DECAY_CHANNEL, DL_RWKV6 = 0, 1, 2
DL_MAX_LOG = 64
ABI_VERSION = 10

EXPORTS = ("dl_gdn_decode_step", "dl_kda_decode_step", "dl_rwkv6_decode_step", "dl_log_append_read", "dl_log_merge",
           "dl_log_merge_read", "dl_log_work_bytes", "dl_log_append_read_noalloc", "dl_pool_step",
           "dl_pool_flush", "dl_state_bytes", "dl_state_to_i8", "dl_state_from_i8", "dl_status_string",
           "dl_last_error", "dl_abi_version", "dl_device_faults", "dl_index_guard_build", "dl_rms_norm",
           "dl_rows_from_8bit", "dl_conv_prompt", "dl_conv_step", "dl_ssm_prompt", "dl_ssm_step", "dl_ssm_work_bytes")
DL_NOALLOC_WORK_BYTES = 16 << 20


class DeltaLogError(RuntimeError):
    def __init__(self, fn: str, status: int, message: str):
        super().__init__(f"{fn}: status {status} ({_status_name(status)}): {message}")
        self.status = status


class dl_log(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("beta", ctypes.c_void_p),
                ("a", ctypes.c_void_p), ("x", ctypes.c_void_p), ("dtype", ctypes.c_int), ("L", ctypes.c_int),
                ("work", ctypes.c_void_p), ("work_bytes", ctypes.c_size_t)]


class dl_pool(ctypes.Structure):
    _fields_ = [("S", ctypes.c_void_p), ("s_dtype", ctypes.c_int), ("P", ctypes.c_int), ("n", ctypes.c_void_p),
                ("status", ctypes.c_void_p), ("log", dl_log)]


class dl_conv(ctypes.Structure):
    _fields_ = [("w", ctypes.c_void_p), ("bias", ctypes.c_void_p), ("channels", ctypes.c_int), ("taps", ctypes.c_int),
                ("dtype", ctypes.c_int), ("silu", ctypes.c_int)]


class dl_ssm(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p), ("x_stride", ctypes.c_longlong), ("dt", ctypes.c_void_p),
                ("dt_stride", ctypes.c_longlong), ("b", ctypes.c_void_p), ("b_stride", ctypes.c_longlong),
                ("c", ctypes.c_void_p), ("c_stride", ctypes.c_longlong), ("z", ctypes.c_void_p),
                ("z_stride", ctypes.c_longlong), ("A", ctypes.c_void_p), ("D", ctypes.c_void_p),
                ("dt_bias", ctypes.c_void_p), ("dtype", ctypes.c_int)]


_lib = None


def load(path: Optional[str] = None) -> ctypes.CDLL:
    """Load libdeltalog.so (raises if it has not been built)."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = path or LIB_PATH
    if not os.path.exists(p):
        raise RuntimeError(f"libdeltalog.so not found at {p}: build it with "
                           "`python -m gated_delta_rule_104_b200.build` (nvcc, sm_100a)")
    lib = ctypes.CDLL(p)
    vp, i, f = ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p
    step = [vp, i, vp, vp, vp, vp, vp, i, f, i, i, i, i, vp]
    lib.dl_gdn_decode_step.argtypes = step
    lib.dl_kda_decode_step.argtypes = step
    lib.dl_rwkv6_decode_step.argtypes = [vp, i, vp, vp, vp, vp, i, f, i, i, i, i, vp]
    lp = ctypes.POINTER(dl_log)
    lib.dl_log_append_read.argtypes = [vp, i, i, lp, i, vp, vp, vp, vp, vp, i, f, i, i, i, i, vp]
    lib.dl_log_merge_read.argtypes = [vp, i, i, lp, i, vp, vp, vp, vp, vp, i, f, i, i, i, i, vp]
    lib.dl_log_append_read_noalloc.argtypes = [vp, i, i, lp, i, vp, vp, vp, vp, vp, i, f, i, i, i, i, vp]
    pp = ctypes.POINTER(dl_pool)
    lib.dl_pool_step.argtypes = [pp, i, vp, vp, vp, vp, vp, vp, i, f, i, i, i, i, vp]
    lib.dl_pool_flush.argtypes = [pp, i, vp, i, i, i, i, vp]
    lib.dl_state_bytes.argtypes = [i, i, i, i, i]
    lib.dl_state_bytes.restype = ctypes.c_size_t
    lib.dl_state_to_i8.argtypes = [vp, i, vp, i, i, i, i, vp]
    lib.dl_state_from_i8.argtypes = [vp, vp, i, i, i, i, i, vp]
    lib.dl_log_merge.argtypes = [vp, i, i, lp, i, i, i, i, i, vp]
    for name in ("dl_gdn_decode_step", "dl_kda_decode_step", "dl_rwkv6_decode_step", "dl_log_append_read",
                 "dl_log_merge", "dl_log_merge_read", "dl_log_append_read_noalloc", "dl_pool_step",
                 "dl_pool_flush", "dl_state_to_i8", "dl_state_from_i8"):
        getattr(lib, name).restype = ctypes.c_int
    ll, sz = ctypes.c_longlong, ctypes.c_size_t
    cp, mp = ctypes.POINTER(dl_conv), ctypes.POINTER(dl_ssm)
    lib.dl_rms_norm.argtypes = [vp, i, ll, vp, vp, i, vp, i, ctypes.c_float, vp, i, vp, i, ll, i, vp]
    lib.dl_rows_from_8bit.argtypes = [vp, i, vp, i, vp, i, ll, i, vp]
    lib.dl_conv_prompt.argtypes = [cp, vp, ll, i, vp, i, vp, i, vp, vp, vp, vp]
    lib.dl_conv_step.argtypes = [cp, vp, ll, i, vp, i, vp, vp, vp, vp]
    lib.dl_ssm_prompt.argtypes = [vp, i, i, vp, vp, mp, vp, i, i, vp, i, i, i, i, vp, sz, vp]
    lib.dl_ssm_step.argtypes = [vp, i, i, vp, vp, mp, vp, i, i, i, i, i, vp]
    lib.dl_ssm_work_bytes.argtypes = [i, i, i, i, i]
    lib.dl_ssm_work_bytes.restype = sz
    for name in ("dl_rms_norm", "dl_rows_from_8bit", "dl_conv_prompt", "dl_conv_step", "dl_ssm_prompt", "dl_ssm_step"):
        getattr(lib, name).restype = ctypes.c_int
    lib.dl_status_string.argtypes = [ctypes.c_int]
    lib.dl_status_string.restype = ctypes.c_char_p
    lib.dl_last_error.argtypes = []
    lib.dl_last_error.restype = ctypes.c_char_p
    lib.dl_log_work_bytes.argtypes = [i, i, i, i]
    lib.dl_log_work_bytes.restype = ctypes.c_size_t
    lib.dl_abi_version.argtypes = []
    lib.dl_abi_version.restype = ctypes.c_int
    lib.dl_device_faults.argtypes = [ctypes.POINTER(ctypes.c_uint), ctypes.c_int]
    lib.dl_device_faults.restype = ctypes.c_int
    lib.dl_index_guard_build.argtypes = []
    lib.dl_index_guard_build.restype = ctypes.c_int
    if lib.dl_abi_version() != ABI_VERSION:
        raise RuntimeError(f"libdeltalog.so ABI {lib.dl_abi_version()} != binding ABI {ABI_VERSION}: rebuild")
    if path is None:
        _lib = lib
    return lib


def _status_name(s: int) -> str:
    return {0: "DL_OK", 1: "DL_ERR_INVALID_ARG", 2: "DL_ERR_UNSUPPORTED", 3: "DL_ERR_LOG_FULL",
            4: "DL_ERR_CUDA"}.get(s, "?")


def check(fn: str, status: int) -> None:
    if status != DL_OK:
        msg = load().dl_last_error().decode(errors="replace")
        raise DeltaLogError(fn, status, msg)


# ------------------------------------------------------------------ tensors

def _torch():
    import torch  # device memory and streams only

    return torch


def _dtype_code(t) -> int:
    torch = _torch()
    if t.dtype == torch.float32:
        return DL_F32
    if t.dtype == torch.bfloat16:
        return DL_BF16
    raise TypeError(f"unsupported dtype {t.dtype} (float32 or bfloat16)")


def _ptr(t, name: str, optional: bool = False) -> Optional[int]:
    if t is None:
        if optional:
            return None
        raise ValueError(f"{name} is required")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _stream(stream) -> int:
    if stream is None:
        return _torch().cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


class I8State:
    """A deferred base in the int8 layout (DL_I8): one device buffer of
    B*H*d_v*d_k int8 codes followed by B*H*d_v float32 row scales; an element's
    value is code * scale. ``codes`` and ``scales`` are views of the buffer."""

    def __init__(self, buf, B: int, H: int, d_k: int, d_v: int):
        self.buf, self.B, self.H, self.d_k, self.d_v = buf, int(B), int(H), int(d_k), int(d_v)
        self.shape = (self.B, self.H, self.d_v, self.d_k)

    @classmethod
    def allocate(cls, B, H, d_k, d_v, device="cuda"):
        torch = _torch()
        n = B * H * d_v * d_k
        return cls(torch.zeros(n + 4 * B * H * d_v, dtype=torch.uint8, device=device), B, H, d_k, d_v)

    @property
    def codes(self):
        torch = _torch()
        n = self.B * self.H * self.d_v * self.d_k
        return self.buf[:n].view(torch.int8).view(self.shape)

    @property
    def scales(self):
        torch = _torch()
        n = self.B * self.H * self.d_v * self.d_k
        return self.buf[n:].view(torch.float32).view(self.B, self.H, self.d_v)

    def data_ptr(self) -> int:
        return self.buf.data_ptr()


def dl_state_to_i8(S, out: "I8State", stream=None) -> None:
    """Round a float32 / bfloat16 state [B,H,d_v,d_k] into ``out``."""
    B, H, dk, dv = _dims(S)
    check("dl_state_to_i8", load().dl_state_to_i8(_ptr(S, "S"), _dtype_code(S), out.data_ptr(), B, H, dk, dv,
                                                  _stream(stream)))


def dl_state_from_i8(S8: "I8State", out, stream=None) -> None:
    """The values of an int8 state into ``out`` (float32 or bfloat16 [B,H,d_v,d_k])."""
    check("dl_state_from_i8", load().dl_state_from_i8(S8.data_ptr(), _ptr(out, "S"), _dtype_code(out), S8.B, S8.H,
                                                      S8.d_k, S8.d_v, _stream(stream)))


def _dims(S):
    if isinstance(S, I8State):
        return S.B, S.H, S.d_k, S.d_v
    if S.dim() != 4:
        raise ValueError("state must be [B, H, d_v, d_k]")
    B, H, dv, dk = S.shape
    return int(B), int(H), int(dk), int(dv)


def _state_code(S) -> int:
    return DL_I8 if isinstance(S, I8State) else _dtype_code(S)


def _state_ptr(S, name: str) -> int:
    if isinstance(S, I8State):
        return _ptr(S.buf, name)
    return _ptr(S, name)


def _in_dtype(*ts) -> int:
    codes = {_dtype_code(t) for t in ts if t is not None}
    if len(codes) != 1:
        raise TypeError("q, k, v, beta and a must share one dtype")
    return codes.pop()


def _check_shapes(B, H, dk, dv, q, k, v, beta, a, o, chan):
    exp = {"q": (q, B * H * dk), "k": (k, B * H * dk), "v": (v, B * H * dv), "beta": (beta, B * H),
           "a": (a, B * H * (dk if chan else 1)), "o": (o, B * H * dv)}
    for name, (t, n) in exp.items():
        if t is None and name == "beta":
            continue
        if t.numel() != n:
            raise ValueError(f"{name} has {t.numel()} elements, expected {n}")
    if o.dtype != _torch().float32:
        raise TypeError("o must be float32")


def dl_gdn_decode_step(S, q, k, v, beta, a, o, stream=None) -> None:
    """Eager GDN step in place on S [B,H,d_v,d_k]; o [B,H,d_v] float32."""
    _eager("dl_gdn_decode_step", S, q, k, v, beta, a, o, stream, chan=False)


def dl_kda_decode_step(S, q, k, v, beta, a, o, stream=None) -> None:
    """Eager KDA step (a [B,H,d_k]) in place on S; o [B,H,d_v] float32."""
    _eager("dl_kda_decode_step", S, q, k, v, beta, a, o, stream, chan=True)


def dl_rwkv6_decode_step(S, q, k, v, a, o, stream=None) -> None:
    """Eager RWKV6 step (a [B,H,d_k]; raw-value update, no beta) in place on S."""
    B, H, dk, dv = _dims(S)
    _check_shapes(B, H, dk, dv, q, k, v, None, a, o, True)
    st = _stream(stream)
    status = load().dl_rwkv6_decode_step(_ptr(S, "S"), _dtype_code(S), _ptr(q, "q"), _ptr(k, "k"), _ptr(v, "v"),
                                         _ptr(a, "a"), _in_dtype(q, k, v, a), _ptr(o, "o"), B, H, dk, dv, st)
    check("dl_rwkv6_decode_step", status)


def _eager(fn, S, q, k, v, beta, a, o, stream, chan):
    if isinstance(S, I8State):
        raise TypeError("the eager step takes a float32 or bfloat16 state")
    B, H, dk, dv = _dims(S)
    _check_shapes(B, H, dk, dv, q, k, v, beta, a, o, chan)
    st = _stream(stream)
    status = getattr(load(), fn)(_ptr(S, "S"), _dtype_code(S), _ptr(q, "q"), _ptr(k, "k"), _ptr(v, "v"),
                                 _ptr(beta, "beta"), _ptr(a, "a"), _in_dtype(q, k, v, beta, a),
                                 _ptr(o, "o"), B, H, dk, dv, st)
    check(fn, status)


class Log:
    """Caller-owned bounded log buffers of a deferred state (device tensors):
    k [B,H,L,d_k], v [B,H,L,d_v], beta [B,H,L], a [B,H,L] or [B,H,L,d_k],
    x [B,H,L,L] float32 (the log's triangular solve matrix), work (fp32 workspace).
    An RWKV6 log (``rwkv6=True``: channel decay, no delta correction) has no
    beta and no x (None)."""

    def __init__(self, k, v, beta, a, x, L: int, channel_decay: bool, work=None, rwkv6: bool = False):
        self.k, self.v, self.beta, self.a, self.x = k, v, beta, a, x
        self.L = int(L)
        self.rwkv6 = bool(rwkv6)
        self.channel_decay = bool(channel_decay) or self.rwkv6
        self.dtype = _in_dtype(k, v, beta, a)
        self.work = work

    @classmethod
    def allocate(cls, B, H, d_k, d_v, L, dtype, channel_decay, device="cuda", rwkv6: bool = False):
        torch = _torch()
        z = lambda *s: torch.zeros(*s, dtype=dtype, device=device)  # noqa: E731
        chan = channel_decay or rwkv6
        a = z(B, H, L, d_k) if chan else z(B, H, L)
        work = torch.empty(B * H * (d_k + d_v), dtype=torch.float32, device=device)
        x = None if rwkv6 else torch.zeros(B, H, L, L, dtype=torch.float32, device=device)
        beta = None if rwkv6 else z(B, H, L)
        return cls(z(B, H, L, d_k), z(B, H, L, d_v), beta, a, x, L, chan, work, rwkv6)

    def struct(self) -> dl_log:
        wp = _ptr(self.work, "log.work") if self.work is not None else None
        wb = self.work.numel() * self.work.element_size() if self.work is not None else 0
        return dl_log(_ptr(self.k, "log.k"), _ptr(self.v, "log.v"), _ptr(self.beta, "log.beta", self.rwkv6),
                      _ptr(self.a, "log.a"), _ptr(self.x, "log.x", self.rwkv6), self.dtype, self.L, wp, wb)

    @property
    def kind(self) -> int:
        if self.rwkv6:
            return DL_RWKV6
        return DL_DECAY_CHANNEL if self.channel_decay else DL_DECAY_HEAD


def dl_log_append_read(S_base, log: Log, n: int, q, k, v, beta, a, o, stream=None) -> None:
    """Append entry n and read o from base + log (base not written)."""
    _log_step("dl_log_append_read", S_base, log, n, q, k, v, beta, a, o, stream)


def dl_log_merge_read(S_base, log: Log, n: int, q, k, v, beta, a, o, stream=None) -> None:
    """Merge log entries 0..n-1 plus this step into the base; o = new base q."""
    _log_step("dl_log_merge_read", S_base, log, n, q, k, v, beta, a, o, stream)


def _log_step(fn, S, log, n, q, k, v, beta, a, o, stream):
    B, H, dk, dv = _dims(S)
    _check_shapes(B, H, dk, dv, q, k, v, beta, a, o, log.channel_decay)
    st = _stream(stream)
    ls = log.struct()
    status = getattr(load(), fn)(_state_ptr(S, "S_base"), _state_code(S), log.kind, ctypes.byref(ls), int(n),
                                 _ptr(q, "q"), _ptr(k, "k"), _ptr(v, "v"), _ptr(beta, "beta", log.rwkv6),
                                 _ptr(a, "a"),
                                 _in_dtype(q, k, v, beta, a), _ptr(o, "o"), B, H, dk, dv, st)
    check(fn, status)


def dl_log_merge(S_base, log: Log, n: int, stream=None) -> None:
    """Merge log entries 0..n-1 into the base in place."""
    B, H, dk, dv = _dims(S_base)
    st = _stream(stream)
    ls = log.struct()
    status = load().dl_log_merge(_state_ptr(S_base, "S_base"), _state_code(S_base), log.kind, ctypes.byref(ls),
                                 int(n), B, H, dk, dv, st)
    check("dl_log_merge", status)


def dl_device_faults(clear: bool = False) -> int:
    """The kernels' fault word on the current device (0: no bounded wait ran
    out and, in the index-guard build, no shared-memory write was out of
    bounds). Synchronises the device."""
    w = ctypes.c_uint(0)
    check("dl_device_faults", load().dl_device_faults(ctypes.byref(w), 1 if clear else 0))
    return int(w.value)


def dl_index_guard_build() -> bool:
    """Whether the loaded library is the index-guard debug build."""
    return bool(load().dl_index_guard_build())


def dl_status_string(status: int) -> str:
    return load().dl_status_string(int(status)).decode()


def dl_log_append_read_noalloc(S_base, log: Log, n: int, q, k, v, beta, a, o, stream=None) -> None:
    """As dl_log_append_read, with the scratch in the library's fixed device
    array instead of ``log.work``: for callers that cannot allocate device
    memory. Calls that overlap on the GPU race on that array."""
    _log_step("dl_log_append_read_noalloc", S_base, log, n, q, k, v, beta, a, o, stream)


# ------------------------------------------------------------------ slot pool

class Pool:
    """A pool of P per-sequence deferred states (device tensors): S [P,H,d_v,d_k],
    ``log`` a Log over the P slots (its workspace covers a batch of up to P
    rows), n [P] int32 log counts, status [1] int32 error word. A new sequence
    taking slot s needs S[s] = its initial state and n[s] = 0 (``reset``)."""

    def __init__(self, S, log: Log, n, status=None):
        self.S, self.log, self.n, self.status = S, log, n, status
        self.P = int(S.shape[0])  # (S may be an I8State: an int8 pool)

    @classmethod
    def allocate(cls, P, H, d_k, d_v, L, s_dtype, in_dtype, channel_decay, rwkv6: bool = False, device="cuda"):
        """``s_dtype``: torch.float32, torch.bfloat16, or torch.int8 for an int8 pool (DL_I8)."""
        torch = _torch()
        if s_dtype == torch.int8:
            S = I8State.allocate(P, H, d_k, d_v, device=device)
        else:
            S = torch.zeros(P, H, d_v, d_k, dtype=s_dtype, device=device)
        log = Log.allocate(P, H, d_k, d_v, L, in_dtype, channel_decay, device=device, rwkv6=rwkv6)
        n = torch.zeros(P, dtype=torch.int32, device=device)
        status = torch.zeros(1, dtype=torch.int32, device=device)
        return cls(S, log, n, status)

    def reset(self, slot: int, S0) -> None:
        """Start a new sequence in ``slot`` from state S0 [H, d_v, d_k] (stream-ordered copies;
        an int8 pool takes S0 rounded to its layout)."""
        if isinstance(self.S, I8State):
            tmp = I8State.allocate(1, self.S.H, self.S.d_k, self.S.d_v, device=self.S.buf.device)
            dl_state_to_i8(S0.reshape(1, *S0.shape).contiguous(), tmp)
            self.S.codes[slot].copy_(tmp.codes[0])
            self.S.scales[slot].copy_(tmp.scales[0])
        else:
            self.S[slot].copy_(S0)
        self.n[slot] = 0

    def struct(self) -> dl_pool:
        if self.n.dtype != _torch().int32:
            raise TypeError("pool.n must be int32")
        return dl_pool(_state_ptr(self.S, "pool.S"), _state_code(self.S), self.P, _ptr(self.n, "pool.n"),
                       _ptr(self.status, "pool.status", True), self.log.struct())


def _slots(slot, B: int) -> int:
    torch = _torch()
    if slot.dtype != torch.int32 or slot.numel() != B:
        raise ValueError(f"slot must be int32 with {B} entries")
    return _ptr(slot, "slot")


def dl_pool_step(pool: Pool, slot, q, k, v, beta, a, o, stream=None) -> None:
    """One decode step of the batch rows ``slot`` [B] int32 of the pool
    (inputs and o are [B,H,...]); each row appends or, on its L-th entry,
    merges, following its own log count."""
    B, H, dk = int(q.shape[0]), int(q.shape[1]), int(q.shape[2])
    dv = int(pool.S.shape[2])  # (an I8State has .shape too)
    _check_shapes(B, H, dk, dv, q, k, v, beta, a, o, pool.log.channel_decay)
    ps = pool.struct()
    status = load().dl_pool_step(ctypes.byref(ps), pool.log.kind, _slots(slot, B), _ptr(q, "q"), _ptr(k, "k"),
                                 _ptr(v, "v"), _ptr(beta, "beta", pool.log.rwkv6), _ptr(a, "a"),
                                 _in_dtype(q, k, v, beta, a), _ptr(o, "o"), B, H, dk, dv, _stream(stream))
    check("dl_pool_step", status)


def dl_pool_flush(pool: Pool, slot, stream=None) -> None:
    """Merge the listed slots' logs into their bases and zero their counts."""
    B = int(slot.numel())
    _, H, dv, dk = (int(x) for x in pool.S.shape)
    ps = pool.struct()
    status = load().dl_pool_flush(ctypes.byref(ps), pool.log.kind, _slots(slot, B), B, H, dk, dv, _stream(stream))
    check("dl_pool_flush", status)


# ------------------------------------------------------------------ norm, short convolution, selective scan

# (These calls take a dozen tensors and a kernel of a few microseconds: what is
# checked of a tensor is checked in one function, by the cheapest queries.)

_found = None


def _queries():
    """torch's dtypes -> dl_dtype, its queries of the current device and of a device's current stream, and its int32:
    looked up once, and set together, so that another thread's first call sees all of them or none."""
    global _found
    torch = _torch()
    codes = {torch.float32: DL_F32, torch.bfloat16: DL_BF16, torch.int8: DL_I8, torch.float8_e4m3fn: DL_E4M3}
    # (torch's own, which cost a microsecond less a call; its public ones where a torch has not these)
    device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
    stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (lambda dev: torch.cuda.current_stream(dev).cuda_stream)
    _found = codes, device, stream, torch.int32
    return _found


def _code_of(t) -> int:
    """dl_dtype of a tensor (as _dtype_code, 8-bit types too)."""
    code = (_found or _queries())[0].get(t.dtype)
    if code is None:
        raise TypeError(f"unsupported dtype {t.dtype}")
    return code


def _float_code(*ts) -> int:
    """The one dl_dtype, float32 or bfloat16, of the tensors that are not None."""
    dtype = ts[0].dtype
    for t in ts:
        if t is not None and t.dtype is not dtype:
            raise TypeError("these operands must share one dtype: " + ", ".join(str(u.dtype) for u in ts if u is not None))
    code = _code_of(ts[0])
    if code > DL_BF16:
        raise TypeError(f"unsupported dtype {dtype} (float32 or bfloat16)")
    return code


def _device() -> int:
    """The current device: a call launches there, and every operand must lie on it."""
    return (_found or _queries())[1]()


def _misplaced(t, name: str, dev: int):
    if not t.is_cuda:
        return ValueError(f"{name} must be a CUDA tensor")
    return ValueError(f"{name} lies on {t.device}, but the current device is cuda:{dev}")


def _raw_stream(stream, dev: int) -> int:
    return (_found or _queries())[2](dev) if stream is None else _stream(stream)


_INT = 0x7fffffff  # the C ABI's largest int: ctypes would drop the upper bits of a larger one


def _too_large(*sizes):
    return ValueError(f"a size of {max(sizes)} exceeds 2^31 - 1")


def _full(t, name: str, shape, dev: int) -> int:
    """Pointer of a contiguous tensor of the given shape on the current device."""
    if t.get_device() == dev and t.shape == shape and t.is_contiguous():
        return t.data_ptr()
    if t.get_device() != dev:
        raise _misplaced(t, name, dev)
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    raise ValueError(f"{name} must be contiguous")


def _f32(t, name: str, shape, dev: int) -> Optional[int]:
    """The same of a float32 tensor, or None."""
    if t is None:
        return None
    if (_found or _queries())[0].get(t.dtype) != DL_F32:
        raise TypeError(f"{name} must be float32, got {t.dtype}")
    return _full(t, name, shape, dev)


def _rows(t, name: str, shape, dev: int, width: int):
    """Pointer and row stride of a tensor whose rows (all dimensions but the first, of `width` elements) are contiguous."""
    if t.get_device() != dev:
        raise _misplaced(t, name, dev)
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    if t.is_contiguous():
        return t.data_ptr(), width or 1
    inner = 1
    strides = t.stride()
    for k in range(len(shape) - 1, 0, -1):
        if shape[k] != 1 and strides[k] != inner:
            raise ValueError(f"the rows of {name} must be contiguous")
        inner *= shape[k]
    return t.data_ptr(), strides[0] if shape[0] > 1 else width or 1


def _index(t, name: str, n: int, dev: int) -> Optional[int]:
    """Pointer of an int32 tensor of n elements, or None."""
    if t is None:
        return None
    if t.dtype is not (_found or _queries())[3]:
        raise TypeError(f"{name} must be int32, got {t.dtype}")
    return _full(t, name, (n,), dev)


def dl_rms_norm(x, weight, eps: float, y, residual=None, residual_out=None, scale=None, group: int = 0,
                stream=None) -> None:
    """y = h / sqrt(mean(h^2) + eps) * weight over the rows of x [rows, width]
    (rows may be strided), h = x or, with ``residual``, x + residual, which
    ``residual_out`` receives (it may be ``residual``). y is float32, bfloat16, or
    int8 / float8_e4m3fn codes with float32 ``scale`` [rows] (``group`` 0) or
    [rows, ceil(width / 128)] (``group`` 128)."""
    if x.dim() != 2:
        raise ValueError("x must be [rows, width]")
    dev = _device() if x.is_cuda else -2
    rows, width = shape = x.shape
    if width > _INT:
        raise _too_large(width)
    xp, xs = _rows(x, "x", shape, dev, width)
    xc, yc = _float_code(x), _code_of(y)
    if (residual is None) != (residual_out is None):
        raise ValueError("residual and residual_out go together")
    rp = rop = sp = None
    rc = DL_F32
    if residual is not None:
        rc = _float_code(residual, residual_out)
        rp, rop = _full(residual, "residual", shape, dev), _full(residual_out, "residual_out", shape, dev)
    if scale is not None:
        sp = _scales(scale, rows, width, group, dev)
    elif yc > DL_BF16:
        raise ValueError("an 8-bit y needs a scale")
    status = load().dl_rms_norm(xp, xc, xs, rp, rop, rc, _full(weight, "weight", (width,), dev), _float_code(weight), eps,
                                _full(y, "y", shape, dev), yc, sp, group, rows, width, _raw_stream(stream, dev))
    if status:
        check("dl_rms_norm", status)


def _scales(scale, rows: int, width: int, group: int, dev: int) -> int:
    n = rows * (-(-width // group) if group > 0 else 1)
    if scale.numel() != n:
        raise ValueError(f"scale has {scale.numel()} elements, expected {n} (rows x groups)")
    return _f32(scale, "scale", scale.shape, dev)


def dl_rows_from_8bit(codes, scale, out, group: int = 0, stream=None) -> None:
    """The values code * scale of dl_rms_norm's 8-bit rows into ``out`` (float32 or bfloat16)."""
    if codes.dim() != 2:
        raise ValueError("codes must be [rows, width]")
    dev = _device() if codes.is_cuda else -2
    rows, width = shape = codes.shape
    if width > _INT:
        raise _too_large(width)
    status = load().dl_rows_from_8bit(_full(codes, "codes", shape, dev), _code_of(codes), _scales(scale, rows, width, group, dev),
                                      group, _full(out, "out", shape, dev), _float_code(out), rows, width,
                                      _raw_stream(stream, dev))
    if status:
        check("dl_rows_from_8bit", status)


def _conv(x, w, bias, state, y, silu, dev):
    if x.dim() != 2 or w.dim() != 2 or state.dim() != 3:
        raise ValueError("x must be [rows, channels], w [channels, taps], state [P, taps - 1, channels]")
    rows, channels = shape = x.shape
    taps, P = w.shape[1], state.shape[0]
    if (rows | channels | taps | P) > _INT:
        raise _too_large(rows, channels, taps, P)
    xp, xs = _rows(x, "x", shape, dev, channels)
    cv = dl_conv(_full(w, "w", (channels, taps), dev), None if bias is None else _full(bias, "bias", (channels,), dev), channels,
                 taps, _float_code(x, w, bias, state, y), 1 if silu else 0)
    return cv, xp, xs, rows, _full(state, "state", (P, taps - 1, channels), dev), P, _full(y, "y", shape, dev)


def dl_conv_prompt(x, w, bias, state, seq_start, slot, y, silu: bool = True, status=None, stream=None) -> None:
    """Short causal convolution over ragged prompts: x [T, channels] (rows may be
    strided), w [channels, taps], bias [channels] or None, state [P, taps - 1,
    channels] (each slot's last inputs, read and replaced), seq_start [n + 1]
    int32, slot [n] int32 or None, y [T, channels]."""
    dev = _device() if x.is_cuda else -2
    cv, xp, xs, T, sp, P, yp = _conv(x, w, bias, state, y, silu, dev)
    n = seq_start.numel() - 1
    if n > _INT:
        raise _too_large(n)
    st = load().dl_conv_prompt(ctypes.byref(cv), xp, xs, T, _index(seq_start, "seq_start", n + 1, dev), n, sp, P,
                               _index(slot, "slot", n, dev), _index(status, "status", 1, dev), yp, _raw_stream(stream, dev))
    if st:
        check("dl_conv_prompt", st)


def dl_conv_step(x, w, bias, state, slot, y, silu: bool = True, status=None, stream=None) -> None:
    """The convolution of one new token per sequence: x, y [B, channels], slot [B] int32 or None."""
    dev = _device() if x.is_cuda else -2
    cv, xp, xs, B, sp, P, yp = _conv(x, w, bias, state, y, silu, dev)
    st = load().dl_conv_step(ctypes.byref(cv), xp, xs, B, sp, P, _index(slot, "slot", B, dev),
                             _index(status, "status", 1, dev), yp, _raw_stream(stream, dev))
    if st:
        check("dl_conv_step", st)


def _ssm(S, x, dt, A, b, c, y, D, dt_bias, z, dev):
    if x.dim() != 3 or b.dim() != 3 or S.dim() != 4:
        raise ValueError("S must be [P, H, d_v, d_k], x [rows, H, d_v], b and c [rows, G, d_k]")
    P, H, dv, dk = s_shape = S.shape
    rows, G = x.shape[0], b.shape[1]
    if (P | H | dv | dk | rows | G) > _INT:
        raise _too_large(P, H, dv, dk, rows, G)
    wide, keys, heads = (rows, H, dv), (rows, G, dk), (H,)
    zp, zs = (None, 0) if z is None else _rows(z, "z", wide, dev, H * dv)
    xp, xs = _rows(x, "x", wide, dev, H * dv)
    tp, ts = _rows(dt, "dt", (rows, H), dev, H)
    bp, bs = _rows(b, "b", keys, dev, G * dk)
    cp, cs = _rows(c, "c", keys, dev, G * dk)
    if A is None:
        raise ValueError("A is required")
    m = dl_ssm(xp, xs, tp, ts, bp, bs, cp, cs, zp, zs, _f32(A, "A", heads, dev), _f32(D, "D", heads, dev),
               _f32(dt_bias, "dt_bias", heads, dev), _float_code(x, dt, b, c, y, z))
    return m, P, H, G, dk, dv, rows, _full(y, "y", wide, dev), _full(S, "S", s_shape, dev), _float_code(S)


def dl_ssm_work_bytes(T: int, n_seq: int, H: int, d_k: int, d_v: int) -> int:
    """Bytes of workspace dl_ssm_prompt needs (0 if none)."""
    if max(T, n_seq, H, d_k, d_v) > _INT:
        raise _too_large(T, n_seq, H, d_k, d_v)
    return int(load().dl_ssm_work_bytes(int(T), int(n_seq), int(H), int(d_k), int(d_v)))


def dl_ssm_prompt(S, seq_start, slot, x, dt, A, b, c, y, D=None, dt_bias=None, z=None, work=None, status=None,
                  stream=None) -> None:
    """Selective scan over ragged prompts from and into the slots' states S
    [P, H, d_v, d_k] (float32 or bfloat16): x, y (and the gate z) [T, H, d_v], dt
    [T, H], b, c [T, G, d_k] (rows may be strided; y is contiguous), A, D, dt_bias
    [H] float32, seq_start [n + 1] int32, slot [n] int32 or None, work a tensor of
    dl_ssm_work_bytes(T, n, H, d_k, d_v) bytes."""
    dev = _device() if x.is_cuda else -2
    m, P, H, G, dk, dv, T, yp, Sp, sc = _ssm(S, x, dt, A, b, c, y, D, dt_bias, z, dev)
    n = seq_start.numel() - 1
    if n > _INT:
        raise _too_large(n)
    wp, wb = None, 0
    if work is not None and work.numel():
        wp, wb = _full(work, "work", work.shape, dev), work.numel() * work.element_size()
    st = load().dl_ssm_prompt(Sp, sc, P, _index(slot, "slot", n, dev), _index(status, "status", 1, dev), ctypes.byref(m),
                              _index(seq_start, "seq_start", n + 1, dev), n, T, yp, H, G, dk, dv, wp, wb,
                              _raw_stream(stream, dev))
    if st:
        check("dl_ssm_prompt", st)


def dl_ssm_step(S, slot, x, dt, A, b, c, y, D=None, dt_bias=None, z=None, status=None, stream=None) -> None:
    """The scan of one new token per sequence: x, y (z) [B, H, d_v], dt [B, H], b, c [B, G, d_k], slot [B] int32 or None."""
    dev = _device() if x.is_cuda else -2
    m, P, H, G, dk, dv, B, yp, Sp, sc = _ssm(S, x, dt, A, b, c, y, D, dt_bias, z, dev)
    st = load().dl_ssm_step(Sp, sc, P, _index(slot, "slot", B, dev), _index(status, "status", 1, dev), ctypes.byref(m), yp, B, H,
                            G, dk, dv, _raw_stream(stream, dev))
    if st:
        check("dl_ssm_step", st)
