"""GPU tests of the norm, the short convolution and the selective scan against
64-bit references (tests/layer_ref.py).

Tolerances count roundings. With u = 2^-24 (half a float32 step) and h half a
step of the output type (u, or 2^-8 for bfloat16):
  norm    y = h r w: h is one rounding, the mean of squares a sum of positive
          terms in chains of at most 32 + 10 additions (halved by the square
          root), two operations of a few units after it: 32 u relative, plus h.
          A code is off by half its step: scale / 2 (int8), 2^-4 of the value or
          2^-10 scale (e4m3, half of its smallest step), each plus 2^-12 of a
          step's size for the float32 value and scale behind it.
  conv    the sum's terms, taps + 1 roundings: (taps + 2) u of their
          magnitudes, times at most 1.1 (the slope of u / (1 + exp(-u))); the
          activation itself 8 u, or 64 u with the fast exponential and division
          (|u| <= 16 here), plus h.
  scan    the reference sums along the recurrence what one relative error unit
          per step makes of each state and output; a step rounds its decay
          (softplus, product, exponential: 8 units), its addend and its sum
          (4): 12 u of that sum, plus d_k u of the magnitudes for the read's
          sum, plus 8 u (64 u when the gate is the fast one) and h of the
          output.
          bfloat16 prompts multiply on tensor cores: there the scores times
          decay, the state read and the decayed addends are rounded to
          bfloat16 (or two of them for the state): 2 * 2^-8 of the magnitudes in
          y and 2 * 2^-17 of them in the state.
"""
import pytest

from tests import layer_ref as R

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16
FAST = {F32: 8, BF16: 64}


@pytest.fixture(scope="module", autouse=True)
def g():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import gated_delta_rule_104_b200 as g

    g.load()
    return g


@pytest.fixture(autouse=True)
def _no_wait_ran_out(request, g):
    yield
    if "ssm" in request.node.name or "layer" in request.node.name:
        assert g.dl_device_faults(clear=True) == 0


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(rng, *shape):
    return torch.randn(*shape, generator=rng, device="cuda")


# ------------------------------------------------------------------ norm

def check_norm(g, x, weight, res, out, group=0, eps=1e-5, in_place=False):
    rows, width = x.shape
    y = torch.zeros(rows, width, dtype=out, device="cuda")
    groups = -(-width // group) if group else 1
    scale = torch.full((rows, groups), -1.0, device="cuda") if out in (torch.int8, torch.float8_e4m3fn) else None
    h, want = R.norm(x, res, weight, eps)
    res_out = None if res is None else (res if in_place else torch.zeros_like(res))
    g.dl_rms_norm(x, weight, eps, y, residual=res, residual_out=res_out, scale=scale, group=group)
    if res is not None:
        R.assert_within(res_out, h, R.half_step(res.dtype) * 1.001 * h.abs() + 1e-40, "residual")
    if scale is None:
        R.assert_within(y, want, (32 * R.U32 + R.half_step(out)) * want.abs() + 1e-38, "y")
        return y
    span = group or width
    padded = torch.nn.functional.pad(want, (0, -width % span)).view(rows, groups, span)
    s_want = padded.abs().amax(2) / (127 if out == torch.int8 else 448)
    R.assert_within(scale, s_want, 40 * R.U32 * s_want + 1e-44, "scale")
    step = s_want.repeat_interleave(span, 1)[:, :width]
    vals = torch.zeros(rows, width, device="cuda")
    g.dl_rows_from_8bit(y, scale, vals, group=group)
    off = 0.5 * step if out == torch.int8 else torch.maximum(2.0 ** -4 * want.abs(), 2.0 ** -10 * step)
    R.assert_within(vals, want, off * (1 + 2.0 ** -12) + 2.0 ** -12 * want.abs() * 2.0 ** -8, "values")
    low = torch.zeros(rows, width, dtype=BF16, device="cuda")
    g.dl_rows_from_8bit(y, scale, low, group=group)
    assert torch.equal(low, vals.to(BF16))
    direct = y.float() * scale.repeat_interleave(span, 1)[:, :width]
    assert torch.equal(vals, direct)
    return y


@pytest.mark.parametrize("out", [F32, BF16, torch.int8, torch.float8_e4m3fn])
@pytest.mark.parametrize("rows,width", [(1, 1), (3, 31), (9, 128), (257, 129), (5, 256), (4, 1000), (3, 4096), (2, 5000),
                                        (2, 8193), (2, 16384), (1, 16385), (1, 32768)])
def test_norm(g, rows, width, out):
    rng = gen(rows * 40000 + width)
    for i, (xt, rt) in enumerate([(BF16, None), (F32, BF16), (BF16, F32), (BF16, BF16)]):
        x = randn(rng, rows, width).to(xt)
        res = None if rt is None else (3 * randn(rng, rows, width)).to(rt)
        w = (1 + 0.2 * randn(rng, width)).to(BF16 if i % 2 else F32)
        for group in ([0, 128] if out in (torch.int8, torch.float8_e4m3fn) else [0]):
            check_norm(g, x, w, res, out, group)


def test_norm_strided_misaligned_and_in_place(g):
    rng = gen(1)
    buf = randn(rng, 70, 700).to(BF16)
    w = randn(rng, 256)
    for first in (0, 8, 1, 3):  # rows of a wider buffer: aligned ones and not
        y0 = check_norm(g, buf[:, first:first + 256], w, None, BF16)
        assert torch.equal(y0, check_norm(g, buf[:, first:first + 256].contiguous(), w, None, BF16))
    res = randn(rng, 70, 256).to(BF16)
    check_norm(g, buf[:, :256], w, res, torch.int8, in_place=True)


def test_norm_rows_of_zeros_and_of_no_number(g):
    x = torch.randn(6, 512, device="cuda")
    x[1] = 0
    x[2, 7], x[3, 300], x[4] = float("nan"), float("inf"), 1e-30
    w = torch.ones(512, device="cuda")
    for out in (F32, torch.int8, torch.float8_e4m3fn):
        for group in (0, 128) if out != F32 else (0,):
            y = torch.zeros(6, 512, dtype=out, device="cuda")
            scale = torch.zeros(6, 4 if group else 1, device="cuda") if out != F32 else None
            g.dl_rms_norm(x, w, 1e-6, y, scale=scale, group=group)
            if out != F32:
                v = torch.zeros(6, 512, device="cuda")
                g.dl_rows_from_8bit(y, scale, v, group=group)
                assert bool(torch.isnan(scale[2]).all()) and bool(torch.isnan(scale[3]).any())
                y = v
            assert bool((y[1] == 0).all()) and bool(torch.isnan(y[2]).all()) and bool(torch.isnan(y[3, 300]))
            assert bool(torch.isfinite(y[[0, 1, 4, 5]]).all())


def test_norm_without_rows(g):
    e = torch.zeros(0, 64, device="cuda")
    g.dl_rms_norm(e, torch.ones(64, device="cuda"), 1e-5, e.clone())


def test_binding_refuses_what_does_not_fit(g):
    x, w, h = torch.zeros(2, 64, device="cuda"), torch.zeros(64, device="cuda"), torch.zeros(2, 64)
    q = torch.zeros(2, 64, dtype=torch.int8, device="cuda")
    bad = [(ValueError, "8-bit y", lambda: g.dl_rms_norm(x, w, 1e-5, q)),
           (ValueError, "go together", lambda: g.dl_rms_norm(x, w, 1e-5, x.clone(), residual=x)),
           (ValueError, "scale has", lambda: g.dl_rms_norm(x, w, 1e-5, q, scale=w)),
           (TypeError, "float32", lambda: g.dl_rms_norm(x, w, 1e-5, q, scale=torch.zeros(2, dtype=BF16, device="cuda"))),
           (ValueError, "CUDA tensor", lambda: g.dl_rms_norm(x, w, 1e-5, h)),
           (ValueError, "contiguous", lambda: g.dl_rms_norm(x.t(), w[:2], 1e-5, torch.zeros(64, 2, device="cuda"))),
           (TypeError, "unsupported", lambda: g.dl_rms_norm(x.half(), w, 1e-5, x.clone())),
           (TypeError, "share one dtype", lambda: g.dl_conv_step(x, torch.zeros(64, 4, device="cuda", dtype=BF16), None,
                                                                 torch.zeros(2, 3, 64, device="cuda"), None, x.clone())),
           (TypeError, "int32", lambda: g.dl_conv_step(x, torch.zeros(64, 4, device="cuda"), None, torch.zeros(2, 3, 64, device="cuda"),
                                                       torch.zeros(2, dtype=torch.int64, device="cuda"), x.clone())),
           (ValueError, "state must be", lambda: g.dl_conv_step(x, torch.zeros(64, 4, device="cuda"), None,
                                                                torch.zeros(2, 2, 64, device="cuda"), None, x.clone())),
           (g.DeltaLogError, "overlaps", lambda: g.dl_rms_norm(x, w, 1e-5, x))]
    for kind, text, call in bad:
        with pytest.raises(kind, match=text):
            call()


# ------------------------------------------------------------------ convolution

def starts(lens, first=0):
    s = [first]
    for n in lens:
        s.append(s[-1] + n)
    return s, torch.tensor(s, dtype=torch.int32, device="cuda")


LENS = [[1], [2, 0, 1, 3], [31, 32, 33], [100, 0, 64, 7, 1, 200]]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("taps", [2, 3, 4])
@pytest.mark.parametrize("channels,stride", [(1, 1), (13, 20), (64, 64), (264, 400)])
def test_conv_prompt(g, channels, stride, taps, dtype):
    for k, lens in enumerate(LENS):
        rng = gen(1000 * channels + 10 * taps + k)
        first = k % 3
        s, seq_start = starts(lens, first)
        T = s[-1] + 2
        x = randn(rng, T, stride).to(dtype)[:, :channels]
        w = randn(rng, channels, taps).to(dtype)
        bias = None if k % 2 else randn(rng, channels).to(dtype)
        act = k != 2
        P = len(lens) + 2
        slot = torch.randperm(P, generator=rng, device="cuda")[:len(lens)].to(torch.int32)
        state = randn(rng, P, taps - 1, channels).to(dtype)
        old = state.clone()
        y = torch.full((T, channels), 7.0, dtype=dtype, device="cuda")
        g.dl_conv_prompt(x, w, bias, state, seq_start, slot, y, silu=act)
        for i, n in enumerate(lens):
            line = torch.cat([old[slot[i].item()], x[s[i]:s[i + 1]]])
            want, mag = R.conv(line, w, bias, act)
            bound = 1.1 * (taps + 2) * R.U32 * mag + (FAST[dtype] * R.U32 + R.half_step(dtype)) * want.abs() + 1e-38
            R.assert_within(y[s[i]:s[i + 1]], want, bound, f"sequence {i}")
            assert torch.equal(state[slot[i].item()], line[n:])
        assert bool((y[:first] == 7).all()) and bool((y[s[-1]:] == 7).all())
        others = [p for p in range(P) if p not in slot.tolist()]
        assert torch.equal(state[others], old[others])


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("taps", [2, 3, 4])
@pytest.mark.parametrize("channels", [1, 13, 64, 264])
def test_conv_steps_continue_a_prompt(g, channels, taps, dtype):
    """A prompt cut anywhere, then single tokens: the same bits as the whole prompt."""
    rng = gen(channels + taps)
    n, B = 40, 3
    x = randn(rng, B, n, channels).to(dtype)
    w, bias = randn(rng, channels, taps).to(dtype), randn(rng, channels).to(dtype)
    whole = torch.zeros(B * n, channels, dtype=dtype, device="cuda")
    state = torch.zeros(B, taps - 1, channels, dtype=dtype, device="cuda")
    last = state.clone()
    _, seq = starts([n] * B)
    g.dl_conv_prompt(x.reshape(B * n, channels), w, bias, last, seq, None, whole)
    cut = [1, 35, 37]
    s, seq = starts(cut)
    part = torch.zeros(s[-1], channels, dtype=dtype, device="cuda")
    g.dl_conv_prompt(torch.cat([x[i, :cut[i]] for i in range(B)]), w, bias, state, seq, None, part)
    got = [[part[s[i] + t] for t in range(cut[i])] for i in range(B)]
    for _ in range(n):
        slot = torch.tensor([i if len(got[i]) < n else -1 for i in range(B)], dtype=torch.int32, device="cuda")
        step = torch.stack([x[i, min(len(got[i]), n - 1)] for i in range(B)])
        y = torch.full((B, channels), 7.0, dtype=dtype, device="cuda")
        g.dl_conv_step(step, w, bias, state, slot, y)
        for i in range(B):
            if len(got[i]) < n:
                got[i].append(y[i])
            else:
                assert bool((y[i] == 7).all())
    assert torch.equal(torch.stack([torch.stack(r) for r in got]).view(B * n, channels), whole)
    assert torch.equal(state, last)


# ------------------------------------------------------------------ scan

def scan_inputs(rng, rows, H, G, dk, dv, dtype, gate, decay=1.0):
    u = randn(rng, rows, H * dv + 2 * G * dk)
    u = (u * torch.sigmoid(u)).to(dtype)
    return dict(x=u[:, :H * dv].view(rows, H, dv), b=u[:, H * dv:H * dv + G * dk].view(rows, G, dk),
                c=u[:, H * dv + G * dk:].view(rows, G, dk), dt=randn(rng, rows, H).to(dtype),
                A=-decay * (0.5 + 8 * torch.rand(H, generator=rng, device="cuda")), D=randn(rng, H),
                dt_bias=randn(rng, H) - 3, z=randn(rng, rows, H, dv).to(dtype) if gate else None)


def scan_bounds(r, dtype, s_dtype, dk, products=False):
    """Tolerances of y and the state; `products`: the bfloat16 prompt's tensor-core products."""
    u = R.U32
    y = 12 * u * r["y_err"] + dk * u * r["y_mag"] + (FAST[dtype] * u + R.half_step(dtype)) * r["y"].abs() + 1e-38
    S = 12 * u * r["S_err"] + R.half_step(s_dtype) * r["S"].abs() + 1e-38
    if products:
        y, S = y + 2 * 2.0 ** -8 * r["y_mag"], S + 2 * 2.0 ** -17 * r["S_mag"]
    return y, S


def run_prompt(g, S, seq_start, slot, m, y, **k):
    T, H, dv = m["x"].shape
    dk, n = m["b"].shape[2], seq_start.numel() - 1
    work = torch.empty(g.dl_ssm_work_bytes(T, n, H, dk, dv), dtype=torch.uint8, device="cuda")
    g.dl_ssm_prompt(S, seq_start, slot, m["x"], m["dt"], m["A"], m["b"], m["c"], y, D=m["D"], dt_bias=m["dt_bias"], z=m["z"],
                    work=work, **k)


def at(m, rows):
    return {k: (v if v is None or k in ("A", "D", "dt_bias") else v[rows]) for k, v in m.items()}


def check_prompt(g, lens, H, G, dk, dv, dtype, s_dtype, gate, seed, decay=1.0, first=0, change=None):
    rng = gen(seed)
    s, seq_start = starts(lens, first)
    T, P = s[-1] + 3, len(lens) + 2
    m = scan_inputs(rng, T, H, G, dk, dv, dtype, gate, decay)
    if change:
        change(m)
    slot = torch.randperm(P, generator=rng, device="cuda")[:len(lens)].to(torch.int32)
    S = (0.5 * randn(rng, P, H, dv, dk)).to(s_dtype)
    old = S.clone()
    y = torch.full((T, H, dv), 7.0, dtype=dtype, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    run_prompt(g, S, seq_start, slot, m, y, status=status)
    assert int(status) == 0
    for i, n in enumerate(lens):
        k = int(slot[i])
        if n == 0:
            assert torch.equal(S[k], old[k])
            continue
        r = R.scan(old[k], **at(m, slice(s[i], s[i + 1])))
        by, bS = scan_bounds(r, dtype, s_dtype, dk, dtype == BF16)
        R.assert_within(y[s[i]:s[i + 1]], r["y"], by, f"y of sequence {i}")
        R.assert_within(S[k], r["S"], bS, f"state of sequence {i}")
    assert bool((y[:first] == 7).all()) and bool((y[s[-1]:] == 7).all())
    others = [p for p in range(P) if p not in slot.tolist()]
    assert torch.equal(S[others], old[others])


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("s_dtype", [F32, BF16])
@pytest.mark.parametrize("dk", [64, 128])
@pytest.mark.parametrize("dv", [64, 128, 256])
def test_ssm_prompt_shapes_and_types(g, dk, dv, dtype, s_dtype):
    check_prompt(g, [70, 1, 0, 130], 4, 2, dk, dv, dtype, s_dtype, gate=dv == 128, seed=dk + dv)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("lens", [[1], [2], [15], [16], [17], [63], [64], [65], [127], [128], [129], [300], [1, 1, 1, 0, 0, 5, 200]],
                         ids=str)
def test_ssm_prompt_lengths(g, lens, dtype):
    check_prompt(g, lens, 3, 1, 128, 64, dtype, F32, gate=len(lens) > 1, seed=sum(lens), first=len(lens) - 1)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("s_dtype", [F32, BF16])
@pytest.mark.parametrize("lens,H,G,dk,dv", [([2600], 2, 1, 128, 128), ([2600], 3, 1, 64, 64), ([3, 2300, 0, 1, 1025, 513, 512, 511], 1, 1, 128, 64),
                                            ([1537, 700, 2048], 2, 2, 64, 256)], ids=str)
def test_ssm_prompt_split_over_its_length(g, lens, H, G, dk, dv, s_dtype, dtype):
    """Few heads and long sequences: segments run side by side from states formed first."""
    if dtype == BF16:
        assert g.dl_ssm_work_bytes(sum(lens) + 3, len(lens), H, dk, dv) > 0
    check_prompt(g, lens, H, G, dk, dv, dtype, s_dtype, gate=dk == 64, seed=H + dv, decay=0.02)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("decay", [1e-6, 0.02, 30.0, 3000.0])
def test_ssm_prompt_weak_and_strong_decay(g, decay, dtype):
    check_prompt(g, [150, 9], 2, 1, 64, 64, dtype, F32, gate=False, seed=5, decay=decay)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_ssm_prompt_without_decay_and_with_one_that_forgets_all(g, dtype):
    def change(m):
        m["A"][0] = 0.0
        m["dt"][3] = 500.0      # exp(dt A) = 0: the state starts again (from a large addend)
        m["dt"][20:30] = -200.0  # dt = 0: those tokens leave the state as it is
        m["D"] = m["dt_bias"] = None

    check_prompt(g, [90], 2, 2, 64, 64, dtype, F32, gate=False, seed=6, change=change)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("at", [0, 3, 40, 127])
def test_ssm_prompt_behind_a_step_of_a_million(g, at, dtype):
    """A step whose log decay is -1e6, then steps of -0.01: sums from the chunk's start must not swallow those."""
    def change(m):
        m["A"][:] = -2000.0
        m["dt"][:] = -12.0  # dt = 6e-6
        m["dt"][at] = 500.0
        m["dt_bias"] = None

    check_prompt(g, [200], 2, 1, 64, 64, dtype, F32, gate=False, seed=21, change=change)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_ssm_prompt_keeps_what_is_no_number_where_it_belongs(g, dtype, bad):
    """A NaN or infinity in x at one token and channel, b, c or dt at others: the
    tokens before, the other channels (for x), heads and sequences stay as they were."""
    rng = gen(9)
    H, dk, dv, lens = 2, 64, 64, [100, 100]
    s, seq_start = starts(lens)
    m = scan_inputs(rng, s[-1] + 60, H, 2, dk, dv, dtype, False)
    S0 = 0.5 * randn(rng, 2, H, dv, dk)

    def run(m):
        S, y = S0.clone(), torch.zeros_like(m["x"]).contiguous()
        run_prompt(g, S, seq_start, None, m, y)
        return S, y

    S, y = run(m)
    for name, head_wide in (("x", False), ("b", True), ("c", True), ("dt", True)):
        m2 = {k: (v.clone() if v is not None else None) for k, v in m.items()}
        m2["x"][s[-1]:] = m2["b"][s[-1]:] = m2["c"][s[-1]:] = float("nan")  # rows behind the last sequence
        m2["dt"][s[-1]:] = float("nan")
        m2[name][40, 0, *([5] if name != "dt" else [])] = bad
        S2, y2 = run(m2)
        assert torch.equal(y2[100:s[-1]], y[100:s[-1]]) and torch.equal(S2[1], S[1]), name
        assert torch.equal(y2[:40], y[:40]) and torch.equal(y2[:, 1], y[:, 1]) and torch.equal(S2[0, 1], S[0, 1]), name
        assert bool((y2[s[-1]:] == 0).all())
        if name == "c":  # a read only: one token
            assert torch.equal(S2, S) and torch.equal(y2[41:], y[41:]) and not bool(torch.isfinite(y2[40, 0]).any())
        if name == "x":
            keep = [e for e in range(dv) if e != 5]
            assert torch.equal(y2[:, 0, keep], y[:, 0, keep]) and torch.equal(S2[0, 0, keep], S[0, 0, keep])
            assert not bool(torch.isfinite(y2[40:100, 0, 5]).any()) and not bool(torch.isfinite(S2[0, 0, 5]).any())
        if name == "b":
            assert not bool(torch.isfinite(S2[0, 0, :, 5]).any()) and torch.equal(S2[0, 0, :, :5], S[0, 0, :, :5])


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("s_dtype", [F32, BF16])
@pytest.mark.parametrize("dk", [64, 128])
@pytest.mark.parametrize("B,H,G,dv", [(1, 1, 1, 64), (3, 6, 2, 128), (37, 5, 5, 64), (2, 4, 1, 256)])
def test_ssm_step(g, B, H, G, dv, dk, s_dtype, dtype):
    rng = gen(B + dv + dk)
    P = B + 3
    S = (0.5 * randn(rng, P, H, dv, dk)).to(s_dtype)
    slot = torch.randperm(P, generator=rng, device="cuda")[:B].to(torch.int32)
    for gate in (False, True):
        old = S.clone()
        m = scan_inputs(rng, B, H, G, dk, dv, dtype, gate)
        y = torch.zeros(B, H, dv, dtype=dtype, device="cuda")
        g.dl_ssm_step(S, slot, m["x"], m["dt"], m["A"], m["b"], m["c"], y, D=m["D"], dt_bias=m["dt_bias"], z=m["z"])
        for i in range(B):
            r = R.scan(old[int(slot[i])], **at(m, slice(i, i + 1)))
            by, bS = scan_bounds(r, dtype, s_dtype, dk)
            R.assert_within(y[i:i + 1], r["y"], by, "y")
            R.assert_within(S[int(slot[i])], r["S"], bS, "state")
        others = [p for p in range(P) if p not in slot.tolist()]
        assert torch.equal(S[others], old[others])


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_ssm_prompt_in_chunks_then_steps(g, dtype):
    """A prompt continued from its slot, then single tokens, against one recurrence."""
    rng = gen(11)
    H, dk, dv, n = 4, 128, 128, 150
    m = scan_inputs(rng, n, H, 1, dk, dv, dtype, True)
    S = 0.5 * randn(rng, 3, H, dv, dk)
    r = R.scan(S[2], **m)
    slot = torch.tensor([2], dtype=torch.int32, device="cuda")
    y = torch.zeros(n, H, dv, dtype=dtype, device="cuda")
    for a, z in ((0, 70), (70, 71), (71, 140)):
        part = at(m, slice(a, z))
        run_prompt(g, S, torch.tensor([0, z - a], dtype=torch.int32, device="cuda"), slot, part, y[a:z])
    for t in range(140, n):
        p = at(m, slice(t, t + 1))
        g.dl_ssm_step(S, slot, p["x"], p["dt"], p["A"], p["b"], p["c"], y[t:t + 1], D=p["D"], dt_bias=p["dt_bias"], z=p["z"])
    by, bS = scan_bounds(r, dtype, F32, dk, dtype == BF16)
    R.assert_within(y, r["y"], by, "y")
    R.assert_within(S[2], r["S"], bS, "state")


# ------------------------------------------------------------------ slots, status, streams, graphs

def test_rows_without_a_slot_are_skipped_and_flagged(g):
    rng = gen(12)
    H, dk, dv, C = 2, 64, 64, 256
    m = scan_inputs(rng, 12, H, 1, dk, dv, F32, False)
    S, state = randn(rng, 2, H, dv, dk), randn(rng, 3, 3, C)
    x, w = randn(rng, 12, C), randn(rng, C, 4)
    for bad in (-1, 9):
        slot = torch.tensor([bad, 1], dtype=torch.int32, device="cuda")
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        _, seq = starts([5, 7])
        S1, c1 = S.clone(), state.clone()
        y, yc = torch.full((12, H, dv), 7.0, device="cuda"), torch.full((12, C), 7.0, device="cuda")
        run_prompt(g, S1, seq, slot, m, y, status=status)
        assert int(status) == 1
        status.zero_()
        g.dl_conv_prompt(x, w, None, c1, seq, slot, yc, status=status)
        assert int(status) == 1
        assert bool((y[:5] == 7).all()) and bool((y[5:] != 7).any()) and bool((yc[:5] == 7).all())
        assert torch.equal(S1[0], S[0]) and not torch.equal(S1[1], S[1])
        assert torch.equal(c1[[0, 2]], state[[0, 2]]) and not torch.equal(c1[1], state[1])
        status.zero_()
        p = at(m, slice(0, 2))
        y, yc = torch.full((2, H, dv), 7.0, device="cuda"), torch.full((2, C), 7.0, device="cuda")
        g.dl_ssm_step(S1, slot, p["x"], p["dt"], p["A"], p["b"], p["c"], y, status=status)
        assert int(status) == 1 and bool((y[0] == 7).all()) and bool((y[1] != 7).any())
        status.zero_()
        g.dl_conv_step(x[:2], w, None, c1, slot, yc, status=status)
        assert int(status) == 1 and bool((yc[0] == 7).all()) and bool((yc[1] != 7).any())


def test_bad_sequence_bounds_are_skipped_and_flagged(g):
    """Bounds outside the rows, or descending (the index arithmetic behind this is replayed on the CPU first)."""
    rng = gen(13)
    H, dk, dv, C = 2, 64, 64, 64
    for dtype in (F32, BF16):
        m = scan_inputs(rng, 40, H, 1, dk, dv, dtype, False)
        x, w = randn(rng, 40, C).to(dtype), randn(rng, C, 3).to(dtype)
        for s in ([0, 41], [-3, 10], [0, 20, 10], [2 ** 31 - 1, 5], [0, 2 ** 31 - 1]):
            seq = torch.tensor(s, dtype=torch.int32, device="cuda")
            n = len(s) - 1
            S, st = torch.zeros(n, H, dv, dk, device="cuda"), torch.zeros(n, 2, C, dtype=dtype, device="cuda")
            for f in (lambda status: run_prompt(g, S, seq, None, m, torch.zeros(40, H, dv, dtype=dtype, device="cuda"), status=status),
                      lambda status: g.dl_conv_prompt(x, w, None, st, seq, None, torch.zeros_like(x), status=status)):
                status = torch.zeros(1, dtype=torch.int32, device="cuda")
                f(status)
                assert int(status) == 2
            assert bool((S[-1] == 0).all()) and bool((st[-1] == 0).all())


def layer(g, bufs, m, w):
    """One layer's operators as they are used together: norm, convolution of the
    normed rows, scan of the convolution's slices, norm of the scan's heads in 8 bits."""
    H, G, dk, dv = 4, 1, 64, 64
    g.dl_rms_norm(m["x"], w["norm"], 1e-5, bufs["n"], residual=m["r"], residual_out=bufs["r"])
    if m["seq"] is not None:
        g.dl_conv_prompt(bufs["n"], w["conv"], w["bias"], bufs["hist"], m["seq"], m["slot"], bufs["u"])
    else:
        g.dl_conv_step(bufs["n"], w["conv"], w["bias"], bufs["hist"], m["slot"], bufs["u"])
    rows = m["x"].shape[0]
    x, b, c = bufs["u"].split([H * dv, G * dk, G * dk], 1)
    args = (x.view(rows, H, dv), m["dt"], w["A"], b.view(rows, G, dk), c.view(rows, G, dk), bufs["y"])
    if m["seq"] is not None:
        g.dl_ssm_prompt(bufs["S"], m["seq"], m["slot"], *args, D=w["D"], dt_bias=w["dtb"], work=bufs["work"])
    else:
        g.dl_ssm_step(bufs["S"], m["slot"], *args, D=w["D"], dt_bias=w["dtb"])
    g.dl_rms_norm(bufs["y"].view(rows * H, dv), w["head"], 1e-5, bufs["q"], scale=bufs["s"])
    g.dl_rows_from_8bit(bufs["q"], bufs["s"], bufs["v"])


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("prompt", [True, False])
def test_a_layer_direct_on_another_stream_and_replayed(g, prompt, dtype):
    """The operators together: against the references chained (each fed with the
    kernels' own previous output), then on a side stream and from a captured
    graph replayed on new inputs, bit for bit."""
    rng = gen(14)
    H, G, dk, dv, C, B = 4, 1, 64, 64, 384, 3
    lens = [90, 1, 33] if prompt else [1] * B
    s, seq = starts(lens)
    rows = s[-1]
    w = dict(norm=1 + 0.1 * randn(rng, C), conv=randn(rng, C, 4).to(dtype), bias=randn(rng, C).to(dtype),
             A=-torch.rand(H, generator=rng, device="cuda"), D=randn(rng, H), dtb=randn(rng, H), head=1 + 0.1 * randn(rng, dv))

    def inputs():
        return dict(x=randn(rng, rows, C).to(dtype), r=randn(rng, rows, C), dt=randn(rng, rows, H).to(dtype),
                    seq=seq if prompt else None, slot=torch.tensor([2, 0, 3], dtype=torch.int32, device="cuda"))

    state0 = dict(S=randn(rng, 4, H, dv, dk), hist=randn(rng, 4, 3, C).to(dtype))

    def buffers():
        z = lambda *sh, t=dtype: torch.zeros(*sh, dtype=t, device="cuda")  # noqa: E731
        return dict(n=z(rows, C), r=z(rows, C, t=F32), u=z(rows, C), y=z(rows, H, dv), q=z(rows * H, dv, t=torch.int8),
                    s=z(rows * H, t=F32), v=z(rows * H, dv, t=F32),
                    work=torch.empty(g.dl_ssm_work_bytes(rows, B, H, dk, dv), dtype=torch.uint8, device="cuda"),
                    **{k: v.clone() for k, v in state0.items()})

    m = inputs()
    bufs = buffers()
    layer(g, bufs, m, w)
    torch.cuda.synchronize()
    h, n = R.norm(m["x"], m["r"], w["norm"], 1e-5)
    R.assert_within(bufs["n"], n, (32 * R.U32 + R.half_step(dtype)) * n.abs(), "norm")
    for i in range(B):
        k = int(m["slot"][i])
        rs = slice(s[i], s[i + 1])
        u, mag = R.conv(torch.cat([state0["hist"][k], bufs["n"][rs]]), w["conv"], w["bias"])
        R.assert_within(bufs["u"][rs], u, 7 * R.U32 * mag + (FAST[dtype] * R.U32 + R.half_step(dtype)) * u.abs() + 1e-38, "conv")
        cu = bufs["u"][rs]
        r = R.scan(state0["S"][k], cu[:, :256].reshape(-1, H, dv), m["dt"][rs], w["A"], cu[:, 256:320].reshape(-1, 1, dk),
                   cu[:, 320:].reshape(-1, 1, dk), w["D"], w["dtb"], None)
        by, bS = scan_bounds(r, dtype, F32, dk, prompt and dtype == BF16)
        R.assert_within(bufs["y"][rs], r["y"], by, "y")
        R.assert_within(bufs["S"][k], r["S"], bS, "S")
    _, n2 = R.norm(bufs["y"].view(rows * H, dv), None, w["head"], 1e-5)
    R.assert_within(bufs["v"], n2, 0.501 * n2.abs().amax(1, keepdim=True) / 127 + 0 * n2, "8-bit heads")

    names = ["n", "r", "u", "y", "q", "s", "v", "S", "hist"]
    side = torch.cuda.Stream()
    again = buffers()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        layer(g, again, m, w)
    side.synchronize()
    for k in names:
        assert torch.equal(again[k], bufs[k]), k
    fixed, cap = {k: (v.clone() if v is not None else None) for k, v in m.items()}, buffers()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        layer(g, cap, fixed, w)
    for turn in range(2):
        new = inputs() if turn else m
        for k in ("x", "r", "dt"):
            fixed[k].copy_(new[k])
        for k, v in state0.items():
            cap[k].copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        want = buffers()
        layer(g, want, new, w)
        torch.cuda.synchronize()
        for k in names:
            assert torch.equal(cap[k], want[k]), (turn, k)
    del graph


# ------------------------------------------------------------------ many rows, far rows

@pytest.mark.parametrize("out", [BF16, torch.int8])
@pytest.mark.parametrize("width", [4097, 5001, 8191, 16383])
def test_norm_of_odd_widths(g, width, out):
    """Rows that no 16-byte access fits, by every number of columns a thread holds."""
    rng = gen(width)
    x, r, w = randn(rng, 3, width).to(BF16), randn(rng, 3, width), 1 + 0.1 * randn(rng, width)
    y = torch.zeros(3, width, dtype=out, device="cuda")
    h = torch.empty_like(r)
    scale = torch.zeros(3, -(-width // 128), device="cuda") if out == torch.int8 else None
    g.dl_rms_norm(x, w, 1e-5, y, residual=r, residual_out=h, scale=scale, group=128 if scale is not None else 0)
    want_h, want = R.norm(x, r, w, 1e-5)
    R.assert_within(h, want_h, R.U32 * want_h.abs(), "residual")
    if scale is None:
        R.assert_within(y, want, (32 * R.U32 + 2.0 ** -8) * want.abs(), "y")
    else:
        got = y.float() * scale.repeat_interleave(128, 1)[:, :width]
        step = torch.nn.functional.pad(want, (0, -width % 128)).view(3, -1, 128).abs().amax(2) / 127
        R.assert_within(scale, step, 2.0 ** -18 * step, "scale")
        step = step.repeat_interleave(128, 1)[:, :width]
        R.assert_within(got, want, 0.5 * step * (1 + 2.0 ** -12) + 2.0 ** -12 * step, "values")


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("channels,tokens", [(301, 9000), (1024, 22000)])
def test_conv_prompt_that_fills_the_gpu(g, channels, tokens, dtype):
    """Long tiles of tokens: a few long sequences among many short and empty ones."""
    rng = gen(channels)
    lens = [tokens // 2, 0, 1, 31, 32, 33, tokens // 2 - 300] + [k % 4 for k in range(60)]
    s, seq = starts(lens)
    T = s[-1] + 5
    x, w = randn(rng, T, channels).to(dtype), randn(rng, channels, 4).to(dtype)
    bias = randn(rng, channels).to(dtype)
    state = randn(rng, len(lens), 3, channels).to(dtype)
    old, y = state.clone(), torch.full((T, channels), 7.0, dtype=dtype, device="cuda")
    g.dl_conv_prompt(x, w, bias, state, seq, None, y)
    for i, n in enumerate(lens):
        line = torch.cat([old[i], x[s[i]:s[i + 1]]])
        assert torch.equal(state[i], line[n:])
        want, mag = R.conv(line, w, bias)
        bound = 1.1 * 6 * R.U32 * mag + (FAST[dtype] * R.U32 + R.half_step(dtype)) * want.abs() + 1e-38
        R.assert_within(y[s[i]:s[i + 1]], want, bound, f"sequence {i}")
    assert bool((y[s[-1]:] == 7).all())


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("H,G,dk,dv", [(5, 1, 128, 64), (6, 2, 64, 64), (3, 3, 64, 128)])
@pytest.mark.parametrize("longest", [6, 90])
def test_ssm_prompt_of_many_sequences(g, longest, H, G, dk, dv, dtype):
    """More sequences than are ordered by length, in few tokens each and in many."""
    lens = [(7 * k) % (longest + 1) for k in range(70)]
    check_prompt(g, lens, H, G, dk, dv, dtype, F32, gate=G == 2, seed=H, first=1)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("gate", [False, True])
def test_ssm_prompt_keeps_what_is_no_number_across_segments(g, dtype, gate):
    """As above, in a sequence whose segments run side by side: one channel's NaN in
    an early segment reaches that channel's later tokens and nothing else."""
    rng = gen(16)
    H, dk, dv, n = 1, 64, 64, 4000
    assert g.dl_ssm_work_bytes(n, 1, H, dk, dv) > 0
    m = scan_inputs(rng, n, H, 1, dk, dv, dtype, gate, 0.02)
    S0 = 0.5 * randn(rng, 1, H, dv, dk)
    _, seq = starts([n])

    def run(m):
        S, y = S0.clone(), torch.zeros(n, H, dv, dtype=dtype, device="cuda")
        run_prompt(g, S, seq, None, m, y)
        return S, y

    S, y = run(m)
    m["x"][700, 0, 5] = float("nan")
    S2, y2 = run(m)
    keep = [e for e in range(dv) if e != 5]
    assert torch.equal(y2[:, :, keep], y[:, :, keep]) and torch.equal(S2[:, :, keep], S[:, :, keep])
    assert torch.equal(y2[:700], y[:700]) and bool(y2[700:, 0, 5].isnan().all()) and bool(S2[0, 0, 5].isnan().all())


@pytest.fixture(scope="module")
def far():
    """2.2e9 bfloat16 elements: rows and slots whose offsets pass 32 bits."""
    buf = torch.empty(2_200_000_000, dtype=BF16, device="cuda")
    yield buf
    del buf
    torch.cuda.empty_cache()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("n", [1, 9, 200])
def test_ssm_slots_behind_32_bits(g, far, n, dtype):
    """The last slots of a large pool, by a prompt (n > 1: token by token, on the
    tensor cores) and by a step."""
    rng = gen(17)
    H, dk, dv = 4, 128, 128
    per = H * dk * dv
    P = far.numel() // per
    assert (P - 2) * per > 2 ** 31
    pool = far[:P * per].view(P, H, dv, dk)
    slot = torch.tensor([P - 1, P - 2], dtype=torch.int32, device="cuda")
    pool[P - 2:] = 0.5 * randn(rng, 2, H, dv, dk).to(BF16)
    old = pool[P - 2:].clone()
    wrapped = [((P - 1 - k) * per - 2 ** 31) // per for k in range(2)] + [((P - 1) * per - 2 ** 31) // per + 1]
    pool[wrapped] = 3.0
    m = scan_inputs(rng, 2 * n, H, 1, dk, dv, dtype, False)
    y = torch.zeros(2 * n, H, dv, dtype=dtype, device="cuda")
    if n == 1:
        g.dl_ssm_step(pool, slot, m["x"], m["dt"], m["A"], m["b"], m["c"], y, D=m["D"], dt_bias=m["dt_bias"])
    else:
        run_prompt(g, pool, torch.tensor([0, n, 2 * n], dtype=torch.int32, device="cuda"), slot, m, y)
    for i in range(2):
        rows = slice(i * n, (i + 1) * n)
        r = R.scan(old[1 - i], **at(m, rows))
        by, bS = scan_bounds(r, dtype, BF16, dk, dtype == BF16 and n > 1)
        R.assert_within(y[rows], r["y"], by, "y")
        R.assert_within(pool[P - 1 - i], r["S"], bS, "state")
    assert bool((pool[wrapped] == 3).all())


def test_norm_conv_and_scan_of_rows_behind_32_bits(g, far):
    """Row strides that put the later rows behind 2^31 elements, and a pool of
    histories as large."""
    rng = gen(18)
    rows, width = 260, 128
    stride = far.numel() // rows // 8 * 8
    assert (rows - 4) * stride > 2 ** 31
    x = torch.as_strided(far, (rows, width), (stride, 1))
    x.copy_(randn(rng, rows, width))
    near = x.clone()
    w = 1 + 0.1 * randn(rng, width)
    a, b = (torch.zeros(rows, width, device="cuda") for _ in range(2))
    g.dl_rms_norm(x, w, 1e-5, a)
    g.dl_rms_norm(near, w, 1e-5, b)
    assert torch.equal(a, b) and bool((b != 0).any())
    f = randn(rng, width, 4).to(BF16)
    _, seq = starts([200, 60])
    st = [torch.zeros(2, 3, width, dtype=BF16, device="cuda") for _ in range(2)]
    y = [torch.zeros(rows, width, dtype=BF16, device="cuda") for _ in range(2)]
    for v, s, o in zip((x, near), st, y):
        g.dl_conv_prompt(v, f, None, s, seq, None, o)
    assert torch.equal(y[0], y[1]) and torch.equal(st[0], st[1])
    m = scan_inputs(rng, rows, 2, 1, 64, 64, BF16, True)
    out = []
    for v in (x, near):
        m["x"] = v.view(rows, 2, 64)
        out.append((torch.zeros(2, 2, 64, 64, device="cuda"), torch.zeros(rows, 2, 64, dtype=BF16, device="cuda")))
        run_prompt(g, out[-1][0], seq, None, m, out[-1][1])
    assert torch.equal(out[0][0], out[1][0]) and torch.equal(out[0][1], out[1][1])
    P = far.numel() // (3 * width)
    pool = far[:P * 3 * width].view(P, 3, width)
    slot = torch.tensor([P - 1, P - 2], dtype=torch.int32, device="cuda")
    pool[P - 2:] = st[0].flip(0)
    o = [torch.zeros(2, width, dtype=BF16, device="cuda") for _ in range(2)]
    g.dl_conv_step(near[:2], f, None, pool, slot, o[0])
    g.dl_conv_step(near[:2], f, None, st[0], None, o[1])
    assert torch.equal(o[0], o[1]) and torch.equal(pool[P - 2:].flip(0), st[0])


def test_layer_graphs_that_share_a_workspace(g):
    """Two captured scans that share their workspace, replayed in turn on one stream."""
    rng = gen(19)
    H, dk, dv, n = 2, 64, 64, 3000
    _, seq = starts([n])
    work = torch.empty(g.dl_ssm_work_bytes(n, 1, H, dk, dv), dtype=torch.uint8, device="cuda")
    assert work.numel() > 0
    calls, graphs = [], []
    for k in range(2):
        m = scan_inputs(rng, n, H, 1, dk, dv, BF16, False, 0.02)
        calls.append((m, torch.zeros(1, H, dv, dk, device="cuda"), torch.zeros(n, H, dv, dtype=BF16, device="cuda")))
    go = lambda m, S, y: g.dl_ssm_prompt(S, seq, None, m["x"], m["dt"], m["A"], m["b"], m["c"], y, work=work)  # noqa: E731
    for c in calls:
        go(*c)
    want = [(S.clone(), y.clone()) for _, S, y in calls]
    for c in calls:
        graphs.append(torch.cuda.CUDAGraph())
        torch.cuda.synchronize()
        with torch.cuda.graph(graphs[-1]):
            go(*c)
    for _, S, y in calls:
        S.zero_(), y.zero_()
    for gr in graphs:
        gr.replay()
    torch.cuda.synchronize()
    for (_, S, y), (S0, y0) in zip(calls, want):
        assert torch.equal(S, S0) and torch.equal(y, y0)
    graphs.clear()
