"""GPU tests of the norm, the short convolution and the selective scan at the
edges of their contract, beside test_layer_ops_gpu.py. References in 64 bits;
u = 2^-24 is half a float32 step, relative, and a rounding to bfloat16 is off by
at most 2^-8 of the value as R.half_step counts it."""
import os
import subprocess
import sys

import pytest

from tests import layer_ref as R

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def g():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import gated_delta_rule_104_b200 as g

    g.load()
    return g


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def starts(lens):
    s = [0]
    for n in lens:
        s.append(s[-1] + n)
    return torch.tensor(s, dtype=torch.int32, device="cuda")


def prompt(g, S, lens, x, dt, A, b, c, **k):
    """The scan over prompts laid end to end; returns y (S is advanced)."""
    T, H, dv = x.shape
    y = torch.full((T, H, dv), 7.0, dtype=x.dtype, device="cuda")
    work = torch.empty(g.dl_ssm_work_bytes(T, len(lens), H, b.shape[2], dv), dtype=torch.uint8, device="cuda")
    g.dl_ssm_prompt(S, starts(lens), None, x, dt, A, b, c, y, work=work, **k)
    return y


# ------------------------------------------------------------------ norm

@pytest.mark.parametrize("out", [torch.int8, torch.float8_e4m3fn])
@pytest.mark.parametrize("width", [512, 511])
def test_norm_scale_of_an_infinite_value(g, width, out):
    """A value behind the weight that is infinite (an infinite weight, a product past float32): its group has scale
    NaN, as with a NaN, and reads back as no number; other groups are as without it."""
    x = torch.randn(4, width, generator=gen(33), device="cuda")
    for group in (0, 128):
        got = []
        for high in (1.0, 3e38, float("inf")):
            w = torch.ones(width, device="cuda")
            w[200] = high
            x[:, 200] = 2.0  # (its norm is above 1.2)
            y = torch.zeros(4, width, dtype=out, device="cuda")
            scale = torch.zeros(4, 4 if group else 1, device="cuda")
            g.dl_rms_norm(x, w, 1e-6, y, scale=scale, group=group)
            v = torch.zeros(4, width, device="cuda")
            g.dl_rows_from_8bit(y, scale, v, group=group)
            got.append((scale, v))
        bad = slice(128, 256) if group else slice(0, width)
        keep = [k for k in range(width) if not (bad.start <= k < bad.stop)]
        for scale, v in got[1:]:
            assert bool(scale[:, 1 if group else 0].isnan().all()) and bool(v[:, bad].isnan().all())
            assert torch.equal(v[:, keep], got[0][1][:, keep])
            if group:
                assert torch.equal(scale[:, [0, 2, 3]], got[0][0][:, [0, 2, 3]])


# ------------------------------------------------------------------ decays of the tensor-core scan

@pytest.mark.parametrize("strong", [16, 40, 100, 112, 120])
def test_ssm_prompt_decays_behind_many_strong_steps(g, strong):
    """`strong` steps that forget all, then weak ones in the same chunk.

    One token has x = 1, the state is zero, and c . b is a number g of 8 bits. So y
    at a later token is the decayed score g exp(l_t - l_s) dt rounded to bfloat16,
    once, and the score's exponential may be off by 2^-10 (and 32 u by the steps and
    products): y lies between the roundings of the ends of that interval.
    """
    H, d, n = 16, 64, 128
    rng = gen(strong)
    dt = (-6 + torch.randn(n, H, generator=rng, device="cuda")).to(BF16)
    dt[:strong] = 500.0
    A = -(1 + 15 * torch.rand(H, generator=rng, device="cuda"))
    b, c = torch.zeros(n, H, d, dtype=BF16, device="cuda"), torch.zeros(n, H, d, dtype=BF16, device="cuda")
    b[:, :, 0] = 1.0
    c[:, :, 0] = (1 + torch.randint(128, (n, H), generator=rng, device="cuda") / 128).to(BF16)
    lost = torch.zeros(n, H, d, dtype=BF16, device="cuda")
    steps = torch.logaddexp(R.f64(dt), torch.zeros(n, H, dtype=torch.float64))
    for s in sorted({strong, (strong + 127) // 2, 125}):
        x = lost.clone()
        x[s] = 1.0
        y = prompt(g, torch.zeros(1, H, d, d, device="cuda"), [n], x, dt, A, b, c)
        decay = (steps * R.f64(A)).cumsum(0)
        want = R.f64(c[:, :, 0]) * torch.exp(decay - decay[s]) * steps[s]
        off = 2.0 ** -10 + 32 * R.U32
        low, high = ((want * f).float().to(BF16).double() for f in (1 - off, 1 + off))
        got = R.f64(y)[s:]
        assert bool((got == got[:, :, :1]).all()) and bool((y[:s] == 0).all())
        outside = (got[:, :, 0] < low[s:]) | (got[:, :, 0] > high[s:])
        assert not bool(outside.any()), (s, int(outside.sum()), outside.nonzero()[0].tolist())


def layer_inputs(seed, n, H, dk, dv, dtype):
    rng = gen(seed)
    randn = lambda *s: torch.randn(*s, generator=rng, device="cuda")  # noqa: E731
    return [randn(n, H, dv).to(dtype), (randn(n, H) - 2).to(dtype), -1 - 8 * torch.rand(H, generator=rng, device="cuda"),
            randn(n, 1, dk).to(dtype), randn(n, 1, dk).to(dtype)]


# a ragged call; few tokens a sequence; one long sequence in segments
CALLS = [[70, 1, 300], [5, 0, 9], [3000]]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("dv", [64, 128])
@pytest.mark.parametrize("lens", CALLS, ids=str)
def test_ssm_prompt_of_a_head_that_forgets_at_once(g, lens, dv, dtype):
    """A of -inf, the strongest decay there is: as any that leaves nothing of the state, to the bit."""
    H, dk = 3, 64
    x, dt, A, b, c = layer_inputs(31, sum(lens), H, dk, dv, dtype)
    out = []
    for a in (-1e30, float("-inf")):
        A[1] = a
        S = torch.ones(len(lens), H, dv, dk, device="cuda")
        out.append((S, prompt(g, S, lens, x, dt, A, b, c)))
    assert torch.equal(out[0][0], out[1][0]) and torch.equal(out[0][1], out[1][1])
    last = sum(lens) - 1  # what is left is the last token's addend
    want = (torch.logaddexp(R.f64(dt[last, 1]), torch.zeros(()).double()) * R.f64(x[last, 1]))[:, None] * R.f64(b[last, 0])
    R.assert_within(out[1][0][-1, 1], want, 16 * R.U32 * want.abs() + 1e-38, "state")


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("dv", [64, 128])
@pytest.mark.parametrize("lens", CALLS, ids=str)
def test_ssm_prompt_of_a_decay_that_is_no_number(g, lens, dv, dtype):
    """A of NaN: nothing of that head is a number. A step size of infinity under A = 0
    (0 times infinity): nothing of it from there on. Other heads and sequences stay as they were."""
    H, dk, T = 3, 64, sum(lens)
    x, dt, A, b, c = layer_inputs(32, T, H, dk, dv, dtype)
    A[0] = 0.0

    def run():
        S = torch.ones(len(lens), H, dv, dk, device="cuda")
        return S, prompt(g, S, lens, x, dt, A, b, c)

    S0, y0 = run()
    used = [i for i, n in enumerate(lens) if n]
    A[1] = float("nan")
    S, y = run()
    assert bool(S[used, 1].isnan().all()) and bool(y[:, 1].isnan().all())
    assert torch.equal(S[:, ::2], S0[:, ::2]) and torch.equal(y[:, ::2], y0[:, ::2])
    A[1] = -1.0
    S0, y0 = run()
    at = T - 3  # in the last sequence
    dt[at, 0] = float("inf")
    S, y = run()
    assert bool(S[-1, 0].isnan().all()) and bool(y[at:, 0].isnan().all()) and torch.equal(y[:at], y0[:at])
    assert torch.equal(S[:, 1:], S0[:, 1:]) and torch.equal(S[:-1], S0[:-1]) and torch.equal(y[:, 1:], y0[:, 1:])


# ------------------------------------------------------------------ accuracy of a float32 state

@pytest.mark.parametrize("dv", [64, 128])
@pytest.mark.parametrize("n", [100, 128, 300, 3000])
def test_ssm_prompt_keeps_a_float32_state_to_its_last_bits(g, n, dv):
    """bfloat16 prompts whose tokens have x = 0 but for one, without decay: the state is that token's addend dt x b^T.

    dt x is one rounding (u), its three parts leave at most 2^-26 of it, their sum in the accumulator at most a whole
    step (2 u); b is a power of two, every other product is zero, and the decays are 1: 4 u of the addend.
    """
    H, dk = 3, 64
    x1, bias, b1, f = R.one_addend(dv, n + dv, H)
    x1, bias = x1.cuda(), bias.cuda()
    b = b1.to(BF16).cuda().expand(n, 1, dk).contiguous()
    dt, A = torch.zeros(n, H, dtype=BF16, device="cuda"), torch.zeros(H, device="cuda")
    assert n != 3000 or g.dl_ssm_work_bytes(n, 1, H, dk, dv) > 0
    for at in sorted({0, 37, n // 2, n - 1}):
        x = torch.zeros(n, H, dv, dtype=BF16, device="cuda")
        x[at] = x1
        S = torch.zeros(1, H, dv, dk, device="cuda")
        prompt(g, S, [n], x, dt, A, b, b, dt_bias=bias)
        want = f[:, :, None] * R.f64(b1)
        R.assert_within(S[0], want, 4 * R.U32 * want.abs(), f"state, token {at} of {n}")


# ------------------------------------------------------------------ strides, alignment, options

@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("dv", [64, 128])
@pytest.mark.parametrize("lens", CALLS + [[1] * 5], ids=str)
def test_ssm_of_slices_of_wider_rows(g, lens, dv, dtype):
    """Every operand a slice of rows that are wider than it, dt at an odd offset of rows of odd width: as
    contiguous ones, to the bit. (Sequences of one token each by the single step too.)"""
    H, G, dk, T = 4, 2, 64, sum(lens)
    rng = gen(34)
    widths = [("x", H, dv), ("z", H, dv), ("b", G, dk), ("c", G, dk)]
    rows = torch.randn(T, 32 + sum(h * d + 8 for _, h, d in widths), generator=rng, device="cuda").to(dtype)
    loose, first = {}, 16
    for name, h, d in widths:
        loose[name] = rows[:, first:first + h * d].unflatten(1, (h, d))
        first += h * d + 8
    loose["dt"] = torch.randn(T, 2 * H + 3, generator=rng, device="cuda").to(dtype)[:, 3:3 + H] - 1
    wide = torch.zeros(T, 2 * H + 3, dtype=dtype, device="cuda")
    wide[:, 3:3 + H] = loose["dt"]
    loose["dt"] = wide[:, 3:3 + H]
    A = -1 - 8 * torch.rand(H, generator=rng, device="cuda")
    D = torch.randn(H, generator=rng, device="cuda")
    assert not any(v.is_contiguous() for v in loose.values())
    tight = {k: v.contiguous() for k, v in loose.items()}
    out = []
    for m in (loose, tight):
        S = torch.ones(len(lens), H, dv, dk, device="cuda")
        y = prompt(g, S, lens, m["x"], m["dt"], A, m["b"], m["c"], D=D, z=m["z"])
        out.append([S, y])
        if max(lens) == 1:
            S, y = torch.ones_like(S), torch.zeros_like(y)
            g.dl_ssm_step(S, None, m["x"], m["dt"], A, m["b"], m["c"], y, D=D, z=m["z"])
            out[-1] += [S, y]
    assert all(torch.equal(a, b) for a, b in zip(*out))
    assert bool((out[0][1] != 7).any()) and bool(out[0][1].isfinite().all())
    r = R.scan(torch.ones(H, dv, dk), *[tight[k][:lens[0]] for k in ("x", "dt")], A, tight["b"][:lens[0]], tight["c"][:lens[0]], D,
               None, tight["z"][:lens[0]])  # (the first sequence; the roundings of the tensor cores' products as elsewhere)
    bound = 12 * R.U32 * r["y_err"] + (dk + 64) * R.U32 * r["y_mag"] + 2 * R.half_step(dtype) * (r["y_mag"] + r["y"].abs()) + 1e-38
    R.assert_within(out[0][1][:lens[0]], r["y"], bound, "y")


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("taps", [2, 3, 4])
@pytest.mark.parametrize("silu", [False, True])
@pytest.mark.parametrize("off", [0, 1])
def test_conv_bias_at_any_alignment_and_no_activation(g, off, silu, taps, dtype):
    """A bias that no 16-byte access fits beside wide rows, and sums without the activation, over prompts and by single tokens."""
    C, n = 264, 21
    rng = gen(35 + taps)
    bias = torch.randn(C + 8, generator=rng, device="cuda").to(dtype)[off:off + C]
    x, w = torch.randn(n, C, generator=rng, device="cuda").to(dtype), torch.randn(C, taps, generator=rng, device="cuda").to(dtype)
    hist = torch.randn(1, taps - 1, C, generator=rng, device="cuda").to(dtype)
    want, mag = R.conv(torch.cat([hist[0], x]), w, bias, silu)
    bound = 1.1 * (taps + 2) * R.U32 * mag + (64 * R.U32 + R.half_step(dtype)) * want.abs() + 1e-38
    y, state = torch.zeros_like(x), hist.clone()
    g.dl_conv_prompt(x, w, bias, state, starts([n]), None, y, silu=silu)
    R.assert_within(y, want, bound, "prompt")
    single, history = torch.zeros_like(x), hist.clone()
    for t in range(n):
        g.dl_conv_step(x[t:t + 1], w, bias, history, None, single[t:t + 1], silu=silu)
    assert torch.equal(single, y) and torch.equal(history, state)


# ------------------------------------------------------------------ two calls at once, first calls in a capture

@pytest.mark.parametrize("dtype", [F32, BF16])
def test_calls_on_two_streams_at_once(g, dtype):
    """Scans, convolutions and norms queued on two streams together, each with its own state and workspace: as one after the other."""
    H, dk, dv = 4, 64, 64
    lens = [[3000], [700, 40, 1500]]
    calls = []
    for k, n in enumerate(lens):
        x, dt, A, b, c = layer_inputs(40 + k, sum(n), H, dk, dv, dtype)
        calls.append((n, x, dt, A, b, c, torch.randn(H * dv, 4, generator=gen(42 + k), device="cuda").to(dtype), starts(n),
                      torch.empty(g.dl_ssm_work_bytes(sum(n), len(n), H, dk, dv), dtype=torch.uint8, device="cuda")))

    def run(n, x, dt, A, b, c, w, seq, work, out):
        rows = x.view(sum(n), H * dv)
        g.dl_rms_norm(rows, torch.ones(H * dv, device="cuda"), 1e-5, out["n"])
        g.dl_conv_prompt(out["n"], w, None, out["h"], seq, None, out["u"])
        g.dl_ssm_prompt(out["S"], seq, None, out["u"].view(sum(n), H, dv), dt, A, b, c, out["y"], work=work)

    def buffers(n):
        z = lambda *s, t=dtype: torch.zeros(*s, dtype=t, device="cuda")  # noqa: E731
        T = sum(n)
        return dict(n=z(T, H * dv), u=z(T, H * dv), h=z(len(n), 3, H * dv), S=z(len(n), H, dv, dk, t=F32), y=z(T, H, dv))

    want = [buffers(n) for n in lens]
    for args, out in zip(calls, want):
        run(*args, out)
    streams = [torch.cuda.Stream() for _ in lens]
    for _ in range(5):
        got = [buffers(n) for n in lens]
        torch.cuda.synchronize()
        for args, out, stream in zip(calls, got, streams):
            with torch.cuda.stream(stream):
                run(*args, out)
        torch.cuda.synchronize()
        assert all(torch.equal(a[k], b[k]) for a, b in zip(got, want) for k in a)


FIRST = """
import torch, sys
import gated_delta_rule_104_b200 as g
dtype = getattr(torch, sys.argv[1])
T, H, d = 300, 2, 64
z = lambda *s, t=dtype: torch.zeros(*s, dtype=t, device="cuda")
x = torch.randn(T, H * d, device="cuda").to(dtype)
seq = torch.tensor([0, 130, T], dtype=torch.int32, device="cuda")
one, w, A, dt, b = torch.ones(H * d, device="cuda"), torch.randn(H * d, 4, device="cuda").to(dtype), -torch.ones(H, device="cuda"), z(T, H), x.view(T, H, d)[:, :1].contiguous()
work = torch.empty(max(1, g.dl_ssm_work_bytes(T, 2, H, d, d)), dtype=torch.uint8, device="cuda")
o = [dict(q=z(T, H * d, t=torch.int8), s=z(T, t=torch.float32), v=z(T, H * d), u=z(T, H * d), h=z(2, 3, H * d), S=z(2, H, d, d, t=torch.float32), y=z(T, H, d), y1=z(2, H, d), u1=z(2, H * d)) for _ in range(2)]
def run(o):
    g.dl_rms_norm(x, one, 1e-5, o["q"], scale=o["s"])
    g.dl_rows_from_8bit(o["q"], o["s"], o["v"])
    g.dl_conv_prompt(o["v"], w, None, o["h"], seq, None, o["u"])
    g.dl_ssm_prompt(o["S"], seq, None, o["u"].view(T, H, d), dt, A, b, b, o["y"], work=work)
    g.dl_conv_step(o["v"][:2], w, None, o["h"], None, o["u1"])
    g.dl_ssm_step(o["S"], None, o["u1"].view(2, H, d), dt[:2], A, b[:2], b[:2], o["y1"])
graph = torch.cuda.CUDAGraph()
torch.cuda.synchronize()
with torch.cuda.graph(graph):
    run(o[0])
graph.replay()
torch.cuda.synchronize()
run(o[1])
torch.cuda.synchronize()
assert all(torch.equal(o[0][k], o[1][k]) for k in o[0]) and g.dl_device_faults() == 0 and bool((o[0]["y1"] != 0).any())
del graph
print("same")
"""


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_the_first_calls_of_a_process_in_a_capture(dtype):
    """Nothing that a first call sets up is forbidden while a graph is captured."""
    out = subprocess.run([sys.executable, "-c", FIRST, dtype], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert out.returncode == 0 and out.stdout.strip() == "same", out.stderr


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("dv", [64, 128])
def test_a_captured_call_replayed_on_other_lengths_and_slots(g, dv, dtype):
    """Lengths and slots are read on the device: a graph captured over some is replayed over others, padding rows and
    sequences without a slot among them, as a call made for those."""
    H, dk, T, P = 2, 64, 3000, 6
    x, dt, A, b, c = layer_inputs(50, T, H, dk, dv, dtype)
    rows, w = x.view(T, H * dv), torch.randn(H * dv, 4, generator=gen(51), device="cuda").to(dtype)
    seq, slot = torch.zeros(5, dtype=torch.int32, device="cuda"), torch.zeros(4, dtype=torch.int32, device="cuda")
    work = torch.empty(g.dl_ssm_work_bytes(T, 4, H, dk, dv), dtype=torch.uint8, device="cuda")
    fresh = lambda: dict(S=torch.ones(P, H, dv, dk, device="cuda"), h=torch.ones(P, 3, H * dv, dtype=dtype, device="cuda"),  # noqa: E731
                         y=torch.full_like(x, 7.0), u=torch.full_like(rows, 7.0),
                         status=torch.zeros(1, dtype=torch.int32, device="cuda"))

    def run(o):
        g.dl_conv_prompt(rows, w, None, o["h"], seq, slot, o["u"], status=o["status"])
        g.dl_ssm_prompt(o["S"], seq, slot, x, dt, A, b, c, o["y"], work=work, status=o["status"])

    calls = [([0, 700, 700, 2900, 3000], [3, 1, 0, 5]), ([0, 2999, 2999, 2999, 2999], [5, -1, -1, -1]),
             ([100, 101, 129, 2000, 2600], [0, 2, 4, 1]), ([0, 0, 0, 0, 0], [0, 1, 2, 3])]
    seq.copy_(torch.tensor(calls[0][0]))
    slot.copy_(torch.tensor(calls[0][1]))
    cap, graph = fresh(), torch.cuda.CUDAGraph()
    run(fresh())
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        run(cap)
    for start, slots in calls:
        seq.copy_(torch.tensor(start))
        slot.copy_(torch.tensor(slots))
        want = fresh()
        for k, v in want.items():
            cap[k].copy_(v)
        run(want)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(cap[k], want[k]) for k in cap) and int(cap["status"]) == (1 if -1 in slots else 0)
        assert bool((cap["y"][:start[0]] == 7).all()) and bool((cap["y"][start[-1]:] == 7).all())
        for i, k in enumerate(slots):
            n = start[i + 1] - start[i]
            if k >= 0 and n:
                at = slice(start[i], start[i + 1])
                r = R.scan(torch.ones(H, dv, dk), x[at], dt[at], A, b[at], c[at], None, None, None)
                off = 12 * R.U32 * r["S_err"] + (2.0 ** -16 if dtype == BF16 else R.U32) * r["S_mag"] + 1e-38
                R.assert_within(cap["S"][k], r["S"], off, "state")
            elif k >= 0:
                assert bool((cap["S"][k] == 1).all())
    del graph
