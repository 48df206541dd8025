"""64-bit references of the norm, the short convolution and the selective scan,
with the sizes of the sums behind each output (for tolerances), on the CPU."""
import torch


def f64(t):
    return None if t is None else t.detach().cpu().double()


def silu(u):
    return u * torch.sigmoid(u)


def norm(x, residual, weight, eps):
    h = f64(x) if residual is None else f64(x) + f64(residual)
    return h, h / torch.sqrt(h.square().mean(1, keepdim=True) + eps) * f64(weight)


def conv(line, w, bias, act=True):
    """Outputs of line[taps - 1:], and the sums of their terms' magnitudes."""
    line, w = f64(line), f64(w)
    taps = w.shape[1]
    n = line.shape[0] - taps + 1
    u = sum(line[j:j + n] * w[:, j] for j in range(taps))
    mag = sum((line[j:j + n] * w[:, j]).abs() for j in range(taps))
    if bias is not None:
        u, mag = u + f64(bias), mag + f64(bias).abs()
    return (silu(u) if act else u), mag


def scan(S0, x, dt, A, b, c, D, dt_bias, z):
    """One sequence: S0 [H, d_v, d_k], x [n, H, d_v], ... Returns y and the last
    state, the magnitudes of the sums that form them (every term positive), and
    the error of the decays: what one relative error unit in each step's dt and
    exp(dt A) makes of a state, summed along the recurrence, and of y through it."""
    S0, x, dt, A, b, c, D, dt_bias, z = map(f64, (S0, x, dt, A, b, c, D, dt_bias, z))
    n, H, dv = x.shape
    per = H // b.shape[1]
    b, c = (t.repeat_interleave(per, 1) for t in (b, c))
    dt = dt + (dt_bias if dt_bias is not None else 0.0)
    dt = torch.logaddexp(dt, torch.zeros_like(dt))
    S, M, E = S0.clone(), S0.abs(), torch.zeros_like(S0)
    y, ym, ye = torch.empty_like(x), torch.empty_like(x), torch.empty_like(x)
    for t in range(n):
        da = torch.exp(dt[t] * A)[:, None, None]
        add = (dt[t][:, None] * x[t])[:, :, None] * b[t][:, None, :]
        E = da * E + da * M * (1.0 + (dt[t] * A).abs())[:, None, None] + add.abs()
        S = da * S + add
        M = da * M + add.abs()
        y[t] = (S * c[t][:, None, :]).sum(2)
        ym[t] = (M * c[t][:, None, :].abs()).sum(2)
        ye[t] = (E * c[t][:, None, :].abs()).sum(2)
    if D is not None:
        y, ym = y + D[:, None] * x, ym + (D[:, None] * x).abs()
    if z is not None:
        g = silu(z)
        y, ym, ye = y * g, ym * g.abs(), ye * g.abs()
    return dict(y=y, S=S, y_mag=ym, S_mag=M, y_err=ye, S_err=E)


def one_addend(dv, seed, H=3):
    """x [H, dv] of bfloat16, steps [H] that are whole float32 numbers of which the softplus is the number itself
    (above 30), powers of two for b [64], and the products dt x in 64 bits."""
    rng = torch.Generator().manual_seed(seed)
    x = torch.randn(H, dv, generator=rng).bfloat16()
    bias = 30 + 10 * torch.rand(H, generator=rng)
    b = torch.ldexp(torch.ones(64), torch.randint(-2, 3, (64,), generator=rng))
    return x, bias, b, f64(x) * f64(bias)[:, None]


U32 = 2.0 ** -24  # half a step of float32, relative


def half_step(dtype):
    return {torch.float32: U32, torch.bfloat16: 2.0 ** -8}[dtype]


def assert_within(got, want, bound, what=""):
    """|got - want| <= bound everywhere."""
    got = f64(got)
    bad = ~((got - want).abs() <= bound)
    assert not bool(bad.any()), (f"{what}: {int(bad.sum())} of {bad.numel()} outside; worst "
                                 f"{float(((got - want).abs() / bound.clamp(min=1e-300))[bad].max()):.3g} of the bound, first at "
                                 f"{bad.nonzero()[0].tolist()}, got {float(got[bad][0])}, want {float(want[bad][0])}")
