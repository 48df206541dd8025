"""Measured cases of the operators around a recurrent layer's decode step.

Five operators, each as a user's program calls it (``own`` true) and in a plain
form of elementary torch operations (``own`` false):

  norm         root-mean-square norm with the residual's addition; the output
               as float32 / bfloat16 or in 8 bits with scales
  conv_prompt  short causal convolution over ragged prompts, with the slots'
               histories
  conv_step    the same for one new token per sequence
  ssm_prompt   selective state space scan over ragged prompts, from and into
               the slots' states
  ssm_step     the same for one new token per sequence

A case is a dict of plain values; ``lens`` is a text of sequence lengths
("300,0,1,37"), ``tail`` counts rows behind the last sequence, which no
operator touches. 8-bit outputs are returned as the values they stand for.
"""
import math

import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "i8": torch.int8, "e4m3": torch.float8_e4m3fn}
SIZE = {"f32": 4, "bf16": 2, "i8": 1, "e4m3": 1}
EPS = 1e-5
CHUNK = 64  # tokens per chunk of the scan's plain form


# ---------------------------------------------------------------- cases


def listed():
    return [
        # a decode step of 256 sequences at 32 heads of 128: the layer's input norm, 8-bit for the projection behind it
        dict(name="norm_step_i8", op="norm", rows=256, width=4096, x="bf16", residual="bf16", out="i8", group=0),
        # the same norm over a batch of prompts: float32 residual stream, e4m3 with a scale per 128 columns
        dict(name="norm_prompt_e4m3", op="norm", rows=16384, width=4096, x="bf16", residual="f32", out="e4m3", group=128),
        # a width and a row count that no vector or tile divides
        dict(name="norm_odd", op="norm", rows=1021, width=2501, x="bf16", residual="bf16", out="bf16", group=0),
        # the prompts of a serving batch, continued and fresh, at 32 value heads of 128 and one key and query group of 128
        dict(name="conv_prompt_ragged", op="conv_prompt", lens="4096,17,2048,1,5000,0,1200,3901", tail=121, channels=4352,
             taps=4, dtype="bf16", bias=True),
        # a few short float32 prompts, three taps, a channel count that no vector divides
        dict(name="conv_prompt_f32", op="conv_prompt", lens="700,2,1,73", tail=1, channels=1541, taps=3, dtype="f32", bias=False),
        # a decode step of 256 sequences
        dict(name="conv_step", op="conv_step", batch=256, channels=4352, taps=4, dtype="bf16", bias=True),
        # the smallest call, where the launch counts: one sequence
        dict(name="conv_step_one", op="conv_step", batch=1, channels=384, taps=4, dtype="f32", bias=True),
        # the prompts of that serving batch, 32 heads of 128 x 128
        dict(name="ssm_prompt_ragged", op="ssm_prompt", lens="4096,17,2048,1,5000,0,1200,3901", tail=121, heads=32, groups=1,
             d_v=128, d_k=128, dtype="bf16", state="f32", gate=False),
        # one long prompt on few heads, which fills the GPU only when its length is split
        dict(name="ssm_prompt_long", op="ssm_prompt", lens="32768", tail=0, heads=16, groups=1, d_v=64, d_k=128, dtype="bf16",
             state="f32", gate=True),
        # short float32 prompts, two groups
        dict(name="ssm_prompt_f32", op="ssm_prompt", lens="257,40", tail=3, heads=16, groups=2, d_v=64, d_k=64, dtype="f32",
             state="f32", gate=False),
        # a decode step of 256 sequences: the whole 512 MiB state is read and written
        dict(name="ssm_step", op="ssm_step", batch=256, heads=32, groups=1, d_v=128, d_k=128, dtype="bf16", state="f32",
             gate=False),
        # the smallest call: one sequence, two heads of 64 x 64
        dict(name="ssm_step_one", op="ssm_step", batch=1, heads=2, groups=1, d_v=64, d_k=64, dtype="f32", state="f32", gate=True),
    ]


def _spread(rng, lo, hi):
    """A whole number in [lo, hi], even over its logarithm."""
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def _lens(rng, most):
    """Lengths of 1 to 12 sequences, short and empty ones among them, at most `most` tokens in all."""
    n = _spread(rng, 1, 12)
    lens = [0 if rng.random() < 0.08 else _spread(rng, 1, max(1, most // n)) for _ in range(n)]
    if sum(lens) == 0:
        lens[0] = 1
    return ",".join(str(x) for x in lens)


def draw(rng):
    op = rng.choice(["norm", "conv_prompt", "conv_step", "ssm_prompt", "ssm_prompt", "ssm_step"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "norm":
        width = _spread(rng, 16, 16384)
        out = rng.choice(["bf16", "f32", "i8", "e4m3"])
        return dict(op=op, rows=_spread(rng, 1, min(16384, 2 ** 25 // width)), width=width, x=dtype,
                    residual=rng.choice(["none", "bf16", "f32"]), out=out,
                    group=rng.choice([0, 128]) if out in ("i8", "e4m3") else 0)
    if op == "conv_prompt":
        channels = _spread(rng, 64, 8192)
        return dict(op=op, lens=_lens(rng, min(16384, 2 ** 25 // channels)), tail=rng.choice([0, 1, 65]), channels=channels,
                    taps=rng.choice([2, 3, 4]), dtype=dtype, bias=rng.random() < 0.5)
    if op == "conv_step":
        return dict(op=op, batch=_spread(rng, 1, 1024), channels=_spread(rng, 64, 8192), taps=rng.choice([2, 3, 4]),
                    dtype=dtype, bias=rng.random() < 0.5)
    d_v, d_k = rng.choice([64, 128, 256]), rng.choice([64, 128])
    groups = rng.choice([1, 1, 2, 4])
    heads = groups * _spread(rng, 1, 32 // groups)
    case = dict(heads=heads, groups=groups, d_v=d_v, d_k=d_k, dtype=dtype, state=rng.choice(["f32", "f32", "bf16"]),
                gate=rng.random() < 0.5)
    if op == "ssm_prompt":
        most = 16384 if dtype == "bf16" else 2048
        return dict(op=op, lens=_lens(rng, min(most, 2 ** 25 // (heads * d_v))), tail=rng.choice([0, 1, 65]), **case)
    return dict(op=op, batch=_spread(rng, 1, min(256, 2 ** 26 // (heads * d_v * d_k))), **case)


# ---------------------------------------------------------------- inputs


def _plan(lens, device):
    """Where the tokens of ragged sequences lie: seq_start as the operators take it, and each token's sequence and position."""
    n = torch.tensor(lens, dtype=torch.int64)
    start = torch.cat([torch.zeros(1, dtype=torch.int64), n.cumsum(0)])
    seq = torch.repeat_interleave(torch.arange(len(lens)), n)
    pos = torch.arange(int(n.sum())) - start[seq]
    chunks = -(-n // CHUNK)
    first = chunks.cumsum(0) - chunks
    return {"seq_start": start.to(torch.int32).to(device), "start": start[:-1].to(device), "n": n.to(device), "seq": seq.to(device),
            "pos": pos.to(device), "chunk_seq": torch.repeat_interleave(torch.arange(len(lens)), chunks).to(device),
            "padded": (first[seq] * CHUNK + pos).to(device), "total": int(n.sum())}


def prepare(case, seed):
    device = "cuda" if torch.cuda.is_available() else "cpu"
    gen = torch.Generator(device=device).manual_seed(int(seed))

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device=device)

    def rand(*shape):
        return torch.rand(*shape, generator=gen, device=device)

    s = {"case": case}
    if case["op"] == "norm":
        rows, width, x = case["rows"], case["width"], TYPES[case["x"]]
        s["x"] = randn(rows, width).to(x)
        s["weight"] = (1.0 + 0.1 * randn(width)).to(x)
        s["residual"] = s["residual_out"] = None
        if case["residual"] != "none":
            s["residual"] = (2.0 * randn(rows, width)).to(TYPES[case["residual"]])
            s["residual_out"] = torch.zeros_like(s["residual"])
        s["y"] = torch.zeros(rows, width, dtype=TYPES[case["out"]], device=device)
        if case["out"] in ("i8", "e4m3"):
            groups = -(-width // case["group"]) if case["group"] else 1
            s["scale"] = torch.zeros(rows, groups, device=device)
            s["values"] = torch.zeros(rows, width, dtype=torch.bfloat16, device=device)
        return s
    if case["op"].startswith("conv"):
        channels, taps, dtype = case["channels"], case["taps"], TYPES[case["dtype"]]
        s["w"] = (randn(channels, taps) / math.sqrt(taps)).to(dtype)
        s["bias"] = (0.1 * randn(channels)).to(dtype) if case["bias"] else None
        if case["op"] == "conv_prompt":
            lens = [int(n) for n in case["lens"].split(",")]
            s["plan"] = _plan(lens, device)
            rows, batch = sum(lens) + case["tail"], len(lens)
        else:
            rows = batch = case["batch"]
        s["x"] = randn(rows, channels).to(dtype)
        s["y"] = torch.zeros(rows, channels, dtype=dtype, device=device)
        slots = batch + 2
        s["slot"] = torch.randperm(slots, generator=gen, device=device)[:batch].to(torch.int32)
        s["state"] = randn(slots, taps - 1, channels).to(dtype)
        return s
    heads, groups, d_v, d_k, dtype = case["heads"], case["groups"], case["d_v"], case["d_k"], TYPES[case["dtype"]]
    if case["op"] == "ssm_prompt":
        lens = [int(n) for n in case["lens"].split(",")]
        s["plan"] = _plan(lens, device)
        rows, batch = sum(lens) + case["tail"], len(lens)
    else:
        rows = batch = case["batch"]
    # x, b and c are slices of the convolution's output row, as the layer has them
    u = randn(rows, heads * d_v + 2 * groups * d_k)
    u = (u * torch.sigmoid(u) + 0.1 * randn(rows, u.shape[1])).to(dtype)
    s["x"] = u[:, :heads * d_v].view(rows, heads, d_v)
    s["b"] = u[:, heads * d_v:heads * d_v + groups * d_k].view(rows, groups, d_k)
    s["c"] = u[:, heads * d_v + groups * d_k:].view(rows, groups, d_k)
    s["dt"] = randn(rows, heads).to(dtype)
    # the usual start of such layers: A in -[1, 16], steps of 0.001 to 0.1 through the inverse of the softplus
    s["A"] = -(1.0 + 15.0 * rand(heads))
    step = torch.exp(math.log(1e-3) + (math.log(1e-1) - math.log(1e-3)) * rand(heads))
    s["dt_bias"] = step + torch.log(-torch.expm1(-step))
    s["D"] = 1.0 + 0.1 * randn(heads)
    s["z"] = randn(rows, heads, d_v).to(dtype) if case["gate"] else None
    s["y"] = torch.zeros(rows, heads, d_v, dtype=dtype, device=device)
    slots = batch + 2
    s["slot"] = torch.randperm(slots, generator=gen, device=device)[:batch].to(torch.int32)
    s["S"] = (0.02 * randn(slots, heads, d_v, d_k)).to(TYPES[case["state"]])
    return s


# ---------------------------------------------------------------- one pass


def run(s):
    return (_own if own else _plain)(s)


def _own(s):
    import gated_delta_rule_104_b200 as g

    op = s["case"]["op"]
    if op == "norm":
        group = s["case"]["group"]
        g.dl_rms_norm(s["x"], s["weight"], EPS, s["y"], residual=s["residual"], residual_out=s["residual_out"],
                      scale=s.get("scale"), group=group)
        if "scale" not in s:
            return {"y": s["y"], "residual": s["residual_out"]}
        g.dl_rows_from_8bit(s["y"], s["scale"], s["values"], group=group)
        return {"y": s["values"], "residual": s["residual_out"]}
    if op == "conv_prompt":
        g.dl_conv_prompt(s["x"], s["w"], s["bias"], s["state"], s["plan"]["seq_start"], s["slot"], s["y"])
        return {"y": s["y"], "state": s["state"]}
    if op == "conv_step":
        g.dl_conv_step(s["x"], s["w"], s["bias"], s["state"], s["slot"], s["y"])
        return {"y": s["y"], "state": s["state"]}
    if op == "ssm_prompt":
        if "work" not in s:  # the caller's workspace, made once
            (rows, heads, d_v), d_k = s["x"].shape, s["b"].shape[2]
            s["work"] = torch.empty(g.dl_ssm_work_bytes(rows, s["slot"].numel(), heads, d_k, d_v), dtype=torch.uint8,
                                    device=s["x"].device)
        g.dl_ssm_prompt(s["S"], s["plan"]["seq_start"], s["slot"], s["x"], s["dt"], s["A"], s["b"], s["c"], s["y"], D=s["D"],
                        dt_bias=s["dt_bias"], z=s["z"], work=s["work"])
        return {"y": s["y"], "S": s["S"]}
    g.dl_ssm_step(s["S"], s["slot"], s["x"], s["dt"], s["A"], s["b"], s["c"], s["y"], D=s["D"], dt_bias=s["dt_bias"], z=s["z"])
    return {"y": s["y"], "S": s["S"]}


def _plain(s):
    return {"norm": _plain_norm, "conv_prompt": _plain_conv_prompt, "conv_step": _plain_conv_step,
            "ssm_prompt": _plain_ssm_prompt, "ssm_step": _plain_ssm_step}[s["case"]["op"]](s)


def _plain_norm(s):
    case = s["case"]
    h = s["x"].float()
    if s["residual"] is not None:
        h = h + s["residual"].float()
        s["residual_out"].copy_(h)
    y = h * torch.rsqrt((h * h).mean(1, keepdim=True) + EPS) * s["weight"].float()
    if case["out"] not in ("i8", "e4m3"):
        s["y"].copy_(y)
        return {"y": s["y"], "residual": s["residual_out"]}
    rows, width = y.shape
    group = case["group"] or width
    y = torch.nn.functional.pad(y, (0, -width % group)).view(rows, -1, group)
    scale = y.abs().amax(2, keepdim=True) / (127.0 if case["out"] == "i8" else 448.0)
    q = torch.where(scale > 0, y / scale, torch.zeros_like(y))
    q = torch.round(q).clamp(-127, 127) if case["out"] == "i8" else q.to(TYPES["e4m3"]).float()
    s["values"].copy_((q * scale).view(rows, -1)[:, :width])
    return {"y": s["values"], "residual": s["residual_out"]}


def _silu(x):
    return x / (1.0 + torch.exp(-x))


def _softplus(x):
    return x.clamp(min=0) + torch.log1p(torch.exp(-x.abs()))


def _plain_conv_prompt(s):
    x, w, state, plan, taps = s["x"], s["w"], s["state"], s["plan"], s["case"]["taps"]
    slot, total, channels = s["slot"].long(), plan["total"], x.shape[1]
    every = torch.cat([x[:total], state[slot].reshape(-1, channels)])  # the tokens, then each sequence's history
    tap = torch.arange(taps, device=x.device) - (taps - 1)

    def rows_at(seq, start, pos):  # rows of `every` at positions from -(taps - 1) on
        return torch.where(pos >= 0, start + pos, total + seq * (taps - 1) + pos + (taps - 1))

    at = rows_at(plan["seq"][:, None], plan["start"][plan["seq"]][:, None], plan["pos"][:, None] + tap)
    out = (every[at].float() * w.float().t()).sum(1)
    if s["bias"] is not None:
        out = out + s["bias"].float()
    s["y"][:total].copy_(_silu(out))
    seq = torch.arange(slot.numel(), device=x.device)
    state[slot] = every[rows_at(seq[:, None], plan["start"][:, None], plan["n"][:, None] + tap[:-1])]
    return {"y": s["y"], "state": state}


def _plain_conv_step(s):
    slot = s["slot"].long()
    window = torch.cat([s["state"][slot], s["x"][:, None]], 1)
    out = (window.float() * s["w"].float().t()).sum(1)
    if s["bias"] is not None:
        out = out + s["bias"].float()
    s["y"].copy_(_silu(out))
    s["state"][slot] = window[:, 1:]
    return {"y": s["y"], "state": s["state"]}


def _plain_ssm_prompt(s):
    """The scan in chunks: products inside a chunk, chunk states joined through a matrix of decays between chunks. Sums of
    log decays, and their differences, in 64 bits."""
    plan, S, total = s["plan"], s["S"], s["plan"]["total"]
    slot, cs, at = s["slot"].long(), plan["chunk_seq"], plan["padded"]
    heads, d_v = s["x"].shape[1:]
    groups, d_k = s["b"].shape[1:]
    nc, per = cs.numel(), heads // groups

    def padded(t):  # [total, ...] -> [chunks, CHUNK, ...], zeros behind each sequence
        return torch.zeros(nc * CHUNK, *t.shape[1:], dtype=t.dtype, device=t.device).index_copy_(0, at, t).view(nc, CHUNK, *t.shape[1:])

    x = s["x"][:total].float()
    dt = _softplus(s["dt"][:total].float() + s["dt_bias"])
    dx = padded(x * dt[..., None]).permute(0, 2, 1, 3)                             # [nc, H, Q, d_v]
    b = padded(s["b"][:total].float()).permute(0, 2, 1, 3)                         # [nc, G, Q, d_k]
    c = padded(s["c"][:total].float()).permute(0, 2, 1, 3)
    ld = padded((dt * s["A"]).double()).permute(0, 2, 1).cumsum(2)                 # [nc, H, Q] log decay since the chunk's start
    causal = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device=x.device).tril()
    diff = (ld[..., :, None] - ld[..., None, :]).masked_fill(~causal, -math.inf)
    m = torch.exp(diff).float().view(nc, groups, per, CHUNK, CHUNK) * (c @ b.transpose(2, 3))[:, :, None]
    y = m.view(nc, heads, CHUNK, CHUNK) @ dx
    # what each chunk adds to the state by its end, and the states before the chunks and behind the sequences
    dec = torch.exp(ld[..., -1:] - ld).float()
    bh = b[:, :, None].expand(nc, groups, per, CHUNK, d_k).reshape(nc, heads, CHUNK, d_k)
    ch = c[:, :, None].expand(nc, groups, per, CHUNK, d_k).reshape(nc, heads, CHUNK, d_k)
    add = (dx * dec[..., None]).transpose(2, 3) @ bh                               # [nc, H, d_v, d_k]
    tot = ld[..., -1]                                                              # [nc, H]
    end = tot.cumsum(0)
    seqs = torch.zeros(slot.numel(), heads, dtype=torch.float64, device=x.device).index_add_(0, cs, tot)
    begin = seqs.cumsum(0) - seqs                                                  # [seqs, H]
    S0 = S[slot].float()
    order = torch.arange(nc, device=x.device)
    before = (cs[:, None] == cs[None, :]) & (order[:, None] > order[None, :])
    mix = torch.exp(((end - tot)[:, None] - end[None]).masked_fill(~before[..., None], -math.inf)).float()   # [nc, nc, H]
    entry = torch.einsum("cdh,dhvk->chvk", mix, add) + torch.exp(end - tot - begin[cs]).float()[..., None, None] * S0[cs]
    y = y + (ch * torch.exp(ld).float()[..., None]) @ entry.transpose(2, 3)
    y = y.permute(0, 2, 1, 3).reshape(nc * CHUNK, heads, d_v)[at] + s["D"][:, None] * x
    if s["z"] is not None:
        y = y * _silu(s["z"][:total].float())
    s["y"][:total].copy_(y)
    mine = cs[None, :] == torch.arange(slot.numel(), device=x.device)[:, None]
    last = torch.exp(((begin + seqs)[:, None] - end[None]).masked_fill(~mine[..., None], -math.inf)).float()
    S[slot] = (torch.einsum("sdh,dhvk->shvk", last, add) + torch.exp(seqs).float()[..., None, None] * S0).to(S.dtype)
    return {"y": s["y"], "S": S}


def _plain_ssm_step(s):
    S, slot = s["S"], s["slot"].long()
    per = s["x"].shape[1] // s["b"].shape[1]
    x = s["x"].float()
    b, c = (t.float().repeat_interleave(per, 1) for t in (s["b"], s["c"]))
    dt = _softplus(s["dt"].float() + s["dt_bias"])
    new = S[slot].float() * torch.exp(dt * s["A"])[..., None, None] + (dt[..., None] * x)[..., None] * b[:, :, None]
    y = (new * c[:, :, None]).sum(3) + s["D"][:, None] * x
    if s["z"] is not None:
        y = y * _silu(s["z"].float())
    s["y"].copy_(y)
    S[slot] = new.to(S.dtype)
    return {"y": s["y"], "S": S}


# ---------------------------------------------------------------- what a pass cannot do without


def work(case):
    if case["op"] == "norm":
        n = case["rows"] * case["width"]
        moved = n * SIZE[case["x"]] + case["width"] * SIZE[case["x"]]
        if case["residual"] != "none":
            moved += 2 * n * SIZE[case["residual"]]
        moved += n * SIZE[case["out"]]
        if case["out"] in ("i8", "e4m3"):  # codes and scales, then their values in bfloat16
            moved += 4 * case["rows"] * (-(-case["width"] // case["group"]) if case["group"] else 1) + 2 * n
        return {"bytes": moved, "flops": 5 * n}
    if case["op"].startswith("conv"):
        size, taps, channels = SIZE[case["dtype"]], case["taps"], case["channels"]
        lens = [int(n) for n in case["lens"].split(",")] if case["op"] == "conv_prompt" else [1] * case["batch"]
        tokens, seqs = sum(lens), sum(n > 0 for n in lens)
        return {"bytes": size * channels * (2 * tokens + 2 * (taps - 1) * seqs + taps + int(case["bias"])),
                "flops": tokens * channels * (2 * taps + 5)}
    lens = [int(n) for n in case["lens"].split(",")] if case["op"] == "ssm_prompt" else [1] * case["batch"]
    tokens, seqs = sum(lens), sum(n > 0 for n in lens)
    heads, groups, d_v, d_k = case["heads"], case["groups"], case["d_v"], case["d_k"]
    row = heads * d_v * (3 if case["gate"] else 2) + 2 * groups * d_k + heads
    return {"bytes": tokens * row * SIZE[case["dtype"]] + 2 * seqs * heads * d_v * d_k * SIZE[case["state"]] + 12 * heads,
            "flops": tokens * heads * 5 * d_v * d_k}


# ---------------------------------------------------------------- the definitions in 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    f = {k: v.double() for k, v in s.items() if isinstance(v, torch.Tensor) and v.is_floating_point() and v.dtype != TYPES["e4m3"]}
    if case["op"] == "norm":
        h = f["x"] + f["residual"] if s["residual"] is not None else f["x"]
        y = h / torch.sqrt(h.square().mean(-1, keepdim=True) + EPS) * f["weight"]
        if case["out"] in ("i8", "e4m3"):
            width = case["width"]
            for lo in range(0, width, case["group"] or width):
                part = y[:, lo:lo + (case["group"] or width)]
                scale = part.abs().max(1, keepdim=True).values / (127 if case["out"] == "i8" else 448)
                q = part / scale.clamp(min=1e-300)
                if case["out"] == "i8":
                    q = q.round()
                else:  # three bits behind the leading one, from 2^-9 on
                    unit = torch.exp2(torch.floor(torch.log2(q.abs().clamp(min=2.0 ** -6))) - 3)
                    q = (q / unit).round() * unit
                part.copy_(q * scale)
        return {"y": y, "residual": None if s["residual"] is None else h}
    if case["op"] == "conv_step":
        y = f["x"] * f["w"][:, -1] + (f["bias"] if s["bias"] is not None else 0.0)
        for j in range(case["taps"] - 1):
            y += f["state"][s["slot"].long(), j] * f["w"][:, j]
        state = f["state"].clone()
        state[s["slot"].long()] = torch.cat([f["state"][s["slot"].long(), 1:], f["x"][:, None]], 1)
        return {"y": y * torch.sigmoid(y), "state": state}
    if case["op"] == "conv_prompt":
        y, state, at, taps = f["y"], f["state"], 0, case["taps"]
        for i, n in enumerate(int(n) for n in case["lens"].split(",")):
            k = int(s["slot"][i])
            line = torch.cat([state[k], f["x"][at:at + n]])
            acc = sum(line[j:j + n] * f["w"][:, j] for j in range(taps))
            acc = acc + f["bias"] if s["bias"] is not None else acc
            y[at:at + n] = acc * torch.sigmoid(acc)
            state[k] = line[n:]
            at += n
        return {"y": y, "state": state}
    per = case["heads"] // case["groups"]
    f["dt"] = torch.logaddexp(f["dt"] + f["dt_bias"], torch.zeros_like(f["dt"]))
    lens = [int(n) for n in case["lens"].split(",")] if case["op"] == "ssm_prompt" else None
    if lens is None:
        steps = [(torch.arange(case["batch"], device=s["x"].device),) * 2]
    else:  # token j of every sequence that has one
        starts = [sum(lens[:i]) for i in range(len(lens))]
        by = sorted(range(len(lens)), key=lambda i: -lens[i])  # the longest first: the active ones are a prefix
        row0 = torch.tensor([starts[i] for i in by], device=s["x"].device)
        sid = torch.tensor(by, device=s["x"].device)
        steps, active = [], len(by)
        for j in range(max(lens)):
            while lens[by[active - 1]] <= j:
                active -= 1
            steps.append((row0[:active] + j, sid[:active]))
    slot, y = s["slot"].long(), f["y"]
    order = sid if lens is not None else steps[0][1]
    state = f["S"][slot[order]]
    a = torch.exp(f["dt"] * f["A"])
    dx = f["x"] * f["dt"][..., None]
    for rows, ids in steps:
        n = rows.numel()
        state[:n].mul_(a[rows][..., None, None])
        state[:n].addcmul_(dx[rows][..., None], f["b"][rows].repeat_interleave(per, 1)[:, :, None])
        y[rows] = torch.matmul(state[:n], f["c"][rows].repeat_interleave(per, 1)[..., None]).squeeze(-1)
    total = y.shape[0] if lens is None else sum(lens)
    y[:total] += f["D"][:, None] * f["x"][:total]
    if s["z"] is not None:
        y[:total] *= f["z"][:total] * torch.sigmoid(f["z"][:total])
    f["S"][slot[order]] = state
    return {"y": y, "S": f["S"]}
