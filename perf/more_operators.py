"""Cases of the operators around the recurrent-state layers: the short causal
convolution over channels, the selective state space scan (both over prompts,
with gradients, and for single tokens on cache pages), and the norms of
queries and keys with the position rotation in the same pass.

``run`` computes a case with elementary torch operations in 32 bits (64 where
those lose what matters; ``own = False``) or through the library's entry
points (``own = True``); ``exact`` is the definition in 64 bits.
"""
from __future__ import annotations

import math

import torch

own = False

F32, F64 = torch.float32, torch.float64
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # the convolution in front of q, k and v (16 heads of 128 each) of a delta-rule layer: a serving prefill of
        # ragged packed prompts that continue cached states, x a view of the layer's fused projection
        dict(name="conv_prompt_packed", op="conv", dtype="bf16", B=1, T=8191, docs=7, D=6144, W=4, act=True,
             bias=False, view=2048, states=True),
        # the same layer's dense training batch, forward and gradients
        dict(name="conv_train", op="conv_train", dtype="bf16", B=4, T=4096, docs=0, D=6144, W=4, act=True, bias=True,
             view=0, states=False),
        # a serving batch of single tokens, some rows without a sequence
        dict(name="conv_step", op="conv_step", dtype="bf16", N=64, D=6144, W=4, act=True, bias=True, empty=2),
        # a short prompt of a small model: latency counts
        dict(name="scan_prompt_short", op="scan", dtype="bf16", B=1, T=61, docs=0, D=512, S=16, G=1, states=True),
        # a serving prefill of ragged packed prompts
        dict(name="scan_prompt_packed", op="scan", dtype="bf16", B=1, T=8192, docs=6, D=4096, S=16, G=1, states=True),
        # a dense training batch, forward and gradients
        dict(name="scan_train", op="scan_train", dtype="bf16", B=2, T=4096, docs=0, D=4096, S=16, G=1, states=False),
        # fp32 fine-tuning on ragged packed documents, two groups, larger states carried between calls
        dict(name="scan_tune_packed", op="scan_train", dtype="fp32", B=1, T=1501, docs=5, D=1536, S=32, G=2,
             states=True),
        # one sequence generating: the smallest call
        dict(name="scan_step_one", op="scan_step", dtype="bf16", N=1, D=2048, S=16, G=1, empty=0),
        # a full serving batch, some rows without a sequence
        dict(name="scan_step_batch", op="scan_step", dtype="bf16", N=256, D=8192, S=16, G=1, empty=3),
        # single tokens far into long contexts
        dict(name="rotary_step", op="rotary", dtype="bf16", B=8, T=1, Hq=16, Hk=16, D=128, R=128, norm="rms",
             interleaved=False, start=900000, scaled=True),
        # a prompt of a model with grouped keys, continued far into a long context
        dict(name="rotary_prompt", op="rotary", dtype="bf16", B=1, T=32768, Hq=32, Hk=8, D=128, R=128, norm="rms",
             interleaved=False, start=200000, scaled=True),
        # a training batch, forward and gradients, half of each head rotated in pairs of neighbours
        dict(name="rotary_train", op="rotary_train", dtype="bf16", B=4, T=4096, Hq=16, Hk=16, D=128, R=64,
             norm="rms", interleaved=True, start=0, scaled=False),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _lengths(rng, tokens):
    """Dense rows or packed documents of about so many tokens."""
    if rng.random() < 0.5:
        return dict(B=1, T=tokens, docs=min(_log_int(rng, 1, 24), tokens))
    B = min(_log_int(rng, 1, 8), tokens)
    return dict(B=B, T=tokens // B, docs=0)


def draw(rng):
    op = rng.choice(["conv", "conv_train", "conv_step", "scan", "scan", "scan_train", "scan_train", "scan_step",
                     "rotary", "rotary_train"])
    c = dict(op=op, dtype=rng.choice(["bf16", "bf16", "fp32"]))
    half = 2 if c["dtype"] == "fp32" else 1
    if op.startswith("conv"):
        c.update(D=8 * _log_int(rng, 1, 1024), W=rng.choice([2, 3, 4, 4]), act=rng.random() < 0.75,
                 bias=rng.random() < 0.5)
        if op == "conv_step":
            N = _log_int(rng, 1, 256)
            return dict(c, N=N, empty=rng.randint(0, min(3, N - 1)))
        most = (48 << 20 if op == "conv" else 96 << 20) // half
        tokens = max(1, min(_log_int(rng, 1, 32768), most // c["D"]))
        return dict(c, **_lengths(rng, tokens), view=8 * rng.choice([0, 0, rng.randint(1, 128)]),
                    states=rng.random() < 0.5)
    if op.startswith("scan"):
        c["S"] = rng.choice([8, 16, 16, 16, 32, 64])
        c["G"] = rng.choice([1, 1, 1, 2, 3])
        c["D"] = 8 * c["G"] * _log_int(rng, 2, 512 // c["G"])
        if op == "scan_step":
            N = max(1, min(_log_int(rng, 1, 256), (1 << 25) // (c["D"] * c["S"])))
            return dict(c, N=N, empty=rng.randint(0, min(3, N - 1)))
        most = (32 << 20 if op == "scan" else 28 << 20) * 16 // (half * max(16, c["S"]))
        tokens = max(1, min(_log_int(rng, 1, 16384), most // c["D"]))
        return dict(c, **_lengths(rng, tokens), states=rng.random() < 0.5)
    D = rng.choice([64, 80, 128, 128, 192, 256])
    Hk = rng.choice([1, 2, 4, 8, 16])
    c.update(D=D, R=rng.choice([D, D, D // 2 // 8 * 8, 16]), Hk=Hk, Hq=Hk * rng.choice([1, 1, 2, 4, 7]),
             norm=rng.choice(["rms", "rms", "l2", "none"]), interleaved=rng.random() < 0.5,
             start=rng.choice([0, rng.randint(1, 1000000)]), scaled=rng.random() < 0.5)
    most = (120 << 20 if op == "rotary" else 60 << 20) // half
    tokens = max(1, min(_log_int(rng, 1, 32768), most // ((c["Hq"] + Hk) * D)))
    B = min(_log_int(rng, 1, 8), tokens)
    return dict(c, B=B, T=tokens // B)


# ------------------------------------------------------------------ inputs
def _gen(seed):
    return torch.Generator("cuda").manual_seed(int(seed))


def _randn(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda", dtype=F32)


def _rand(gen, *shape):
    return torch.rand(*shape, generator=gen, device="cuda", dtype=F32)


def _units(case):
    """Token offsets of the sequences: rows, or documents of ragged lengths."""
    if not case["docs"]:
        return [b * case["T"] for b in range(case["B"] + 1)]
    n, T = case["docs"], case["T"]
    rnd = torch.rand(n, generator=torch.Generator().manual_seed(17 * n + T)) + 0.05
    cuts = (rnd.cumsum(0) / rnd.sum() * (T - n)).floor().to(torch.int64) + torch.arange(1, n + 1)
    return [0] + cuts[:-1].tolist() + [T]


def _lead(case):
    return (case["T"],) if case["docs"] else (case["B"], case["T"])


def _pages(gen, n, n_pages, empty):
    """A page for every one of n rows in shuffled order; `empty` rows have none."""
    p = torch.randperm(n_pages, generator=gen, device="cuda")[:n].to(torch.int32)
    if empty:
        p[torch.randperm(n, generator=gen, device="cuda")[:empty]] = -1
    return p


def _frequencies(R, scaled):
    """Radians a token of the R / 2 pairs (64 bits). Scaled for long contexts:
    slow pairs turn 8 times slower, fast ones as before, with a blend of both
    between 1 and 4 turns in 8192 tokens."""
    f = 500000.0 ** (-torch.arange(0, R, 2, dtype=F64) / R)
    if scaled:
        turns = 8192 * f / (2 * math.pi)
        keep = ((turns - 1) / 3).clamp(0, 1)
        f = f * (keep + (1 - keep) / 8)
    return f.cuda()


def prepare(case, seed):
    gen, op, dt = _gen(seed), case["op"], DTYPES[case["dtype"]]
    s = dict(case=case, meta=None)
    if op in ("conv", "conv_train", "scan", "scan_train"):
        s["offsets"] = _units(case)
        if own and case["docs"]:
            from chunked_gated_delta_05_amd import binding
            s["meta"] = binding.make_meta(s["offsets"], s["offsets"][-1], "cuda")
        offs = torch.tensor(s["offsets"], device="cuda")
        s["first"], s["last"] = offs[:-1], offs[1:] - 1
        s["unit"] = torch.repeat_interleave(torch.arange(len(offs) - 1, device="cuda"), offs[1:] - offs[:-1])
    if op.startswith("conv"):
        D, W = case["D"], case["W"]
        s["weight"] = (_randn(gen, D, W) / math.sqrt(W)).to(dt)
        s["bias"] = (0.1 * _randn(gen, D)).to(dt) if case["bias"] else None
        if op == "conv_step":
            n_pages = case["N"] + case["N"] // 8 + 1
            s["pages"] = _pages(gen, case["N"], n_pages, case["empty"])
            s["live"] = (s["pages"] >= 0).nonzero().flatten()
            s["x"] = _randn(gen, case["N"], D).to(dt)
            s["state"] = _randn(gen, n_pages, W - 1, D).to(dt)
            return s
        n = len(s["offsets"]) - 1
        s["x"] = _randn(gen, *_lead(case), D + case["view"]).to(dt)[..., :D]
        s["s0"] = _randn(gen, n, W - 1, D).to(dt) if case["states"] else None
        if op == "conv_train":
            s["dout"] = _randn(gen, *_lead(case), D).to(dt)
            s["dfinal"] = _randn(gen, n, W - 1, D).to(dt) if case["states"] else None
        return s
    if op.startswith("scan"):
        D, S, G = case["D"], case["S"], case["G"]
        # decays of -1 to -S a unit of time, time steps of 0.001 to 0.1 a token
        s["A"] = -torch.arange(1, S + 1, device="cuda").float() * torch.exp(0.1 * _randn(gen, D, S))
        step = torch.exp(math.log(1e-3) + math.log(100.0) * _rand(gen, D))
        s["dt_bias"] = torch.log(torch.expm1(step))
        s["skip"] = 1 + 0.1 * _randn(gen, D)
        lead = (case["N"],) if op == "scan_step" else _lead(case)
        s["u"], s["gate"] = _randn(gen, *lead, D).to(dt), _randn(gen, *lead, D).to(dt)
        s["dt"] = (0.5 * _randn(gen, *lead, D)).to(dt)
        s["B"], s["C"] = _randn(gen, *lead, G, S).to(dt), _randn(gen, *lead, G, S).to(dt)
        if op == "scan_step":
            n_pages = case["N"] + case["N"] // 8 + 1
            s["pages"] = _pages(gen, case["N"], n_pages, case["empty"])
            s["live"] = (s["pages"] >= 0).nonzero().flatten()
            s["state"] = _randn(gen, n_pages, D, S)
            return s
        n = len(s["offsets"]) - 1
        s["s0"] = _randn(gen, n, D, S) if case["states"] else None
        if op == "scan_train":
            s["dout"] = _randn(gen, *lead, D).to(dt)
            s["dht"] = _randn(gen, n, D, S) if case["states"] else None
        return s
    B, T, D = case["B"], case["T"], case["D"]
    s["q"] = _randn(gen, B, T, case["Hq"], D).to(dt)
    s["k"] = _randn(gen, B, T, case["Hk"], D).to(dt)
    weights = case["norm"] == "rms"
    s["q_weight"] = (1 + 0.1 * _randn(gen, D)).to(dt) if weights else None
    s["k_weight"] = (1 + 0.1 * _randn(gen, D)).to(dt) if weights else None
    s["freqs"] = _frequencies(case["R"], case["scaled"])
    s["amplitude"] = 0.1 * math.log(8) + 1 if case["scaled"] else 1.0
    at = case["start"] + torch.arange(T, device="cuda")[None] + 1009 * torch.arange(B, device="cuda")[:, None]
    s["positions"] = at.contiguous()
    if op == "rotary_train":
        s["dq"] = _randn(gen, B, T, case["Hq"], D).to(dt)
        s["dk"] = _randn(gen, B, T, case["Hk"], D).to(dt)
    return s


# ------------------------------------------------------------------ plain form: convolution
def _silu_slope(z):
    p = torch.sigmoid(z)
    return p * (1 + z * (1 - p))


def _tap(x, s0, s, back):
    """x `back` tokens earlier in the same sequence: [tokens, D], before its
    start from the state s0 [units, W - 1, D] (or zero)."""
    if back == 0:
        return x
    N = x.shape[0]
    at = torch.arange(N, device=x.device)
    p = at - s["first"][s["unit"]] - back                 # position in the sequence
    y = x[(at - back).clamp(min=0)] * (p >= 0)[:, None]
    if s0 is not None:
        row = (p + s0.shape[1]).clamp(0, s0.shape[1] - 1)
        y = y + s0[s["unit"], row] * (p < 0)[:, None]
    return y


def _conv_linear(s, x, s0):
    W, w = s["case"]["W"], s["weight"].float()
    z = _tap(x, s0, s, 0) * w[:, W - 1]
    for j in range(W - 1):
        z = z + _tap(x, s0, s, W - 1 - j) * w[:, j]
    return z if s["bias"] is None else z + s["bias"].float()


def _conv_final(s, x, s0):
    """The last W - 1 inputs of every sequence, its entry state before them."""
    n = s["case"]["W"] - 1
    back = torch.arange(n - 1, -1, -1, device=x.device)
    p = (s["last"] - s["first"])[:, None] - back           # [units, W - 1]
    y = x[(s["first"][:, None] + p).clamp(min=0)] * (p >= 0)[..., None]
    if s0 is not None:
        u = torch.arange(p.shape[0], device=x.device)[:, None].expand_as(p)
        y = y + s0[u, (p + n).clamp(0, n - 1)] * (p < 0)[..., None]
    return y


def _plain_conv(s):
    case, dt = s["case"], s["x"].dtype
    x = s["x"].reshape(-1, case["D"]).float()
    s0 = None if s["s0"] is None else s["s0"].float()
    z = _conv_linear(s, x, s0)
    y = z * torch.sigmoid(z) if case["act"] else z
    r = {"y": y.to(dt).view(*_lead(case), -1)}
    if case["states"]:
        r["final"] = _conv_final(s, x, s0).to(dt)
    if case["op"] == "conv":
        return r
    W, w = case["W"], s["weight"].float()
    dz = s["dout"].reshape(-1, case["D"]).float()
    if case["act"]:
        dz = dz * _silu_slope(z)
    N, at = x.shape[0], torch.arange(x.shape[0], device=x.device)
    dx = dz * w[:, W - 1]
    for back in range(1, W):                               # token t + back reads token t
        inside = at + back <= s["last"][s["unit"]]
        dx = dx + dz[(at + back).clamp(max=N - 1)] * w[:, W - 1 - back] * inside[:, None]
    r["dweight"] = torch.stack([(dz * _tap(x, s0, s, W - 1 - j)).sum(0, dtype=F64) for j in range(W)], 1).float()
    if s["bias"] is not None:
        r["dbias"] = dz.sum(0, dtype=F64).float()
    if case["states"]:
        n, df = W - 1, s["dfinal"].float()
        length = s["last"] - s["first"] + 1
        d0 = torch.zeros_like(s0)
        for i in range(n):                                 # row i is position i - n
            for t in range(i + 1):                         # read by the tap j = i - t of token t
                d0[:, i] += dz[(s["first"] + t).clamp(max=N - 1)] * w[:, i - t] * (t < length)[:, None]
        p = length[:, None] - n + torch.arange(n, device=x.device)
        for i in range(n):
            inside = p[:, i] >= 0
            dx = dx.index_add(0, s["first"] + p[:, i].clamp(min=0), df[:, i] * inside[:, None])
            u = torch.arange(len(length), device=x.device)
            d0 = d0.index_put((u, (p[:, i] + n).clamp(0, n - 1)), df[:, i] * (~inside)[:, None], accumulate=True)
        r["dinitial"] = d0.to(dt)
    r["dx"] = dx.to(dt).view(*_lead(case), -1)
    return r


def _plain_conv_step(s):
    live, w = s["live"], s["weight"].float()
    at = s["pages"][live].long()
    seen = torch.cat([s["state"][at], s["x"][live][:, None]], 1)
    z = (seen.float() * w.t()).sum(1)
    if s["bias"] is not None:
        z = z + s["bias"].float()
    y = torch.zeros_like(s["x"])
    y[live] = (z * torch.sigmoid(z) if s["case"]["act"] else z).to(y.dtype)
    s["state"][at] = seen[:, 1:]
    return {"y": y, "state": s["state"]}


# ------------------------------------------------------------------ plain form: scan
def _scan(a, b):
    """h_i = a_i h_{i-1} + b_i along the first axis, h_{-1} = 0: by doubling
    within blocks of 64, then over the blocks' ends."""
    N, L = a.shape[0], 64
    blocks = -(-N // L)
    pad = blocks * L - N
    if pad:
        a, b = torch.cat([a, a.new_zeros(pad, *a.shape[1:])]), torch.cat([b, b.new_zeros(pad, *b.shape[1:])])
    a, b = a.view(blocks, L, *a.shape[1:]), b.view(blocks, L, *b.shape[1:])
    step = 1
    while step < L:
        a, b = (torch.cat([a[:, :step], a[:, step:] * a[:, :-step]], 1),
                torch.cat([b[:, :step], b[:, step:] + a[:, step:] * b[:, :-step]], 1))
        step *= 2
    if blocks > 1:
        ends = _scan(a[:, -1], b[:, -1])
        b = torch.cat([b[:1], b[1:] + a[1:] * ends[:-1, None]])
    return b.reshape(blocks * L, *b.shape[2:])[:N]


def _softplus(x):
    return x.clamp(min=0) + torch.log1p(torch.exp(-x.abs()))


def _scan_inputs(s):
    """fp32, channels of a group apart: u, dt, gate [tokens, G, D / G]; B, C
    [tokens, G, S]; A [G, D / G, S]; dt after its bias and softplus."""
    case = s["case"]
    G, S, D = case["G"], case["S"], case["D"]
    f = lambda n: s[n].reshape(-1, G, D // G).float()
    raw = f("dt") + s["dt_bias"].view(G, -1)
    rows = lambda n: s[n].reshape(-1, G, S).float()
    return f("u"), raw, _softplus(raw), f("gate"), rows("B"), rows("C"), s["A"].view(G, -1, S)


def _plain_scan(s):
    case, dtype, lead = s["case"], s["u"].dtype, _lead(s["case"])
    G, S, D = case["G"], case["S"], case["D"]
    u, raw, dt, gate, B, C, A = _scan_inputs(s)
    first = s["first"]
    a = torch.exp(dt[..., None] * A)                       # [tokens, G, D / G, S]
    b = (dt * u)[..., None] * B[:, :, None]
    if s["s0"] is not None:
        b[first] += a[first] * s["s0"].view(-1, G, D // G, S)
    keep = torch.ones(a.shape[0], 1, 1, 1, device=a.device)
    keep[first] = 0                                        # a sequence starts anew
    h = _scan(a * keep, b)
    y = (h * C[:, :, None]).sum(-1) + s["skip"].view(G, -1) * u
    p = torch.sigmoid(gate)
    r = {"out": (y * gate * p).to(dtype).view(*lead, D)}
    if case["states"]:
        r["final"] = h[s["last"]].reshape(-1, D, S)
    if case["op"] == "scan":
        return r
    dout = s["dout"].reshape(-1, G, D // G).float()
    dy = dout * gate * p
    # gradients of the states, in reversed time: the decay of the next token, none past a sequence's end
    after = torch.cat([a[1:] * keep[1:], a.new_zeros(1, *a.shape[1:])])
    c = dy[..., None] * C[:, :, None]
    if s["s0"] is not None:
        c[s["last"]] += s["dht"].view(-1, G, D // G, S)
    g = _scan(after.flip(0), c.flip(0)).flip(0)
    del after, c
    before = torch.cat([h.new_zeros(1, *h.shape[1:]), h[:-1]]) * keep
    if s["s0"] is not None:
        before[first] += s["s0"].view(-1, G, D // G, S)
    r["dB"] = ((dt * u)[..., None] * g).sum(2).to(dtype).view(*lead, G, S)
    r["dC"] = (dy[..., None] * h).sum(2).to(dtype).view(*lead, G, S)
    if s["s0"] is not None:
        r["dh0"] = (a[first] * g[first]).reshape(-1, D, S)
    ddu = (g * B[:, :, None]).sum(-1)
    w = g * a * before
    del a, before, h, g
    ddt = (ddu * u + (w * A).sum(-1)) * torch.sigmoid(raw)
    r["dA"] = (w * dt[..., None]).sum(0, dtype=F64).float().view(D, S)
    r["du"] = (ddu * dt + dy * s["skip"].view(G, -1)).to(dtype).view(*lead, D)
    r["ddt"] = ddt.to(dtype).view(*lead, D)
    r["dgate"] = (dout * y * _silu_slope(gate)).to(dtype).view(*lead, D)
    r["dskip"] = (dy * u).sum(0, dtype=F64).float().view(D)
    r["ddt_bias"] = ddt.sum(0, dtype=F64).float().view(D)
    return r


def _plain_scan_step(s):
    case, live = s["case"], s["live"]
    G, S, D = case["G"], case["S"], case["D"]
    at = s["pages"][live].long()
    u, _, dt, gate, B, C, A = (x if i == 6 else x[live] for i, x in enumerate(_scan_inputs(s)))
    h = s["state"][at].view(-1, G, D // G, S)
    h = torch.exp(dt[..., None] * A) * h + (dt * u)[..., None] * B[:, :, None]
    y = ((h * C[:, :, None]).sum(-1) + s["skip"].view(G, -1) * u) * gate * torch.sigmoid(gate)
    out = torch.zeros_like(s["u"])
    out[live] = y.reshape(-1, D).to(out.dtype)
    s["state"][at] = h.reshape(-1, D, S)
    return {"out": out, "state": s["state"]}


# ------------------------------------------------------------------ plain form: norm and rotation
EPS = 1e-6


def _turned(x, cos, sin, interleaved, R):
    """Pairs of the first R values of every row turned by the angle."""
    rest = x[..., R:]
    if interleaved:
        a, b = x[..., 0:R:2], x[..., 1:R:2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., :R // 2], x[..., R // 2:R]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([y, rest], -1)


def _norm(x, kind):
    """1 / norm of every row."""
    if kind == "none":
        return torch.ones_like(x[..., :1])
    return torch.rsqrt(((x * x).mean(-1, keepdim=True) if kind == "rms" else (x * x).sum(-1, keepdim=True)) + EPS)


def _rotary_one(s, name, ft):
    case, x = s["case"], s[name].to(ft)
    R, kind = case["R"], case["norm"]
    angle = s["positions"].double()[..., None, None] * s["freqs"]     # [B, T, 1, R / 2]
    cos, sin = (torch.cos(angle) * s["amplitude"]).to(ft), (torch.sin(angle) * s["amplitude"]).to(ft)
    w = s[name + "_weight"]
    r = _norm(x, kind)
    n = x * r
    y = _turned(n if w is None else n * w.to(ft), cos, sin, case["interleaved"], R)
    if case["op"] == "rotary":
        return y, None, None
    d = _turned(s["d" + name].to(ft), cos, -sin, case["interleaved"], R)   # the transposed rotation
    dw = None if w is None else (d * n).sum((0, 1, 2), dtype=F64)
    if w is not None:
        d = d * w.to(ft)
    if kind != "none":
        dot = (d * n).mean(-1, keepdim=True) if kind == "rms" else (d * n).sum(-1, keepdim=True)
        d = r * (d - n * dot)
    return y, d, dw


def _rotary(s, ft):
    out = {}
    for name in ("q", "k"):
        y, d, dw = _rotary_one(s, name, ft)
        cast = (lambda t: t) if ft == F64 else (lambda t: t.to(s[name].dtype))
        out[name] = cast(y)
        if d is not None:
            out["d" + name] = cast(d)
            if dw is not None:
                out["d" + name + "_weight"] = dw if ft == F64 else dw.float()
    return out


# ------------------------------------------------------------------ a pass
def run(state):
    s, op = state, state["case"]["op"]
    if not own:
        if op.startswith("conv"):
            return _plain_conv_step(s) if op == "conv_step" else _plain_conv(s)
        if op.startswith("scan"):
            return _plain_scan_step(s) if op == "scan_step" else _plain_scan(s)
        return _rotary(s, F32)
    from chunked_gated_delta_05_amd import binding
    case = s["case"]
    if op.startswith("conv"):
        act = "silu" if case["act"] else None
        if op == "conv_step":
            y = binding.gdn_conv_step(s["x"], s["weight"], s["state"], s["bias"], activation=act, pages=s["pages"])
            return {"y": y, "state": s["state"]}
        y, final = binding.gdn_conv_fwd(s["x"], s["weight"], s["bias"], activation=act, meta=s["meta"],
                                        initial_state=s["s0"], output_final_state=case["states"])
        r = {"y": y, "final": final} if case["states"] else {"y": y}
        if op == "conv_train":
            r.update(binding.gdn_conv_bwd(s["x"], s["weight"], s["bias"], s["dout"], activation=act, meta=s["meta"],
                                          initial_state=s["s0"], dfinal=s["dfinal"], want_dinitial=case["states"]))
        return r
    if op == "scan_step":
        out = binding.gdn_scan_step(s["u"], s["dt"], s["A"], s["B"], s["C"], s["state"], s["skip"], s["gate"],
                                    dt_bias=s["dt_bias"], dt_softplus=True, pages=s["pages"])
        return {"out": out, "state": s["state"]}
    if op.startswith("scan"):
        train = op == "scan_train"
        out, final, h = binding.gdn_scan_fwd(s["u"], s["dt"], s["A"], s["B"], s["C"], s["skip"], s["gate"],
                                             dt_bias=s["dt_bias"], dt_softplus=True, meta=s["meta"],
                                             initial_state=s["s0"], output_final_state=case["states"], want_h=train)
        r = {"out": out, "final": final} if case["states"] else {"out": out}
        if train:
            r.update(binding.gdn_scan_bwd(s["u"], s["dt"], s["A"], s["B"], s["C"], s["skip"], s["gate"], s["dout"], h,
                                          dt_bias=s["dt_bias"], dt_softplus=True, meta=s["meta"], dht=s["dht"],
                                          want_dh0=case["states"]))
        return r
    norm = None if case["norm"] == "none" else case["norm"]
    kw = dict(norm=norm, q_weight=s["q_weight"], k_weight=s["k_weight"], eps=EPS, interleaved=case["interleaved"],
              amplitude=s["amplitude"])
    q, k = binding.gdn_qk_rotary_fwd(s["q"], s["k"], s["freqs"], s["positions"], **kw)
    r = {"q": q, "k": k}
    if op == "rotary_train":
        r.update(binding.gdn_qk_rotary_bwd(s["q"], s["k"], s["freqs"], s["positions"], s["dq"], s["dk"], **kw))
    return r


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    c, op = case, case["op"]
    es = 2 if c["dtype"] == "bf16" else 4
    if op.startswith("conv"):
        D, W = c["D"], c["W"]
        if op == "conv_step":
            n = (c["N"] - c["empty"]) * D
            return {"bytes": n * es * (2 + 2 * (W - 1)) + D * (W + 1) * es, "flops": 2.0 * n * W}
        n, units = c["B"] * c["T"] * D, c["docs"] or c["B"]
        state = units * (W - 1) * D * es if c["states"] else 0
        if op == "conv":
            return {"bytes": 2 * n * es + 2 * state, "flops": 2.0 * n * W}
        # x, dout read, y, dx written; the forward's and two products of the gradient
        return {"bytes": 4 * n * es + 4 * state, "flops": 6.0 * n * W}
    if op.startswith("scan"):
        D, S, G = c["D"], c["S"], c["G"]
        if op == "scan_step":
            n = c["N"] - c["empty"]
            return {"bytes": n * (D * (8.0 * S + 4 * es) + 2 * G * S * es) + D * S * 4, "flops": 7.0 * n * D * S}
        tokens, units = c["B"] * c["T"], c["docs"] or c["B"]
        state = units * D * S * 4 if c["states"] else 0
        if op == "scan":
            # a decay's product and exponential, the input's product, the update and the sum with C
            return {"bytes": tokens * (4 * D + 2 * G * S) * es + 2 * state, "flops": 7.0 * tokens * D * S}
        # gradients: g, its decay, and the sums for u, B, C, dt and A
        return {"bytes": tokens * (8 * D + 4 * G * S) * es + 4 * state, "flops": (7.0 + 14.0) * tokens * D * S}
    n = c["B"] * c["T"] * (c["Hq"] + c["Hk"]) * c["D"]
    return {"bytes": n * es * (2 if op == "rotary" else 4), "flops": n * (7.0 if op == "rotary" else 19.0)}


# ------------------------------------------------------------------ the definitions in 64 bits
def _conv_exact(s):
    """By sequences: the state's rows, the tokens, one window a token."""
    case, W = s["case"], s["case"]["W"]
    D, dt = case["D"], s["x"].dtype
    x, w = s["x"].reshape(-1, D).double(), s["weight"].double()
    b = torch.zeros(D, dtype=F64, device="cuda") if s["bias"] is None else s["bias"].double()
    train = case["op"] == "conv_train"
    ys, finals, dxs, d0s = [], [], [], []
    dw, db = torch.zeros_like(w), torch.zeros_like(b)
    for n, (lo, hi) in enumerate(zip(s["offsets"], s["offsets"][1:])):
        head = x.new_zeros(W - 1, D) if s["s0"] is None else s["s0"][n].double()
        seq = torch.cat([head, x[lo:hi]])
        L = hi - lo
        z = b.expand(L, D).clone()
        for j in range(W):
            z += seq[j:j + L] * w[:, j]
        sg = 1 / (1 + torch.exp(-z))
        ys.append(z * sg if case["act"] else z)
        finals.append(seq[L:].to(dt))
        if train:
            dz = s["dout"].reshape(-1, D)[lo:hi].double()
            if case["act"]:
                dz = dz * (sg + z * sg * (1 - sg))
            dseq = torch.zeros_like(seq)
            for j in range(W):
                dseq[j:j + L] += dz * w[:, j]
                dw[:, j] += (dz * seq[j:j + L]).sum(0)
            db += dz.sum(0)
            if case["states"]:
                dseq[L:] += s["dfinal"][n].double()
            dxs.append(dseq[W - 1:])
            d0s.append(dseq[:W - 1])
    lead = _lead(case)
    r = {"y": torch.cat(ys).view(*lead, D)}
    if case["states"]:
        r["final"] = torch.stack(finals)
    if train:
        r["dweight"] = dw
        if s["bias"] is not None:
            r["dbias"] = db
        if case["states"]:
            r["dinitial"] = torch.stack(d0s)
        r["dx"] = torch.cat(dxs).view(*lead, D)
    return r


def _scan_exact(s):
    """Token by token over all sequences at once (padded to the longest)."""
    case = s["case"]
    D, S, G, offs = case["D"], case["S"], case["G"], s["offsets"]
    n, length = len(offs) - 1, [b - a for a, b in zip(offs, offs[1:])]
    T = max(length)

    def pad(x):
        x = x.double().reshape(-1, *((G, S) if x.dim() == s["B"].dim() else (D,)))
        out = x.new_zeros(T, n, *x.shape[1:])
        for i, (a, b) in enumerate(zip(offs, offs[1:])):
            out[:b - a, i] = x[a:b]
        return out

    def unpad(x):
        return torch.cat([x[:b - a, i] for i, (a, b) in enumerate(zip(offs, offs[1:]))])

    each = lambda x: x.repeat_interleave(D // G, dim=-2)   # a group's row for each of its channels
    u, gate = pad(s["u"]), pad(s["gate"])
    raw = pad(s["dt"]) + s["dt_bias"].double()
    dt = torch.logaddexp(raw, torch.zeros_like(raw))
    B, C, A, skip = pad(s["B"]), pad(s["C"]), s["A"].double(), s["skip"].double()
    h = torch.zeros(n, D, S, dtype=F64, device="cuda") if s["s0"] is None else s["s0"].double()
    live = torch.arange(T, device="cuda")[:, None] < torch.tensor(length, device="cuda")
    train = case["op"] == "scan_train"
    y = torch.zeros_like(u)
    kept = []
    for t in range(T):
        if train:
            kept.append(h)
        new = torch.exp(dt[t, ..., None] * A) * h + (dt[t] * u[t])[..., None] * each(B[t])
        y[t] = (new * each(C[t])).sum(-1) + skip * u[t]
        h = torch.where(live[t][:, None, None], new, h)
    p = 1 / (1 + torch.exp(-gate))
    lead = _lead(case)
    r = {"out": unpad(y * gate * p).view(*lead, D)}
    if case["states"]:
        r["final"] = h
    if not train:
        return r
    dout = pad(s["dout"])
    dy = dout * gate * p
    E = torch.zeros_like(h) if s["dht"] is None else s["dht"].double()
    du, ddt = torch.zeros_like(u), torch.zeros_like(u)
    dB, dC = torch.zeros_like(B), torch.zeros_like(C)
    dA = torch.zeros_like(A)
    sums = lambda x: x.view(n, G, D // G, S).sum(2)
    for t in reversed(range(T)):
        on = live[t][:, None, None]
        before = kept.pop()
        a = torch.exp(dt[t, ..., None] * A)
        g = torch.where(on, dy[t][..., None] * each(C[t]) + E, torch.zeros_like(E))
        now = a * before + (dt[t] * u[t])[..., None] * each(B[t])
        dC[t], dB[t] = sums(dy[t][..., None] * now), sums((dt[t] * u[t])[..., None] * g)
        ddu = (g * each(B[t])).sum(-1)
        w = a * g * before
        dA += (w * dt[t][..., None]).sum(0)
        du[t] = dt[t] * ddu + skip * dy[t]
        ddt[t] = (u[t] * ddu + (w * A).sum(-1)) / (1 + torch.exp(-raw[t]))
        E = torch.where(on, a * g, E)
    r["dB"], r["dC"] = unpad(dB).view(*lead, G, S), unpad(dC).view(*lead, G, S)
    if s["s0"] is not None:
        r["dh0"] = E
    r["dA"], r["du"], r["ddt"] = dA, unpad(du).view(*lead, D), unpad(ddt).view(*lead, D)
    r["dgate"] = unpad(dout * y * p * (1 + gate * (1 - p))).view(*lead, D)
    r["dskip"], r["ddt_bias"] = unpad(dy * u).sum(0), unpad(ddt).sum(0)
    return r


def _rotary_exact(s):
    """The rotation as a product of complex numbers, gradients by autograd."""
    case = s["case"]
    R, D, train = case["R"], case["D"], case["op"] == "rotary_train"
    turn = torch.polar(torch.full((case["B"], case["T"], 1, R // 2), float(s["amplitude"]), dtype=F64, device="cuda"),
                       s["positions"].double()[..., None, None] * s["freqs"])
    out = {}
    for name in ("q", "k"):
        x = s[name].double().requires_grad_(train)
        w = s[name + "_weight"]
        w = None if w is None else w.double().requires_grad_(train)
        y = x
        if case["norm"] != "none":
            size = (x ** 2).sum(-1, keepdim=True) / (D if case["norm"] == "rms" else 1)
            y = x / torch.sqrt(size + EPS)
        if w is not None:
            y = y * w
        pairs = y[..., :R].unflatten(-1, (R // 2, 2)) if case["interleaved"] else \
            y[..., :R].unflatten(-1, (2, R // 2)).transpose(-1, -2)
        z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
        z = z.flatten(-2) if case["interleaved"] else z.transpose(-1, -2).flatten(-2)
        y = torch.cat([z, y[..., R:]], -1)
        if train:
            grads = torch.autograd.grad(y, [x] if w is None else [x, w], s["d" + name].double())
            out["d" + name] = grads[0]
            if w is not None:
                out["d" + name + "_weight"] = grads[1]
        out[name] = y.detach()
    return out


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op in ("rotary", "rotary_train"):
        return _rotary_exact(s)
    if op == "conv_step":
        live = s["live"].tolist()
        y = torch.zeros(case["N"], case["D"], dtype=F64, device="cuda")
        state, w = s["state"].clone(), s["weight"].double()
        for n in live:
            page = int(s["pages"][n])
            seen = torch.cat([s["state"][page], s["x"][n][None]])
            z = (seen.double() * w.t()).sum(0) + (0 if s["bias"] is None else s["bias"].double())
            y[n] = z / (1 + torch.exp(-z)) if case["act"] else z
            state[page] = seen[1:]
        return {"y": y, "state": state}
    if op == "scan_step":
        D, G = case["D"], case["G"]
        state, A = s["state"].double(), s["A"].double()
        out = torch.zeros(case["N"], D, dtype=F64, device="cuda")
        for n in s["live"].tolist():
            page = int(s["pages"][n])
            raw = s["dt"][n].double() + s["dt_bias"].double()
            dt = torch.logaddexp(raw, torch.zeros_like(raw))
            B, C = (s[x][n].double().repeat_interleave(D // G, dim=0) for x in "BC")
            u, gate = s["u"][n].double(), s["gate"][n].double()
            h = torch.exp(dt[:, None] * A) * state[page] + (dt * u)[:, None] * B
            out[n] = ((h * C).sum(-1) + s["skip"].double() * u) * gate / (1 + torch.exp(-gate))
            state[page] = h
        return {"out": out, "state": state}
    if op.startswith("conv"):
        return _conv_exact(s)
    # the states that a gradient in 64 bits keeps, and the time of its tokens one by one
    longest = max(b - a for a, b in zip(s["offsets"], s["offsets"][1:]))
    kept = 8.0 * longest * (len(s["offsets"]) - 1) * case["D"] * case["S"]
    if (op == "scan_train" and kept > 40e9) or longest > 20000:
        return None
    return _scan_exact(s)
