"""The operators around the recurrent layers against 64-bit references, at the
sizes and options where they can go wrong.

Tolerances. An output in bf16 is rounded once, by half a step, 2^-8 of the value
(eps / 2); an fp32 one by 2^-24. What the kernels compute before that is fp32,
and its error is bounded by a multiple n of 2^-24 of the same formula over
absolute values ("scale"):
* convolution: W products and sums and the exponential, reciprocal and products
  of silu: n = 24; sums over tokens add one for each token.
* scan: a decay e^(t A) is off by the rounding of A log2(e), of the product and
  of t (softplus: 6 steps) times the exponent, |t A| <= 2 here, and by the
  exponential's own step: at most 20 steps, and the update rounds twice more;
  these add up over a sequence's L tokens, and in gradients over both directions
  and the sums over tokens or channels (D, N): n = 24 L + 64 for states and
  outputs, twice that + D + N for gradients.
* norms and rotation: a row's sum, root, products, the angle's cosine and sine
  (each to 2^-23) and their products: n = 32 of the row's largest magnitude
  (times sqrt D for gradients, whose projection sums D terms); sums over rows add
  one for each row.
"""
import math

import pytest
import torch

import mixer_ref as ref
from chunked_gated_delta_05_amd import binding as gb

pytestmark = pytest.mark.gpu
BF, F32, F64, I32 = torch.bfloat16, torch.float32, torch.float64, torch.int32
DT = {"bf16": BF, "fp32": F32}


def gen(seed):
    return torch.Generator().manual_seed(seed)


def randn(g, *shape, dtype=F32):
    return torch.randn(*shape, generator=g).to(dtype).cuda()


def near(got, want, scale, n, what):
    """|got - want| <= half a step of got's type + n 2^-24 scale"""
    got, eps = got.detach().cpu(), torch.finfo(got.dtype).eps
    err = (got.double() - want.reshape(got.shape)).abs()
    tol = eps / 2 * want.abs().reshape(got.shape) * 1.01 + n * 2.0 ** -24 * scale.reshape(got.shape) + 1e-37
    assert torch.isfinite(got).all(), what
    bad = (err > tol).nonzero()
    assert not len(bad), f"{what}: {len(bad)} of {err.numel()}, worst {float((err / tol).max()):.3g} tolerances, first at {bad[0].tolist()}"


def layout(lead):
    """Token axes, offsets, meta of dense rows (B, T) or packed lengths [..]."""
    if isinstance(lead, tuple):
        return lead, [b * lead[1] for b in range(lead[0] + 1)], None
    offs = [0]
    for n in lead:
        offs.append(offs[-1] + n)
    return (offs[-1],), offs, gb.make_meta(offs, offs[-1], "cuda")


# ------------------------------------------------------------------ convolution
CONV = [((1, 1), 8), ((2, 3), 16), ((3, 7), 40), ((1, 8), 24), ((2, 9), 136), ((1, 65), 520), ((2, 130), 64),
        ([1], 8), ([1, 2, 3, 1], 24), ([5, 1, 64, 2, 129], 72), ([300, 8, 16], 16)]


def conv_case(lead, D, W, dtype, bias=True, states=True, pad=0, seed=0, w_dtype=None):
    g = gen(seed)
    ld, offs, meta = layout(lead)
    n = len(offs) - 1
    dt = DT[dtype]
    x = randn(g, *ld, D + pad, dtype=dt)[..., :D]
    w = randn(g, D, W, dtype=w_dtype or dt)
    b = randn(g, D, dtype=w_dtype or dt) if bias else None
    s0 = randn(g, n, W - 1, D, dtype=dt) if states else None
    return dict(x=x, w=w, b=b, s0=s0, offs=offs, meta=meta, dout=randn(g, *ld, D, dtype=dt),
                dfinal=randn(g, n, W - 1, D, dtype=dt) if states else None)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("lead,D", CONV)
def test_conv(lead, D, W, dtype):
    for i, (bias, states, act, pad) in enumerate([(True, True, "silu", 0), (False, False, None, 8)]):
        c = conv_case(lead, D, W, dtype, bias, states, pad, seed=i)
        y, final = gb.gdn_conv_fwd(c["x"], c["w"], c["b"], activation=act, meta=c["meta"], initial_state=c["s0"],
                                   output_final_state=True)
        r = gb.gdn_conv_bwd(c["x"], c["w"], c["b"], c["dout"], activation=act, meta=c["meta"], initial_state=c["s0"],
                            dfinal=c["dfinal"])
        a = (c["x"], c["w"], c["b"], act == "silu", c["offs"], c["s0"], c["dout"], c["dfinal"])
        want, scale = ref.conv(*a), ref.conv(*a, absolute=True)
        near(y, want[0], scale[0], 24, "y")
        assert torch.equal(final.cpu().double(), want[1])
        assert ("dbias" in r) == bias
        for k, t in r.items():
            tokens = c["offs"][-1] if k in ("dweight", "dbias") else 0
            near(t, want[2][k], scale[2][k], 24 + tokens, k)


@pytest.mark.parametrize("dtype,w_dtype", [("bf16", F32), ("fp32", BF)])
def test_conv_parameters_of_another_type(dtype, w_dtype):
    c = conv_case((2, 33), 48, 3, dtype, w_dtype=w_dtype)
    y, _ = gb.gdn_conv_fwd(c["x"], c["w"], c["b"], initial_state=c["s0"])
    a = (c["x"], c["w"], c["b"], False, c["offs"], c["s0"])
    near(y, ref.conv(*a)[0], ref.conv(*a, absolute=True)[0], 24, "y")


def test_conv_of_nothing_keeps_the_state():
    s0 = randn(gen(1), 3, 3, 16, dtype=BF)
    x, w = torch.zeros(3, 0, 16, dtype=BF, device="cuda"), randn(gen(2), 16, 4, dtype=BF)
    y, final = gb.gdn_conv_fwd(x, w, initial_state=s0, output_final_state=True)
    assert y.shape == x.shape and torch.equal(final, s0)
    r = gb.gdn_conv_bwd(x, w, None, x, initial_state=s0, dfinal=s0)
    assert torch.equal(r["dinitial"], s0) and not r["dweight"].any()


@pytest.mark.parametrize("lead", [(3, 130), (3, 2), [4, 1, 200]])
def test_conv_pages_in_place(lead):
    # states come from and go to pages; a page that no sequence names stays, and -1 means zeros and nothing written
    c = conv_case(lead, 64, 4, "bf16", seed=3)
    pool = randn(gen(4), 6, 3, 64, dtype=BF)
    before = pool.clone()
    src, dst = torch.tensor([4, -1, 2], dtype=I32, device="cuda"), torch.tensor([4, 0, -1], dtype=I32, device="cuda")
    s0 = before[[4, 0, 2]].clone()
    s0[1] = 0
    y, final = gb.gdn_conv_fwd(c["x"], c["w"], c["b"], activation="silu", meta=c["meta"], initial_state=pool,
                               initial_pages=src, final_out=pool, final_pages=dst)
    a = (c["x"], c["w"], c["b"], True, c["offs"], s0)
    want = ref.conv(*a)
    near(y, want[0], ref.conv(*a, absolute=True)[0], 24, "y")
    assert final is pool or final.data_ptr() == pool.data_ptr()
    assert torch.equal(pool[[4, 0]].cpu().double(), want[1][[0, 1]])
    assert torch.equal(pool[[1, 2, 3, 5]], before[[1, 2, 3, 5]])


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("N,D", [(1, 8), (3, 24), (7, 520), (70, 64)])
def test_conv_step(N, D, W, dtype):
    g = gen(N + D + W)
    x, w = randn(g, N, D + 16, dtype=DT[dtype])[:, :D], randn(g, D, W, dtype=DT[dtype])
    b = randn(g, D, dtype=DT[dtype])
    pool = randn(g, N + 2, W - 1, D, dtype=DT[dtype])
    before = pool.clone()
    pages = torch.randperm(N + 2, generator=g)[:N].to(I32)
    if N > 2:
        pages[1] = -1
        pages[2] = N + 2
    live = (pages >= 0) & (pages < N + 2)
    y = gb.gdn_conv_step(x, w, pool, b, activation="silu", pages=pages.cuda())
    at = pages[live].long()
    want, scale, state = ref.conv_step(x[live.cuda()], w, b, True, before[at.cuda()])
    near(y[live.cuda()], want, scale, 24, "y")
    assert not y[~live.cuda()].any()
    assert torch.equal(pool[at.cuda()].cpu().double(), state)
    rest = [p for p in range(N + 2) if p not in at.tolist()]
    assert torch.equal(pool[rest], before[rest])
    # the same rows as prompts of one token
    y2, _ = gb.gdn_conv_fwd(x[live.cuda()][:, None].contiguous(), w, b, activation="silu", initial_state=before[at.cuda()])
    assert torch.equal(y2[:, 0], y[live.cuda()])


# ------------------------------------------------------------------ scan
def scan_case(lead, D, S, G, dtype, full=True, seed=0, pad=0, rate=1.0):
    """full: skip, gate, time bias through softplus and states; else none."""
    g = gen(seed)
    ld, offs, meta = layout(lead) if lead is not None else (None, None, None)
    n, dt = len(offs) - 1, DT[dtype]
    wide = randn(g, *ld, 3 * D + 2 * G * S + pad, dtype=dt)     # views of one projection
    u, t, z = (wide[..., i * D:(i + 1) * D] for i in range(3))
    rows = wide[..., 3 * D:3 * D + 2 * G * S].unflatten(-1, (2 * G, S))
    A = -torch.rand(D, S, generator=g).cuda() * rate
    c = dict(u=u, dt=t, A=A, B=rows[..., :G, :], C=rows[..., G:, :], skip=None, gate=None, dt_bias=None, softplus=full,
             s0=None, dht=None, offs=offs, meta=meta, dout=randn(g, *ld, D, dtype=dt))
    if full:
        c.update(skip=randn(g, D), gate=z, dt_bias=randn(g, D) - 2, s0=randn(g, n, D, S), dht=randn(g, n, D, S))
    else:
        c["dt"] = (t.float().abs() * 0.2).to(dt).contiguous()
    return c


def scan_gpu(c, **kw):
    return gb.gdn_scan_fwd(c["u"], c["dt"], c["A"], c["B"], c["C"], c["skip"], c["gate"], dt_bias=c["dt_bias"],
                           dt_softplus=c["softplus"], meta=c["meta"], initial_state=c["s0"], output_final_state=True, **kw)


def scan_gpu_bwd(c, h, **kw):
    return gb.gdn_scan_bwd(c["u"], c["dt"], c["A"], c["B"], c["C"], c["skip"], c["gate"], c["dout"], h,
                           dt_bias=c["dt_bias"], dt_softplus=c["softplus"], meta=c["meta"], dht=c["dht"], **kw)


def scan_args(c):
    return (c["u"], c["dt"], c["A"], c["B"], c["C"], c["skip"], c["gate"], c["dt_bias"], c["softplus"], c["offs"],
            c["s0"], c["dout"], c["dht"])


def check_scan(c):
    out, final, h = scan_gpu(c, want_h=True)
    r = scan_gpu_bwd(c, h)
    want, scale = ref.scan(*scan_args(c)), ref.scan(*scan_args(c), absolute=True)
    L = max(b - a for a, b in zip(c["offs"], c["offs"][1:]))
    n = 24 * L + 64
    near(out, want[0], scale[0], n, "out")
    near(final, want[1], scale[1], n, "final")
    assert set(r) == {k for k in want[2] if (k != "dskip" or c["skip"] is not None)
                      and (k != "ddt_bias" or c["dt_bias"] is not None)}
    for k, t in r.items():
        near(t, want[2][k], scale[2][k], 2 * n + c["u"].shape[-1] + c["offs"][-1], k)
    return out, final, r


SCAN = [((1, 1), 8, 1), ((2, 2), 24, 1), ((1, 15), 64, 1), ((2, 16), 72, 1), ((1, 17), 64, 2), ((3, 31), 16, 2),
        ((1, 32), 128, 1), ((2, 33), 40, 1), ((1, 100), 136, 1), ((1, 257), 48, 3), ([1], 8, 1), ([1, 1, 2], 16, 1),
        ([33, 1, 64, 15, 100], 72, 1), ([16, 16, 40], 48, 2), ([130, 70], 200, 1)]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("S", [8, 16, 32, 64])
@pytest.mark.parametrize("lead,D,G", SCAN)
def test_scan(lead, D, G, S, dtype):
    check_scan(scan_case(lead, D, S, G, dtype, full=True, seed=S))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("S", [8, 16, 64])
@pytest.mark.parametrize("lead,D,G", [((2, 40), 72, 1), ([5, 70, 1], 48, 2)])
def test_scan_without_options(lead, D, G, S, dtype):
    check_scan(scan_case(lead, D, S, G, dtype, full=False, seed=S, pad=8))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_scan_of_many_sequences_is_not_cut(dtype):
    check_scan(scan_case((260, 70), 16, 16, 1, dtype))


def test_scan_of_nothing_keeps_the_state():
    c = scan_case((2, 1), 16, 16, 1, "bf16")
    for k in ("u", "dt", "gate", "B", "C", "dout"):
        c[k] = c[k][:, :0].contiguous()
    out, final, h = scan_gpu(c, want_h=True)
    assert out.shape == (2, 0, 16) and torch.equal(final, c["s0"])
    r = scan_gpu_bwd(c, h)
    assert torch.equal(r["dh0"], c["dht"]) and not r["dA"].any() and not r["dskip"].any() and not r["ddt_bias"].any()


def test_scan_forgets_at_once():
    # decays that underflow: h is the last input alone
    c = scan_case((1, 40), 64, 16, 1, "fp32", rate=0.0)
    c["A"] -= 1e6
    c["dt"] = torch.ones_like(c["dt"])
    out, final, h = scan_gpu(c, want_h=True)
    c["softplus"], c["dt_bias"] = False, None
    c2 = dict(c, s0=torch.zeros_like(c["s0"]))
    one, fin, _ = scan_gpu(dict(c2, u=c["u"][:, -1:], dt=c["dt"][:, -1:], B=c["B"][:, -1:], C=c["C"][:, -1:],
                                gate=c["gate"][:, -1:]))
    c["softplus"] = False
    out, final, h = scan_gpu(c, want_h=True)
    assert torch.equal(final, fin) and torch.equal(out[:, -1:], one)
    r = scan_gpu_bwd(c, h)
    assert not r["dh0"].any() and all(torch.isfinite(t).all() for t in r.values())


@pytest.mark.parametrize("lead", [(3, 100), (3, 5), [130, 1, 40]])
def test_scan_pages_in_place(lead):
    c = scan_case(lead, 72, 16, 1, "bf16")
    pool = randn(gen(9), 6, 72, 16)
    before = pool.clone()
    src, dst = torch.tensor([4, -1, 2], dtype=I32, device="cuda"), torch.tensor([4, 0, -1], dtype=I32, device="cuda")
    s0 = before[[4, 0, 2]].clone()
    s0[1] = 0
    c["s0"] = pool
    out, final, _ = scan_gpu(c, initial_pages=src, final_out=pool, final_pages=dst)
    c["s0"] = s0
    want, wfinal, _ = scan_gpu(c)
    assert torch.equal(out, want) and torch.equal(pool[[4, 0]], wfinal[[0, 1]])
    assert torch.equal(pool[[1, 2, 3, 5]], before[[1, 2, 3, 5]])


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("S", [8, 16, 32, 64])
@pytest.mark.parametrize("N,D,G", [(1, 8, 1), (3, 24, 1), (5, 48, 2), (70, 136, 1)])
def test_scan_step(N, D, G, S, dtype):
    c = scan_case((N, 1), D, S, G, dtype, seed=N)
    g = gen(N + 1)
    pool = randn(g, N + 2, D, S)
    before = pool.clone()
    pages = torch.randperm(N + 2, generator=g)[:N].to(I32)
    if N > 2:
        pages[1] = -1
        pages[2] = N + 2
    live = ((pages >= 0) & (pages < N + 2)).cuda()
    row = lambda k: c[k][:, 0]
    out = gb.gdn_scan_step(row("u"), row("dt"), c["A"], row("B"), row("C"), pool, c["skip"], row("gate"),
                           dt_bias=c["dt_bias"], dt_softplus=True, pages=pages.cuda())
    at = pages.cuda()[live].long()
    a = [x[live] if i in (0, 1, 3, 4, 6) else x for i, x in enumerate(scan_args(c)[:9])]
    a += [list(range(int(live.sum()) + 1)), before[at]]
    want, scale = ref.scan(*a), ref.scan(*a, absolute=True)
    near(out[live], want[0], scale[0], 88, "out")
    near(pool[at], want[1], scale[1], 88, "state")
    assert not out[~live].any()
    rest = [p for p in range(N + 2) if p not in at.tolist()]
    assert torch.equal(pool[rest], before[rest])


# ------------------------------------------------------------------ norms and rotation
ROT = [((1, 1), 1, 1, 64, 64), ((2, 3), 4, 2, 128, 128), ((1, 7), 7, 1, 80, 40), ((3, 5), 2, 2, 256, 256),
       ((2, 9), 3, 3, 192, 64), ((1, 33), 5, 1, 8, 8), ((9,), 16, 4, 128, 64), ((2, 11), 2, 2, 128, 0),
       ((1, 2100), 2, 1, 64, 16)]


def rotary_case(lead, Hq, Hk, D, R, dtype, seed=0, weights=True):
    g = gen(seed)
    dt = DT[dtype]
    qkv = randn(g, *lead, Hq + 2 * Hk, D, dtype=dt)
    freqs = gb.rotary_frequencies(R, 500000.0, factor=8, scaling="by_turns", original_length=8192, device="cuda") if R else None
    pos = torch.randint(-50, 1000000, lead, generator=g).cuda()
    w = [1 + 0.2 * randn(g, D) for _ in range(2)] if weights else [None, None]
    return dict(q=qkv[..., :Hq, :], k=qkv[..., Hq:Hq + Hk, :], freqs=freqs, pos=pos, w=w,
                dq=randn(g, *lead, Hq, D, dtype=dt), dk=randn(g, *lead, Hk, D, dtype=dt))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("norm,weights", [("rms", True), ("l2", False), (None, True)])
@pytest.mark.parametrize("lead,Hq,Hk,D,R", ROT)
def test_rotary(lead, Hq, Hk, D, R, norm, weights, interleaved, dtype):
    c = rotary_case(lead, Hq, Hk, D, R, dtype, seed=D + R, weights=weights)
    kw = dict(norm=norm, q_weight=c["w"][0], k_weight=c["w"][1], eps=1e-5, interleaved=interleaved, amplitude=1.25)
    q, k = gb.gdn_qk_rotary_fwd(c["q"], c["k"], c["freqs"], c["pos"], **kw)
    r = gb.gdn_qk_rotary_bwd(c["q"], c["k"], c["freqs"], c["pos"], c["dq"], c["dk"], **kw)
    want = ref.rotary(c["q"], c["k"], c["freqs"], c["pos"], norm, *c["w"], 1e-5, interleaved, 1.25, c["dq"], c["dk"])
    rows = lambda x: x.abs().amax(-1, keepdim=True).expand_as(x)
    tokens = c["pos"].numel()
    for name, got in (("q", q), ("k", k)):
        near(got, want[name], rows(want[name]), 32, name)
    heads = {"q": Hq, "k": Hk}
    for name, got in r.items():
        if name.endswith("weight"):
            n = name[1]
            x = ref.f64(c[n])
            y = ref.rotary(c["q"], c["k"], None, c["pos"], norm, None, None, 1e-5, False, 1.0)[n]
            scale = (rows(y) * 1.25 * rows(ref.f64(c["d" + n])) * 2).flatten(0, -2).sum(0)
            near(got, want[name], scale, 32 + tokens * heads[n], name)
        else:
            # r (dn - n <dn, n>): at most (1 + D / D) of the row's r |d| |w| sqrt(D)
            x, d = ref.f64(c[name[1]]), ref.f64(c[name])
            size = {"rms": (x * x).mean(-1, keepdim=True), "l2": (x * x).sum(-1, keepdim=True)}
            inv = 1.0 if norm is None else 1 / torch.sqrt(size[norm] + 1e-5)
            scale = (inv * d.norm(dim=-1, keepdim=True) * 1.25 * 2 * (2 if weights else 1)).expand_as(x)
            near(got, want[name], scale, 32, name)


def test_rotary_positions_of_rows_and_in_place():
    c = rotary_case((3, 6), 2, 2, 64, 64, "bf16")
    q, k = c["q"].contiguous(), c["k"].contiguous()
    at = torch.arange(6, device="cuda").expand(3, 6)
    want = gb.gdn_qk_rotary_fwd(q, k, c["freqs"], at.contiguous())
    got = gb.gdn_qk_rotary_fwd(q, k, c["freqs"])
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    got = gb.gdn_qk_rotary_fwd(q, k, c["freqs"], at.to(I32).contiguous(), q_out=q, k_out=k)
    assert got[0].data_ptr() == q.data_ptr() and torch.equal(q, want[0]) and torch.equal(k, want[1])


def test_rotary_turns_whole_turns_exactly():
    # a quarter turn a token, exactly: x -> (-b, a) and so on, far out as well
    freqs = torch.full((4,), math.pi / 2, dtype=F64, device="cuda")
    q = randn(gen(0), 1, 8, 1, 8)
    # (a position that pi / 2 in 64 bits still resolves to 2^-24 of a turn)
    at = torch.arange(8, device="cuda")[None] + 4000000
    got, _ = gb.gdn_qk_rotary_fwd(q, q, freqs, at, norm=None)
    a, b = q[..., :4], q[..., 4:]
    for t in range(8):
        want = [(a, b), (-b, a), (-a, -b), (b, -a)][t % 4]
        want = torch.cat([want[0][0, t], want[1][0, t]], -1)
        assert (got[0, t] - want).abs().max() <= 2.0 ** -22 * want.abs().max()
