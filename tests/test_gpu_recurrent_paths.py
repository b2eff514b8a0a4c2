"""Paths of the recurrent-state operators that only some sizes take, on the
GPU against 64-bit references (the bounds are those of test_gpu_recurrent.py,
where they are derived)."""
import ctypes

import pytest
import torch

import recurrent_ref as ref
from chunked_gated_delta_05_amd import binding as gb
from test_gpu_recurrent import DEV, DT, prompt, within
from test_recurrent_checks import LinattnDesc, status_of

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ dh0 in place of dht or the entry states
def bwd(x, dh0, s_in, dht):
    """gdn_linattn_bwd with the caller's dh0, through the C ABI."""
    B, T, H, K = x["q"].shape
    V = x["v"].shape[-1]
    code = 1 if x["q"].dtype == torch.bfloat16 else 0
    d = LinattnDesc(B=B, T=T, H=H, Hq=H, Hk=H, Hv=H, K=K, V=V, dtype=code, o_dtype=code, scale=x["scale"])
    for n, w in (("q", K), ("k", K), ("v", V)):
        getattr(d, n + "_stride")[:] = (H * w, w)
    grads = [torch.empty_like(x[n]) for n in "qkv"]
    p = lambda t: ctypes.c_void_p(t.data_ptr())
    nb = ctypes.c_size_t(0)
    stream = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)

    def call(ws):
        return status_of("gdn_linattn_bwd", ctypes.byref(d), p(x["q"]), p(x["k"]), p(x["v"]), p(x["decay"]), p(s_in),
                         p(x["dout"]), p(dht), *(p(g) for g in grads), p(dh0), ws, ctypes.byref(nb), stream)

    assert call(ctypes.c_void_p(None)) == gb.GDN_OK
    ws = torch.empty(nb.value, dtype=torch.uint8, device=DEV)
    assert call(p(ws)) == gb.GDN_OK
    torch.cuda.synchronize()
    return grads


@pytest.mark.parametrize("over", ["dht", "S0"])
@pytest.mark.parametrize("K,V", [(128, 128), (64, 128)])
@pytest.mark.parametrize("dtype,B,T", [("bf16", 3, 90), ("bf16", 2, 500), ("fp32", 2, 250), ("bf16", 1, 1500)])
def test_an_entry_state_gradient_in_place(dtype, B, T, K, V, over):
    # uncut, in few segments, in many: the same bits as with a buffer of its own
    x = prompt(("", [T] * B, False, 2, 2, 2, 2), dtype, K, V, "spread")
    want = gb.gdn_linattn_bwd(x["q"], x["k"], x["v"], x["decay"], x["dout"], x["scale"], initial_state=x["S0"],
                              dht=x["dht"])
    for _ in range(3):
        state = {"dht": x["dht"].clone(), "S0": x["S0"].clone()}
        got = bwd(x, state[over], state["S0"], state["dht"])
        assert torch.equal(state[over], want["dh0"])
        for g, n in zip(got, ("dq", "dk", "dv")):
            assert torch.equal(g, want[n]), n


# ------------------------------------------------------------------ decays over many tokens
def awkward(n, lo=-1e-3, hi=-1e-4):
    """n log decays whose e^g lies almost half a step beside the nearest fp32 number."""
    g = torch.linspace(lo, hi, 20001)
    d = torch.exp(g.double())
    off = (d.float().double() - d).abs() / d
    return g[off.argsort(descending=True)[:n]].sort().values


def remaining(S0, S, g, n, exp2=False):
    """How far S is from b^{g n} S0, relative to it, over its bound. Every step
    rounds an element once, by at most 2^-24, here or there by chance: 8
    standard deviations of n such errors, 2^-24 / sqrt(3) each, hold for all
    elements; b^g - 1 to 2^-22 adds n |g| 2^-22."""
    g = g.detach().cpu().double()
    want = S0.cpu().double() * (torch.exp2(g * n) if exp2 else torch.exp(g * n))
    bound = 8 * 2.0 ** -24 * (n / 3) ** 0.5 + n * g.abs() * 2.0 ** -22
    return (((S.cpu().double() - want) / want).abs() / bound).max().item()


def test_a_weak_decay_does_not_drift_over_linear_steps():
    n, H = 4096, 4
    decay = awkward(H).to(DEV)
    S0 = torch.randn(1, H, 128, 64, generator=torch.Generator().manual_seed(1)).to(DEV)
    S, zero, v = S0.clone(), torch.zeros(1, H, 128, device=DEV), torch.ones(1, H, 64, device=DEV)
    for _ in range(n):
        gb.gdn_linattn_step(zero, zero, v, decay, S)
    assert remaining(S0, S, decay.view(1, H, 1, 1), n) <= 1


@pytest.mark.parametrize("per_key,exp2", [(False, False), (False, True), (True, False), (True, True)])
def test_a_weak_decay_does_not_drift_over_delta_steps(per_key, exp2):
    n, H = 4096, 4
    g = awkward(H * 128 if per_key else H).view(1, H, -1)
    g = (g if per_key else g[..., 0]).contiguous().to(DEV)
    S0 = torch.randn(1, H, 128, 128, generator=torch.Generator().manual_seed(2)).to(DEV)
    S, zero, v = S0.clone(), torch.zeros(1, H, 128, device=DEV), torch.ones(1, H, 128, device=DEV)
    beta = torch.ones(1, H, device=DEV)
    for _ in range(n):
        gb.gdn_recurrent_step(zero, zero, v, g, beta, S, use_exp2=exp2)
    assert remaining(S0, S, g.view(1, H, -1, 1), n, exp2) <= 1


# ------------------------------------------------------------------ autograd sees what is written in place
def writers():
    """name, the tensors it writes, the call."""
    H, N = 2, 2
    z = lambda *s: torch.zeros(*s, device=DEV)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device=DEV)
    q, decay, pool = z(N, H, 128), z(H), z(3, H, 128, 128)
    out, p4 = z(N, H, 128), z(1, 4, 2, 8)
    yield "linear step", (pool, out), lambda: gb.gdn_linattn_step(q, q, q, decay, pool, out=out)
    yield "delta step", (pool, out), lambda: gb.gdn_recurrent_step(q, q, q, z(N, H), z(N, H), pool, out=out)
    x, o, fin = z(1, 5, H, 128), z(1, 5, H, 128), z(1, H, 128, 128)
    yield "prompt", (o, fin), lambda: gb.gdn_linattn_fwd(x, x, x, decay, out=o, final_out=fin)
    yield "prompt to a page", (pool,), lambda: gb.gdn_linattn_fwd(x, x, x, decay, final_out=pool, final_pages=i32(1))
    yield "copy", (p4,), lambda: gb.gdn_pages_copy(p4, p4.clone(), i32(1), i32(0))
    yield "fork", (p4,), lambda: gb.gdn_pages_fork(p4, i32(0, 1), i32(0, 0))
    yield "compact", (p4,), lambda: gb.gdn_pages_compact(p4, i32(3))


@pytest.mark.parametrize("i", range(7))
def test_a_write_in_place_is_seen_by_autograd(i):
    name, written, call = list(writers())[i]
    for t in written:
        w = torch.ones_like(t, requires_grad=True)
        y = (w * t).sum()       # saves t
        call()
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            y.backward()


@pytest.mark.parametrize("i", range(7))
def test_tensors_of_inference_mode_are_written_inside_and_outside(i):
    with torch.inference_mode():
        name, written, call = list(writers())[i]
        call()
    call()
    torch.cuda.synchronize()


# ------------------------------------------------------------------ devices
@pytest.mark.skipif(torch.cuda.device_count() < 2, reason="needs two GPUs")
def test_calls_run_on_their_tensors_device():
    # a tensor of a device that is not the current one
    def both(dev):
        gen = torch.Generator().manual_seed(3)
        x = [torch.randn(1, 70, 2, 128, generator=gen).to(dev) for _ in range(3)]
        decay, pool = torch.full((2,), -0.1, device=dev), torch.zeros(2, 2, 128, 128, device=dev)
        o, _ = gb.gdn_linattn_fwd(*x, decay)
        return o, gb.gdn_linattn_step(*(t[:, 0] for t in x), decay, pool), pool

    with torch.cuda.device(0):
        for a, b in zip(both("cuda:1"), both("cuda:0")):
            assert torch.equal(a.cpu(), b.cpu())


# ------------------------------------------------------------------ errors
def test_memory_that_is_not_there_raises_as_from_torch():
    x = torch.zeros(1, 1, 1, 64, dtype=torch.bfloat16, device=DEV).expand(1, 2 ** 21, 1, 64)
    with pytest.raises(torch.OutOfMemoryError):   # o alone is 1 TiB
        gb.gdn_linattn_fwd(x, x, x, torch.zeros(4096, device=DEV))


def test_a_flag_without_a_truth_value_raises_its_own_error():
    x, pool = torch.zeros(1, 2, 128, device=DEV), torch.zeros(1, 2, 128, 128, device=DEV)
    with pytest.raises(RuntimeError, match="ambiguous"):
        gb.gdn_recurrent_step(x, x, x, torch.zeros(1, 2, device=DEV), torch.zeros(1, 2, device=DEV), pool,
                              use_exp2=torch.zeros(2))
    assert not pool.any()


# ------------------------------------------------------------------ full-width walks
# From 129 segments' heads on (n below), a workgroup takes all 128 value
# columns; up to there two share them. Everything here has n >= 256 in the
# forward, where it is one walk a segment and head, and checks that.
def walks(x):
    """n: segments x heads of a call, from the workspace that it asks for."""
    q, k, v, offs = x["q"], x["k"], x["v"], x["offs"]
    H, K, V = x["decay"].shape[0], q.shape[-1], v.shape[-1]
    code = 1 if q.dtype == torch.bfloat16 else 0
    d = LinattnDesc(B=1, T=offs[-1], H=H, Hq=q.shape[-2], Hk=k.shape[-2], Hv=v.shape[-2], K=K, V=V, dtype=code,
                    o_dtype=code, scale=0.1)
    if x["meta"] is None:
        d.B, d.T = q.shape[0], q.shape[1]
    else:
        d.n_units = len(offs) - 1
        d.offsets_host = ctypes.cast(x["meta"].host, ctypes.POINTER(ctypes.c_int32))
        d.offsets_dev = x["meta"].offsets_dev.data_ptr()
    for n, t in (("q", q), ("k", k), ("v", v)):
        getattr(d, n + "_stride")[:] = (t.shape[-2] * t.shape[-1], t.shape[-1])
    nb, none = ctypes.c_size_t(0), ctypes.c_void_p(None)
    assert status_of("gdn_linattn_fwd", ctypes.byref(d), *[none] * 8, 0, none, none, ctypes.byref(nb), none) == gb.GDN_OK
    segs = nb.value // (H * K * V * 4) if nb.value > 256 else len(offs) - 1
    return segs * H, segs > len(offs) - 1


def chunked(q, k, v, decay, scale, offsets, S0, late=0, reverse=False, absolute=False):
    """o and final states of the recurrence in 64 bits on the GPU, 32 tokens at
    a time by its own definition: o_i = scale (sum_{j <= i} d^{i-j} (q_i . k_j)
    v_j + d^{i+1-late} q_i S); late: the decay follows a token's k v^T. [tokens,
    H, D] each, S0 [units, H, K, V]."""
    if absolute:
        q, k, v, S0, scale = q.abs(), k.abs(), v.abs(), S0.abs(), abs(scale)
    d = torch.exp(decay.double())
    power = lambda n: torch.where(n == 0, torch.ones_like(n), d[:, None] ** n)      # [H, n]; 0^0 = 1
    o, final = torch.empty(q.shape[0], q.shape[1], v.shape[2], dtype=torch.float64, device=DEV), S0.clone()
    for u, (a, b) in enumerate(zip(offsets, offsets[1:])):
        at = torch.arange(a, b, device=DEV)
        at = at.flip(0) if reverse else at
        for c in at.split(32):
            n, S = len(c), final[u]
            i = torch.arange(n, device=DEV, dtype=torch.float64)
            qc, kc, vc = (t[c].transpose(0, 1) for t in (q, k, v))                     # [H, n, D]
            gap = (i[:, None] - i[None, :]).clamp(min=0)
            inside = power(gap.flatten()[None].expand(len(d), -1)).view(-1, n, n).tril()
            y = ((qc @ kc.transpose(1, 2).contiguous()) * inside) @ vc
            y = y + power((i + 1 - late)[None].expand(len(d), -1))[..., None] * (qc @ S)
            o[c] = scale * y.transpose(0, 1)
            left = power((n - 1 + late - i)[None].expand(len(d), -1))[..., None]
            final[u] = power(torch.full((len(d), 1), float(n), dtype=torch.float64, device=DEV))[..., None] * S + \
                (left * kc).transpose(1, 2).contiguous() @ vc
    return o, final


def on_gpu(x, absolute=False):
    """The forward's and the backward's results in 64 bits."""
    H, scale, offs, decay = x["decay"].shape[0], x["scale"], x["offs"], x["decay"]
    flat = lambda t: t.double().reshape(-1, *t.shape[-2:])
    q, k, v, do = (flat(x[n]).repeat_interleave(H // x[n].shape[-2], dim=1) for n in ("q", "k", "v", "dout"))
    zero = torch.zeros(len(offs) - 1, H, q.shape[2], v.shape[2], dtype=torch.float64, device=DEV)
    S0 = zero if x["S0"] is None else x["S0"].double()
    D = zero if x["dht"] is None else x["dht"].double()
    T = lambda t: t.transpose(-1, -2).contiguous()
    o, fin = chunked(q, k, v, decay, scale, offs, S0, absolute=absolute)
    dq, _ = chunked(do, v, k, decay, scale, offs, T(S0), absolute=absolute)
    dk, _ = chunked(v, scale * do, q, decay, 1.0, offs, T(D), late=1, reverse=True, absolute=absolute)
    dv, dh0 = chunked(k, scale * q, do, decay, 1.0, offs, D, late=1, reverse=True, absolute=absolute)
    return {"o": o, "fin": fin, "dq": dq, "dk": dk, "dv": dv, "dh0": dh0}


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_the_reference_in_chunks_is_the_one_by_tokens(dtype):
    x = prompt(("", [1, 32, 33, 70], True, 4, 4, 2, 1), dtype, 64, 128, "mixed")
    args = (x["q"], x["k"], x["v"], x["decay"], x["scale"], x["offs"], x["S0"])
    for absolute in (False, True):
        got = on_gpu(x, absolute)
        want = dict(zip(("o", "fin"), ref.linattn(*args, absolute=absolute)))
        want.update(zip(("dq", "dk", "dv", "dh0"),
                        ref.linattn_grads(*args, x["dout"], x["dht"], absolute=absolute)))
        for n in want:
            torch.testing.assert_close(got[n].cpu(), want[n], rtol=1e-11, atol=1e-11)


# name, lengths, packed, H, Hq, Hk, Hv, and whether the forward cuts them
WIDE = [
    ("rows, joined", [1000] * 4, False, 16, 16, 16, 16, True),
    ("rows", [200] * 17, False, 16, 16, 8, 16, False),
    ("row, merged", [2040], False, 32, 8, 32, 32, True),
    ("documents", [1 + 37 * i % 331 for i in range(20)], True, 16, 16, 4, 4, False),
    ("documents, joined", [1000] + [499, 500] * 12, True, 8, 8, 8, 4, True),
    ("documents, merged", [2600, 130, 1, 64, 300], True, 32, 32, 32, 32, True),
]


@pytest.mark.parametrize("states", [True, False], ids=["states", "no states"])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("K", [128, 64])
@pytest.mark.parametrize("case", WIDE, ids=lambda c: c[0])
def test_linattn_full_width(case, K, dtype, states):
    x = prompt(case[:-1], dtype, K, 128, "mixed", seed=7, states=states)
    n, cut = walks(x)
    assert n >= 256 and cut == case[-1]
    o, fin = gb.gdn_linattn_fwd(x["q"], x["k"], x["v"], x["decay"], x["scale"], meta=x["meta"],
                                initial_state=x["S0"], output_final_state=states)
    r = gb.gdn_linattn_bwd(x["q"], x["k"], x["v"], x["decay"], x["dout"], x["scale"], meta=x["meta"],
                           initial_state=x["S0"], dht=x["dht"], want_dh0=states)
    want, A = ({m: t.cpu() for m, t in on_gpu(x, absolute).items()} for absolute in (False, True))
    within(o, want["o"], A["o"], 2.0 ** -14, o.dtype, "o")
    for m, t in (("dq", "q"), ("dk", "k"), ("dv", "v")):
        h = x[t].shape[-2]
        within(r[m], ref.shared(want[m], h), ref.shared(A[m], h), 2.0 ** -14, r[m].dtype, m)
    if states:
        within(fin, want["fin"], A["fin"], 2.0 ** -17, fin.dtype, "final state")
        within(r["dh0"], want["dh0"], A["dh0"], 2.0 ** -17, torch.float32, "dh0")


# ------------------------------------------------------------------ beyond the last-level cache
# Steps on more than 256 MB of states, and page calls that walk through more,
# go around the caches, in kernels of their own.
BEYOND = 2 ** 28


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("K,V,N,H", [(128, 128, 131, 32), (64, 64, 515, 33), (64, 128, 260, 32), (128, 64, 260, 32)])
def test_a_linear_step_around_the_caches(K, V, N, H, dtype):
    assert N * H * K * V * 4 > BEYOND
    gen = torch.Generator(DEV).manual_seed(K + V)
    r = lambda *s: torch.randn(*s, generator=gen, device=DEV)
    q, k, v = (r(N, H, w).to(DT[dtype]) for w in (K, K, V))
    decay, pool = -torch.rand(H, generator=gen, device=DEV), r(N + 2, H, K, V)
    pages = torch.randperm(N + 2, generator=gen, device=DEV)[:N].to(torch.int32)
    pages[0], pages[N - 1] = -1, N + 2       # no page
    before = pool.clone()
    o = gb.gdn_linattn_step(q, k, v, decay, pool, pages=pages)
    assert not o[0].any() and not o[N - 1].any()
    rest = torch.ones(N + 2, dtype=torch.bool, device=DEV)
    rest[pages[1:-1].long()] = False
    assert rest.sum() == 4 and torch.equal(pool[rest], before[rest])
    for rows in torch.arange(1, N - 1).split(64):
        rows = rows.to(DEV)
        at = pages[rows].long()
        args = (q[rows], k[rows], v[rows], decay, K ** -0.5, before[at])
        want, S = ref.linattn_step(*args)
        A, AS = ref.linattn_step(*args, absolute=True)
        within(o[rows], want, A, 2.0 ** -16, o.dtype, "o")
        within(pool[at], S, AS, 2.0 ** -21, torch.float32, "state")


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("per_key", [False, True])
def test_a_delta_step_around_the_caches(per_key, dtype):
    N, H = 133, 32
    assert N * H * 128 * 128 * 4 > BEYOND
    gen = torch.Generator(DEV).manual_seed(5)
    r = lambda *s: torch.randn(*s, generator=gen, device=DEV)
    unit = lambda t: t / t.norm(dim=-1, keepdim=True)
    q, k, v = (t.to(DT[dtype]) for t in (unit(r(N, 8, 128)), unit(r(N, 8, 128)), r(N, H, 128)))
    g = -torch.rand(*((N, H, 128) if per_key else (N, H)), generator=gen, device=DEV)
    beta = torch.rand(N, H, generator=gen, device=DEV).to(DT[dtype])
    pool = r(N + 1, H, 128, 128)
    pages = torch.randperm(N + 1, generator=gen, device=DEV)[:N].to(torch.int32)
    pages[7] = -1
    before = pool.clone()
    o = gb.gdn_recurrent_step(q, k, v, g, beta, pool, pages=pages)
    assert not o[7].any()
    on = (pages >= 0).nonzero().flatten()
    rest = torch.ones(N + 1, dtype=torch.bool, device=DEV)
    rest[pages[on].long()] = False
    assert torch.equal(pool[rest], before[rest])
    for rows in on.split(48):
        at = pages[rows].long()
        args = (q[rows], k[rows], v[rows], g[rows], beta[rows], 128 ** -0.5, before[at])
        want, S = ref.delta_step(*args)
        A, AS = ref.delta_step(*args, absolute=True)
        within(o[rows], want, A, 2.0 ** -15, o.dtype, "o")
        within(pool[at], S, AS, 2.0 ** -16, torch.float32, "state")


def large_pool(pages, page_bytes, layers=2):
    """Every 4 bytes of a pool different."""
    return torch.arange(layers * pages * page_bytes // 4, dtype=torch.int32, device=DEV).view(layers, pages, -1)


def after(pool, copies):
    want = pool.clone()
    if copies:
        s, d = (torch.tensor(x, device=DEV) for x in zip(*copies))
        want[:, d] = pool[:, s]
    return want


@pytest.mark.parametrize("n,pages,page_bytes", [
    (40, 70, 4 << 20), (200, 230, (1 << 20) + 16), (500, 600, (1 << 19) + 4096),      # around the caches
    (6, 70, 4 << 20), (300, 600, 1 << 18)])                                             # few of a large pool: through them
def test_forks_and_compactions_of_large_pools(n, pages, page_bytes):
    gen = torch.Generator().manual_seed(n)
    order = torch.randperm(pages, generator=gen).tolist()
    table, spare = order[:n], order[n:n + 9]
    parent = torch.randint(-1, n // 2, (n,), generator=gen).tolist()
    table[2] = -1
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)
    pool = large_pool(pages, page_bytes)
    assert pool.nbytes > BEYOND
    new, copies, left = ref.fork(table, parent, spare, pages)
    want = after(pool, copies)
    got, gleft = gb.gdn_pages_fork(pool, i32(table), i32(parent), spare=i32(spare))
    assert got.tolist() == new and gleft.tolist() == left and torch.equal(pool, want)
    new, moves, count = ref.compact(table, pages)
    assert moves
    want = after(pool, moves)
    got, c = gb.gdn_pages_compact(pool, i32(table))
    assert got.tolist() == new and c.tolist() == [count] and torch.equal(pool, want)


def test_a_compaction_of_many_large_pages():
    # more pages than one kernel's plan holds
    pages, n = 1100, 700
    gen = torch.Generator().manual_seed(1)
    table = torch.randperm(pages, generator=gen)[:n].tolist()
    pool = large_pool(pages, 1 << 18)
    assert n * 2 * (1 << 18) > BEYOND
    new, moves, count = ref.compact(table, pages)
    want = after(pool, moves)
    got, c = gb.gdn_pages_compact(pool, torch.tensor(table, dtype=torch.int32, device=DEV))
    assert got.tolist() == new and c.tolist() == [count] and torch.equal(pool, want)


@pytest.mark.parametrize("n", [3, 60])      # through and around the caches
def test_copies_of_large_pages(n):
    src, dst = large_pool(80, (2 << 20) + 48), torch.zeros(2, 70, ((2 << 20) + 48) // 4, dtype=torch.int32, device=DEV)
    assert src.nbytes > BEYOND
    gen = torch.Generator().manual_seed(n)
    d, s = torch.randperm(70, generator=gen)[:n].tolist(), torch.randint(0, 80, (n,), generator=gen).tolist()
    s[1], d[2] = s[0], 70      # a page twice; none
    want = dst.clone()
    for a, b in zip(s, d):
        if b < 70:
            want[:, b] = src[:, a]
    gb.gdn_pages_copy(dst, src, *(torch.tensor(x, dtype=torch.int32, device=DEV) for x in (d, s)))
    assert torch.equal(dst, want)
