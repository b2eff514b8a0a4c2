"""What only larger or odder calls of the operators around the recurrent layers
reach: both widths of the scan's walks, cut and whole, many pieces, large steps,
values beyond 2^31, streams, graphs, versions, autograd, values that are not
finite, and a run of them together."""
import ctypes
import os
import sys

import pytest
import torch

import mixer_ref as ref
import test_gpu_mixer as small
from chunked_gated_delta_05_amd import binding as gb
from test_gpu_mixer import BF, F32, F64, I32, check_scan, gen, near, randn, scan_args, scan_case, scan_gpu, scan_gpu_bwd

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ scan
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("lead,D,S", [((520, 40), 16, 16),            # uncut, two channels a lane
                                      ((300, 20), 128, 16),            # one
                                      ((1, 600), 136, 16), ((1, 900), 40, 64), ((1, 900), 40, 32), ((1, 900), 72, 8),   # cut, one
                                      ([1] * 300 + [40, 3], 16, 16),   # sums over more than 256 pieces
                                      ([700, 1, 300], 64, 8)])
def test_scan_paths(lead, D, S, dtype):
    check_scan(scan_case(lead, D, S, 1, dtype, seed=7))


def test_scan_cut_with_two_channels_a_lane():
    # 512 workgroups in segments of 32 tokens
    c = scan_case((1, 2048), 1024, 16, 1, "bf16", seed=8)
    c["dout"] = None
    out, final, h = scan_gpu(c, want_h=True)
    a = scan_args(c)
    want, scale = ref.scan(*a), ref.scan(*a, absolute=True)
    near(out, want[0], scale[0], 24 * 2048 + 64, "out")
    near(final, want[1], scale[1], 24 * 2048 + 64, "final")


@pytest.mark.parametrize("S", [8, 16, 32, 64])
def test_scan_of_one_sequence_alone_and_among_others(S):
    # 520 sequences (two channels a lane), 300 (one) and one (one state a lane, or so): the same states; sums over
    # states in another order, within S + 2 steps of fp32 on either side and a rounding to bf16
    D = 128 if S == 8 else 2048 // S
    c = scan_case((520, 37), D, S, 1, "bf16", seed=9)
    out, final, h = scan_gpu(c, want_h=True)
    some = dict(c, **{k: c[k][:300].contiguous() for k in ("u", "dt", "gate", "B", "C", "s0")})
    o, f, hh = scan_gpu(some, want_h=True)
    assert torch.equal(o, out[:300]) and torch.equal(f, final[:300]) and torch.equal(hh, h[:900])
    one = dict(c, **{k: c[k][77:78].contiguous() for k in ("u", "dt", "gate", "B", "C", "s0")})
    o, f, hh = scan_gpu(one, want_h=True)
    assert torch.equal(f[0], final[77]) and torch.equal(hh, h[77 * 3:78 * 3])
    a = [x if x is None or not torch.is_tensor(x) or x.dim() < 3 else x[77:78] for x in scan_args(c)]
    a[9], a[11], a[12] = [0, 37], None, None
    _, scale = ref.scan(*a)[0], ref.scan(*a, absolute=True)[0]
    near(o[0], out[77].double().cpu(), 2 * (S + 2) * scale + out[77].double().cpu().abs() * 2 ** 16, 1, "out")


@pytest.mark.parametrize("lead", [(2, 400), [400, 1, 90]])
def test_scan_cut_pages_in_place(lead):
    # cut sequences whose states are replaced where they were read
    c = scan_case(lead, 72, 16, 1, "bf16", seed=11)
    n = len(c["offs"]) - 1
    pool = randn(gen(12), n + 2, 72, 16)
    before = pool.clone()
    pages = torch.arange(n, 0, -1, dtype=I32, device="cuda")
    c["s0"], c["dout"] = pool, None
    out, _, _ = scan_gpu(c, initial_pages=pages, final_out=pool, final_pages=pages)
    c["s0"] = before[pages.long()]
    a = scan_args(c)
    want, scale = ref.scan(*a), ref.scan(*a, absolute=True)
    near(out, want[0], scale[0], 24 * 400 + 64, "out")
    near(pool[pages.long()], want[1], scale[1], 24 * 400 + 64, "final")
    assert torch.equal(pool[[0, n + 1]], before[[0, n + 1]])


class ScanDesc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("B", "T", "D", "G", "S", "dtype", "softplus", "n_units")] + \
               [(n, ctypes.c_int64) for n in ("u_stride", "dt_stride", "gate_stride", "b0", "b1", "c0", "c1")] + \
               [("offsets_host", ctypes.c_void_p), ("offsets_dev", ctypes.c_void_p)]


@pytest.mark.parametrize("T", [400, 1500])     # segments joined and merged
def test_entry_gradients_replace_those_of_the_final_states(T):
    c = scan_case((2, T), 72, 16, 1, "fp32", seed=13)
    for k in ("u", "dt", "gate", "B", "C"):
        c[k] = c[k].contiguous()
    h = scan_gpu(c, want_h=True)[2]
    r = scan_gpu_bwd(c, h)
    d = ScanDesc(2, T, 72, 1, 16, 0, 1, 0, 72, 72, 72, 16, 16, 16, 16, None, None)
    p = lambda t: ctypes.c_void_p(t.data_ptr())
    dh = c["dht"].clone()
    got = {k: torch.empty_like(t) for k, t in r.items()}
    ins = [p(c[k]) for k in ("u", "dt", "A", "B", "C", "skip", "gate", "dt_bias")] + [p(h), p(c["dout"]), p(dh)]
    outs = [p(got[k]) for k in ("du", "ddt", "dA", "dB", "dC", "dskip", "dgate", "ddt_bias")] + [p(dh)]
    f, size = gb.lib().gdn_scan_bwd, ctypes.c_size_t(0)
    stream = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    assert f(ctypes.byref(d), *ins, *outs, None, ctypes.byref(size), stream) == 0
    ws = torch.empty(size.value, dtype=torch.uint8, device="cuda")
    assert f(ctypes.byref(d), *ins, *outs, p(ws), ctypes.byref(size), stream) == 0
    got["dh0"] = dh
    a = scan_args(c)
    want, scale = ref.scan(*a)[2], ref.scan(*a, absolute=True)[2]
    for k, t in got.items():
        near(t, want[k], scale[k], 2 * (24 * T + 64) + 72 + 2 * T, k)


@pytest.mark.parametrize("N", [259, 1030])   # four sequences a workgroup; states around the caches
def test_scan_large_steps(N):
    D, S = 512, 64
    g = gen(N)
    x = {k: randn(g, N, *s) for k, s in (("u", (D,)), ("dt", (D,)), ("B", (1, S)), ("C", (1, S)), ("gate", (D,)))}
    A, skip, pool = -torch.rand(D, S, generator=g).cuda(), randn(g, D), randn(g, N + 3, D, S)
    pages = torch.randperm(N + 3, generator=g)[:N].to(I32)
    pages[5], pages[N - 1] = -1, -1
    before = pool.clone()
    out = gb.gdn_scan_step(x["u"], x["dt"], A, x["B"], x["C"], pool, skip, x["gate"], dt_softplus=True, pages=pages.cuda())
    for n in (0, 1, 2, 3, 4, 6, N - 2):
        a = [x["u"][n:n + 1], x["dt"][n:n + 1], A, x["B"][n:n + 1], x["C"][n:n + 1], skip, x["gate"][n:n + 1], None, True, [0, 1],
             before[int(pages[n])][None]]
        want, scale = ref.scan(*a), ref.scan(*a, absolute=True)
        near(out[n], want[0][0], scale[0][0], 88, "out")
        near(pool[int(pages[n])], want[1][0], scale[1][0], 88, "state")
    assert not out[5].any() and not out[N - 1].any()
    used = set(pages.tolist())
    rest = [p for p in range(N + 3) if p not in used]
    assert torch.equal(pool[rest], before[rest])


def test_steps_without_a_page_list_use_the_first_pages():
    c = scan_case((3, 1), 24, 16, 1, "fp32")
    row = lambda k: c[k][:, 0]
    pool = randn(gen(1), 5, 24, 16)
    a, b = pool.clone(), pool.clone()
    args = lambda p: (row("u"), row("dt"), c["A"], row("B"), row("C"), p, c["skip"], row("gate"))
    one = gb.gdn_scan_step(*args(a))
    two = gb.gdn_scan_step(*args(b), pages=torch.arange(3, dtype=I32, device="cuda"))
    assert torch.equal(one, two) and torch.equal(a, b) and torch.equal(a[3:], pool[3:])
    x, w, s = randn(gen(2), 3, 24), randn(gen(3), 24, 4), randn(gen(4), 5, 3, 24)
    a, b = s.clone(), s.clone()
    assert torch.equal(gb.gdn_conv_step(x, w, a), gb.gdn_conv_step(x, w, b, pages=torch.arange(3, dtype=I32, device="cuda")))
    assert torch.equal(a, b) and torch.equal(a[3:], s[3:]) and torch.equal(a[:3, 2], x)


def test_prompts_continue_as_steps():
    # a prompt, then single tokens: the same as the whole as a prompt
    T, D = 50, 72
    c = scan_case((2, T), D, 16, 1, "fp32", seed=3)
    whole, final, _ = scan_gpu(c)
    first = dict(c, **{k: c[k][:, :40].contiguous() for k in ("u", "dt", "gate", "B", "C")})
    out, state, _ = scan_gpu(first)
    rows = [gb.gdn_scan_step(c["u"][:, t].contiguous(), c["dt"][:, t].contiguous(), c["A"], c["B"][:, t].contiguous(),
                             c["C"][:, t].contiguous(), state, c["skip"], c["gate"][:, t].contiguous(), dt_bias=c["dt_bias"],
                             dt_softplus=True) for t in range(40, T)]
    got = torch.cat([out, torch.stack(rows, 1)], 1)
    want, scale = ref.scan(*scan_args(c)[:11]), ref.scan(*scan_args(c)[:11], absolute=True)
    near(got, want[0], scale[0], 24 * T + 64, "out")
    near(state, want[1], scale[1], 24 * T + 64, "state")


# ------------------------------------------------------------------ beyond 2^31 values
def test_conv_and_scan_beyond_two_to_the_31():
    T, D, tail = 270000, 8192, 50
    offs = [0, T - tail, T]
    meta, own = gb.make_meta(offs, T, "cuda"), gb.make_meta([0, tail], tail, "cuda")
    g = torch.Generator("cuda").manual_seed(5)
    big = lambda *s: torch.randn(*s, generator=g, device="cuda", dtype=BF)
    x, w = big(T, D), big(D, 4)
    y, final = gb.gdn_conv_fwd(x, w, activation="silu", meta=meta, output_final_state=True)
    y2, f2 = gb.gdn_conv_fwd(x[-tail:].contiguous(), w, activation="silu", meta=own, output_final_state=True)
    assert torch.equal(y[-tail:], y2) and torch.equal(final[1], f2[0])
    r = gb.gdn_conv_bwd(x, w, None, y, activation="silu", meta=meta)
    r2 = gb.gdn_conv_bwd(x[-tail:].contiguous(), w, None, y2, activation="silu", meta=own)
    assert torch.equal(r["dx"][-tail:], r2["dx"])
    del r, r2, final
    dt, A = y, -torch.rand(D, 16, generator=g, device="cuda")
    B, C = big(T, 1, 16), big(T, 1, 16)
    out, fin, h = gb.gdn_scan_fwd(x, dt, A, B, C, dt_softplus=True, meta=meta, output_final_state=True, want_h=True)
    part = [t[-tail:].contiguous() for t in (x, dt, B, C)]
    o2, fin2, h2 = gb.gdn_scan_fwd(part[0], part[1], A, part[2], part[3], dt_softplus=True, meta=own, output_final_state=True,
                                   want_h=True)
    same = lambda a, b, n: near(a, b.cpu().double(), b.cpu().double().abs().amax().expand(b.shape), n, "tail")
    same(out[-tail:], o2, 24 * tail + 64)
    same(fin[1], fin2[0], 24 * tail + 64)
    r = gb.gdn_scan_bwd(x, dt, A, B, C, None, None, out, h, dt_softplus=True, meta=meta)
    r2 = gb.gdn_scan_bwd(part[0], part[1], A, part[2], part[3], None, None, out[-tail:].contiguous(), h2, dt_softplus=True,
                         meta=own)
    for k in ("du", "ddt", "dB", "dC"):
        same(r[k][-tail:], r2[k], 2 * (24 * tail + 64) + D)


def test_rotary_beyond_two_to_the_31():
    T, H, D = 300000, 57, 128
    q = torch.randn(T, H, D, generator=torch.Generator("cuda").manual_seed(1), device="cuda", dtype=BF)
    k, at = q[:, :1].contiguous(), torch.arange(T, device="cuda")
    f = gb.rotary_frequencies(D, device="cuda")
    a, b = gb.gdn_qk_rotary_fwd(q, k, f, at)
    c, d = gb.gdn_qk_rotary_fwd(q[-9:], k[-9:], f, at[-9:].clone())
    assert torch.equal(a[-9:], c) and torch.equal(b[-9:], d)
    r = gb.gdn_qk_rotary_bwd(q, k, f, at, a, b)
    s = gb.gdn_qk_rotary_bwd(q[-9:], k[-9:], f, at[-9:].clone(), c, d)
    assert torch.equal(r["dq"][-9:], s["dq"]) and torch.equal(r["dk"][-9:], s["dk"])


# ------------------------------------------------------------------ values that are not finite
def test_not_finite_values_stay_in_their_sequence_and_channel():
    c = scan_case([20, 33, 40], 72, 16, 1, "fp32", seed=4)
    clean, final, h = scan_gpu(c, want_h=True)
    grads = scan_gpu_bwd(c, h)
    bad = dict(c, u=c["u"].clone())
    bad["u"][30, 5] = float("nan")     # in the second sequence
    out, fin, h = scan_gpu(bad, want_h=True)
    r = scan_gpu_bwd(bad, h)
    hit = torch.zeros(93, 72, dtype=torch.bool, device="cuda")
    hit[30:53, 5] = True
    assert torch.isnan(out[hit]).all() and torch.equal(out[~hit], clean[~hit])
    assert torch.equal(fin[[0, 2]], final[[0, 2]])
    others = torch.ones(93, dtype=torch.bool, device="cuda")
    others[20:53] = False
    for k in ("du", "ddt", "dgate", "dB", "dC"):
        assert torch.equal(r[k][others], grads[k][others]), k
    x, w = randn(gen(1), 60, 16), randn(gen(2), 16, 4)
    m = gb.make_meta([0, 20, 60], 60, "cuda")
    y, _ = gb.gdn_conv_fwd(x, w, meta=m)
    x[19, 3], x[30, 4] = float("inf"), float("nan")
    z, _ = gb.gdn_conv_fwd(x, w, meta=m)
    hit = torch.zeros(60, 16, dtype=torch.bool, device="cuda")
    hit[19, 3] = True
    hit[30:34, 4] = True
    assert torch.equal(z[~hit], y[~hit]) and not torch.isfinite(z[hit]).any()


# ------------------------------------------------------------------ streams, graphs, repeats
def calls():
    """name -> a call on fixed tensors that returns its outputs (states reset first)."""
    c = scan_case([70, 300, 1], 136, 16, 1, "bf16", seed=6)
    h = scan_gpu(c, want_h=True)[2]
    x, w, b, s0 = randn(gen(1), 371, 136, dtype=BF), randn(gen(2), 136, 4, dtype=BF), randn(gen(3), 136, dtype=BF), \
        randn(gen(4), 3, 3, 136, dtype=BF)
    m = c["meta"]
    q, k, f = randn(gen(5), 2, 40, 4, 64, dtype=BF), randn(gen(6), 2, 40, 2, 64, dtype=BF), gb.rotary_frequencies(64, device="cuda")
    wt = randn(gen(7), 64)
    pool, cpool = randn(gen(8), 3, 136, 16), randn(gen(9), 3, 3, 136, dtype=BF)
    state, cstate = pool.clone(), cpool.clone()

    def steps():
        state.copy_(pool)
        cstate.copy_(cpool)
        y = gb.gdn_conv_step(x[:3], w, cstate, b, activation="silu")
        return [y, gb.gdn_scan_step(y, c["dt"][:3], c["A"], c["B"][:3], c["C"][:3], state, c["skip"]), state, cstate]

    return {"scan_fwd": lambda: [t for t in scan_gpu(c, want_h=True)[:2]],
            "scan_bwd": lambda: list(scan_gpu_bwd(c, h).values()),
            "conv_fwd": lambda: list(gb.gdn_conv_fwd(x, w, b, activation="silu", meta=m, initial_state=s0, output_final_state=True)),
            "conv_bwd": lambda: list(gb.gdn_conv_bwd(x, w, b, x, activation="silu", meta=m, initial_state=s0, dfinal=s0).values()),
            "rotary_fwd": lambda: list(gb.gdn_qk_rotary_fwd(q, k, f, q_weight=wt, k_weight=wt)),
            "rotary_bwd": lambda: list(gb.gdn_qk_rotary_bwd(q, k, f, None, q, k, q_weight=wt, k_weight=wt).values()),
            "steps": steps}


NAMES = ["scan_fwd", "scan_bwd", "conv_fwd", "conv_bwd", "rotary_fwd", "rotary_bwd", "steps"]


@pytest.mark.parametrize("name", NAMES)
def test_repeats_streams_and_graphs_agree_bit_for_bit(name):
    f = calls()[name]
    want = [t.clone() for t in f()]
    for got in (f(), f()):
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = [t.clone() for t in f()]
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = f()
    for _ in range(3):
        for t in got:
            t.zero_()
        f()                      # eager work between the replays
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_two_graphs_replayed_in_turn():
    fs = calls()
    graphs = []
    for n in ("scan_bwd", "conv_bwd"):
        want = [t.clone() for t in fs[n]()]
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = fs[n]()
        graphs.append((graph, got, want))
    for _ in range(3):
        for graph, _, _ in graphs:
            graph.replay()
        torch.cuda.synchronize()
        for _, got, want in graphs:
            assert all(torch.equal(a, b) for a, b in zip(got, want))


# ------------------------------------------------------------------ autograd
def test_versions_of_tensors_written_in_place():
    x, w = randn(gen(1), 2, 8, 16), randn(gen(2), 16, 4)
    out, state = torch.empty_like(x), randn(gen(3), 2, 3, 16)
    v = out._version, state._version
    gb.gdn_conv_fwd(x, w, out=out, final_out=state)
    assert (out._version, state._version) == (v[0] + 1, v[1] + 1)
    gb.gdn_conv_step(x[:, 0], w, state)
    assert state._version == v[1] + 2
    c = scan_case((2, 3), 16, 16, 1, "fp32")
    fin = c["s0"].clone()
    n = fin._version
    scan_gpu(c, final_out=fin)
    assert fin._version == n + 1
    q = randn(gen(4), 1, 3, 1, 64)
    k, n = q.clone(), q._version
    gb.gdn_qk_rotary_fwd(q, k, q_out=q)
    assert q._version == n + 1 and k._version == 0


def test_autograd_ops_match_the_calls():
    c = scan_case([20, 45], 72, 16, 1, "bf16", seed=2)
    leaves = {k: c[k].detach().clone().requires_grad_() for k in ("u", "dt", "A", "B", "C", "skip", "gate", "dt_bias", "s0")}
    out, final = gb.SelectiveScan.apply(*leaves.values(), True, c["meta"])
    grads = torch.autograd.grad([out, final], list(leaves.values()), [c["dout"], c["dht"]])
    d = dict(c, **{k: t.detach() for k, t in leaves.items()})
    r = scan_gpu_bwd(d, scan_gpu(d, want_h=True)[2])
    for name, g in zip(("du", "ddt", "dA", "dB", "dC", "dskip", "dgate", "ddt_bias", "dh0"), grads):
        assert torch.equal(g, r[name]), name
    x, w, b, s0 = (t.requires_grad_() for t in (randn(gen(1), 2, 30, 16), randn(gen(2), 16, 3), randn(gen(3), 16), randn(gen(4), 2, 2, 16)))
    y, fin = gb.CausalConv.apply(x, w, b, s0, "silu")
    dy, df = randn(gen(5), 2, 30, 16), randn(gen(6), 2, 2, 16)
    grads = torch.autograd.grad([y, fin], [x, w, b, s0], [dy, df])
    r = gb.gdn_conv_bwd(x.detach(), w.detach(), b.detach(), dy, activation="silu", initial_state=s0.detach(), dfinal=df)
    for g, name in zip(grads, ("dx", "dweight", "dbias", "dinitial")):
        assert torch.equal(g, r[name]), name
    only, = torch.autograd.grad(gb.CausalConv.apply(x, w, b, s0, "silu")[1], [s0], [df])     # the final state alone
    assert only.shape == s0.shape
    q, k, wt = randn(gen(7), 1, 9, 2, 64).requires_grad_(), randn(gen(8), 1, 9, 1, 64).requires_grad_(), \
        randn(gen(9), 64, dtype=BF).requires_grad_()
    f = gb.rotary_frequencies(64, device="cuda")
    a, b2 = gb.QKRotary.apply(q, k, f, None, wt, wt)
    grads = torch.autograd.grad([a, b2], [q, k, wt], [a.detach(), b2.detach()])
    r = gb.gdn_qk_rotary_bwd(q.detach(), k.detach(), f, None, a.detach(), b2.detach(), q_weight=wt.detach(), k_weight=wt.detach())
    assert torch.equal(grads[0], r["dq"]) and torch.equal(grads[1], r["dk"])
    assert torch.equal(grads[2], r["dq_weight"].to(BF) + r["dk_weight"].to(BF))


def hybrid_leaves():
    shapes = dict(x=(2, 70, 72), w=(72, 4), dt=(2, 70, 72), A=(72, 16), B=(2, 70, 1, 16), C=(2, 70, 1, 16), skip=(72,),
                  k=(2, 70, 3, 24), wt=(24,))
    return {n: (randn(gen(i), *s) if n != "A" else -randn(gen(i), *s).abs()).requires_grad_() for i, (n, s) in enumerate(shapes.items())}


def hybrid_outputs(p, f):
    y, s1 = gb.CausalConv.apply(p["x"], p["w"], None, None, "silu")
    o, s2 = gb.SelectiveScan.apply(y, p["dt"], p["A"], p["B"], p["C"], p["skip"], y, None, None, True)
    q, k = gb.QKRotary.apply(o.unflatten(-1, (3, 24)), p["k"], f, None, p["wt"], p["wt"])
    return [q, k, s1, s2]


def test_captured_training_step_repeats_the_eager_one():
    p, f = hybrid_leaves(), gb.rotary_frequencies(24, device="cuda")

    def step():
        outs = hybrid_outputs(p, f)
        return [o.detach() for o in outs] + list(torch.autograd.grad(outs, list(p.values()), [torch.ones_like(o) for o in outs]))

    want = [t.clone() for t in step()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for _ in range(3):
        for t in got:
            t.zero_()
        step()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_gradients_may_arrive_expanded_or_off_alignment():
    p, f = hybrid_leaves(), gb.rotary_frequencies(24, device="cuda")
    outs, leaves = hybrid_outputs(p, f), list(p.values())
    want = torch.autograd.grad(outs, leaves, [torch.ones_like(o) for o in outs], retain_graph=True)
    expanded = torch.autograd.grad([o.sum() for o in outs], leaves, retain_graph=True)
    odd = []
    for o in outs:
        room = torch.ones(o.numel() + 1, dtype=o.dtype, device="cuda")
        odd.append(room[1:].view(o.shape))
        assert odd[-1].data_ptr() % 16
    shifted = torch.autograd.grad(outs, leaves, odd)
    for a, b, c in zip(want, expanded, shifted):
        assert torch.equal(a, b) and torch.equal(a, c)


def test_second_order_gradients_and_constants_raise():
    x, w = randn(gen(1), 1, 9, 16).requires_grad_(), randn(gen(2), 16, 4)
    y, _ = gb.CausalConv.apply(x, w)
    g, = torch.autograd.grad(y.square().sum(), x, create_graph=True)
    with pytest.raises(RuntimeError):
        g.sum().backward()
    q = randn(gen(3), 1, 4, 1, 64).requires_grad_()
    f = gb.rotary_frequencies(64, device="cuda").requires_grad_()
    a, b = gb.QKRotary.apply(q, q, f)
    with pytest.raises(NotImplementedError, match="freqs"):
        (a.sum() + b.sum()).backward()


# ------------------------------------------------------------------ together
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def test_prompts_steps_and_forks_of_a_hybrid_model():
    import hybrid_decoding as ex
    # fp32 throughout: chunked prompts and steps differ by the 1e-4 of the delta rule's fp32 bar, over three layers
    assert ex.decode() < 1e-3
    assert ex.decode(lengths=(1, 2, 3, 400), beams=2, steps=5, seed=3) < 1e-3


def test_gradients_of_the_example_against_differences():
    import hybrid_decoding as ex
    losses, grads, p, rest = ex.train(steps=2)
    assert all(torch.isfinite(g).all() for g in grads.values()) and len(losses) == 2
    # along the gradient itself: the loss is fp32 (2^-24 of about 2), the difference 1e-2 of it or more
    for name, g in grads.items():
        n = float(g.double().square().sum().sqrt())
        step = 0.02 / n
        side = []
        for sign in (1, -1):
            q = {k: t.detach() for k, t in p.items()}
            q[name] = q[name] + sign * step * g
            side.append(float(ex.loss(q, *rest)))
        slope = (side[0] - side[1]) / (2 * step)
        assert abs(slope - n * n) <= 0.05 * n * n + 2e-6 / step, (name, slope, n * n)
