"""Calls of the operators around the recurrent layers between those of
test_gpu_mixer.py and test_gpu_mixer_paths.py, with their references and
tolerances."""
import pytest
import torch

import mixer_ref as ref
from chunked_gated_delta_05_amd import binding as gb
from test_gpu_mixer import DT, layout, near, scan_args, scan_case, scan_gpu, scan_gpu_bwd

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ cut gradients
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("states", [False, True])
@pytest.mark.parametrize("lead", [(2, 400), [400, 1, 90], (2, 1500)])   # segments joined, joined, merged
def test_cut_gradients_with_and_without_states(lead, states, dtype):
    c = scan_case(lead, 72, 16, 1, dtype, seed=21)
    if not states:
        c["s0"] = c["dht"] = None
    h = gb.gdn_scan_fwd(c["u"], c["dt"], c["A"], c["B"], c["C"], c["skip"], c["gate"], dt_bias=c["dt_bias"],
                        dt_softplus=True, meta=c["meta"], initial_state=c["s0"], want_h=True)[2]
    r = scan_gpu_bwd(c, h, want_dh0=states)
    a = scan_args(c)
    want, scale = ref.scan(*a)[2], ref.scan(*a, absolute=True)[2]
    L = max(b - a for a, b in zip(c["offs"], c["offs"][1:]))
    assert ("dh0" in r) == states
    for k, t in r.items():
        near(t, want[k], scale[k], 2 * (24 * L + 64) + 72 + c["offs"][-1], k)


# ------------------------------------------------------------------ long prompts
def scan_with_errors(u, dt, A, B, C, skip, gate, bias, s0, offs, S, decay_steps):
    """The scan in 64 bits on the GPU, all sequences side by side, and with every
    value the error that fp32 arithmetic may have by then, to first order, in
    steps of 2^-24: out, its error, final states, their error.

    t = softplus(raw): raw is rounded (slope sigmoid), and e^-|raw| is off by the
    rounding of |raw| log2(e) twice, its own step (2) and that of what becomes of
    it. A decay is off by t's error times |A|, by `decay_steps` of its exponent (A
    log2(e), the product; where segments are joined their sums as well) and by
    two steps of its own; the update and du B round three times and once; y rounds
    S + 2 times, the gate like e^-|raw|."""
    n, length = len(offs) - 1, [b - a for a, b in zip(offs, offs[1:])]
    T, D = max(length), u.shape[-1]
    at = torch.zeros(T, n, dtype=torch.int64, device="cuda")
    live = torch.zeros(T, n, dtype=torch.bool, device="cuda")
    for i, (a, b) in enumerate(zip(offs, offs[1:])):
        at[:b - a, i] = torch.arange(a, b, device="cuda")
        live[:b - a, i] = True
    flat = lambda x, k: x.double().reshape(-1, *x.shape[x.dim() - k:])
    u, raw, gate = flat(u, 1), flat(dt, 1) + bias.double(), flat(gate, 1)
    B, C, A, skip = flat(B, 2)[:, 0], flat(C, 2)[:, 0], A.double(), skip.double()
    t = torch.nn.functional.softplus(raw, threshold=60)
    e = torch.exp(-raw.abs())
    et = 2 * torch.sigmoid(raw) * raw.abs() + e * (2 * raw.abs() + 4) + 4 * t
    y, ey = torch.zeros_like(u), torch.zeros_like(u)
    h = s0.double().clone()
    eh = torch.zeros_like(h)
    for i in range(T):
        p, on = at[i], live[i]
        p, hh, ehh = p[on], h[on], eh[on]
        tt, ett, uu, b, c = t[p, :, None], et[p, :, None], u[p, :, None], B[p, None], C[p, None]
        a = torch.exp(tt * A)
        ea = a * (A.abs() * ett + (tt * A).abs() * decay_steps + 2)
        new = a * hh + tt * uu * b
        ehh = a * ehh + ea * hh.abs() + (uu * b).abs() * ett + 3 * (tt * uu * b).abs() + new.abs()
        y[p] = (c * new).sum(-1) + skip * uu[..., 0]
        ey[p] = (c.abs() * (ehh + (S + 2) * new.abs())).sum(-1) + 2 * (skip * uu[..., 0]).abs()
        h[on], eh[on] = new, ehh
    sg = torch.sigmoid(gate)
    out = y * gate * sg
    return out, (gate * sg).abs() * ey + out.abs() * (2 * gate.abs() + 8), h, eh


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("lead,D,decay_steps", [
    ([700, 2900, 1, 1500, 2211, 880], 4096, 2),      # one state a lane
    ((2, 4096), 4096, 2),                            # likewise
    ((1, 4096), 1024, 32)])                          # segments of 96 tokens at most: sums of 96 / 8 + 8 terms and 3 more
def test_long_prompts_within_their_own_error(lead, D, decay_steps, dtype):
    S, dt = 16, DT[dtype]
    g = torch.Generator("cuda").manual_seed(51)
    ld, offs, meta = layout(lead)
    randn = lambda *s: torch.randn(*s, generator=g, device="cuda")
    u, gate, raw = (randn(*ld, D).to(dt) for _ in range(3))
    B, C = randn(*ld, 1, S).to(dt), randn(*ld, 1, S).to(dt)
    A = -torch.arange(1, S + 1, device="cuda").float() * torch.exp(0.1 * randn(D, S))
    skip, bias, s0 = randn(D), randn(D) - 5, randn(len(offs) - 1, D, S)
    out, final, _ = gb.gdn_scan_fwd(u, raw, A, B, C, skip, gate, dt_bias=bias, dt_softplus=True, meta=meta, initial_state=s0,
                                    output_final_state=True)
    want, e, state, es = scan_with_errors(u, raw, A, B, C, skip, gate, bias, s0, offs, S, decay_steps)
    for got, w, err, what in ((out.view(-1, D), want, e, "out"), (final, state, es, "final")):
        tol = torch.finfo(got.dtype).eps / 2 * w.abs() * 1.01 + 1.05 * 2.0 ** -24 * err + 1e-37
        worst = ((got.double() - w).abs() / tol).max()
        assert worst <= 1, (what, float(worst))


# ------------------------------------------------------------------ what lies around the tensors
def walled(x, wall):
    """A copy of x with `wall` of 4096 elements on either side; the whole."""
    whole = torch.full((x.numel() + 8192,), wall, dtype=x.dtype, device="cuda")
    inner = whole[4096:4096 + x.numel()].view(x.shape)
    inner.copy_(x)
    return inner, whole


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("lead,D,S", [
    ((520, 37), 128, 16), ((520, 33), 128, 8), ((520, 41), 64, 32), ((520, 37), 32, 64),     # two channels a lane
    ((300, 37), 128, 16), ((300, 35), 128, 8), ((300, 37), 32, 64),                          # one
    ((1, 61), 40, 16), ((1, 67), 40, 8), ((1, 70), 24, 32), ((1, 61), 24, 64),               # one state a lane
    ((1, 901), 72, 16), ((1, 913), 72, 8), ((2, 905), 24, 64)])                              # cut
def test_scan_reads_and_writes_nothing_around_its_tensors(lead, D, S, dtype):
    # NaN on either side of what is read, and what is on either side of the outputs stays
    c = scan_case(lead, D, S, 1, dtype, seed=61)
    want, wfinal, h = scan_gpu(c, want_h=True)
    grads = scan_gpu_bwd(c, h)
    w = dict(c)
    for k in ("u", "dt", "gate", "B", "C", "A", "skip", "dt_bias", "s0", "dout", "dht"):
        w[k] = walled(c[k], float("nan"))[0]
    out, around = walled(torch.zeros_like(want), 7.0)
    final, around_final = walled(torch.zeros_like(wfinal), 7.0)
    _, _, h2 = scan_gpu(w, want_h=True, out=out, final_out=final)
    assert torch.equal(out, want) and torch.equal(final, wfinal) and torch.equal(h2, h)
    for whole in (around, around_final):
        assert (whole[:4096] == 7).all() and (whole[-4096:] == 7).all()
    got = scan_gpu_bwd(w, walled(h2, float("nan"))[0])
    for k, t in grads.items():
        assert torch.equal(got[k], t), k


# ------------------------------------------------------------------ rotation without a norm
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("interleaved", [False, True])
def test_gradients_without_a_norm_do_not_depend_on_the_rows(interleaved, dtype):
    # dq is the gradient turned back, whatever q holds: rows that are not finite (padding that was never
    # written), and products with the gradient beyond fp32
    g = torch.Generator().manual_seed(31)
    q, k, dq, dk = (torch.randn(2, 9, h, 80, generator=g).to(dtype).cuda() for h in (3, 1, 3, 1))
    f = gb.rotary_frequencies(48, device="cuda")
    dq[0, 2] *= 1e20
    call = lambda x: gb.gdn_qk_rotary_bwd(x, k, f, None, dq, dk, norm=None, interleaved=interleaved)
    want = call(q)
    bad = q.clone()
    bad[0, 2] *= 1e20
    bad[1, 5] = float("nan")
    bad[1, 7, 1, 3] = float("inf")
    bad[0, 4, 2, 70] = -float("inf")
    got = call(bad)
    assert torch.isfinite(want["dq"]).all()
    assert torch.equal(got["dq"], want["dq"]) and torch.equal(got["dk"], want["dk"])
    # a gradient that is not finite stays in its pair
    dq[1, 1, 0, 5] = float("inf")
    hit = torch.zeros_like(dq, dtype=torch.bool)
    hit[1, 1, 0, [4, 5] if interleaved else [5, 29]] = True
    got = call(bad)
    assert torch.equal(got["dq"][~hit], want["dq"][~hit]) and not torch.isfinite(got["dq"][hit]).any()


@pytest.mark.parametrize("dtype", [torch.int32, torch.int64])
def test_positions_and_frequencies_may_be_slices(dtype):
    g = torch.Generator().manual_seed(32)
    q, k = (torch.randn(37, h, 64, generator=g).cuda() for h in (3, 1))
    f = gb.rotary_frequencies(56, device="cuda")
    at = torch.randint(0, 100000, (40,), generator=g).to(dtype).cuda()
    for first in (1, 2, 3):
        own = (f[first:first + 24].clone(), at[first:first + 37].clone())
        part = (f[first:first + 24], at[first:first + 37])
        assert first == 2 or (part[0].data_ptr() % 16 and part[1].data_ptr() % 16)
        want, got = gb.gdn_qk_rotary_fwd(q, k, *own), gb.gdn_qk_rotary_fwd(q, k, *part)
        assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
        want, got = gb.gdn_qk_rotary_bwd(q, k, *own, q, k), gb.gdn_qk_rotary_bwd(q, k, *part, q, k)
        assert torch.equal(want["dq"], got["dq"]) and torch.equal(want["dk"], got["dk"])


def test_rotation_of_no_tokens_with_strided_heads():
    wide = torch.zeros(2, 0, 6, 128, device="cuda")
    q, k, f = wide[:, :, :4, :64], wide[:, :, 4:, :64], gb.rotary_frequencies(64, device="cuda")
    a, b = gb.gdn_qk_rotary_fwd(q, k, f)
    assert a.shape == q.shape and b.shape == k.shape
    w = torch.ones(64, device="cuda")
    r = gb.gdn_qk_rotary_bwd(q, k, f, None, a, b, q_weight=w, k_weight=w)
    assert r["dq"].shape == q.shape and not r["dq_weight"].any() and not r["dk_weight"].any()


# ------------------------------------------------------------------ autograd
def test_scan_without_gradients_takes_no_room_for_states():
    c = scan_case((1, 2048), 1024, 16, 1, "bf16", seed=41)
    args = [c[k] for k in ("u", "dt", "A", "B", "C", "skip", "gate", "dt_bias", "s0")]
    args[2] = args[2].clone().requires_grad_()
    call = lambda: gb.SelectiveScan.apply(*args, True)
    room = []
    for off in (False, True):
        torch.cuda.synchronize()
        torch.cuda.reset_peak_memory_stats()
        before = torch.cuda.memory_allocated()
        with torch.set_grad_enabled(not off):
            got = call()
        room.append(torch.cuda.max_memory_allocated() - before)
        if not off:
            want = [t.detach().clone() for t in got]
            del got
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert room[0] - room[1] >= 2048 // 16 * 1024 * 16 * 4 and not got[0].requires_grad
