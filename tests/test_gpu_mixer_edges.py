"""Calls of the operators around the recurrent layers between those of
test_gpu_mixer.py and test_gpu_mixer_paths.py, with their references and
tolerances."""
import pytest
import torch

import mixer_ref as ref
from chunked_gated_delta_05_amd import binding as gb
from test_gpu_mixer import near, scan_args, scan_case, scan_gpu, scan_gpu_bwd

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
