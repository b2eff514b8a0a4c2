"""Calls of the operators around the recurrent layers that have to be taken, or
refused, on the CPU: a call that the binding takes is rejected last, for not
being on the GPU."""
import ctypes

import pytest
import torch

from chunked_gated_delta_05_amd import binding as gb

BF, F32, F64, I32, I64 = torch.bfloat16, torch.float32, torch.float64, torch.int32, torch.int64
OK, INVALID = 0, 1


def z(*shape, dtype=BF):
    return torch.zeros(*shape, dtype=dtype)


def fake(i, off=0):
    return ctypes.c_void_p((1 << 40) + (i << 32) + off)


# ------------------------------------------------------------------ norms and rotation
class RotaryDesc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("B", "T", "Hq", "Hk", "D", "R", "dtype", "w_dtype", "norm", "interleaved", "pos_i64")] + \
               [("eps", ctypes.c_float), ("amplitude", ctypes.c_float)] + \
               [(n, ctypes.c_int64) for n in ("q0", "q1", "k0", "k1")]


@pytest.mark.parametrize("dtype", [I32, I64])
@pytest.mark.parametrize("first", [0, 1, 2, 3])
def test_positions_and_frequencies_may_be_slices(first, dtype):
    # both are read one by one
    q, k = z(9, 4, 64), z(9, 2, 64)
    at, f = torch.arange(first + 9).to(dtype)[first:], gb.rotary_frequencies(2 * (24 + first))[first:]
    for call in (lambda: gb.gdn_qk_rotary_fwd(q, k, f, at), lambda: gb.gdn_qk_rotary_bwd(q, k, f, at, q, k)):
        with pytest.raises(ValueError, match="GPU tensors"):
            call()


@pytest.mark.parametrize("pos_i64,off,ok", [(0, 4, True), (0, 2, False), (1, 8, True), (1, 4, False)])
def test_positions_are_aligned_to_their_own_size(pos_i64, off, ok):
    # no tokens: what is accepted launches nothing
    d = RotaryDesc(2, 0, 4, 2, 64, 64, 1, 0, 1, 0, pos_i64, 1e-6, 1.0, 256, 64, 128, 64)
    f = gb.lib().gdn_qk_rotary_fwd
    call = lambda pos, freqs: f(ctypes.byref(d), fake(0), fake(1), freqs, pos, None, None, fake(4), fake(5), None)
    assert call(fake(3, off), fake(2)) == (OK if ok else INVALID)
    assert call(fake(3), fake(2, 8)) == OK and call(fake(3), fake(2, 4)) == INVALID
    size = ctypes.c_size_t(256)
    b = gb.lib().gdn_qk_rotary_bwd
    call = lambda pos, freqs: b(ctypes.byref(d), fake(0), fake(1), freqs, pos, None, None, fake(4), fake(5), fake(6), fake(7),
                                None, None, fake(8), ctypes.byref(size), None)
    assert call(fake(3, off), fake(2)) == (OK if ok else INVALID)
    assert call(fake(3), fake(2, 8)) == OK and call(fake(3), fake(2, 4)) == INVALID


def test_rotation_of_no_tokens_with_strided_heads():
    # empty tensors have no address: NULL in and out is not "in place"
    d = RotaryDesc(2, 0, 4, 2, 64, 64, 1, 0, 1, 0, 0, 1e-6, 1.0, 512, 128, 256, 128)
    f = gb.lib().gdn_qk_rotary_fwd
    assert f(ctypes.byref(d), None, None, fake(2), None, None, None, None, None, None) == OK
    assert f(ctypes.byref(d), fake(0), fake(1), fake(2), None, None, None, fake(3), fake(4), None) == OK
    d.T = 3                                   # in place means contiguous, as before
    assert f(ctypes.byref(d), fake(0), fake(1), fake(2), None, None, None, fake(0), fake(4), None) == INVALID
    assert f(ctypes.byref(d), fake(0), fake(1), fake(2), None, None, None, fake(3), fake(1), None) == INVALID


# ------------------------------------------------------------------ states
@pytest.mark.parametrize("first", [0, 1, 2])
def test_states_may_not_overlap_by_part(first):
    # two sequences: pool[:2] to pool[1:3] would let one read what the other has written
    msg = "out overlaps initial_state" if first == 1 else "GPU tensors"
    pool = z(5, 3, 64)
    with pytest.raises(ValueError, match=msg):
        gb.gdn_conv_fwd(z(2, 7, 64), z(64, 4), initial_state=pool[:2], final_out=pool[first:first + 2])
    pool = z(5, 64, 16, dtype=F32)
    x, rows, A = z(2, 7, 64), z(2, 7, 1, 16), z(64, 16, dtype=F32)
    with pytest.raises(ValueError, match=msg):
        gb.gdn_scan_fwd(x, x, A, rows, rows, initial_state=pool[:2], final_out=pool[first:first + 2])
    with pytest.raises(ValueError, match="GPU tensors"):     # by pages it is the caller's tables that matter
        gb.gdn_scan_fwd(x, x, A, rows, rows, initial_state=pool[:3], initial_pages=z(2, dtype=I32),
                        final_out=pool[1:4], final_pages=z(2, dtype=I32))


# ------------------------------------------------------------------ autograd
@pytest.fixture
def scans(monkeypatch):
    """want_h of the calls that SelectiveScan makes, which are replaced."""
    seen = []

    def fwd(u, *rest, initial_state=None, output_final_state=False, want_h=False, **kw):
        seen.append(want_h)
        return u.clone(), u.new_zeros(1) if output_final_state else None, u.new_zeros(1) if want_h else None

    monkeypatch.setattr(gb, "gdn_scan_fwd", fwd)
    return seen


@pytest.mark.parametrize("off", [torch.no_grad, torch.inference_mode])
def test_scan_keeps_states_for_gradients_alone(scans, off):
    u, A = z(1, 4, 64, dtype=F32), z(64, 16, dtype=F32).requires_grad_()      # A: a parameter
    rows = z(1, 4, 1, 16, dtype=F32)
    with off():
        out, final = gb.SelectiveScan.apply(u, u, A, rows, rows)
        assert not out.requires_grad and final is not None
        gb.SelectiveScan.apply(u, u, A, rows, rows, None, u, None, None, True, None)
    out, _ = gb.SelectiveScan.apply(u, u, A.detach(), rows, rows)
    assert not out.requires_grad and scans == [False] * 3
    out, final = gb.SelectiveScan.apply(u, u, A, rows, rows)
    assert out.requires_grad and final.requires_grad and scans[3:] == [True]
