"""The argument checks and C ABI of the operators around the recurrent layers on
the CPU: every mismatch raises before anything touches a GPU, and a consistent
call on CPU tensors is rejected last, for not being on the GPU."""
import ctypes
import os
import re
import shutil

import pytest
import torch

from chunked_gated_delta_05_amd import binding as gb
from test_host_sanitizers import SAN, _build_and_run

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "chunked_gated_delta_05_amd", "csrc")
BF, F32, F64, I32 = torch.bfloat16, torch.float32, torch.float64, torch.int32
B, T, D, W, S, G = 2, 30, 64, 4, 16, 2


def test_library_exports_every_declared_function():
    src = open(os.path.join(ROOT, "include", "gdn_mixer.h")).read()
    names = sorted(set(re.findall(r"^(?:gdn_status|int64_t)\s+(gdn_\w+)\s*\(", src, re.M)))
    assert names == ["gdn_conv_bwd", "gdn_conv_fwd", "gdn_conv_step", "gdn_qk_rotary_bwd", "gdn_qk_rotary_fwd",
                     "gdn_scan_bwd", "gdn_scan_fwd", "gdn_scan_h_rows", "gdn_scan_step"]
    for n in names:
        assert hasattr(gb.lib(), n), n


def test_native_calls_launch_on_their_tensors_device():
    src = open(os.path.join(CSRC, "gdn_mixer_torch.cpp")).read()
    calls = [f for f in re.split(r"\n}\n", src) if "stream_of(" in f]
    assert len(calls) == 8
    for f in calls:
        assert f.index("const Guard guard(") < f.index("stream_of("), f


def meta():
    return gb.UnitMeta([0, 10, 30], (ctypes.c_int32 * 3)(0, 10, 30), torch.zeros(3, dtype=I32),
                       torch.zeros(3, dtype=I32), torch.zeros(3, 2, dtype=I32), 3)


def z(*shape, dtype=BF):
    return torch.zeros(*shape, dtype=dtype)


def raises(f, msg, kind=ValueError):
    with pytest.raises(kind, match=msg):
        f()


# ------------------------------------------------------------------ convolution
def conv_args(**kw):
    return dict(dict(x=z(B, T, D), weight=z(D, W), bias=z(D)), **kw)


def conv_calls(x):
    a = (x["x"], x["weight"], x["bias"])
    yield lambda **kw: gb.gdn_conv_fwd(*a, **kw)
    yield lambda **kw: gb.gdn_conv_bwd(*a, z(B, T, D), **kw)


@pytest.mark.parametrize("bad,msg", [
    ({}, "GPU tensors"),
    ({"x": z(B, T, D + 8)[..., :D]}, "GPU tensors"),
    ({"weight": z(D, W, dtype=F32), "bias": z(D, dtype=F32)}, "GPU tensors"),
    ({"x": None}, "x must have shape"), ({"x": z(D)}, "x must have shape"), ({"x": z(1, B, T, D)}, "x must have shape"),
    ({"x": z(T, D)}, "need meta"),
    ({"x": z(B, T, D, dtype=torch.float16)}, "unsupported dtype torch.float16"),
    ({"x": z(B, T, D).tolist()}, "x must be a tensor"),
    ({"x": z(B, T, 60), "weight": z(60, W), "bias": z(60)}, "60 channels, not a multiple of 8"),
    ({"x": z(B, T, D + 4)[..., :D]}, "16-byte aligned"),
    ({"x": z(T, B, D).transpose(0, 1)}, "batch rows must follow"),
    ({"x": z(B, D, T).transpose(1, 2)}, "values of a row must be contiguous"),
    ({"weight": None}, r"weight must be \[D,W\]"), ({"weight": z(D)}, r"weight must be \[D,W\]"),
    ({"weight": z(D + 8, W)}, "weight must have shape"), ({"weight": z(W, D).t()}, "weight must be contiguous"),
    ({"weight": z(D, W, dtype=F64), "bias": None}, "unsupported dtype"),
    ({"bias": z(D, dtype=F32)}, "bias must be torch.bfloat16"), ({"bias": z(D + 8)}, "bias must have shape"),
])
def test_conv_mismatches_raise(bad, msg):
    for f in conv_calls(conv_args(**bad)):
        raises(f, msg)


@pytest.mark.parametrize("taps", [1, 5])
def test_conv_of_other_taps_is_not_implemented(taps):
    for f in conv_calls(conv_args(weight=z(D, taps))):
        raises(f, "taps", NotImplementedError)


@pytest.mark.parametrize("kw,msg", [
    ({"activation": "gelu"}, "activation must be"), ({"activation": "silu"}, "GPU tensors"),
    ({"meta": meta()}, "meta goes with packed"),
    ({"initial_state": z(B, W, D)}, "initial_state must have shape"),
    ({"initial_state": z(B, W - 1, D, dtype=F32)}, "initial_state must be torch.bfloat16"),
])
def test_conv_option_mismatches_raise(kw, msg):
    for f in conv_calls(conv_args()):
        raises(lambda: f(**kw), msg)


def test_conv_states_and_outputs():
    f, b = conv_calls(conv_args())
    for kw, msg in (({"initial_pages": z(B, dtype=I32)}, "must be a pool"),
                    ({"initial_state": z(5, W - 1, D), "initial_pages": z(B + 1, dtype=I32)}, "initial_pages must have"),
                    ({"initial_state": z(5, W - 1, D), "initial_pages": z(B)}, "initial_pages must be torch.int32"),
                    ({"initial_state": z(5, W - 1, D), "initial_pages": z(B, dtype=I32), "final_out": z(6, W - 1, D),
                      "final_pages": z(B, dtype=I32)}, "pools have 5 and 6 pages"),
                    ({"out": z(B, T, D, dtype=F32)}, "out must be torch.bfloat16"),
                    ({"out": z(B, D, T).transpose(1, 2)}, "out must be contiguous")):
        raises(lambda: f(**kw), msg)
    x = z(B, T, D)
    raises(lambda: gb.gdn_conv_fwd(x, z(D, W), out=x), "out overlaps x")
    flat = z(B * (W - 1) * D)
    raises(lambda: gb.gdn_conv_fwd(x, z(D, W), out=flat.new_zeros(B * T * D).view(B, T, D), initial_state=None,
                                   final_out=x.view(-1)[:B * (W - 1) * D].view(B, W - 1, D)), "out overlaps x")
    for kw, msg in (({"dfinal": z(B, W - 1, D, dtype=F32)}, "dfinal must be torch.bfloat16"),
                    ({"dfinal": z(B, W, D)}, "dfinal must have shape")):
        raises(lambda: b(**kw), msg)
    a = (x, z(D, W), None)
    raises(lambda: gb.gdn_conv_bwd(*a, None), "dout is required")
    raises(lambda: gb.gdn_conv_bwd(*a, z(B, T, D, dtype=F32)), "dout must be torch.bfloat16")


@pytest.mark.parametrize("kw,msg", [
    ({}, "GPU tensors"), ({"x": z(3, T, D)}, r"x must have shape \[N,D\]"), ({"state": z(5, W, D)}, "state must have shape"),
    ({"state": z(2, W - 1, D)}, "2 pages for 3 rows"), ({"state": z(5, W - 1, D, dtype=F32)}, "state must be torch.bfloat16"),
    ({"state": z(5, W - 1, D + 8)[..., :D]}, "state must be contiguous"), ({"pages": z(3)}, "pages must be torch.int32"),
    ({"pages": z(4, dtype=I32)}, "pages must have shape"), ({"out": z(3, D + 8)}, "out must have shape"),
])
def test_conv_step_mismatches_raise(kw, msg):
    x = dict(dict(x=z(3, D), weight=z(D, W), state=z(5, W - 1, D)), **kw)
    raises(lambda: gb.gdn_conv_step(**x), msg)


# ------------------------------------------------------------------ scan
def scan_args(lead=(B, T), **kw):
    x = dict(u=z(*lead, D), dt=z(*lead, D), A=z(D, S, dtype=F32), B=z(*lead, G, S), C=z(*lead, G, S),
             skip=z(D, dtype=F32), gate=z(*lead, D))
    x.update(kw)
    return x


def scan_fwd(x, **kw):
    return gb.gdn_scan_fwd(x["u"], x["dt"], x["A"], x["B"], x["C"], x["skip"], x["gate"], **kw)


def scan_bwd(x, dout=None, h=None, **kw):
    dout = z(B, T, D) if dout is None else dout
    h = z(B * 2, D, S, dtype=F32) if h is None else h
    return gb.gdn_scan_bwd(x["u"], x["dt"], x["A"], x["B"], x["C"], x["skip"], x["gate"], dout, h, **kw)


SCAN_BAD = [
    ({}, "GPU tensors"),
    ({"B": z(B, T, 2 * G, S)[:, :, :G], "C": z(B, T, 2 * G, S)[:, :, G:]}, "GPU tensors"),
    ({"u": None}, "u must have shape"), ({"u": z(B, T, D, 1)}, "u must have shape"),
    ({"dt": None}, "dt is required"), ({"dt": z(B, T, D, dtype=F32)}, "dt must be torch.bfloat16"),
    ({"dt": z(B, T + 1, D)}, "dt must have shape"), ({"gate": z(B, T, D + 8)}, "gate must have shape"),
    ({"A": None}, r"A must be fp32 \[D,S\]"), ({"A": z(D, S)}, "A must be torch.float32"),
    ({"A": z(D + 8, S, dtype=F32)}, "A must have shape"), ({"A": z(S, D, dtype=F32).t()}, "A must be contiguous"),
    ({"B": None}, r"B must have shape \[..,G,S\]"), ({"B": z(B, T, S)}, "B must have shape"),
    ({"B": z(B, T, G, S + 8)}, "B must have shape"), ({"C": z(B, T, 1, S)}, "C must have shape"),
    ({"B": z(B, T, 3, S), "C": z(B, T, 3, S)}, "do not divide into 3 groups"),
    ({"B": z(B, T, 16, S), "C": z(B, T, 16, S)}, "groups of a multiple of 8"),
    ({"C": z(B, T, G, S + 4)[..., :S]}, "16-byte aligned"), ({"u": z(B, T, D + 4)[..., :D]}, "16-byte aligned"),
    ({"skip": z(D)}, "skip must be torch.float32"), ({"skip": z(D + 8, dtype=F32)}, "skip must have shape"),
    ({"u": z(B, T, D, dtype=F64)}, "unsupported dtype|must be"),
]


@pytest.mark.parametrize("bad,msg", SCAN_BAD)
def test_scan_mismatches_raise(bad, msg):
    x = scan_args(**bad)
    raises(lambda: scan_fwd(x), msg)
    raises(lambda: scan_bwd(x), msg)


def test_scan_options_and_states():
    x = scan_args()
    p = {n: t[0] if n in ("u", "dt", "B", "C", "gate") else t for n, t in scan_args().items()}
    raises(lambda: scan_fwd(p), "need meta")
    raises(lambda: scan_fwd(p, meta=meta()), "GPU tensors")
    for kw, msg in (({"dt_bias": z(D)}, "dt_bias must be torch.float32"), ({"meta": meta()}, "meta goes with packed"),
                    ({"initial_state": z(B, D, S)}, "initial_state must be torch.float32"),
                    ({"initial_state": z(B, S, D, dtype=F32)}, "initial_state must have shape"),
                    ({"final_out": z(4, D, S, dtype=F32), "final_pages": z(B)}, "final_pages must be torch.int32"),
                    ({"initial_pages": z(B, dtype=I32)}, "must be a pool"),
                    ({"out": x["u"]}, "out overlaps u"), ({"out": z(B, T, D, dtype=F32)}, "out must be torch.bfloat16")):
        raises(lambda: scan_fwd(x, **kw), msg)
    y = scan_args(A=z(D, 12, dtype=F32), B=z(B, T, G, 12), C=z(B, T, G, 12))
    raises(lambda: scan_fwd(y), "scans of 12 states", NotImplementedError)
    raises(lambda: gb.gdn_scan_bwd(x["u"], x["dt"], x["A"], x["B"], x["C"], None, None, z(B, T, D), None), "h is required")
    raises(lambda: gb.gdn_scan_bwd(x["u"], x["dt"], x["A"], x["B"], x["C"], None, None, None, None), "dout is required")
    raises(lambda: scan_bwd(x, h=z(B * 2 + 1, D, S, dtype=F32)), "h must have shape")
    raises(lambda: scan_bwd(x, dout=z(B, T, D, dtype=F32)), "dout must be torch.bfloat16")
    raises(lambda: scan_bwd(x, dht=z(B, D, S)), "dht must be torch.float32")


@pytest.mark.parametrize("kw,msg", [
    ({}, "GPU tensors"), ({"u": z(3, 1, D)}, r"u must have shape \[N,D\]"), ({"state": z(5, S, D, dtype=F32)}, "state must have shape"),
    ({"state": z(2, D, S, dtype=F32)}, "2 pages for 3 rows"), ({"state": z(5, D, S)}, "state must be torch.float32"),
    ({"pages": z(3)}, "pages must be torch.int32"), ({"out": z(3, D, dtype=F32)}, "out must be torch.bfloat16"),
    ({"dt": z(2, D)}, "dt must have shape"),
])
def test_scan_step_mismatches_raise(kw, msg):
    x = dict(scan_args((3,)), state=z(5, D, S, dtype=F32), **{k: v for k, v in kw.items() if k in ("pages", "out")})
    x.update({k: v for k, v in kw.items() if k not in ("pages", "out")})
    raises(lambda: gb.gdn_scan_step(**x), msg)


# ------------------------------------------------------------------ norms and rotation
def rot_args(**kw):
    x = dict(q=z(B, T, 4, 64), k=z(B, T, 2, 64), freqs=z(32, dtype=F64), positions=None)
    x.update(kw)
    return x


@pytest.mark.parametrize("bad,kw,msg", [
    ({}, {}, "GPU tensors"), ({"q": z(T, 4, 64), "k": z(T, 2, 64)}, {}, "need positions"),
    ({"q": z(T, 4, 64), "k": z(T, 2, 64), "positions": z(T, dtype=I32)}, {}, "GPU tensors"),
    ({"q": z(T, 4, 64), "k": z(T, 2, 64), "freqs": None}, {}, "GPU tensors"),
    ({"q": None}, {}, "q must have shape"), ({"k": None}, {}, "q's tokens and width"), ({"k": z(T, 2, 64)}, {}, "q's tokens"),
    ({"k": z(B, T, 2, 128)}, {}, "k must have shape"), ({"k": z(B, T, 2, 64, dtype=F32)}, {}, "k must be torch.bfloat16"),
    ({"k": z(B, T, 0, 64)}, {}, "need heads"),
    ({"freqs": z(32, dtype=F32)}, {}, "freqs must be torch.float64"), ({"freqs": z(36, dtype=F64)}, {}, "turn 72 of 64"),
    ({"positions": z(B, T)}, {}, "positions must be torch.int32 or torch.int64"),
    ({"positions": z(B, T + 1, dtype=I32)}, {}, "positions must have shape"),
    ({"q": z(B, T, 4, 68)[..., :64]}, {}, "16-byte aligned"),
    ({}, {"norm": "layer"}, "norm must be"), ({}, {"q_weight": z(32)}, "q_weight must have shape"),
    ({}, {"q_weight": z(64), "k_weight": z(64, dtype=F32)}, "k_weight must be torch.bfloat16"),
    ({}, {"q_weight": z(64, dtype=F64)}, "unsupported dtype"), ({}, {"eps": "x"}, "eps must be a number"),
    ({}, {"amplitude": None}, "amplitude must be a number"),
])
def test_rotary_mismatches_raise(bad, kw, msg):
    x = rot_args(**bad)
    raises(lambda: gb.gdn_qk_rotary_fwd(**x, **kw), msg)
    d = [z(*t.shape) if t is not None else None for t in (x["q"], x["k"])]
    raises(lambda: gb.gdn_qk_rotary_bwd(*x.values(), *d, **kw), msg)


def test_rotary_limits_outputs_and_gradients():
    for kw in (dict(q=z(B, T, 1, 60), k=z(B, T, 1, 60), freqs=None), dict(q=z(B, T, 1, 264), k=z(B, T, 1, 264), freqs=None),
               dict(freqs=z(30, dtype=F64))):
        raises(lambda: gb.gdn_qk_rotary_fwd(**rot_args(**kw)), "rows of|rotations of", NotImplementedError)
    x = rot_args()
    raises(lambda: gb.gdn_qk_rotary_fwd(**x, q_out=x["q"], k_out=x["k"]), "GPU tensors")      # in place is fine
    qk = z(B, T, 6, 64)
    y = rot_args(q=qk[:, :, :4], k=qk[:, :, 4:])
    raises(lambda: gb.gdn_qk_rotary_fwd(**y, q_out=qk.view(-1)[:B * T * 4 * 64].view(B, T, 4, 64)), "out overlaps q")
    raises(lambda: gb.gdn_qk_rotary_fwd(**rot_args(k=z(B, T, 4, 64)), q_out=x["q"], k_out=x["q"]), "out overlaps")
    raises(lambda: gb.gdn_qk_rotary_fwd(**x, k_out=z(B, T, 2, 64, dtype=F32)), "k_out must be torch.bfloat16")
    raises(lambda: gb.gdn_qk_rotary_bwd(*x.values(), None, x["k"]), "dq_out is required")
    raises(lambda: gb.gdn_qk_rotary_bwd(*x.values(), x["q"], None), "dk_out is required")
    raises(lambda: gb.gdn_qk_rotary_bwd(*x.values(), x["q"], x["q"]), "dk_out must have shape")


def test_rotary_frequencies():
    f = gb.rotary_frequencies(64, 10000.0)
    assert f.dtype == F64 and f[0] == 1 and torch.allclose(f[1:] / f[:-1], torch.full((31,), 10000.0 ** (-1 / 32), dtype=F64))
    assert torch.equal(gb.rotary_frequencies(64, factor=4, scaling="linear"), f / 4)
    b = gb.rotary_frequencies(64, factor=4, scaling="base")
    assert b[0] == 1 and abs(float(b[-1] * 4 / f[-1]) - 1) < 1e-12
    t = gb.rotary_frequencies(64, factor=8, scaling="by_turns", original_length=8192)
    turns = 8192 * f / 6.283185307179586
    assert torch.equal(t[turns >= 4], f[turns >= 4]) and torch.allclose(t[turns <= 1], f[turns <= 1] / 8, rtol=1e-15)
    mid = (turns > 1) & (turns < 4)
    assert mid.any() and ((t[mid] > f[mid] / 8) & (t[mid] < f[mid])).all()
    for bad in (dict(width=7), dict(width=0), dict(width=64, scaling="x"), dict(width=64, factor=0),
                dict(width=2, scaling="base"), dict(width=64, scaling="by_turns"),
                dict(width=64, scaling="by_turns", original_length=8, slow=4, fast=4)):
        with pytest.raises(ValueError):
            gb.rotary_frequencies(**bad)


# ------------------------------------------------------------------ the C ABI's own checks
@pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")
def test_abi_fuzz_under_sanitizers(tmp_path):
    out = _build_and_run(tmp_path, ["g++", "-std=c++17", *SAN, "-D__HIP_PLATFORM_AMD__", "-I", os.path.join(ROOT, "include"),
                                    "-I", CSRC, "-I", "/opt/rocm/include", os.path.join(CSRC, "gdn_mixer_host.cpp"),
                                    os.path.join(ROOT, "tests", "sanitize", "fuzz_mixer.cpp")], "fuzz_mixer")
    assert "statuses:" in out
    print(out)
