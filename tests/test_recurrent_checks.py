"""The recurrent-state operators' argument checks and C ABI on the CPU: every
mismatch raises before anything touches a GPU, and a consistent call on CPU
tensors is rejected last, for not being on the GPU."""
import ctypes
import os
import re

import pytest
import torch

from chunked_gated_delta_05_amd import binding as gb

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32
B, T, H, K, V = 2, 70, 4, 128, 64


def test_library_exports_every_declared_function():
    src = open(os.path.join(ROOT, "include", "gdn_recurrent.h")).read()
    names = sorted(set(re.findall(r"^(?:gdn_status|size_t)\s+(gdn_\w+)\s*\(", src, re.M)))
    assert names == ["gdn_linattn_bwd", "gdn_linattn_fwd", "gdn_linattn_step", "gdn_pages_compact", "gdn_pages_copy",
                     "gdn_pages_fork", "gdn_pages_workspace_ints", "gdn_recurrent_step"]
    for n in names:
        assert hasattr(gb.lib(), n), n


# ------------------------------------------------------------------ prompts
def prompt(**kw):
    x = {"q": torch.zeros(B, T, H, K, dtype=BF), "k": torch.zeros(B, T, 2, K, dtype=BF),
         "v": torch.zeros(B, T, 1, V, dtype=BF), "decay": torch.zeros(H)}
    x.update(kw)
    return x


def fwd(x, **kw):
    return gb.gdn_linattn_fwd(x["q"], x["k"], x["v"], x["decay"], **kw)


def meta():
    return gb.UnitMeta([0, 30, 70], (ctypes.c_int32 * 3)(0, 30, 70), torch.zeros(3, dtype=I32),
                       torch.zeros(3, dtype=I32), torch.zeros(3, 2, dtype=I32), 3)


def test_consistent_cpu_calls_are_rejected_for_the_device():
    with pytest.raises(ValueError, match="GPU tensors"):
        fwd(prompt())
    with pytest.raises(ValueError, match="GPU tensors"):
        fwd({n: t[0] if t.dim() == 4 else t for n, t in prompt().items()}, meta=meta())
    x = prompt()
    with pytest.raises(ValueError, match="GPU tensors"):
        gb.gdn_linattn_bwd(x["q"], x["k"], x["v"], x["decay"], torch.zeros(B, T, H, V, dtype=BF))
    with pytest.raises(ValueError, match="GPU tensors"):   # views of one projection are accepted
        qkv = torch.zeros(B, T, 3 * H * K, dtype=BF)
        fwd(prompt(**{n: qkv[..., i * H * K:(i + 1) * H * K].unflatten(-1, (H, K)) for i, n in enumerate("qkv")}))


@pytest.mark.parametrize("bad,msg", [
    ({"q": torch.zeros(B, T, H, K)}, "q must be torch.bfloat16"),
    ({"v": torch.zeros(B, T, 1, V)}, "v must be torch.bfloat16"),
    ({"k": torch.zeros(B, T, 2, K, dtype=torch.float16)}, "unsupported dtype torch.float16"),
    ({"k": None}, "must have shape"),
    ({"q": None}, "q must have shape"),
    ({"k": torch.zeros(T, 2, dtype=BF)}, "must have shape"),
    ({"q": torch.zeros(B, T - 1, H, K, dtype=BF)}, "q must have shape"),
    ({"q": torch.zeros(B, T, 3, K, dtype=BF)}, "3 heads, which do not divide 4"),
    ({"v": torch.zeros(B, T, 0, V, dtype=BF)}, "0 heads"),
    ({"q": torch.zeros(B, T, H, 64, dtype=BF)}, "k's width 128"),
    ({"decay": torch.zeros(H, 1)}, "decay must be fp32"),
    ({"decay": None}, "decay must be fp32"),
    ({"decay": torch.zeros(H, dtype=BF)}, "decay must be torch.float32"),
    ({"q": torch.zeros(B, T, K, H, dtype=BF).transpose(-1, -2)}, "values of a row must be contiguous"),
    ({"q": torch.zeros(B, T, H, K + 4, dtype=BF)[..., :K]}, "16-byte aligned"),
    ({"q": torch.zeros(B * T * H * K + 8, dtype=BF)[1:1 + B * T * H * K].view(B, T, H, K)}, "16-byte aligned"),
    ({"q": torch.zeros(T, B, H, K, dtype=BF).transpose(0, 1)}, "batch rows must follow"),
])
def test_prompt_mismatches_raise(bad, msg):
    x = prompt(**bad)
    with pytest.raises(ValueError, match=msg):
        fwd(x)
    with pytest.raises(ValueError, match=msg):
        gb.gdn_linattn_bwd(x["q"], x["k"], x["v"], x["decay"], torch.zeros(B, T, H, V, dtype=BF))


@pytest.mark.parametrize("kw,msg", [
    ({"out": torch.zeros(B, T, H, V, dtype=BF), "o_dtype": F32}, "out must be torch.float32"),
    ({"out": torch.zeros(B, T, H, V - 1, dtype=BF)}, "out must have shape"),
    ({"out": torch.zeros(B, T, V, H, dtype=BF).transpose(-1, -2)}, "out must be contiguous"),
    ({"o_dtype": torch.float16}, "unsupported output dtype"),
    ({"o_dtype": "bf16"}, "o_dtype must be a torch dtype"),
    ({"initial_state": torch.zeros(B, H, K, V, dtype=BF)}, "initial_state must be torch.float32"),
    ({"initial_state": torch.zeros(B + 1, H, K, V)}, "initial_state must have shape"),
    ({"initial_pages": torch.zeros(B, dtype=I32)}, "must be a pool"),
    ({"initial_state": torch.zeros(5, H, K, V), "initial_pages": torch.zeros(B + 1, dtype=I32)}, "initial_pages must have"),
    ({"initial_state": torch.zeros(5, H, K, V), "initial_pages": torch.zeros(B)}, "initial_pages must be torch.int32"),
    ({"final_out": torch.zeros(B, H, V, K)}, "final_out must have shape"),
    ({"initial_state": torch.zeros(5, H, K, V), "initial_pages": torch.zeros(B, dtype=I32),
      "final_out": torch.zeros(6, H, K, V), "final_pages": torch.zeros(B, dtype=I32)}, "pools have 5 and 6 pages"),
    ({"meta": meta()}, "meta goes with packed"),
    ({"scale": "x"}, "scale must be a number"),
])
def test_prompt_option_mismatches_raise(kw, msg):
    with pytest.raises(ValueError, match=msg):
        fwd(prompt(), **kw)


def test_packed_prompts_need_meta_and_gradients_their_shapes():
    x = prompt()
    with pytest.raises(ValueError, match="need meta"):
        fwd({n: t[0] if t.dim() == 4 else t for n, t in x.items()})
    bwd = lambda dout, **kw: gb.gdn_linattn_bwd(x["q"], x["k"], x["v"], x["decay"], dout, **kw)
    ok = torch.zeros(B, T, H, V, dtype=BF)
    for dout, kw, msg in ((None, {}, "dout is required"), (ok.float(), {}, "dout must be torch.bfloat16"),
                          (ok[:, :, :1], {}, "dout must have shape"),
                          (ok, {"dht": torch.zeros(B, H, V, K)}, "dht must have shape"),
                          (ok, {"initial_state": torch.zeros(1, H, K, V)}, "initial_state must have shape")):
        with pytest.raises(ValueError, match=msg):
            bwd(dout, **kw)


# ------------------------------------------------------------------ single tokens
N = 3


def rows(**kw):
    x = {"q": torch.zeros(N, 2, 128, dtype=BF), "k": torch.zeros(N, 2, 128, dtype=BF),
         "v": torch.zeros(N, H, 128, dtype=BF), "decay": torch.zeros(H), "state": torch.zeros(5, H, 128, 128),
         "g": torch.zeros(N, H), "beta": torch.zeros(N, H, dtype=BF)}
    x.update(kw)
    return x


def steps(x, **kw):
    yield lambda: gb.gdn_linattn_step(x["q"], x["k"], x["v"], x["decay"], x["state"], **kw)
    yield lambda: gb.gdn_recurrent_step(x["q"], x["k"], x["v"], x["g"], x["beta"], x["state"], **kw)


def test_consistent_cpu_steps_are_rejected_for_the_device():
    for f in steps(rows(), pages=torch.zeros(N, dtype=I32)):
        with pytest.raises(ValueError, match="GPU tensors"):
            f()


@pytest.mark.parametrize("bad,kw,msg", [
    ({"k": torch.zeros(N, 2, dtype=BF)}, {}, "step inputs must have shape"),
    ({"q": torch.zeros(N + 1, 2, 128, dtype=BF)}, {}, "q must have shape"),
    ({"v": torch.zeros(N, H, 128)}, {}, "v must be torch.bfloat16"),
    ({"q": torch.zeros(N, 3, 128, dtype=BF)}, {}, "do not divide 4"),
    ({"state": torch.zeros(5, H, 128)}, {}, r"state must be \[n_pages"),
    ({"state": torch.zeros(5, H, 128, 64)}, {}, "state must have shape"),
    ({"state": torch.zeros(5, H, 128, 128, dtype=BF)}, {}, "state must be torch.float32"),
    ({"state": torch.zeros(5, H, 128, 256)[..., ::2]}, {}, "state must be contiguous"),
    ({"state": torch.zeros(2, H, 128, 128)}, {}, "2 pages for 3 rows"),
    ({}, {"pages": torch.zeros(N)}, "pages must be torch.int32"),
    ({}, {"pages": torch.zeros(N + 1, dtype=I32)}, "pages must have shape"),
    ({}, {"out": torch.zeros(N, H, 64, dtype=BF)}, "out must have shape"),
    ({"q": torch.zeros(N, 2, 132, dtype=BF)[..., :128]}, {}, "16-byte aligned"),
])
def test_step_mismatches_raise(bad, kw, msg):
    for f in steps(rows(**bad), **kw):
        with pytest.raises(ValueError, match=msg):
            f()


@pytest.mark.parametrize("bad,msg", [
    ({"g": torch.zeros(N, H, 64)}, "g must have shape"), ({"g": torch.zeros(N)}, "g must be"),
    ({"g": torch.zeros(N, H, dtype=BF)}, "g must be torch.float32"),
    ({"beta": torch.zeros(N, H)}, "beta must be torch.bfloat16"), ({"beta": torch.zeros(N)}, "beta must be"),
])
def test_delta_step_mismatches_raise(bad, msg):
    x = rows(**bad)
    with pytest.raises(ValueError, match=msg):
        gb.gdn_recurrent_step(x["q"], x["k"], x["v"], x["g"], x["beta"], x["state"])


# ------------------------------------------------------------------ pages
def test_pages_mismatches_raise():
    pool, ids = torch.zeros(2, 6, 4, 4), torch.zeros(3, dtype=I32)
    for f in (lambda p, t: gb.gdn_pages_fork(p, t, ids), gb.gdn_pages_compact,
              lambda p, t: gb.gdn_pages_copy(p, p, t, ids)):
        for p, t, msg in ((torch.zeros(2, 6), ids, "must be \\[n_layers"), (pool.transpose(0, 1), ids, "contiguous"),
                          (torch.zeros(2, 6, 3), ids, "multiple of 16 bytes"), (pool, ids.long(), "must be torch.int32"),
                          (pool, ids, "GPU tensors")):
            with pytest.raises(ValueError, match=msg):
                f(p, t)
    with pytest.raises(ValueError, match="parent must have shape"):
        gb.gdn_pages_fork(pool, ids, ids[:2])
    with pytest.raises(ValueError, match="pools differ"):
        gb.gdn_pages_copy(pool, torch.zeros(2, 6, 4, 8), ids, ids)
    with pytest.raises(ValueError, match="pools differ"):
        gb.gdn_pages_copy(pool, torch.zeros(3, 6, 4, 4), ids, ids)


# ------------------------------------------------------------------ the C ABI's own checks
class LinattnDesc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("B", "T", "H", "Hq", "Hk", "Hv", "K", "V", "dtype", "o_dtype")] + [
        ("scale", ctypes.c_float), ("n_units", ctypes.c_int32), ("q_stride", ctypes.c_int64 * 2),
        ("k_stride", ctypes.c_int64 * 2), ("v_stride", ctypes.c_int64 * 2),
        ("offsets_host", ctypes.POINTER(ctypes.c_int32)), ("offsets_dev", ctypes.c_void_p)]


def query(**kw):
    d = LinattnDesc(B=2, T=100, H=4, Hq=4, Hk=2, Hv=1, K=128, V=64, dtype=1, o_dtype=1, scale=0.1)
    d.q_stride[:], d.k_stride[:], d.v_stride[:] = (512, 128), (256, 128), (64, 64)
    offs = kw.pop("offsets", None)
    if offs is not None:
        kw["offsets_host"] = (ctypes.c_int32 * len(offs))(*offs)
        kw.setdefault("offsets_dev", 1 << 20)
    for n, x in kw.items():
        if n.endswith("stride"):
            getattr(d, n)[:] = x
        else:
            setattr(d, n, x)
    nb = ctypes.c_size_t(0)
    vp = ctypes.c_void_p(None)
    f = gb.lib().gdn_linattn_fwd
    f.restype = ctypes.c_int
    st = f(ctypes.byref(d), vp, vp, vp, vp, vp, vp, vp, vp, ctypes.c_int32(0), vp, vp, ctypes.byref(nb), vp)
    return st, nb.value


@pytest.mark.parametrize("kw,status", [
    ({}, gb.GDN_OK), ({"T": 0}, gb.GDN_OK), ({"B": 1, "n_units": 2, "offsets": [0, 40, 100]}, gb.GDN_OK),
    ({"K": 96}, gb.GDN_ERR_UNSUPPORTED), ({"V": 256}, gb.GDN_ERR_UNSUPPORTED), ({"B": 0}, gb.GDN_ERR_INVALID),
    ({"T": -1}, gb.GDN_ERR_INVALID), ({"H": 0}, gb.GDN_ERR_INVALID), ({"Hk": 3}, gb.GDN_ERR_INVALID),
    ({"Hv": 0}, gb.GDN_ERR_INVALID), ({"dtype": 2}, gb.GDN_ERR_INVALID), ({"o_dtype": -1}, gb.GDN_ERR_INVALID),
    ({"scale": float("nan")}, gb.GDN_ERR_INVALID), ({"q_stride": (12, 128)}, gb.GDN_ERR_INVALID),
    ({"q_stride": (-512, 128)}, gb.GDN_ERR_INVALID), ({"k_stride": (1 << 62, 128)}, gb.GDN_ERR_INVALID),
    ({"q_stride": (1 << 25, 128)}, gb.GDN_ERR_UNSUPPORTED), ({"n_units": -1}, gb.GDN_ERR_INVALID),
    ({"n_units": 2, "offsets": [0, 40, 200]}, gb.GDN_ERR_INVALID),              # documents of one row only
    ({"B": 1, "n_units": 2, "offsets": [0, 40, 99]}, gb.GDN_ERR_INVALID),
    ({"B": 1, "n_units": 2, "offsets": [0, 0, 100]}, gb.GDN_ERR_INVALID),
    ({"B": 1, "n_units": 2, "offsets": [1, 40, 100]}, gb.GDN_ERR_INVALID),
    ({"B": 1, "n_units": 2, "offsets": [0, 40, 100], "offsets_dev": 0}, gb.GDN_ERR_INVALID),
])
def test_prompt_descriptor(kw, status):
    assert query(**kw)[0] == status


def test_workspace_is_the_states_between_segments():
    # one segment a sequence: the least workspace; cut sequences: a state a segment
    assert query(T=64)[1] == 256
    st, nb = query(T=4096)
    assert st == gb.GDN_OK and nb % (2 * 4 * 128 * 64 * 4) == 0 and nb > 256


@pytest.mark.parametrize("T,status", [(2 ** 31 - 1 - 2 ** 26, gb.GDN_OK), (2 ** 31 - 1, gb.GDN_ERR_UNSUPPORTED)])
def test_a_segments_end_is_an_int(T, status):
    one = (64, 64)
    kw = dict(B=1, T=T, H=1, Hq=1, Hk=1, Hv=1, K=64, V=64, q_stride=one, k_stride=one, v_stride=one)
    assert query(**kw)[0] == status
    assert query(n_units=1, offsets=[0, T], **kw)[0] == status


# ------------------------------------------------------------------ launch sizes
def status_of(f, *args):
    fn = getattr(gb.lib(), f)
    fn.restype = ctypes.c_int
    return fn(*args)


NONE = ctypes.c_void_p(None)


def bwd_query(**kw):
    d = LinattnDesc(B=1, T=4, H=1, Hq=1, Hk=1, Hv=1, K=64, V=64, dtype=1, o_dtype=1, scale=0.1)
    for n, x in kw.items():
        setattr(d, n, x)
    for n, h, w in (("q", d.Hq, d.K), ("k", d.Hk, d.K), ("v", d.Hv, d.V)):
        getattr(d, n + "_stride")[:] = (h * w, w)
    nb = ctypes.c_size_t(0)
    return status_of("gdn_linattn_bwd", ctypes.byref(d), *[NONE] * 12, ctypes.byref(nb), NONE)


# a launch has fewer than 2^32 threads along x: 256 for a row's head, in the
# backward for each of three passes; a quarter of the values where shared heads are summed
def test_forward_launches_of_2_to_the_32_threads_are_refused():
    one = dict(T=1, H=32, Hq=1, Hk=1, Hv=1, K=64, V=64, q_stride=(64, 64), k_stride=(64, 64), v_stride=(64, 64))
    assert query(B=2 ** 19 - 1, **one)[0] == gb.GDN_OK
    assert query(B=2 ** 19, **one)[0] == gb.GDN_ERR_UNSUPPORTED


def test_backward_launches_of_2_to_the_32_threads_are_refused():
    most = (2 ** 32 - 1) // (3 * 256 * 32)
    assert bwd_query(B=most, H=32, Hq=32, Hk=32, Hv=32) == gb.GDN_OK
    assert bwd_query(B=most + 1, H=32, Hq=32, Hk=32, Hv=32) == gb.GDN_ERR_UNSUPPORTED
    # tokens x shared heads x width / 4
    for n in ("Hq", "Hk", "Hv"):
        kw = {"Hq": 64, "Hk": 64, "Hv": 64, n: 32}
        assert bwd_query(B=1, T=2 ** 23 - 1, H=64, **kw) == gb.GDN_OK
        assert bwd_query(B=1, T=2 ** 23, H=64, **kw) == gb.GDN_ERR_UNSUPPORTED


def test_whole_workgroups_of_sums_of_shared_heads_count():
    # 2^32 - 16 values in fours fill the 2^24th workgroup of 256 in part
    assert bwd_query(B=1, T=2 ** 28 - 1, H=2, Hq=1, Hk=2, Hv=2) == gb.GDN_ERR_UNSUPPORTED


def test_merges_of_2_to_the_32_threads_are_refused():
    # one long document among many of one token is cut; the merge has K V / 4 threads a document and head
    one = dict(B=1, H=16, Hq=16, Hk=16, Hv=16, K=128, V=128, q_stride=(2048, 128), k_stride=(2048, 128),
               v_stride=(2048, 128))
    for docs, status in ((2 ** 16 - 1, gb.GDN_OK), (2 ** 16, gb.GDN_ERR_UNSUPPORTED)):
        offs = [*range(docs), docs - 1 + 2 ** 22]
        st, need = query(T=offs[-1], n_units=docs, offsets=offs, **one)
        assert st == status
        if st == gb.GDN_OK:   # cut: a state for each segment
            assert need // (16 * 128 * 128 * 4) > docs + 4


class StepDesc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("N", "H", "Hq", "Hk", "Hv", "K", "V", "dtype", "o_dtype")] + [
        ("scale", ctypes.c_float), ("n_pages", ctypes.c_int32), ("q_stride", ctypes.c_int64 * 2),
        ("k_stride", ctypes.c_int64 * 2), ("v_stride", ctypes.c_int64 * 2)]


def test_step_launches_of_2_to_the_32_threads_are_refused():
    for N, status in ((2 ** 19 - 1, gb.GDN_ERR_INVALID), (2 ** 19, gb.GDN_ERR_UNSUPPORTED)):   # INVALID: no pointers given
        d = StepDesc(N=N, H=32, Hq=32, Hk=32, Hv=32, K=128, V=128, dtype=1, o_dtype=1, scale=0.1, n_pages=1)
        for s in (d.q_stride, d.k_stride, d.v_stride):
            s[:] = (32 * 128, 128)
        assert status_of("gdn_linattn_step", ctypes.byref(d), *[NONE] * 8) == status
        assert status_of("gdn_recurrent_step", ctypes.byref(d), 0, 0, *[NONE] * 7, 0, NONE) == status


# ------------------------------------------------------------------ outputs that are inputs
I64 = ctypes.c_int64
AT = 1 << 30      # addresses that nothing may touch: a refused call enqueues nothing


def fork_status(n, m, **at):
    """The plan's buffers lie 1 MiB apart unless placed elsewhere."""
    p = {b: AT + (i << 20) for i, b in enumerate(("table", "parent", "spare", "new_table", "left", "workspace"))}
    p.update({b: p[x] + d for b, (x, d) in at.items()})
    p = {b: ctypes.c_void_p(x) for b, x in p.items()}
    return status_of("gdn_pages_fork", ctypes.c_void_p(AT << 4), 1, 600, I64(1024), p["table"], p["parent"], n, p["spare"],
                     m, p["new_table"], p["left"], p["workspace"], NONE)


@pytest.mark.parametrize("n,m", [(8, 4), (300, 260)])
@pytest.mark.parametrize("out,at", [
    ("left", ("spare", 0)),            # an in-place list of free pages
    ("new_table", ("parent", 0)), ("new_table", ("table", 4)), ("new_table", ("table", -4)),
    ("left", ("parent", -16)), ("left", ("table", 28)), ("left", ("new_table", 12)),
    ("workspace", ("spare", 8)), ("workspace", ("new_table", -8)), ("workspace", ("left", 0)),
])
def test_a_fork_refuses_outputs_over_its_inputs(out, at, n, m):
    assert fork_status(n, m, **{out: at}) == gb.GDN_ERR_INVALID


@pytest.mark.parametrize("out,at", [
    ("new_table", ("table", 0)), ("new_table", ("table", 4)), ("count", ("table", 28)), ("count", ("new_table", 0)),
    ("workspace", ("table", 0)), ("workspace", ("new_table", -8)), ("workspace", ("count", -400)),
])
def test_a_compaction_refuses_outputs_over_its_inputs(out, at):
    p = {b: AT + (i << 20) for i, b in enumerate(("table", "new_table", "count", "workspace"))}
    p[out] = p[at[0]] + at[1]
    p = {b: ctypes.c_void_p(x) for b, x in p.items()}
    assert status_of("gdn_pages_compact", ctypes.c_void_p(AT << 4), 1, 60, I64(1024), p["table"], 8, p["new_table"],
                     p["count"], p["workspace"], NONE) == gb.GDN_ERR_INVALID


# shifted against a state that another walk reads: no order of the sequences would do
@pytest.mark.parametrize("over", ["dht", "s_in"])
@pytest.mark.parametrize("shift", [16, -16, 1 << 18])
@pytest.mark.parametrize("T", [40, 2000])      # uncut, cut
def test_a_gradient_shifted_against_its_states_is_refused(over, shift, T):
    d = LinattnDesc(B=2, T=T, H=4, Hq=4, Hk=4, Hv=4, K=128, V=128, dtype=1, o_dtype=1, scale=0.1)
    for s in (d.q_stride, d.k_stride, d.v_stride):
        s[:] = (512, 128)
    at = {n: AT + (i << 26) for i, n in enumerate(("q", "k", "v", "decay", "s_in", "dout", "dht", "dq", "dk", "dv"))}
    at["dh0"] = at[over] + shift
    nb = ctypes.c_size_t(1 << 30)
    assert status_of("gdn_linattn_bwd", ctypes.byref(d), *(ctypes.c_void_p(x) for x in at.values()),
                     ctypes.c_void_p(AT << 4), ctypes.byref(nb), NONE) == gb.GDN_ERR_INVALID


# ------------------------------------------------------------------ unit metadata
@pytest.mark.parametrize("change,msg", [
    ({"offsets_dev": torch.zeros(2, dtype=I32)}, "offsets must have shape"),     # the kernels read one for every document
    ({"offsets_dev": torch.zeros(3)}, "offsets must be torch.int32"),
    ({"offsets_dev": torch.zeros(6, dtype=I32)[::2]}, "offsets must be contiguous"),
    ({"offsets": [0, 30, 50, 70], "offsets_dev": torch.zeros(4, dtype=I32)}, "host copy"),
    ({"offsets": [0], "offsets_dev": torch.zeros(1, dtype=I32), "host": (ctypes.c_int32 * 1)(0)}, "no documents"),
])
def test_unit_metadata_is_checked(change, msg):
    x = {n: t[0] if t.dim() == 4 else t for n, t in prompt().items()}
    m = meta()
    for n, y in change.items():
        setattr(m, n, y)
    with pytest.raises(ValueError, match=msg):
        fwd(x, meta=m)
    with pytest.raises(ValueError, match=msg):
        gb.gdn_linattn_bwd(x["q"], x["k"], x["v"], x["decay"], torch.zeros(T, H, V, dtype=BF), meta=m)


# ------------------------------------------------------------------ out over an input
@pytest.mark.parametrize("over", ["q", "k", "v", "initial_state", "final_out"])
def test_a_prompts_out_over_an_input_is_refused(over):
    # a head's value columns may be two workgroups' work, and each reads all of q and k
    n, h = 60, 2
    buf = {m: torch.zeros(n * h * 64 + 64) for m in "qkv"}
    x = {m: t[:n * h * 64].view(1, n, h, 64) for m, t in buf.items()}
    states = {m: torch.zeros(1, h, 64, 64) for m in ("initial_state", "final_out")}
    if over not in states:
        out = buf[over][64:].view(1, n, h, 64)    # shifted by a row: contiguous, 16-byte aligned
    else:                                          # one token that ends inside the state
        x = {m: t[:, :1, :1] for m, t in x.items()}
        states = {m: torch.zeros(1, 1, 64, 64) for m in states}
        out = states[over].flatten()[-64:].view(1, 1, 1, 64)
    with pytest.raises(ValueError, match=f"out overlaps {over}"):
        gb.gdn_linattn_fwd(x["q"], x["k"], x["v"], torch.zeros(x["q"].shape[2]), out=out, **states)
    with pytest.raises(ValueError, match="GPU tensors"):
        gb.gdn_linattn_fwd(x["q"], x["k"], x["v"], torch.zeros(x["q"].shape[2]), out=out.clone(), **states)


@pytest.mark.parametrize("over", ["q", "k", "v", "state"])
def test_a_steps_out_over_an_input_is_refused(over):
    x = rows(q=torch.zeros(N, H, 128), k=torch.zeros(N, H, 128), v=torch.zeros(N, H, 128), beta=torch.zeros(N, H))
    out = x["state"].flatten()[:N * H * 128].view(N, H, 128) if over == "state" else x[over]
    for f in steps(x, out=out):
        with pytest.raises(ValueError, match=f"out overlaps {over}"):
            f()
