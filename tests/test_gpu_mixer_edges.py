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
