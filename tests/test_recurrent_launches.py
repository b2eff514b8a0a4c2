"""What the host code of the recurrent-state operators hands to the kernels
(gdn_recurrent_host.cpp with launch stubs), for random valid calls: segments
that cover the sequences, launches within HIP's limit, no state replaced while
a walk may read it, no plan that writes what it reads. Built with g++ alone."""
import os
import shutil

import pytest

from test_host_sanitizers import ROOT, SAN, _build_and_run


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")
def test_launches_of_valid_calls(tmp_path):
    csrc = os.path.join(ROOT, "chunked_gated_delta_05_amd", "csrc")
    out = _build_and_run(tmp_path, ["g++", "-O1", "-std=c++17", *SAN, "-D__HIP_PLATFORM_AMD__", "-I",
                                    os.path.join(ROOT, "include"), "-I", csrc, "-I", "/opt/rocm/include",
                                    os.path.join(csrc, "gdn_recurrent_host.cpp"),
                                    os.path.join(ROOT, "tests", "sanitize", "fuzz_recurrent_launches.cpp")],
                         "fuzz_recurrent_launches")
    assert "launches:" in out
