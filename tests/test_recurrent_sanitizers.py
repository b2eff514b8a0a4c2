"""The host code of the recurrent-state operators (gdn_recurrent_host.cpp, with
launch stubs that check what it hands them) driven by a fuzzer under
AddressSanitizer and UndefinedBehaviorSanitizer. Built with g++ alone; no
device code is involved."""
import os
import shutil

import pytest

from test_host_sanitizers import ROOT, SAN, _build_and_run


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")
def test_recurrent_abi_fuzz_under_sanitizers(tmp_path):
    csrc = os.path.join(ROOT, "chunked_gated_delta_05_amd", "csrc")
    out = _build_and_run(tmp_path, ["g++", "-std=c++17", *SAN, "-D__HIP_PLATFORM_AMD__", "-I",
                                    os.path.join(ROOT, "include"), "-I", csrc, "-I", "/opt/rocm/include",
                                    os.path.join(csrc, "gdn_recurrent_host.cpp"),
                                    os.path.join(ROOT, "tests", "sanitize", "fuzz_recurrent.cpp")], "fuzz_recurrent")
    print(out)
    assert "statuses:" in out
