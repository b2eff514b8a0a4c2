"""What the host code of the operators around the recurrent layers hands to the
kernels for chosen calls (gdn_mixer_host.cpp with launch stubs). Built with g++
alone."""
import os
import shutil
import subprocess

import pytest

from test_host_sanitizers import ROOT, SAN

CSRC = os.path.join(ROOT, "chunked_gated_delta_05_amd", "csrc")


@pytest.fixture(scope="module")
def plans(tmp_path_factory):
    if shutil.which("g++") is None:
        pytest.skip("needs g++")
    exe = str(tmp_path_factory.mktemp("plans") / "mixer_plans")
    subprocess.run(["g++", "-std=c++17", *SAN, "-D__HIP_PLATFORM_AMD__", "-I", os.path.join(ROOT, "include"), "-I", CSRC,
                    "-I", "/opt/rocm/include", os.path.join(CSRC, "gdn_mixer_host.cpp"),
                    os.path.join(ROOT, "tests", "sanitize", "mixer_plans.cpp"), "-o", exe], check=True)

    def run(what):
        env = {k: v for k, v in os.environ.items() if k != "LD_PRELOAD"}
        r = subprocess.run([exe, what], capture_output=True, text=True, timeout=120, env=env)
        assert r.returncode == 0 and f"{what}: ok" in r.stdout, r.stdout + r.stderr

    return run


def test_gradients_of_few_segments_are_joined_with_and_without_states(plans):
    plans("joins")


def test_states_may_not_overlap_by_part(plans):
    plans("states")


def test_sums_that_share_a_launch_fit_into_it(plans):
    plans("limits")
