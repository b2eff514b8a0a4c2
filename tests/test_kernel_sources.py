"""What inline assembly in the kernels has to declare, read from the sources."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "chunked_gated_delta_05_amd", "csrc")
ASM = re.compile(r"asm\s+volatile\s*\((.*?)\);", re.S)


@pytest.mark.parametrize("path", sorted(glob.glob(os.path.join(CSRC, "*.h*"))), ids=os.path.basename)
def test_assembly_that_writes_m0_says_so(path):
    for block in ASM.findall(open(path).read()):
        if re.search(r"s_mov_b32\s+m0\s*,", block):
            assert '"m0"' in block.rsplit(":", 1)[1], block


def test_native_calls_launch_on_their_tensors_device():
    # every function that asks for a stream has made the stream's device current
    src = open(os.path.join(CSRC, "gdn_torch.cpp")).read()
    calls = [f for f in re.split(r"\n}\n", src) if "stream_of(" in f and "PyObject* " in f]
    assert len(calls) == 7
    for f in calls:
        assert "const Guard guard(" in f and f.index("const Guard guard(") < f.index("stream_of("), f
