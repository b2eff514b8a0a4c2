"""What the inline assembly of the scan has to declare, read from its source."""
import os
import re

from test_host_sanitizers import ROOT


def test_assembly_that_writes_before_it_has_read_says_so():
    # results that the first instructions write may not share registers with inputs of the later ones
    src = open(os.path.join(ROOT, "chunked_gated_delta_05_amd", "csrc", "gdn_scan.hip")).read()
    blocks = [b for b in re.findall(r"\basm\s*(?:volatile\s*)?\((.*?)\)\s*;", src, re.S) if "GDN_HALVES" in b]
    assert len(blocks) == 2
    for b in blocks:
        results, inputs = re.split(r"\n\s*: ", b)[1:]
        assert '"v"(' in inputs and '"+&v"(' in results and '"+v"(' not in results, b
