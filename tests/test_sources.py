"""What the kernels' sources may not contain."""
import glob
import os
import re

import pytest

from causal_gqa_attention_rope_gb300 import _build


@pytest.mark.parametrize("path", sorted(glob.glob(os.path.join(_build.CSRC, "*.cu*"))), ids=os.path.basename)
def test_no_multicast_load(path):
    """Nothing says that a caller's buffer is this GPU's own memory, and replicas on several GPUs load
    the same library: no copy is sent to several CTAs of a cluster.  (What tells several
    CTAs of the end of a product, tcgen05.commit, reads no memory.)"""
    with open(path) as f:
        text = re.sub(r'"\s*"', "", f.read())  # adjacent literals are one
    for literal in re.findall(r'"([^"\n]*)"', text):
        for instruction in literal.split(";"):
            assert not ("cp.async.bulk" in instruction and "multicast" in instruction), instruction
