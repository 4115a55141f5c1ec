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


@pytest.mark.parametrize("path", sorted(glob.glob(os.path.join(_build.CSRC, "*.cu*"))), ids=os.path.basename)
def test_what_is_told_across_ctas_is_released(path):
    """st.async orders the word that it stores and nothing else, so it stores what is read and never a word
    that only stands for other writes; an arrival without a release of its own follows a fence."""
    with open(path) as f:
        text = f.read()
    assert not re.search(r"store_async\([^;]*,\s*0(\.0?f)?\);", text)
    asm = [x for x in re.findall(r'"([^"\n]*)"', re.sub(r'"\s*"', "", text)) if "." in x]  # instructions
    for before, this in zip([""] + asm, asm):
        if "mbarrier.arrive.relaxed" in this:
            assert "fence.release" in before
