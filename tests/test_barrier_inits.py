"""Kernels whose mbarriers take asynchronous arrivals (copies, tensor-core commits) fence the barriers' initialisation."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "gated_deltanet_linear_decode_gb300", "csrc")
FILES = [f for f in sorted(glob.glob(os.path.join(CSRC, "*.cu*"))) if re.search(r"\btc::mbar_init\(", open(f).read())]


@pytest.mark.parametrize("path", FILES, ids=os.path.basename)
def test_the_inits_are_fenced(path):
    src = re.sub(r"//.*", "", open(path).read())
    last = [m.end() for m in re.finditer(r"\bmbar_init\(", src)][-1]
    rest = src[last:]
    fence = rest.find("fence.mbarrier_init.release.cluster")
    assert fence >= 0, "no fence"
    barrier = re.search(r"__syncthreads\(\)|cluster_sync|my_share", rest)
    assert barrier is None or fence < barrier.start(), "the block's barrier comes before the fence"
