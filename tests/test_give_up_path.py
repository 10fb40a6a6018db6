"""A wait that runs out is not made to happen on a GPU for the delta rule's kernels: what their give-up paths wait for
before they return is read from the source."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "causal_depthwise_conv1d_gb300", "csrc")
FILES = [p for p in sorted(glob.glob(os.path.join(CSRC, "gdr_*.cu"))) if "mbar_wait(" in open(p).read()]


def give_up_paths(text):
    """The blocks, up to their return, of the conditions that follow a failed wait in a kernel."""
    for m in re.finditer(r"if \((?:late|!mbar_wait\([^;]*?\))\) \{(.*?)\breturn;", text, re.S):
        yield m.group(1)


@pytest.mark.parametrize("path", FILES, ids=[os.path.basename(p) for p in FILES])
def test_stores_and_loads_of_the_block_are_waited_for(path):
    text = open(path).read()
    paths = list(give_up_paths(text))
    assert paths
    for block in paths:
        assert "g_fault" in block
        assert block.count("mbar_wait(") >= 1  # copies into the other stages
        if "bulk_store(" in text:
            assert "bulk_wait_all();" in block  # copies out of the block's shared memory
        if "cp_async16(" in text:
            assert "cp_async_wait_all();" in block
