"""The recorded DRAM traffic belongs to the sources whose hash it is keyed by: all of them are in it."""
import os
import re

import bench


def test_every_included_header_is_hashed():
    names = {os.path.basename(p) for p in bench.kernel_sources()}
    assert {"ccv_fwd_time.cu", "ccv_update.cu", "ccv_common.cuh"} <= names
    for p in bench.kernel_sources():
        assert set(re.findall(r'#include "([^"]+)"', open(p).read())) <= names, p
