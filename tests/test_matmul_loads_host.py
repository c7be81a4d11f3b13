"""Every process of a job on several GPUs may call every kernel of the library, so none loads
tiles into several blocks' shared memory at once."""

import glob
import os
import re

import padding_free_packed_gb300.build as build


def test_no_bulk_load_names_several_blocks():
    paths = glob.glob(os.path.join(build.CSRC, "*.cu*"))
    assert paths
    for path in paths:
        with open(path) as fh:
            text = re.sub(r'"\s*\n\s*"', "", fh.read())      # joined string literals
        for load in re.findall(r"cp\.(?:reduce\.)?async\.bulk[^\"]*", text):
            assert "multicast" not in load, f"{os.path.basename(path)}: {load}"
