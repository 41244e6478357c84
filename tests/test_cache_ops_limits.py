"""Rules of the cache operators that hold without a GPU."""
import os

import pytest

import medusa_speculative_decoding_02_gb300 as m
from medusa_speculative_decoding_02_gb300 import build as mbuild


def test_rotation_in_place_reads_no_read_only_path():
    """q_out may be q: the rows must not come through loads that PTX allows only for
    data that nothing writes during the kernel."""
    with open(os.path.join(mbuild.CSRC, "rope.cu")) as f:
        src = f.read()
    for load in ("ld.global.nc", "ld_stream16", "__ldg"):
        assert load not in src, load
