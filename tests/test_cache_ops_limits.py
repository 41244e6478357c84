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


@pytest.mark.parametrize("kv4", [False, True])
def test_integers_past_32_bits_are_refused(kv4):
    """ctypes would take them modulo 2^32: a window of 2^32 + 3 would be one of 3."""
    mbuild.build()
    size = m.tree_attention_window_workspace_size
    assert size(m.BF16, 1, 65, 8, 8, 128, 5000, 2 ** 31 - 1, 2 ** 31 - 1, kv4) >= m.WS_HEADER
    for P_max, window, sinks in ((5000, 2 ** 32 + 3, 0), (5000, 2 ** 31, 0), (2 ** 32 + 7, 0, 0),
                                 (5000, 64, 2 ** 32 + 1), (5000, -2 ** 31 - 1, 0)):
        with pytest.raises(ValueError):
            size(m.BF16, 1, 65, 8, 8, 128, P_max, window, sinks, kv4)
    for bad in (2 ** 31, -2 ** 31 - 1, 2 ** 40):
        with pytest.raises(ValueError):
            m._ints(0, bad)
    m._ints(2 ** 31 - 1, -2 ** 31)
