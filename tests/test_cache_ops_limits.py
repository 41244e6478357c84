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


def test_rows_of_the_4bit_calls_stay_in_the_division():
    """launch_kv4_rows divides a block's index by the blocks of a slot as a product
    and a shift: right up to the last index of the largest call of every size."""
    import numpy as np
    rows = 65535
    for dh in (64, 128):
        for Hkv in [*range(1, 1024, 7), 512, 1024]:
            d = 2 * Hkv * dh // 16
            s = 0
            while (2 << s) < d:
                s += 1
            magic = (1 << (32 + s)) // d + 1
            assert magic < 1 << 32
            blocks = rows * d
            assert blocks <= (1 << 30) - 256  # the last CTA's threads past the end included
            r = np.unique(np.r_[np.arange(3), np.linspace(3, rows, 97).astype(np.uint64)]).astype(np.uint64)
            for i in (r * np.uint64(d), r * np.uint64(d) + np.uint64(d - 1)):
                assert ((i * np.uint64(magic) >> np.uint64(32 + s)) == i // np.uint64(d)).all(), (dh, Hkv)
