"""Attention over the caches at the row counts where its kernels change (rows a
KV head has: up to 8, up to 16, more) against a 64-bit reference, with the
tolerances of test_gpu_cache_ops."""
import math

import numpy as np
import pytest
import torch

import cache_ops_ref as ref
import medusa_speculative_decoding_02_gb300 as m
from test_gpu_cache_ops import BF, attn_inputs, call_attn, check_attn, dev, status  # noqa: F401 (dev: fixture)

pytestmark = pytest.mark.gpu

# R, H, Hkv: 1, 7, 8, 9, 16, 17 and 64 rows a KV head
ROWS = [(1, 3, 3), (7, 1, 1), (2, 8, 2), (9, 2, 2), (4, 4, 1), (17, 1, 1), (16, 8, 2)]
LENGTHS = [0, 1, 7, 8, 9, 14, 15, 16, 17, 30, 31, 32, 33, 47, 62, 63, 64, 65, 100, 127, 128, 129, 191, 193]


@pytest.mark.parametrize("kv4", [False, True])
@pytest.mark.parametrize("dh", [64, 128])
@pytest.mark.parametrize("R,H,Hkv", ROWS)
def test_every_length(dev, kv4, dh, R, H, Hkv):
    a = attn_inputs(len(LENGTHS), R, H, Hkv, dh, LENGTHS, BF, kv4, dev, seed=R + H)
    for window, sinks in ((0, 0), (1, 0), (15, 3), (63, 17), (64, 16), (129, 65)):
        check_attn(call_attn(a, window, sinks, Hkv, kv4, dev), a, window, sinks, kv4=kv4)


@pytest.mark.parametrize("kv4", [False, True])
@pytest.mark.parametrize("B", [2, 8, 32, 33])
@pytest.mark.parametrize("R,H,Hkv", [(1, 4, 2), (5, 2, 1), (17, 2, 1)])
def test_ragged_batches_in_many_ranges(dev, kv4, B, R, H, Hkv):
    """A few long sequences among short and empty ones, and a P_max far above all."""
    prefix = [(53 * b * b) % 300 for b in range(B)]
    prefix[0], prefix[-1], prefix[B // 2] = 2900, 1700, 0
    a = attn_inputs(B, R, H, Hkv, 64, prefix, BF, kv4, dev, seed=B + R)
    check_attn(call_attn(a, 0, 0, Hkv, kv4, dev), a, 0, 0, kv4=kv4)
    tight = call_attn(a, 700, 20, Hkv, kv4, dev)
    check_attn(tight, a, 700, 20, kv4=kv4)
    a["P_max"] = 200000  # only bounds the prefixes
    check_attn(call_attn(a, 0, 0, Hkv, kv4, dev), a, 0, 0, kv4=kv4)
    check_attn(call_attn(a, 700, 20, Hkv, kv4, dev), a, 700, 20, kv4=kv4)


@pytest.mark.parametrize("kv4", [False, True])
@pytest.mark.parametrize("R,H,Hkv", [(1, 4, 1), (3, 5, 1), (17, 4, 1)])
def test_long_with_peaked_and_flat_scores(dev, kv4, R, H, Hkv):
    for std, scale in ((0.1, None), (8.0, None), (1.0, 1.0)):
        a = attn_inputs(2, R, H, Hkv, 128, [9001, 6000], BF, kv4, dev, seed=13, std=std)
        check_attn(call_attn(a, 0, 0, Hkv, kv4, dev, scale=scale), a, 0, 0, scale, kv4=kv4)
        check_attn(call_attn(a, 4097, 130, Hkv, kv4, dev, scale=scale), a, 4097, 130, scale, kv4=kv4)


@pytest.mark.parametrize("kv4", [False, True])
@pytest.mark.parametrize("R,H", [(6, 1), (6, 2), (20, 2)])
def test_queries_of_very_different_size(dev, kv4, R, H):
    a = attn_inputs(1, R, H, 1, 128, [100], BF, kv4, dev, seed=3)
    a["q"][0, 1] *= 1e-30
    a["q"][0, 2] *= 200.0
    a["q"][0, 3] = 0
    a["q"][0, 5, 0] *= 2.0 ** 100
    got = call_attn(a, 0, 0, 1, kv4, dev)
    check_attn(got, a, 0, 0, rows=[r for r in range(R) if r != 5], kv4=kv4)
    assert torch.isfinite(got[0, 5]).all()
    a["q"][0, 5, 0, 0] = math.inf
    got = call_attn(a, 0, 0, 1, kv4, dev)
    assert torch.isnan(got[0, 5, 0]).all() and torch.isfinite(got[0, :5]).all()


@pytest.mark.parametrize("kv4", [False, True])
@pytest.mark.parametrize("R,H", [(3, 1), (12, 1), (20, 1)])
def test_scale_below_the_normal_numbers(dev, kv4, R, H):
    """Every visible key weighs the same; the masked ones still nothing."""
    a = attn_inputs(1, R, H, 1, 64, [70], BF, kv4, dev, seed=4)
    a["q"] *= 1e-36
    scale = 1e-44
    check_attn(call_attn(a, 30, 4, 1, kv4, dev, scale=scale), a, 30, 4, scale, kv4=kv4)


@pytest.mark.parametrize("kv4", [False, True])
@pytest.mark.parametrize("dh", [64, 128])
@pytest.mark.parametrize("R,H", [(8, 1), (16, 1), (8, 2), (32, 1)])
@pytest.mark.parametrize("prefix", [0, 40, 150])
def test_infinities_reach_only_the_rows_that_see_them(dev, kv4, dh, R, H, prefix):
    """V: an infinity, or in 4 bits a block of NaNs, in a tree slot and in a prefix
    slot that leaves some rows' window; K: a NaN."""
    a = attn_inputs(1, R, H, 1, dh, [prefix], BF, kv4, dev, seed=9)
    slots = [prefix + 4] + ([prefix - 1] if prefix else [])
    a["mask"][0, 6] &= ~(1 << 4)
    for j, s in enumerate(slots):
        if kv4:
            a["vc"][0][s, dh // 2 + j] = 0x7f
            a["vs"][0][s, 0, 16 * j:16 * j + 16] = math.nan
        else:
            a["vc"][0][s, 0, 3 + j] = -math.inf
            a["vs"][0][s, 0, 3 + j] = -math.inf
    window = 2
    see = ref.visible(prefix, R, a["mask"][0], a["depth"][0], window, 0)
    assert see[:, slots].any() and not see[:, slots].all(0).any()
    check_attn(call_attn(a, window, 0, 1, kv4, dev), a, window, 0, kv4=kv4)
    if kv4:
        a["kc"][0][prefix + 4, dh // 2] = 0x7f
    else:
        a["kc"][0][prefix + 4, 0, 0] = math.nan
    got = call_attn(a, window, 0, 1, kv4, dev)
    hit = torch.from_numpy(see[:, prefix + 4]).to(dev)
    assert torch.isnan(got[0, hit]).all()
    unseen = torch.from_numpy(~see[:, slots].any(1)).to(dev)
    assert unseen.any() and torch.isfinite(got[0, unseen]).all()


@pytest.mark.parametrize("kv4", [False, True])
@pytest.mark.parametrize("R", [1, 9, 17])
def test_rows_that_see_nothing_and_stale_slots(dev, kv4, R):
    """A padded batch: sequence 1 has one row, the slots behind it hold NaNs."""
    a = attn_inputs(2, R, 2, 2, 64, [90, 40], BF, kv4, dev, seed=5)
    a["mask"][1, 1:] = 0
    for b, first in ((0, 90 + R), (1, 41)):
        for c in (a["kc"][b], a["vc"][b]):
            c[first:] = 0x7f if kv4 else math.nan
        for v in (a["ks"][b], a["vs"][b]):
            v[first:] = math.nan
    got = call_attn(a, 0, 0, 2, kv4, dev)
    check_attn(got, a, 0, 0, kv4=kv4)
    assert torch.isfinite(got).all()
    a["prefix"] = [0, 0]
    a["mask"][:] = 0
    assert not call_attn(a, 0, 0, 2, kv4, dev).any()


@pytest.mark.parametrize("kv4", [False, True])
@pytest.mark.parametrize("R", [1, 5, 17])
def test_bad_sequences_among_long_ones(dev, kv4, R):
    """Several ranges a sequence: a bad one gives zeros and its status, the others
    what they give without it (their ranges may differ, so within two tolerances)."""
    a = attn_inputs(3, R, 2, 2, 64, [3000, 2000, 700], BF, kv4, dev, seed=1, slack=0)
    good = call_attn(a, 0, 0, 2, kv4, dev)
    check_attn(good, a, 0, 0, kv4=kv4)
    kp, vp = m.cache_pointers(a["kc"], dev), m.cache_pointers(a["vc"], dev)
    fn = m.tree_attention_kv4 if kv4 else m.tree_attention_window
    q, mask = a["q"].to(dev), a["mask"].to(dev)
    for bad, name in ((3001, "bad prefix"), (-1, "bad prefix"), (None, "bad cache")):
        ws = m.new_workspace(1 << 24)
        P = torch.tensor([3000, 2000 if bad is None else bad, 700], dtype=torch.int32, device=dev)
        holes = kp.clone()
        if bad is None:
            holes[1] = 0
        got = fn(q, holes, vp, P, 3000, mask, 2, ws=ws)
        assert status(ws) == name and not got[1].any()
        keep = [0, 2]
        sub = {k: ([v[b] for b in keep] if isinstance(v, list) else v) for k, v in a.items()}
        sub.update(q=a["q"][keep], mask=a["mask"][keep], depth=a["depth"][keep])
        check_attn(got[keep], sub, 0, 0, kv4=kv4)


@pytest.mark.parametrize("kv4", [False, True])
@pytest.mark.parametrize("window", [0, 500])
def test_single_tokens_on_a_side_stream_replayed_and_repeated(dev, kv4, window):
    a = attn_inputs(3, 1, 8, 2, 128, [2000, 30, 900], BF, kv4, dev, seed=6)
    eager = call_attn(a, window, 3 if window else 0, 2, kv4, dev)
    q, kp, vp = a["q"].to(dev), m.cache_pointers(a["kc"], dev), m.cache_pointers(a["vc"], dev)
    P = torch.tensor(a["prefix"], dtype=torch.int32, device=dev)
    mask, depth = a["mask"].to(dev), a["depth"].to(dev)
    fn = m.tree_attention_kv4 if kv4 else m.tree_attention_window

    def call(**kw):
        return fn(q, kp, vp, P, a["P_max"], mask, 2, depth=depth if window else None, window=window,
                  sinks=3 if window else 0, **kw)

    for _ in range(3):
        assert torch.equal(call(), eager)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    out = call(stream=side)
    side.synchronize()
    assert torch.equal(out, eager)
    ws = m.new_workspace(1 << 24)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = call(ws=ws)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, eager)
    # lengths are read when the graph runs
    P.copy_(torch.tensor([100, 1500, 0], dtype=torch.int32))
    a["prefix"] = [100, 900, 0]
    P.copy_(torch.tensor(a["prefix"], dtype=torch.int32))
    g.replay()
    torch.cuda.synchronize()
    check_attn(out, a, window, 3 if window else 0, kv4=kv4)
