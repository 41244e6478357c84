"""The cache operators at the sizes where their kernels change, against a 64-bit
reference with the tolerances of test_gpu_cache_ops: attention by the rows a
KV head has (up to 8, up to 16, more), rotation of many rows, 4-bit rows of every
size of element."""
import math

import numpy as np
import pytest
import torch

import cache_ops_ref as ref
import medusa_speculative_decoding_02_gb300 as m
from test_gpu_cache_ops import (BF, attn_inputs, call_attn, check_attn, check_rope, dev, inv_freqs, np64,  # noqa: F401
                                randn, status)

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


# Enough rows that a CTA takes several of them, numbers of rows that do not fill
# the last CTA, vectors that fill one group of passes, more, and a part.
@pytest.mark.parametrize("dtype", [BF, torch.float32])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("B,R,H,Hkv,dh,rot,rows", [
    (2, 1303, 3, 1, 64, 64, [1303, 1102]), (3, 822, 3, 1, 128, 32, [821, 1, 0]),
    (1, 701, 40, 5, 128, 96, [698]), (1, 2500, 1, 1, 64, 0, [2500])])
def test_rotation_of_many_rows(dev, dtype, inter, B, R, H, Hkv, dh, rot, rows):
    """Slices of a projection, ragged, with norms: to dense outputs, in place, and
    with K and V into their slots; rows past a sequence's stay as they were."""
    g = torch.Generator().manual_seed(R)
    qkv = randn(g, B, R, H + 2 * Hkv, dh, dtype=dtype)
    q, k, v = qkv[:, :, :H], qkv[:, :, H:H + Hkv], qkv[:, :, H + Hkv:]
    qw, kw = (1 + 0.3 * randn(g, dh)).to(dtype), (1 + 0.3 * randn(g, dh)).to(dtype)
    pos = torch.randint(0, 100000, (B, R), generator=g, dtype=torch.int32)
    f, x = inv_freqs(rot), qkv.to(dev)
    dq, dk, dv = x[:, :, :H], x[:, :, H:H + Hkv], x[:, :, H + Hkv:]
    kw_ = dict(q_weight=qw.to(dev), k_weight=kw.to(dev), eps=1e-5, interleaved=inter,
               n_rows=torch.tensor(rows, dtype=torch.int32, device=dev))
    out = tuple(torch.full((B, R, h, dh), 7.0, dtype=dtype, device=dev) for h in (H, Hkv))
    qo, ko = m.qk_norm_rope(dq, dk, pos.to(dev), f.to(dev), out=out, **kw_)
    check_rope(qo, q, pos, f, qw, 1e-5, True, inter, rows)
    check_rope(ko, k, pos, f, kw, 1e-5, True, inter, rows)
    prefix = [5 + 3 * b for b in range(B)]
    P = torch.tensor(prefix, dtype=torch.int32, device=dev)
    kc = [torch.full((max(prefix) + R, Hkv, dh), 3.0, dtype=dtype, device=dev) for _ in range(B)]
    vc = [c.clone() for c in kc]
    ws = m.new_workspace(256)
    q2 = m.qk_norm_rope_append(dq, dk, dv, pos.to(dev), f.to(dev), m.cache_pointers(kc, dev),
                               m.cache_pointers(vc, dev), P, max(prefix), ws=ws, **kw_)
    qd, kd = dq.contiguous(), dk.contiguous()
    m.qk_norm_rope(qd, kd, pos.to(dev), f.to(dev), out=(qd, kd), **kw_)
    for b, r in enumerate(rows):
        p = prefix[b]
        assert (qo[b, r:] == 7).all() and (ko[b, r:] == 7).all()
        assert torch.equal(q2[b, :r], qo[b, :r]) and torch.equal(kc[b][p:p + r], ko[b, :r])
        assert torch.equal(vc[b][p:p + r], dv[b, :r])
        for c in (kc[b], vc[b]):
            assert (c[:p] == 3).all() and (c[p + r:] == 3).all()
        assert torch.equal(qd[b, :r], qo[b, :r]) and torch.equal(kd[b, :r], ko[b, :r])
        assert torch.equal(qd[b, r:], dq[b, r:]) and torch.equal(kd[b, r:], dk[b, r:])
    assert status(ws) == "ok"


def test_rotation_of_many_rows_leaves_bad_sequences_alone(dev):
    B, R, H, dh = 3, 900, 2, 64
    g = torch.Generator().manual_seed(2)
    x = randn(g, B, R, H, dh, dtype=BF).to(dev)
    pos, f = torch.zeros(B, R, dtype=torch.int32, device=dev), inv_freqs(64).to(dev)
    kc = [torch.zeros(R + 9, H, dh, dtype=BF, device=dev) for _ in range(B)]
    vc = [c.clone() for c in kc]
    for P, bad, name in (([4, 10, 9], 1, "bad prefix"), ([4, -1, 9], 1, "bad prefix"), ([4, 5, 9], 2, "bad cache")):
        ws = m.new_workspace(256)
        kp = m.cache_pointers(kc, dev)
        if name == "bad cache":
            kp[bad] = 0
        for c in kc + vc:
            c.zero_()
        out = torch.full((B, R, H, dh), 7.0, dtype=BF, device=dev)
        m.qk_norm_rope_append(x, x, x, pos, f, kp, m.cache_pointers(vc, dev),
                              torch.tensor(P, dtype=torch.int32, device=dev), 9, norm=False, out=out, ws=ws)
        assert status(ws) == name and (out[bad] == 7).all() and not kc[bad].any() and not vc[bad].any()
        for b in {0, 1, 2} - {bad}:
            assert torch.equal(out[b], x[b]) and torch.equal(vc[b][P[b]:P[b] + R], x[b])


@pytest.mark.parametrize("Hkv,dh", [(1, 64), (3, 64), (5, 128), (7, 128)])
def test_4bit_rows_of_every_size_of_element(dev, Hkv, dh):
    """Blocks from the smallest to the largest bf16 magnitudes, ties and values next
    to ties, bit for bit, rows of an odd number of blocks."""
    g = torch.Generator().manual_seed(Hkv)
    R = 301
    x = randn(g, 1, R, Hkv, dh)
    x *= torch.pow(2.0, torch.randint(-20, 20, (1, R, Hkv, dh // 16), generator=g).float()).repeat_interleave(16, 3)
    k = x.to(BF)
    # the midpoints between codes times a scale, a step above and below, both signs
    s = torch.tensor([2.0 ** -6, 0.3125, 1.0, 1.875, 448.0])
    mid = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])
    row = 0
    for sc in s:
        for e in (-1, 0, 1):
            t = ((mid * sc).to(BF).view(torch.int16) + e).view(BF)
            k[0, row, 0, :16] = torch.cat([(6 * sc).to(BF)[None], t, -t, torch.tensor([-0.0], dtype=BF)])
            row += 1
    kd = k.to(dev)
    cap = [torch.zeros(R, m.kv4_row_bytes(Hkv, dh), dtype=torch.uint8, device=dev) for _ in range(2)]
    P = torch.zeros(1, dtype=torch.int32, device=dev)
    m.kv4_append(kd, -kd, m.cache_pointers(cap[:1], dev), m.cache_pointers(cap[1:], dev), P, 0,
                 ws=m.new_workspace(256))
    used = Hkv * dh * 9 // 16
    for c, y in zip(cap, (k, -k)):
        assert (c.cpu().numpy()[:, :used] == ref.pack_rows(np64(y)[0])[:, :used]).all()


@pytest.mark.parametrize("kv4", [False, True])
@pytest.mark.parametrize("R", [1, 17])
def test_slots_past_four_gigabytes(dev, kv4, R):
    """Rows written and read behind byte 2^32 of a cache: what the same calls give
    in a small one (a window without sinks only sees differences of positions)."""
    B, H, dh, window, near = 1, 256, 128, 100, 150
    row = m.kv4_row_bytes(H, dh) if kv4 else H * dh * 2
    P = 2 ** 32 // row + 300
    g = torch.Generator().manual_seed(R)
    q = randn(g, B, R, H, dh, dtype=BF).to(dev)
    k, v = (randn(g, B, near + R, H, dh, dtype=BF).to(dev) for _ in range(2))
    mask, depth = ref.tree(B, R, np.random.RandomState(R))
    outs, stored = [], []
    for prefix in (near, P):
        slots = prefix + near + R
        c = [m.kv4_cache(slots, H, dh, device=dev) if kv4
             else torch.zeros(slots, H, dh, dtype=BF, device=dev) for _ in range(2)]
        kp, vp = m.cache_pointers(c[:1], dev), m.cache_pointers(c[1:], dev)
        start = torch.tensor([prefix - near], dtype=torch.int32, device=dev)
        n = torch.tensor([prefix], dtype=torch.int32, device=dev)
        if kv4:
            m.kv4_append(k, v, kp, vp, start, prefix)
            back = m.kv4_unpack(kp, vp, start, prefix, near + R, H, dh)
        else:
            m.qk_norm_rope_append(k, k, v, torch.zeros(B, near + R, dtype=torch.int32, device=dev),
                                  inv_freqs(dh).to(dev), kp, vp, start, prefix, norm=False)
            back = (c[0][prefix - near:prefix + R][None], c[1][prefix - near:prefix + R][None])
        fn = m.tree_attention_kv4 if kv4 else m.tree_attention_window
        outs.append(fn(q, kp, vp, n, prefix, mask.to(dev), H, depth=depth.to(dev), window=window))
        stored.append([x.clone() for x in back])
        assert prefix == near or (prefix - near) * row > 2 ** 32
        del c, back
    assert torch.equal(outs[0], outs[1]) and outs[0].any() and torch.isfinite(outs[0]).all()
    for x, y in zip(*stored):
        assert torch.equal(x, y) and x.any()
    torch.cuda.empty_cache()
