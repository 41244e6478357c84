"""The cache operators where two stages, two streams or the ends of a type meet,
against a 64-bit reference with the tolerances of test_gpu_cache_ops."""
import math

import numpy as np
import pytest
import torch

import cache_ops_ref as ref
import medusa_speculative_decoding_02_gb300 as m
from test_gpu_cache_ops import (BF, attn_inputs, call_attn, check_attn, check_rope, dev, inv_freqs, np64, randn,  # noqa: F401
                                status)

pytestmark = pytest.mark.gpu


def pack_mask(bits):
    """bool [B,R,R] as the words of anc_mask, int64 [B,R,W]."""
    B, R = bits.shape[:2]
    full = np.zeros((B, R, (R + 63) // 64 * 64), bool)
    full[..., :R] = bits
    return torch.from_numpy(np.packbits(full, axis=-1, bitorder="little").view(np.int64))


@pytest.mark.parametrize("kv4", [False, True])
@pytest.mark.parametrize("dh", [64, 128])
@pytest.mark.parametrize("R,G,prefix", [(32, 1, 50), (24, 1, 45), (129, 1, 0), (200, 1, 40), (256, 1, 0),
                                        (65, 4, 40), (150, 2, 17)])
def test_infinities_in_adjacent_stages(dev, kv4, dh, R, G, prefix):
    """Whole V rows that are not finite in several adjacent stages of 64 keys, all
    partly visible: even rows see the first stage's, odd rows a single one of the
    second or the third (or none).  More than 16 rows a KV head and at most six
    stages: one CTA works through all of them."""
    B, Hkv = 2, 4
    a = attn_inputs(B, R, G * Hkv, Hkv, dh, [prefix] * B, BF, kv4, dev, seed=R + prefix, slack=0)
    rs = np.random.RandomState(R)
    stage = (prefix + np.arange(R)) // 64
    stages = sorted(set(stage))
    assert len(stages) >= 2
    first = np.flatnonzero(stage == stages[0])[:32]
    single = [np.flatnonzero(stage == s)[-1] for s in stages[1:3]]
    bits = rs.rand(B, R, R) < 0.3
    bits[:, :, first] = False
    bits[:, :, single] = False
    bits[:, 0::2, first[0]] = True
    for i, t in enumerate(single):
        bits[:, 1 + 2 * i::2 * (len(single) + 1), t] = True
    a["mask"] = pack_mask(bits)
    for b in range(B):
        for t in [*first, *single]:
            s, value = prefix + int(t), math.nan if kv4 or t in first else -math.inf
            if kv4:
                a["vc"][b][s, Hkv * dh // 2:Hkv * dh // 2 + Hkv * dh // 16] = 0x7f
            else:
                a["vc"][b][s] = value
            a["vs"][b][s] = value
    ws = m.new_workspace(m.tree_attention_window_workspace_size(m.BF16, B, R, G * Hkv, Hkv, dh, prefix,
                                                                kv4=kv4))
    assert ws.numel() == m.WS_HEADER  # a single range
    got = call_attn(a, 0, 0, Hkv, kv4, dev, ws=ws)
    check_attn(got, a, 0, 0, kv4=kv4)
    plain = torch.from_numpy(~bits[:, :, [*first, *single]].any(2)).to(dev)
    assert plain.any() and torch.isfinite(got[plain]).all()
    for _ in range(30):
        again = call_attn(a, 0, 0, Hkv, kv4, dev, ws=ws)
        assert torch.equal(torch.nan_to_num(again, 7.0, 8.0, 9.0), torch.nan_to_num(got, 7.0, 8.0, 9.0))


@pytest.mark.parametrize("dtype", [BF, torch.float32])
@pytest.mark.parametrize("dh", [64, 128])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("R", [20, 3000])
def test_norms_over_the_stated_range(dev, dtype, dh, inter, R):
    """Rows of every magnitude that the header allows: with eps 0 from 2^-60 to 2^60,
    with an eps every smaller one as well; infinities and NaNs stay in their vector."""
    g = torch.Generator().manual_seed(dh)
    for eps, least in ((0.0, -57), (1e-30, -110), (1e-6, -110)):
        size = torch.linspace(least, 57, R).round()
        q = randn(g, 1, R, 3, dh).double() * torch.exp2(size.double())[None, :, None, None]
        q[0, :, 1] = randn(g, R, dh)  # an ordinary vector beside
        q[0, 9, 2] = 0
        q[0, 9, 2, 5] = 2.0 ** 60
        q = q.to(dtype)
        pos, f = torch.arange(R, dtype=torch.int32)[None], inv_freqs(dh)
        w = (1 + 0.3 * randn(g, dh)).to(dtype)
        qo, ko = m.qk_norm_rope(q.to(dev), q.to(dev), pos.to(dev), f.to(dev), q_weight=w.to(dev), eps=eps,
                                interleaved=inter)
        check_rope(qo, q, pos, f, w, eps, True, inter)
        check_rope(ko, q, pos, f, None, eps, True, inter)
    bad = q.clone()
    bad[0, 8, 0, 1], bad[0, 8, 2, 3] = math.inf, math.nan
    got, _ = m.qk_norm_rope(bad.to(dev), q.to(dev), pos.to(dev), f.to(dev), q_weight=w.to(dev), eps=eps,
                            interleaved=inter)
    assert torch.isnan(got[0, 8, 0, 1]) and torch.isnan(got[0, 8, 2]).all()
    rest = torch.ones(1, R, 3, dtype=torch.bool, device=dev)
    rest[0, 8, 0] = rest[0, 8, 2] = False
    assert torch.equal(got[rest], qo[rest])


@pytest.mark.parametrize("dtype", [BF, torch.float32])
@pytest.mark.parametrize("kv4", [False, True])
@pytest.mark.parametrize("R", [3, 20])
def test_bad_depth_is_reported_behind_every_window(dev, dtype, kv4, R):
    """A window that no slot falls out of does not use the depths, and reports a bad
    one all the same; without a window they are not looked at."""
    a = attn_inputs(2, R, 2, 1, 64, [30, 20], dtype, kv4, dev, seed=3)
    want = call_attn(a, 0, 0, 1, kv4, dev)
    fn = m.tree_attention_kv4 if kv4 else m.tree_attention_window
    args = (a["q"].to(dev), m.cache_pointers(a["kc"], dev), m.cache_pointers(a["vc"], dev),
            torch.tensor(a["prefix"], dtype=torch.int32, device=dev), a["P_max"], a["mask"].to(dev), 1)
    for bad in (-1, R):
        depth = a["depth"].clone()
        depth[1, R - 1] = bad
        for window, word in ((0, "ok"), (a["P_max"] + R, "bad depth"), (2 ** 31 - 1, "bad depth")):
            ws = m.new_workspace(1 << 22)
            got = fn(*args, depth=depth.to(dev), window=window, ws=ws)
            assert status(ws) == word, window
            assert torch.equal(got, want)


@pytest.mark.parametrize("dtype", [BF, torch.float32])
def test_4bit_rows_up_to_the_largest_call(dev, dtype):
    """65535 rows, and a ragged sequence beside: every slot is written and read."""
    B, R, Hkv, dh = 2, 65535, 1, 64
    g = torch.Generator().manual_seed(1)
    k, v = randn(g, B, R, Hkv, dh, dtype=dtype, std=3.0), randn(g, B, R, Hkv, dh, dtype=dtype)
    rows = [R, 65000]
    kc = [torch.zeros(R, m.kv4_row_bytes(Hkv, dh), dtype=torch.uint8, device=dev) for _ in range(B)]
    vc = [c.clone() for c in kc]
    kp, vp = m.cache_pointers(kc, dev), m.cache_pointers(vc, dev)
    P = torch.zeros(B, dtype=torch.int32, device=dev)
    n = torch.tensor(rows, dtype=torch.int32, device=dev)
    m.kv4_append(k.to(dev), v.to(dev), kp, vp, P, 0, n_rows=n)
    ko, vo = m.kv4_unpack(kp, vp, P, 0, R, Hkv, dh, dtype=dtype, n_rows=n)
    used = Hkv * dh // 2 + Hkv * dh // 16
    for b, r in enumerate(rows):
        for x, c, y in ((k, kc, ko), (v, vc, vo)):
            want = ref.pack_rows(np64(x)[b, :r])
            assert (c[b].cpu().numpy()[:r, :used] == want[:, :used]).all() and not c[b][r:].any()
            assert (np64(y)[b, :r] == ref.unpack_rows(want, Hkv, dh)).all()


def test_commit_of_4bit_rows_leaves_bad_sequences_alone(dev):
    """A negative prefix, a missing or unaligned cache and a path outside the tree:
    the status says so, the others are committed."""
    B, R, Hkv, dh = 3, 9, 1, 64
    g = torch.Generator().manual_seed(4)
    x = randn(g, B, R, Hkv, dh, dtype=BF).to(dev)
    base = torch.tensor([4, 2, 0], dtype=torch.int32, device=dev)
    path = torch.tensor([[0, 2, 5, 8], [0, 3, -1, -1], [0, 1, 4, -1]], dtype=torch.int32, device=dev)
    acc = torch.tensor([3, 1, 2], dtype=torch.int32, device=dev)
    for fault, word in (("prefix", "bad prefix"), ("hole", "bad cache"), ("odd", "bad cache"),
                        ("path", "bad path"), ("length", "bad path")):
        kc = [torch.zeros(4 + R, m.kv4_row_bytes(Hkv, dh), dtype=torch.uint8, device=dev) for _ in range(B)]
        vc = [c.clone() for c in kc]
        kp, vp = m.cache_pointers(kc, dev), m.cache_pointers(vc, dev)
        m.kv4_append(x, -x, kp, vp, base, 4)
        before = [c.clone() for c in kc + vc]
        P, pth, n = base.clone(), path.clone(), acc.clone()
        if fault == "prefix":
            P[1] = -1
        elif fault == "hole":
            vp[1] = 0
        elif fault == "odd":
            kp[1] += 8
        elif fault == "path":
            pth[1, 1] = R
        else:
            n[1] = 4
        ws = m.new_workspace(256)
        new = m.commit_kv4(kp, vp, P, pth, n, R, Hkv, dh, ws=ws)
        assert status(ws) == word, fault
        assert new.tolist() == [8, int(P[1]), 3]
        for c, old in zip(kc + vc, before):
            b = [i for i in range(B) if c is kc[i] or c is vc[i]][0]
            p, L = int(base[b]), int(acc[b])
            if b == 1:
                assert torch.equal(c, old)
            else:
                for q in range(L + 1):
                    assert torch.equal(c[p + q], old[p + int(path[b, q])])


@pytest.mark.parametrize("dtype", [BF, torch.float32])
@pytest.mark.parametrize("kv4", [False, True])
@pytest.mark.parametrize("R,prefix", [(6, 100), (6, 3000), (30, 100), (30, 3000)])
def test_queries_that_are_not_finite_stay_in_their_rows(dev, dtype, kv4, R, prefix):
    a = attn_inputs(1, R, 2, 1, 64, [prefix], dtype, kv4, dev, seed=7)
    a["q"][0, 1, 0, 3], a["q"][0, 3, 1, 0], a["q"][0, 4, 0] = math.inf, math.nan, -math.inf
    for window, sinks in ((0, 0), (40, 3)):
        got = call_attn(a, window, sinks, 1, kv4, dev)
        check_attn(got, a, window, sinks, kv4=kv4)
        for r, h in ((1, 0), (3, 1), (4, 0)):
            assert not torch.isfinite(got[0, r, h]).any()
            assert torch.isfinite(got[0, r, 1 - h]).all()
        assert torch.isfinite(got[0, [0, 2, 5]]).all()


@pytest.mark.parametrize("kv4", [False, True])
@pytest.mark.parametrize("R", [1, 17])
def test_calls_at_the_same_time_on_two_streams(dev, kv4, R):
    """Each stream with a workspace of its own, the caches shared; and calls whose
    workspace and outputs are made by the call and dropped at once."""
    a = attn_inputs(4, R, 8, 2, 128, [3000, 100, 0, 1700], BF, kv4, dev, seed=R)
    fn = m.tree_attention_kv4 if kv4 else m.tree_attention_window
    kp, vp = m.cache_pointers(a["kc"], dev), m.cache_pointers(a["vc"], dev)
    P = torch.tensor(a["prefix"], dtype=torch.int32, device=dev)
    mask, depth = a["mask"].to(dev), a["depth"].to(dev)
    qs = [a["q"].to(dev), (a["q"] * -0.5).to(dev)]
    kinds = ((0, 0), (700, 9))

    def call(i, stream=None, ws=None):
        window, sinks = kinds[i]
        return fn(qs[i], kp, vp, P, a["P_max"], mask, 2, depth=depth, window=window, sinks=sinks, ws=ws,
                  stream=stream)

    want = [call(0), call(1)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    spaces = [m.new_workspace(1 << 26) for _ in range(2)]
    torch.cuda.synchronize()
    outs = []
    for n in range(40):
        for i in range(2):
            call(i, streams[i])  # dropped: its memory goes to the next call of this stream
            outs.append((i, call(i, streams[i], spaces[i])))
    torch.cuda.synchronize()
    for i, got in outs:
        assert torch.equal(got, want[i])
    assert [status(ws) for ws in spaces] == ["ok", "ok"]
