"""Rotation, 4-bit cache and windowed tree attention on the GPU, against the
64-bit references of cache_ops_ref.

Tolerances, elementwise, derived from the arithmetic (u = half a step of the
output type: bf16 2^-8, fp32 2^-24):
  * rotation: y = a cos t -+ b sin t from fp32 a, b, cos, sin.  Norm: the
    mean of dh squares loses at most (dh/8 + 4 + 3) roundings (eight terms in
    a chain, then a shuffle tree), halved by the square root, plus division
    and two products; cos and sin are off by 2 steps plus the angle's own
    2 pi 2^-25; two products and a sum.  24 * 2^-24 * (|a| + |b|) covers
    them all; then u |y| for the rounding to the output type.
  * 4-bit rows: bit-exact.
  * attention: a score's fp32 dot product of dh terms is off by at most
    (dh + 8) 2^-24 E, E = scale * sum |q k| (the + 8: scaling, the subtraction
    of the maximum and the conversion to base 2, whose own size is at most
    2 E); weights are thus off by a relative 2 (dh + 8) 2^-24 E and by the
    exponential's 2^-21.  The weights of the matrix product are rounded to
    bf16 or fp16, at most u_p = 2^-8 (none on fp32 paths), and sums of N
    terms lose N 2^-24 at the worst.  A = sum w |v| / sum w carries all of
    this: |error| <= A (u_p + 4 (dh + 8) 2^-24 E + 2^-20 + 2 N 2^-24) + u |y|,
    and weights under 2^-126 of a row's largest are lost altogether: at most
    N 2^-126 max |v| < 1e-30 more.  bf16 queries over a 4-bit cache round
    their weights to fp16 with the row's reference at 2^7: half of fp16's
    smallest step, 2^-25, is 2^-32 of a reference that the sum reaches at
    least, so each key may lose 2^-32 |v| on top: N 2^-32 max |v|.
"""
import math

import numpy as np
import pytest
import torch

import cache_ops_ref as ref
import medusa_speculative_decoding_02_gb300 as m
from medusa_speculative_decoding_02_gb300 import build as mbuild

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def dev():
    mbuild.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    d = torch.device("cuda:0")
    torch.cuda.set_device(d)
    return d


def half_step(dt):
    return torch.finfo(dt).eps / 2


def randn(g, *shape, std=1.0, dtype=F32):
    return (torch.randn(shape, generator=g) * std).to(dtype)


def np64(t):
    return t.detach().double().cpu().numpy()


def status(ws):
    return m.DEVICE_STATUS[m.read_device_status(ws)]


# ---------------------------------------------------------------- rotation ---

def check_rope(got, x, pos, inv_freq, w, eps, norm, inter, rows=None):
    y, mag = ref.rope(np64(x), pos.cpu().numpy(), np64(inv_freq), None if w is None else np64(w), eps,
                      norm, inter)
    tol = 24 * 2.0 ** -24 * mag + half_step(x.dtype) * np.abs(y) * 1.01 + 1e-37
    err = np.abs(np64(got) - y)
    if rows is not None:
        for b, n in enumerate(rows):
            assert (err[b, :n] <= tol[b, :n]).all(), (b, (err[b, :n] / tol[b, :n]).max())
    else:
        assert (err <= tol).all(), (err / tol).max()


def inv_freqs(rot, base=10000.0):
    return torch.pow(torch.tensor(base, dtype=torch.float64),
                     -torch.arange(0, rot, 2).double() / max(rot, 1)).float()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("B,R,H,Hkv,dh,rot", [
    (1, 1, 1, 1, 64, 64), (1, 1, 32, 32, 128, 128), (8, 1, 32, 8, 128, 128), (1, 65, 32, 32, 128, 128),
    (3, 7, 6, 3, 64, 32), (2, 129, 5, 1, 128, 16), (2, 5, 4, 2, 128, 0), (1, 300, 40, 40, 128, 96),
    (5, 3, 28, 4, 64, 48)])
@pytest.mark.parametrize("norm,inter", [(True, False), (False, True), (False, False), (True, True)])
def test_rope(dev, dtype, B, R, H, Hkv, dh, rot, norm, inter):
    g = torch.Generator().manual_seed(B * 1000 + R * 10 + H + rot)
    q, k = randn(g, B, R, H, dh, dtype=dtype, std=2.0), randn(g, B, R, Hkv, dh, dtype=dtype)
    qw, kw = (1 + 0.3 * randn(g, dh)).to(dtype), (1 + 0.3 * randn(g, dh)).to(dtype)
    pos = torch.randint(0, 5000, (B, R), generator=g, dtype=torch.int32)
    f = inv_freqs(rot)
    kwargs = dict(q_weight=qw.to(dev), k_weight=kw.to(dev), eps=1e-5) if norm else {}
    qo, ko = m.qk_norm_rope(q.to(dev), k.to(dev), pos.to(dev), f.to(dev), norm=norm, interleaved=inter,
                            **kwargs)
    check_rope(qo, q, pos, f, qw, 1e-5, norm, inter)
    check_rope(ko, k, pos, f, kw, 1e-5, norm, inter)


@pytest.mark.parametrize("inter", [False, True])
def test_rope_far_and_negative_positions(dev, inter):
    """Angles of 10^5 and of 2^31 turns keep their fraction."""
    g = torch.Generator().manual_seed(3)
    q = randn(g, 1, 6, 2, 128)
    pos = torch.tensor([[0, -1, 1 << 20, 10 ** 9, 2 ** 31 - 1, -2 ** 31]], dtype=torch.int32)
    f = inv_freqs(128)
    qo, ko = m.qk_norm_rope(q.to(dev), q.to(dev), pos.to(dev), f.to(dev), norm=False, interleaved=inter)
    check_rope(qo, q, pos, f, None, 0, False, inter)
    assert torch.equal(qo, ko)


def test_rope_norm_without_weights_zero_and_large_rows(dev):
    q = torch.zeros(1, 3, 2, 64)
    q[0, 1] = 1e15
    q[0, 2, :, 0] = 1e-15
    pos, f = torch.tensor([[5, 6, 7]], dtype=torch.int32), inv_freqs(64)
    qo, _ = m.qk_norm_rope(q.to(dev), q.to(dev), pos.to(dev), f.to(dev), eps=1e-6)
    check_rope(qo, q, pos, f, None, 1e-6, True, False)
    # a row of zeros with eps 0 has no norm: NaN, as the formula gives
    qo, _ = m.qk_norm_rope(q.to(dev), q.to(dev), pos.to(dev), f.to(dev), eps=0.0)
    assert torch.isnan(qo[0, 0]).all() and torch.isfinite(qo[0, 1]).all()


def test_rope_unrotated_elements_pass_through(dev):
    """Elements from rot on are copied, infinities and NaNs too, and change no other."""
    g = torch.Generator().manual_seed(4)
    for inter in (False, True):
        q = randn(g, 1, 2, 1, 128, dtype=BF)
        q[..., 40], q[..., 41], q[..., 90] = math.inf, math.nan, -math.inf
        pos, f = torch.tensor([[3, 9]], dtype=torch.int32), inv_freqs(32)
        qo, _ = m.qk_norm_rope(q.to(dev), q.to(dev), pos.to(dev), f.to(dev), norm=False, interleaved=inter)
        # equal values, NaN where NaN (which NaN's bits is not part of the result)
        assert torch.equal(torch.nan_to_num(qo[..., 32:].cpu(), 77.0), torch.nan_to_num(q[..., 32:], 77.0))
        assert torch.isnan(qo[..., 41]).all() and torch.isfinite(qo[..., :32]).all()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_rope_slices_of_a_projection_in_place_and_ragged(dev, dtype):
    g = torch.Generator().manual_seed(7)
    B, R, H, Hkv, dh = 3, 9, 6, 2, 64
    qkv = randn(g, B, R, H + 2 * Hkv, dh, dtype=dtype).to(dev)
    q, k, v = qkv[:, :, :H], qkv[:, :, H:H + Hkv], qkv[:, :, H + Hkv:]
    pos = torch.randint(0, 999, (B, R), generator=g, dtype=torch.int32).to(dev)
    f, rows = inv_freqs(64).to(dev), [9, 0, 4]
    n = torch.tensor(rows, dtype=torch.int32, device=dev)
    out = (torch.full_like(q, 7.0, memory_format=torch.contiguous_format),
           torch.full_like(k, 7.0, memory_format=torch.contiguous_format))
    qo, ko = m.qk_norm_rope(q, k, pos, f, n_rows=n, out=out)
    check_rope(qo, q, pos, f, None, 1e-6, True, False, rows)
    check_rope(ko, k, pos, f, None, 1e-6, True, False, rows)
    for b, r in enumerate(rows):
        assert (qo[b, r:] == 7).all() and (ko[b, r:] == 7).all()
    # into caches: the rows' slots only
    P = torch.tensor([5, 0, 2], dtype=torch.int32, device=dev)
    kc = [torch.full((5 + R, Hkv, dh), 3.0, dtype=dtype, device=dev) for _ in range(B)]
    vc = [c.clone() for c in kc]
    ws = m.new_workspace(256)
    q2 = m.qk_norm_rope_append(q, k, v, pos, f, m.cache_pointers(kc, dev), m.cache_pointers(vc, dev), P, 5,
                               n_rows=n, ws=ws)
    for b, r in enumerate(rows):
        p = int(P[b])
        assert torch.equal(q2[b, :r], qo[b, :r])
        assert torch.equal(kc[b][p:p + r], ko[b, :r]) and torch.equal(vc[b][p:p + r], v[b, :r])
        for c in (kc[b], vc[b]):
            assert (c[:p] == 3).all() and (c[p + r:] == 3).all()
    # dense tensors in place
    qd, kd = q.contiguous(), k.contiguous()
    a, b = m.qk_norm_rope(qd, kd, pos, f, n_rows=n, out=(qd, kd))
    assert a is qd and torch.equal(qd[0], qo[0]) and torch.equal(kd[2, :4], ko[2, :4])
    assert torch.equal(qd[1], q[1]) and status(ws) == "ok"


def test_rope_append_bad_sequences_are_left_alone(dev):
    g = torch.Generator().manual_seed(8)
    q = randn(g, 3, 2, 2, 64, dtype=BF).to(dev)
    pos = torch.zeros((3, 2), dtype=torch.int32, device=dev)
    kc = [torch.zeros((6, 2, 64), dtype=BF, device=dev) for _ in range(3)]
    ptrs = m.cache_pointers(kc, dev)
    for bad, word in ((4, "bad prefix"), (-1, "bad prefix")):
        ws = m.new_workspace(256)
        P = torch.tensor([0, bad, 3], dtype=torch.int32, device=dev)
        out = torch.full_like(q, 9.0)
        m.qk_norm_rope_append(q, q, q, pos, inv_freqs(64).to(dev), ptrs, ptrs, P, 3, norm=False, out=out,
                              ws=ws)
        assert status(ws) == word
        assert (out[1] == 9).all() and (kc[1] == 0).all() and torch.equal(out[0], q[0])
    ws = m.new_workspace(256)
    holes = ptrs.clone()
    holes[1] = 0
    m.qk_norm_rope_append(q, q, q, pos, inv_freqs(64).to(dev), holes, ptrs,
                          torch.zeros(3, dtype=torch.int32, device=dev), 3, ws=ws)
    assert status(ws) == "bad cache" and (kc[1] == 0).all()


# ------------------------------------------------------------- 4-bit cache ---

def caches4(B, slots, Hkv, dh, dev, fill=0):
    c = [torch.full((slots, m.kv4_row_bytes(Hkv, dh)), fill, dtype=torch.uint8, device=dev)
         for _ in range(B)]
    return c, m.cache_pointers(c, dev)


def ties(dtype):
    """Blocks of 16 whose elements sit on and next to every midpoint of the codes,
    for scales over the whole e4m3 range, and blocks whose maximum sits on and
    next to the midpoints between scales."""
    blocks = []
    u = 2.0 ** -7 if dtype == BF else 2.0 ** -23
    mids = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]
    for s in ref.E4M3[[1, 2, 3, 7, 8, 15, 16, 40, 57, 90, 113, 126]]:
        row = [6 * s] + [x * s for x in mids] + [x * s * (1 + u) for x in mids] + [0.0]
        blocks.append(row)
        blocks.append([6 * s] + [-x * s * (1 - u) for x in mids] + [-x * s for x in mids] + [-0.0])
    for a, b in zip(ref.E4M3[:126:5], ref.E4M3[1:127:5]):
        for f in (1 - u, 1.0, 1 + u):
            top = 3 * (a + b) * f
            blocks.append([top] + [top * x / 17 for x in range(1, 16)])
    return torch.tensor(blocks, dtype=torch.float64).to(dtype)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_kv4_ties_zero_and_extremes_are_exact(dev, dtype):
    x = ties(dtype)
    more = torch.zeros(6, 16, dtype=dtype)
    more[1] = 1e30            # past the largest scale
    more[2, 3] = 2.0 ** -11   # rounds to scale 0 or the smallest one
    more[3, 0] = math.inf
    more[4, 5], more[4, 6] = math.nan, 3.0
    more[5] = -448.0 * 6
    x = torch.cat([x, more])
    x = torch.cat([x, x.new_zeros((-len(x)) % 8, 16)]).reshape(1, -1, 1, 128)
    R = x.shape[1]
    (kc, kp), (vc, vp) = caches4(1, R, 1, 128, dev), caches4(1, R, 1, 128, dev)
    zero = torch.zeros(1, dtype=torch.int32, device=dev)
    m.kv4_append(x.to(dev), -x.to(dev), kp, vp, zero, 0)
    want = ref.pack_rows(np64(x)[0])
    got = kc[0].cpu().numpy()
    n = 72  # code and scale bytes
    assert (got[:, :n] == want[:, :n]).all(), np.argwhere(got[:, :n] != want[:, :n])[:5]
    want = ref.pack_rows(-np64(x)[0])
    assert (vc[0].cpu().numpy()[:, :n] == want[:, :n]).all()
    for dt in (BF, F32):
        k, v = m.kv4_unpack(kp, vp, zero, 0, R, 1, 128, dtype=dt)
        np.testing.assert_array_equal(np64(k)[0], ref.unpack_rows(got, 1, 128))
        assert torch.isnan(k).sum() == 32  # the two blocks that hold an infinity and a NaN


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("B,R,Hkv,dh,P", [(1, 1, 1, 64, 0), (1, 65, 32, 128, 100), (3, 7, 3, 64, 5),
                                          (2, 130, 5, 128, 33), (1, 2, 40, 128, 1)])
def test_kv4_rows(dev, dtype, B, R, Hkv, dh, P):
    g = torch.Generator().manual_seed(R + Hkv)
    wide = randn(g, B, R, 2 * Hkv, dh, dtype=dtype, std=3.0).to(dev)
    wide[..., ::17] *= 30
    k, v = wide[:, :, :Hkv], wide[:, :, Hkv:]
    prefix = [max(0, P - 2 * b) for b in range(B)]
    rows = [R if b == 0 else R // (b + 1) for b in range(B)]
    pl = torch.tensor(prefix, dtype=torch.int32, device=dev)
    n = torch.tensor(rows, dtype=torch.int32, device=dev)
    (kc, kp), (vc, vp) = caches4(B, P + R, Hkv, dh, dev, 0xA5), caches4(B, P + R, Hkv, dh, dev, 0x5A)
    ws = m.new_workspace(256)
    m.kv4_append(k, v, kp, vp, pl, P, n_rows=n, ws=ws)
    used = Hkv * dh // 2 + Hkv * dh // 16
    out = (torch.full((B, R, Hkv, dh), 5.0, dtype=dtype, device=dev),
           torch.full((B, R, Hkv, dh), 5.0, dtype=dtype, device=dev))
    ko, vo = m.kv4_unpack(kp, vp, pl, P, R, Hkv, dh, n_rows=n, out=out, ws=ws)
    for b in range(B):
        p, r = prefix[b], rows[b]
        for x, c, fill, y in ((k, kc, 0xA5, ko), (v, vc, 0x5A, vo)):
            want = ref.pack_rows(np64(x)[b, :r])
            got = c[b].cpu().numpy()
            assert (got[p:p + r, :used] == want[:, :used]).all()
            assert (got[:p] == fill).all() and (got[p + r:] == fill).all() and (got[:, used:] == fill).all()
            np.testing.assert_array_equal(np64(y)[b, :r], ref.unpack_rows(want, Hkv, dh))
            assert (y[b, r:] == 5).all()
    assert status(ws) == "ok"


def test_kv4_bad_sequences(dev):
    (kc, kp), (vc, vp) = caches4(2, 4, 1, 64, dev), caches4(2, 4, 1, 64, dev)
    x = torch.ones((2, 2, 1, 64), dtype=BF, device=dev)
    ws = m.new_workspace(256)
    m.kv4_append(x, x, kp, vp, torch.tensor([3, 1], dtype=torch.int32, device=dev), 2, ws=ws)
    assert status(ws) == "bad prefix" and not kc[0].any() and kc[1].any()
    ws = m.new_workspace(256)
    kp[1] += 8
    m.kv4_append(x, x, kp, vp, torch.zeros(2, dtype=torch.int32, device=dev), 2, ws=ws)
    assert status(ws) == "bad cache" and not vc[1][0].any()


def test_kv4_commit_moves_rows(dev):
    g = torch.Generator().manual_seed(5)
    B, R, Hkv, dh, K = 2, 9, 3, 64, 3
    x = randn(g, B, R, Hkv, dh, dtype=BF).to(dev)
    (kc, kp), (vc, vp) = caches4(B, 4 + R, Hkv, dh, dev), caches4(B, 4 + R, Hkv, dh, dev)
    pl = torch.tensor([4, 2], dtype=torch.int32, device=dev)
    m.kv4_append(x, -x, kp, vp, pl, 4)
    before = [c.clone() for c in kc]
    path = torch.tensor([[0, 2, 5, 8], [0, 3, -1, -1]], dtype=torch.int32, device=dev)
    acc = torch.tensor([3, 1], dtype=torch.int32, device=dev)
    new = m.commit_kv4(kp, vp, pl, path, acc, R, Hkv, dh)
    assert new.tolist() == [8, 4]
    for b, (p, nodes) in enumerate([(4, [0, 2, 5, 8]), (2, [0, 3])]):
        for q, node in enumerate(nodes):
            assert torch.equal(kc[b][p + q], before[b][p + node])


# --------------------------------------------------------------- attention ---

def attn_inputs(B, R, H, Hkv, dh, prefix, dtype, kv4, dev, seed=0, std=1.5, slack=3):
    g = torch.Generator().manual_seed(seed)
    rs = np.random.RandomState(seed)
    q = randn(g, B, R, H, dh, std=std, dtype=dtype)
    mask, depth = ref.tree(B, R, rs)
    P_max = max(prefix) + slack
    ks, vs, kc, vc = [], [], [], []
    for b in range(B):
        for vals, cache in ((ks, kc), (vs, vc)):
            x = randn(g, P_max + R, Hkv, dh, dtype=dtype)
            if kv4:
                rows = ref.pack_rows(np64(x))
                cache.append(torch.from_numpy(rows).to(dev))
                vals.append(torch.from_numpy(ref.unpack_rows(rows, Hkv, dh)))
            else:
                cache.append(x.to(dev))
                vals.append(x.double())
    return dict(q=q, mask=mask, depth=depth, P_max=P_max, ks=ks, vs=vs, kc=kc, vc=vc, prefix=prefix)


def call_attn(a, window, sinks, Hkv, kv4, dev, **kw):
    fn = m.tree_attention_kv4 if kv4 else m.tree_attention_window
    return fn(a["q"].to(dev), m.cache_pointers(a["kc"], dev), m.cache_pointers(a["vc"], dev),
              torch.tensor(a["prefix"], dtype=torch.int32, device=dev), a["P_max"], a["mask"].to(dev), Hkv,
              depth=a["depth"].to(dev) if window else None, window=window, sinks=sinks, **kw)


def check_attn(got, a, window, sinks, scale=None, rows=slice(None), kv4=False):
    dh, dt = a["q"].shape[3], a["q"].dtype
    y, A, E = ref.attention(a["q"], a["ks"], a["vs"], a["prefix"], a["mask"], a["depth"], window, sinks,
                            1 / math.sqrt(dh) if scale is None else scale)
    n = max(a["prefix"]) + a["q"].shape[1]
    up = 2.0 ** -8 if dt == BF else 0.0
    rel = up + 4 * (dh + 8) * 2.0 ** -24 * E[..., None] + 2.0 ** -20 + 2 * n * 2.0 ** -24
    lost = 1e-30
    if kv4 and dt == BF:
        lost = n * 2.0 ** -32 * max(float(torch.nan_to_num(v).abs().max()) for v in a["vs"])
    tol = (A * rel + half_step(dt) * 1.01 * y.abs() + lost)[:, rows]
    got, y = got.double().cpu()[:, rows], y[:, rows]
    nan = torch.isnan(y)
    assert torch.equal(torch.isnan(got), nan)
    inf = torch.isinf(y)
    assert torch.equal(got[inf], y[inf]) and torch.equal(torch.isinf(got), inf)
    err = (got - y).abs()
    ok = (err <= tol) | nan | inf
    assert ok.all(), (err / tol)[~ok].max()


SHAPES = [
    # B, R, H, Hkv, dh, prefix
    (1, 1, 1, 1, 64, [0]), (1, 1, 4, 1, 128, [63]), (2, 15, 4, 2, 64, [37, 0]),
    (1, 65, 2, 2, 128, [200]), (3, 17, 6, 3, 128, [129, 64, 1]), (1, 129, 2, 1, 128, [70]),
    (1, 256, 1, 1, 64, [5]), (2, 64, 2, 2, 64, [64, 128]), (1, 130, 3, 1, 128, [300]),
    (2, 1, 8, 2, 128, [1000, 511]),
]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("kv4", [False, True])
@pytest.mark.parametrize("B,R,H,Hkv,dh,prefix", SHAPES)
@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (2, 3), (50, 4), (64, 100), (5000, 7)])
def test_attention(dev, dtype, kv4, B, R, H, Hkv, dh, prefix, window, sinks):
    a = attn_inputs(B, R, H, Hkv, dh, prefix, dtype, kv4, dev, seed=R + dh)
    ws = m.new_workspace(m.tree_attention_window_workspace_size(
        m.BF16 if dtype == BF else m.F32, B, R, H, Hkv, dh, a["P_max"], window, sinks, kv4))
    check_attn(call_attn(a, window, sinks, Hkv, kv4, dev, ws=ws), a, window, sinks, kv4=kv4)
    assert status(ws) == "ok"


@pytest.mark.parametrize("kv4", [False, True])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_attention_every_length_around_a_tile(dev, dtype, kv4):
    """Prefix lengths around the key tiles, in one ragged batch; R = 2."""
    prefix = [0, 1, 29, 30, 31, 61, 62, 63, 64, 125, 126, 127, 189, 190, 191, 192]
    a = attn_inputs(len(prefix), 2, 2, 1, 128, prefix, dtype, kv4, dev, seed=2)
    for window, sinks in ((0, 0), (63, 2), (128, 0), (129, 65)):
        check_attn(call_attn(a, window, sinks, 1, kv4, dev), a, window, sinks, kv4=kv4)


@pytest.mark.parametrize("kv4", [False, True])
@pytest.mark.parametrize("B", [2, 31, 32, 33, 70])
@pytest.mark.parametrize("window,sinks", [(0, 0), (100, 7)])
def test_attention_many_ragged(dev, kv4, B, window, sinks):
    """Batches split by their real lengths (up to 32) and evenly (more): a few long
    sequences among short ones and one without a prefix."""
    prefix = [(37 * b * b) % 190 for b in range(B)]
    prefix[0], prefix[-1], prefix[B // 2] = 2500, 1700, 0
    a = attn_inputs(B, 3, 2, 2, 64, prefix, BF, kv4, dev, seed=B)
    check_attn(call_attn(a, window, sinks, 2, kv4, dev), a, window, sinks, kv4=kv4)


@pytest.mark.parametrize("kv4", [False, True])
def test_attention_long(dev, kv4):
    """Long contexts in many key ranges, peaked and flat scores, a scale of its own."""
    for std, scale in ((0.1, None), (8.0, None), (1.0, 1.0)):
        a = attn_inputs(2, 5, 4, 2, 128, [9001, 6000], BF, kv4, dev, seed=11, std=std)
        check_attn(call_attn(a, 0, 0, 2, kv4, dev, scale=scale), a, 0, 0, scale, kv4=kv4)
        check_attn(call_attn(a, 4097, 130, 2, kv4, dev, scale=scale), a, 4097, 130, scale, kv4=kv4)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("kv4", [False, True])
@pytest.mark.parametrize("R", [20, 70])
def test_attention_rows_that_see_nothing_and_stale_slots(dev, dtype, kv4, R):
    """A padded batch: sequence 1 has three rows, the others' masks are empty and
    their slots hold NaNs; slots past the tree and out of the window hold NaNs
    as well; a mask may leave out the row itself."""
    a = attn_inputs(2, R, 4, 2, 64, [90, 40], dtype, kv4, dev, seed=5)
    a["mask"][1, 3:] = 0
    a["mask"][0, 5] = 0           # still sees the prefix
    a["mask"][0, 7, 0] = 1        # the root only
    P0, P1 = a["prefix"]
    nan_at = {0: list(range(P0 + R, a["P_max"] + R)) + list(range(6, 30)),
              1: list(range(P1 + 3, a["P_max"] + R))}
    for b, slots in nan_at.items():
        for c in (a["kc"][b], a["vc"][b]):
            if kv4:
                c[slots] = 0x7f
            else:
                c[slots] = math.nan
        for v in (a["ks"][b], a["vs"][b]):
            v[slots] = math.nan
    window, sinks = 60, 5
    see = ref.visible(P0, R, a["mask"][0], a["depth"][0], window, sinks)
    assert not see[:, 6:30].any()
    got = call_attn(a, window, sinks, 2, kv4, dev)
    check_attn(got, a, window, sinks, kv4=kv4)
    assert torch.isfinite(got).all()
    # no prefix, no bit: zeros
    a["prefix"] = [0, 0]
    a["mask"][:] = 0
    assert not call_attn(a, 0, 0, 2, kv4, dev).any()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("kv4", [False, True])
@pytest.mark.parametrize("prefix", [0, 40, 150])
def test_attention_infinities_reach_only_the_rows_that_see_them(dev, dtype, kv4, prefix):
    """An infinity (4-bit: a NaN block) in V of a tree slot, and of a prefix slot
    that leaves some rows' window, changes the rows that see it, in its own
    elements, and no other row."""
    R = 33
    a = attn_inputs(1, R, 2, 1, 64, [prefix], dtype, kv4, dev, seed=9)
    slots = [prefix + 4] + ([prefix - 3] if prefix else [])
    for j, s in enumerate(slots):
        if kv4:
            a["vc"][0][s, 32 + j] = 0x7f    # one block of 16 elements
            a["vs"][0][s, 0, 16 * j:16 * j + 16] = math.nan
        else:
            a["vc"][0][s, 0, 3 + j] = -math.inf
            a["vs"][0][s, 0, 3 + j] = -math.inf
    window = 4
    see = ref.visible(prefix, R, a["mask"][0], a["depth"][0], window, 0)
    assert see[:, slots].any() and not see[:, slots].all(0).any()
    check_attn(call_attn(a, window, 0, 1, kv4, dev), a, window, 0, kv4=kv4)
    # a NaN key: rows that see it are NaN, the others as before
    k = a["ks"][0]
    if kv4:
        a["kc"][0][prefix + 4, 32] = 0x7f
        k[prefix + 4, 0, :16] = math.nan
    else:
        a["kc"][0][prefix + 4, 0, 0] = math.nan
        k[prefix + 4, 0, 0] = math.nan
    got = call_attn(a, window, 0, 1, kv4, dev)
    hit = torch.from_numpy(see[:, prefix + 4])
    assert torch.isnan(got[0, hit.to(dev)]).all()
    if not prefix:
        assert torch.isfinite(got[0, ~hit.to(dev)]).all()


@pytest.mark.parametrize("kv4", [False, True])
def test_attention_extreme_queries(dev, kv4):
    """Rows of very different size: tiny, large, zero and infinite queries."""
    a = attn_inputs(1, 6, 2, 1, 128, [100], BF, kv4, dev, seed=3)
    a["q"][0, 1] *= 1e-30
    a["q"][0, 2] *= 200.0
    a["q"][0, 3] = 0
    a["q"][0, 5, 0] *= 2.0 ** 100
    got = call_attn(a, 0, 0, 1, kv4, dev)
    check_attn(got, a, 0, 0, rows=slice(0, 5), kv4=kv4)
    assert torch.isfinite(got[0, 5]).all()


@pytest.mark.parametrize("kv4", [False, True])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_attention_bad_sequences_give_zeros(dev, kv4, dtype):
    a = attn_inputs(3, 4, 2, 2, 64, [20, 30, 10], dtype, kv4, dev, seed=1, slack=0)
    good = call_attn(a, 0, 0, 2, kv4, dev)
    fn = m.tree_attention_kv4 if kv4 else m.tree_attention_window
    q, mask, depth = a["q"].to(dev), a["mask"].to(dev), a["depth"].to(dev)
    kp, vp = m.cache_pointers(a["kc"], dev), m.cache_pointers(a["vc"], dev)
    for bad in (31, -1):
        ws = m.new_workspace(1 << 22)
        P = torch.tensor([20, bad, 10], dtype=torch.int32, device=dev)
        got = fn(q, kp, vp, P, 30, mask, 2, ws=ws)
        assert status(ws) == "bad prefix" and not got[1].any()
        assert torch.equal(got[0], good[0]) and torch.equal(got[2], good[2])
    ws = m.new_workspace(1 << 22)
    holes = vp.clone()
    holes[2] = 0
    P = torch.tensor([20, 30, 10], dtype=torch.int32, device=dev)
    got = fn(q, kp, holes, P, 30, mask, 2, ws=ws)
    assert status(ws) == "bad cache" and not got[2].any() and torch.equal(got[1], good[1])
    ws = m.new_workspace(1 << 22)
    depth[0, 2] = 4
    fn(q, kp, vp, P, 30, mask, 2, depth=depth, window=8, ws=ws)
    assert status(ws) == "bad depth"


def test_attention_agrees_with_tree_attention(dev):
    """Without a window and with as many KV heads, the existing call's result."""
    a = attn_inputs(2, 65, 4, 4, 128, [500, 90], BF, False, dev, seed=4)
    kp, vp = m.cache_pointers(a["kc"], dev), m.cache_pointers(a["vc"], dev)
    P = torch.tensor(a["prefix"], dtype=torch.int32, device=dev)
    old = m.tree_attention(a["q"].to(dev), kp, vp, P, a["P_max"], a["mask"].to(dev))
    new = call_attn(a, 0, 0, 4, False, dev)
    _, A, _ = ref.attention(a["q"], a["ks"], a["vs"], a["prefix"], a["mask"], a["depth"], 0, 0,
                            1 / math.sqrt(128))
    assert ((old.double() - new.double()).abs().cpu() <= 2.0 ** -7 * 1.1 * (A + old.abs().double().cpu())).all()


@pytest.mark.parametrize("kv4", [False, True])
def test_attention_repeats_bit_for_bit(dev, kv4):
    a = attn_inputs(2, 65, 8, 2, 128, [3000, 700], BF, kv4, dev, seed=6)
    ws = m.new_workspace(1 << 27)
    first = call_attn(a, 0, 0, 2, kv4, dev, ws=ws)
    for _ in range(5):
        assert torch.equal(call_attn(a, 0, 0, 2, kv4, dev, ws=ws), first)


@pytest.mark.parametrize("kv4", [False, True])
@pytest.mark.parametrize("prefix,window", [(0, 0), (40, 4), (3000, 0), (3000, 700)])
def test_attention_wait_timeout_leaves_the_context_usable(dev, kv4, prefix, window):
    """With no polls every bounded wait gives up at once: the status reads
    "timeout", the output is zero, and the next call is right again."""
    a = attn_inputs(1, 17, 4, 2, 128, [prefix], BF, kv4, dev, seed=8)
    ws = m.new_workspace(1 << 24)
    good = call_attn(a, window, 0, 2, kv4, dev, ws=ws)
    default = m.wait_budget()
    m.set_wait_budget(0)
    try:
        got = call_attn(a, window, 0, 2, kv4, dev, ws=ws)
        assert status(ws) == "timeout" and not got.any()
    finally:
        m.set_wait_budget(default)
    m.clear_device_status(ws)
    assert torch.equal(call_attn(a, window, 0, 2, kv4, dev, ws=ws), good) and status(ws) == "ok"


# ---------------------------------------------------- streams, graphs, run ---

def test_streams_and_graphs(dev):
    """Calls on a side stream and captured into two graphs that share one
    workspace (replayed one after the other) give the eager results."""
    a = attn_inputs(2, 17, 8, 2, 128, [700, 300], BF, True, dev, seed=12)
    q = a["q"].to(dev)
    kp, vp = m.cache_pointers(a["kc"], dev), m.cache_pointers(a["vc"], dev)
    P = torch.tensor(a["prefix"], dtype=torch.int32, device=dev)
    mask, depth = a["mask"].to(dev), a["depth"].to(dev)
    pos = (P[:, None] + depth).int().contiguous()
    f = inv_freqs(128).to(dev)
    k = torch.randn((2, 17, 2, 128), device=dev).to(BF)
    ws = m.new_workspace(1 << 25)

    def rotate(stream=None):
        return m.qk_norm_rope(q, k, pos, f, stream=stream)

    def attend(stream=None, ws=ws):
        return m.tree_attention_kv4(q, kp, vp, P, a["P_max"], mask, 2, depth=depth, window=333, sinks=4,
                                    ws=ws, stream=stream)

    eager = (*rotate(), attend())
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    on_side = (*rotate(side), attend(side, ws=None))
    side.synchronize()
    for x, y in zip(eager, on_side):
        assert torch.equal(x, y)
    graphs, outs = [], []
    for call in (rotate, attend, attend):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(call())
        graphs.append(g)
    for _ in range(3):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    for x, y in zip(eager, (*outs[0], outs[1])):
        assert torch.equal(x, y)
    assert torch.equal(outs[2], eager[2])


@pytest.mark.parametrize("kv4", [False, True])
def test_verification_pass(dev, kv4):
    """The calls in the order of a step, twice in a row: tree, rotation, rows into
    the cache, windowed attention, posterior, commit; the second step reads what
    the first committed."""
    g = torch.Generator().manual_seed(21)
    B, H, Hkv, dh, K, V, n = 2, 4, 2, 64, 3, 64, 14
    R, s, window, sinks = n + 1, (2, 2, 2), 24, 2
    P_max = 64
    prefix = [30, 11]
    kc = [randn(g, P_max + R, Hkv, dh, dtype=BF) for _ in range(B)]
    vc = [randn(g, P_max + R, Hkv, dh, dtype=BF) for _ in range(B)]
    if kv4:
        rows = [[torch.from_numpy(ref.pack_rows(np64(x))).to(dev) for x in c] for c in (kc, vc)]
        kcd, vcd = rows
        value = lambda c: torch.from_numpy(ref.unpack_rows(c.cpu().numpy(), Hkv, dh))
    else:
        kcd, vcd = [x.to(dev) for x in kc], [x.to(dev) for x in vc]
        value = lambda c: c.double().cpu()
    kp, vp = m.cache_pointers(kcd, dev), m.cache_pointers(vcd, dev)
    P = torch.tensor(prefix, dtype=torch.int32, device=dev)
    ws = m.new_workspace(1 << 22)
    f = inv_freqs(dh).to(dev)
    for step in range(2):
        logp = torch.log_softmax(randn(g, B, K, 2), -1).to(dev)
        ids = torch.randint(0, V, (B, K, 2), generator=g, dtype=torch.int32).to(dev)
        root = torch.randint(0, V, (B,), generator=g, dtype=torch.int32).to(dev)
        t = m.build_tree(root, ids, logp.contiguous(), s, n, prefix_len=P, ws=ws)
        q, k, v = (randn(g, B, R, h, dh, dtype=BF).to(dev) for h in (H, Hkv, Hkv))
        if kv4:
            qr, kr = m.qk_norm_rope(q, k, t.pos_id, f)
            m.kv4_append(kr, v, kp, vp, P, P_max, ws=ws)
            out = m.tree_attention_kv4(qr, kp, vp, P, P_max, t.anc_mask, Hkv, depth=t.depth, window=window,
                                       sinks=sinks, ws=ws)
        else:
            qr = m.qk_norm_rope_append(q, k, v, t.pos_id, f, kp, vp, P, P_max, ws=ws)
            out = m.tree_attention_window(qr, kp, vp, P, P_max, t.anc_mask, Hkv, depth=t.depth,
                                          window=window, sinks=sinks, ws=ws)
        check_rope(qr, q, t.pos_id, f, None, 1e-6, True, False)
        a = dict(q=qr.cpu(), ks=[value(c) for c in kcd], vs=[value(c) for c in vcd], prefix=P.tolist(),
                 mask=t.anc_mask.cpu(), depth=t.depth.cpu())
        check_attn(out, a, window, sinks, kv4=kv4)
        logits = randn(g, B, R, V, std=2.0)
        for b in range(B):  # plant an accepted chain of two nodes below the root
            node = 0
            for _ in range(2):
                kids = [i for i in range(R) if int(t.parent[b, i]) == node]
                if not kids:
                    break
                logits[b, node, int(t.tokens[b, kids[0]])] = 50.0
                node = kids[0]
        post = m.evaluate_posterior(logits.to(BF).to(dev), t.tokens, t.parent, t.depth, K, ws=ws)
        before = [c.clone() for c in kcd]
        if kv4:
            new = m.commit_kv4(kp, vp, P, post.path, post.accept_len, R, Hkv, dh, ws=ws)
        else:
            new = m.commit_kv(m.BF16, kp, vp, P, post.path, post.accept_len, R, Hkv, dh, ws=ws)
        for b in range(B):
            p, L = int(P[b]), int(post.accept_len[b])
            assert L >= 1 and int(new[b]) == p + L + 1
            for j in range(L + 1):
                assert torch.equal(kcd[b][p + j], before[b][p + int(post.path[b, j])])
        P = new
    assert status(ws) == "ok"
