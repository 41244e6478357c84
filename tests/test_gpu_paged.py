"""Calls on a cache in pages, on the GPU, against the 64-bit references of
paged_ref.

Tolerances, elementwise, derived from the arithmetic (u = half a step of the
output type: bf16 2^-8, fp32 2^-24).  Rows that are moved are equal bit for bit.
Attention: a score's fp32 dot product of dh terms is off by at most
(dh + 8) 2^-24 E, E = scale * sum |q k| (the + 8: scaling, the subtraction of the
maximum and the conversion to base 2, whose own size is at most 2 E); weights are
thus off by a relative 2 (dh + 8) 2^-24 E and by the exponential's 2^-21.  Weights
over a bf16 cache are rounded to bf16 for the product, at most u_p = 2^-8 (fp32: not
at all), and sums of N terms lose N 2^-24 at the worst.  A = sum w |v| / sum w carries all of
this: |error| <= A (u_p + 4 (dh + 8) 2^-24 E + 2^-20 + 2 N 2^-24) + u |y|, and weights
under 2^-126 of a row's largest are lost altogether: less than 1e-30 more.
"""
import math

import numpy as np
import pytest
import torch

import cache_ops_ref
import medusa_speculative_decoding_02_gb300 as m
import paged_ref as ref
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


def status(ws):
    return m.DEVICE_STATUS[m.read_device_status(ws)]


def same(a, b):
    return torch.equal(a.cpu().contiguous().view(torch.uint8), b.cpu().contiguous().view(torch.uint8))


def i32(*x):
    return torch.tensor(x, dtype=torch.int32)


class Case:
    """A cache in pages with B sequences: prefixes, rows, pools, page table."""

    def __init__(self, seed, prefix, rows, Hkv, dh, page, dtype, R=None, std=1.0):
        self.g = torch.Generator().manual_seed(seed)
        self.prefix, self.rows, self.page = list(prefix), list(rows), page
        self.B, self.R, self.P_max = len(prefix), R or max(rows), max(prefix)
        need = [-(-(P + n) // page) for P, n in zip(prefix, rows)]
        self.tab, self.pages = ref.table(self.g, need)
        wide = -(-(self.P_max + self.R) // page)
        if self.tab.shape[1] < wide:
            self.tab = torch.nn.functional.pad(self.tab, (0, wide - self.tab.shape[1]), value=-77)
        self.kp = ref.pool(self.g, self.pages, page, Hkv, dh, dtype, std)
        self.vp = ref.pool(self.g, self.pages, page, Hkv, dh, dtype)
        self.dtype, self.Hkv, self.dh = dtype, Hkv, dh

    def randn(self, *shape, std=1.0):
        return (torch.randn(shape, generator=self.g) * std).to(self.dtype)

    def to(self, dev):
        """(k pool, v pool, table, prefixes, P_max) on the device"""
        return (self.kp.to(dev), self.vp.to(dev), self.tab.to(dev), i32(*self.prefix).to(dev), self.P_max)


# ------------------------------------------------------------------ append ---

@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("prefix,rows,R,Hkv,dh,page", [
    ((0,), (1,), 1, 1, 64, 16), ((15,), (2,), 2, 8, 128, 16), ((1000, 0, 31), (65, 7, 33), 65, 32, 128, 64),
    ((5,) * 9, tuple(range(9)), 9, 5, 64, 32), ((3,), (1025,), 1025, 3, 128, 1024),
    ((100, 17), (300, 0), 301, 40, 128, 16)])
def test_append(dev, dtype, prefix, rows, R, Hkv, dh, page):
    c = Case(R + Hkv, prefix, rows, Hkv, dh, page, dtype, R)
    wide = c.randn(c.B, R, 3 * Hkv, dh)  # k and v as slices of one projection
    k, v = wide[:, :, :Hkv], wide[:, :, 2 * Hkv:]
    want_k, want_v = c.kp.clone(), c.vp.clone()
    for b in range(c.B):
        i, r = ref.spots(c.tab, b, page, prefix[b], rows[b])
        want_k[i, r], want_v[i, r] = k[b, :rows[b]], v[b, :rows[b]]
    ws = m.new_workspace(m.WS_HEADER)
    w = wide.to(dev)
    for src in ((w[:, :, :Hkv], w[:, :, 2 * Hkv:]), (k.contiguous().to(dev), v.contiguous().to(dev))):
        kp, vp, tab, pl, P_max = c.to(dev)
        m.paged_append(*src, kp, vp, tab, pl, P_max, n_rows=i32(*rows).to(dev), ws=ws)
        assert same(kp, want_k) and same(vp, want_v) and status(ws) == "ok"


def test_append_bad_pages_and_prefixes(dev):
    """Rows in a bad page and sequences with a bad prefix change nothing; the others do."""
    c = Case(3, (10, 20, 5), (40, 40, 40), 2, 64, 16, BF)
    k, v = c.randn(3, 40, 2, 64), c.randn(3, 40, 2, 64)
    for bad, code in ((-1, "bad page"), (c.pages, "bad page"), (2 ** 31 - 1, "bad page"), (None, "bad prefix")):
        tab, prefix = c.tab.clone(), list(c.prefix)
        want = c.kp.clone()
        if bad is None:
            prefix[1] = 21  # past P_max
        else:
            tab[1, 2] = bad  # slots 32 .. 47
        for b in range(3):
            if b == 1 and bad is None:
                continue
            keep = [i for i in range(40) if not (b == 1 and (c.prefix[b] + i) // 16 == 2)]
            i, r = ref.spots(c.tab, b, 16, c.prefix[b], 40)
            want[i[keep], r[keep]] = k[b, keep]
        ws = m.new_workspace(m.WS_HEADER)
        kp, vp, _, _, _ = c.to(dev)
        m.paged_append(k.to(dev), v.to(dev), kp, vp, tab.to(dev), i32(*prefix).to(dev), 20, ws=ws)
        assert same(kp, want) and status(ws) == code
    ws = m.new_workspace(m.WS_HEADER)
    kp, vp, tab, pl, P_max = c.to(dev)
    m.paged_append(k.to(dev), v.to(dev), kp, vp, tab, pl, P_max, n_rows=i32(0, -3, 0).to(dev), ws=ws)
    assert same(kp, c.kp) and same(vp, c.vp) and status(ws) == "ok"


# ------------------------------------------------------------------ commit ---

@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("B,R,K,Hkv,dh,page,P", [
    (1, 1, 1, 1, 64, 16, 0), (1, 65, 5, 32, 128, 64, 1000), (7, 65, 5, 8, 128, 16, 47), (40, 15, 8, 3, 64, 32, 100),
    (2, 256, 8, 40, 128, 16, 15), (3, 9, 0, 2, 64, 16, 31)])
def test_commit(dev, dtype, B, R, K, Hkv, dh, page, P):
    prefix = [max(0, P - 3 * b) for b in range(B)]
    c = Case(B * R + K, prefix, [R] * B, Hkv, dh, page, dtype)
    rs = np.random.RandomState(R)
    L = rs.randint(0, min(K, R - 1) + 1, B)
    path = np.full((B, K + 1), -1, np.int32)
    want_k, want_v = c.kp.clone(), c.vp.clone()
    for b in range(B):
        path[b, 0] = 0  # any ascending nodes: sources and targets overlap
        path[b, 1:L[b] + 1] = np.sort(rs.choice(np.arange(1, R), L[b], replace=False)) if L[b] else []
        i, r = ref.spots(c.tab, b, page, prefix[b], R)
        src = path[b, :L[b] + 1].tolist()
        n = len(src)
        want_k[i[:n], r[:n]], want_v[i[:n], r[:n]] = c.kp[i[src], r[src]], c.vp[i[src], r[src]]
    ws = m.new_workspace(m.WS_HEADER)
    kp, vp, tab, pl, P_max = c.to(dev)
    new = m.commit_paged(kp, vp, tab, pl, P_max, torch.from_numpy(path).to(dev),
                         torch.from_numpy(L.astype(np.int32)).to(dev), R, ws=ws)
    assert same(kp, want_k) and same(vp, want_v) and status(ws) == "ok"
    assert new.cpu().tolist() == [P + n + 1 for P, n in zip(prefix, L)]


def test_commit_refuses_bad_paths_pages_and_prefixes(dev):
    c = Case(5, (14, 14), (20, 20), 2, 64, 16, BF)
    ok_path, ok_len = [0, 4, 9, 19], 3
    for what, code in (("len", "bad path"), ("node", "bad path"), ("page", "bad page"), ("prefix", "bad prefix"),
                       ("neg", "bad prefix")):
        path, length = torch.tensor([ok_path, ok_path], dtype=torch.int32), i32(ok_len, ok_len)
        tab, prefix = c.tab.clone(), i32(14, 14)
        if what == "len":
            length[1] = 4
        elif what == "node":
            path[1, 2] = 20
        elif what == "page":
            tab[1, 2] = c.pages  # slot 33 of node 19
        else:
            prefix[1] = 15 if what == "prefix" else -1
        want = c.kp.clone()
        i, r = ref.spots(c.tab, 0, 16, 14, 20)
        want[i[:4], r[:4]] = c.kp[i[ok_path], r[ok_path]]
        ws = m.new_workspace(m.WS_HEADER)
        kp, vp, _, _, _ = c.to(dev)
        new = m.commit_paged(kp, vp, tab.to(dev), prefix.to(dev), 14, path.to(dev), length.to(dev), 20, ws=ws)
        assert same(kp, want) and status(ws) == code
        assert new.cpu().tolist() == [18, int(prefix[1])]


# --------------------------------------------------------------- attention ---

def check(got, q, c, sees, scale=None, kp=None, vp=None):
    """got [B,R,H,dh] against 64 bits; sees(b): bool [n, slots]."""
    dh = q.shape[3]
    scale = dh ** -0.5 if scale is None else scale
    u = torch.finfo(q.dtype).eps / 2
    u_p = 2.0 ** -8 if q.dtype == BF else 0.0
    got = got.double().cpu()
    for b in range(c.B):
        see = sees(b)
        n, N = see.shape
        k, v = (ref.sequence(p, c.tab, b, N) for p in (c.kp if kp is None else kp, c.vp if vp is None else vp))
        y, A, E = ref.attention(q[b, :n].double(), k, v, see, scale)
        tol = A * (u_p + 4 * (dh + 8) * 2.0 ** -24 * E[..., None] + 2.0 ** -20 + 2 * N * 2.0 ** -24) \
            + u * y.abs() + 1e-30
        err = (got[b, :n] - y).abs()
        # (infinities and NaNs have no distance: they are there or not)
        ok = (y == got[b, :n]) | (torch.isnan(y) & torch.isnan(got[b, :n])) | (torch.isfinite(y) & (err <= tol))
        assert ok.all(), (b, float((err / tol).nan_to_num().max()), (~ok).nonzero()[:4].tolist())


SHAPES = [  # prefixes, rows, H, Hkv, dh, page
    ((0,), (1,), 1, 1, 64, 16),
    ((1,), (1,), 4, 4, 128, 16),
    ((1000, 37, 0), (1, 1, 1), 32, 8, 128, 64),
    ((513,), (1,), 28, 4, 64, 32),
    ((300, 301), (4, 4), 16, 4, 128, 16),
    ((63,), (17,), 5, 1, 128, 32),
    ((255, 0), (33, 33), 6, 3, 64, 16),
    ((0, 129, 5), (129, 1, 77), 8, 2, 128, 128),
    ((200,), (130,), 4, 4, 128, 256),
    ((0,), (513,), 7, 1, 64, 64),
    ((2100, 11), (65, 40), 8, 8, 128, 1024),
    ((77,), (300,), 12, 4, 128, 16),
]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("prefix,rows,H,Hkv,dh,page", SHAPES)
def test_chunk_attention(dev, dtype, prefix, rows, H, Hkv, dh, page):
    c = Case(sum(prefix) + sum(rows) + H, prefix, rows, Hkv, dh, page, dtype, R=max(rows) + 2, std=1.5)
    # what no row sees: the tails of the last pages, and pages of nobody
    used = torch.zeros((c.pages, page), dtype=torch.bool)
    for b in range(c.B):
        used[ref.spots(c.tab, b, page, 0, prefix[b] + rows[b])] = True
    c.kp[~used], c.vp[~used] = math.nan, math.inf
    q = c.randn(c.B, c.R, H, dh)
    for b in range(c.B):
        q[b, rows[b]:] = math.nan  # rows behind a sequence are not read
    out = torch.full_like(q, 7.0).to(dev)
    ws = m.new_workspace(m.paged_attention_workspace_size(m.BF16 if dtype == BF else m.F32, c.B, c.R, H, Hkv, dh,
                                                          c.P_max))
    got = m.chunk_attention_paged(q.to(dev), *c.to(dev), n_rows=i32(*rows).to(dev), out=out, ws=ws)
    assert got is out and status(ws) == "ok"
    for b in range(c.B):
        assert (out[b, rows[b]:] == 7).all()
    check(out, q, c, lambda b: ref.causal(prefix[b], rows[b]))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("prefix,R,H,Hkv,dh,page", [
    ((0,), 1, 2, 2, 64, 16), ((1024,), 65, 4, 4, 128, 64), ((300, 17, 0), 65, 8, 2, 128, 16),
    ((129,), 256, 3, 3, 64, 32), ((500, 499), 130, 4, 1, 128, 128), ((40, 900, 0, 3), 15, 4, 2, 64, 16),
    ((5000,), 2, 32, 8, 128, 256), ((64,), 64, 2, 1, 128, 64)])
def test_tree_attention(dev, dtype, prefix, R, H, Hkv, dh, page):
    c = Case(sum(prefix) + R + H, prefix, [R] * len(prefix), Hkv, dh, page, dtype, std=1.5)
    mask, _ = cache_ops_ref.tree(c.B, R, np.random.RandomState(R))
    q = c.randn(c.B, R, H, dh)
    got = m.tree_attention_paged(q.to(dev), *c.to(dev), mask.to(dev))
    check(got, q, c, lambda b: ref.tree_sees(prefix[b], R, mask[b]))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("R,H,Hkv", [(9, 4, 2), (65, 4, 2), (65, 2, 2), (200, 2, 1)])
def test_unseen_slots_and_empty_rows(dev, dtype, R, H, Hkv):
    """Infinities and NaNs in K and V of nodes change only the rows that see them, and a
    row whose mask and prefix leave nothing gets zeros."""
    for P in (0, 70):
        c = Case(P + R, (P,), (R,), Hkv, 128, 16, dtype)
        mask, _ = cache_ops_ref.tree(1, R, np.random.RandomState(R))
        rs = np.random.RandomState(7)
        odd = rs.choice(np.arange(1, R), 3, replace=False)
        for j, x in zip(odd, (math.nan, math.inf, -math.inf)):
            i, r = ref.spots(c.tab, 0, 16, P + int(j), 1)
            c.vp[i, r, :, int(j) % 128] = x
        mask[0, 5] = 0  # no ancestor, itself not either
        q = c.randn(1, R, H, 128)
        got = m.tree_attention_paged(q.to(dev), *c.to(dev), mask.to(dev))
        check(got, q, c, lambda b: ref.tree_sees(P, R, mask[b]))
        if P == 0:
            assert (got[0, 5] == 0).all()
        # the same slots in a chunk: rows before them do not see them
        got = m.chunk_attention_paged(q.to(dev), *c.to(dev))
        check(got, q, c, lambda b: ref.causal(P, R))
        for j in odd:
            i, r = ref.spots(c.tab, 0, 16, P + int(j), 1)
            c.kp[i, r] = math.nan
        got = m.chunk_attention_paged(q.to(dev), *c.to(dev))
        first = int(min(odd))
        assert torch.isnan(got[0, first:]).all()
        check(got[:, :first], q[:, :first], c, lambda b: ref.causal(P, R)[:first, :P + first])


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("R,H,Hkv,ns", [(1, 8, 2, 0), (3, 4, 4, 0), (40, 4, 2, 0), (200, 4, 1, 0)])
def test_bad_pages_are_not_seen(dev, dtype, R, H, Hkv, ns):
    c = Case(R + H, (600, 333), (R, R), Hkv, 128, 16, dtype)
    q = c.randn(2, R, H, 128)
    kp, vp, tab, pl, P_max = c.to(dev)
    for at, bad in ((0, -1), (7, c.pages), (20, 2 ** 31 - 1), ((333 + R - 1) // 16, -2 ** 31)):
        t = c.tab.clone()
        t[1, at] = bad
        ws = m.new_workspace(m.paged_attention_workspace_size(m.BF16 if dtype == BF else m.F32, 2, R, H, Hkv, 128,
                                                              P_max))
        got = m.chunk_attention_paged(q.to(dev), kp, vp, t.to(dev), pl, P_max, ws=ws)
        assert status(ws) == "bad page"

        def sees(b):
            see = ref.causal(c.prefix[b], R)
            if b == 1:
                see[:, at * 16:at * 16 + 16] = False
            return see
        check(got, q, c, sees)
    t = torch.full_like(c.tab, -5)  # no page at all: nothing is seen
    got = m.chunk_attention_paged(q.to(dev), kp, vp, t.to(dev), pl, P_max)
    assert (got == 0).all()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("R", [1, 70])
def test_bad_prefix_and_rows(dev, dtype, R):
    c = Case(R, (50, 60, 70), (R,) * 3, 2, 64, 16, dtype)
    q = c.randn(3, R, 4, 64)
    kp, vp, tab, pl, P_max = c.to(dev)
    ws = m.new_workspace(m.paged_attention_workspace_size(m.BF16 if dtype == BF else m.F32, 3, R, 4, 2, 64, 70))
    for bad in (-1, 71, 2 ** 31 - 1):
        pl[1] = bad
        out = torch.full((3, R, 4, 64), 3.0, dtype=dtype, device=dev)
        m.chunk_attention_paged(q.to(dev), kp, vp, tab, pl, P_max, out=out, ws=ws)
        assert (out[1] == 0).all() and status(ws) == "bad prefix"
        keep = Case.__new__(Case)
        keep.__dict__.update(c.__dict__, B=1)
        check(out[:1], q[:1], keep, lambda b: ref.causal(50, R))
        m.clear_device_status(ws)
    pl[1] = 60
    out = torch.full((3, R, 4, 64), 3.0, dtype=dtype, device=dev)
    m.chunk_attention_paged(q.to(dev), kp, vp, tab, pl, P_max, n_rows=i32(0, -4, R + 9).to(dev), out=out, ws=ws)
    assert (out[:2] == 3).all() and status(ws) == "ok"  # no rows: not touched


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("R", [1, 60])
def test_scores_at_the_ends(dev, dtype, R):
    """Large scores, equal scores, and queries that are not finite."""
    c = Case(R, (90,), (R,), 1, 64, 16, dtype)
    q = c.randn(1, R, 2, 64) * 200
    got = m.chunk_attention_paged(q.to(dev), *c.to(dev), scale=1.0)
    check(got, q, c, lambda b: ref.causal(90, R), scale=1.0)
    z = torch.zeros_like(q)
    got = m.chunk_attention_paged(z.to(dev), *c.to(dev))
    check(got, z, c, lambda b: ref.causal(90, R))
    q[0, R // 2, 1] = math.nan
    got = m.chunk_attention_paged(q.to(dev), *c.to(dev))
    assert torch.isnan(got[0, R // 2, 1]).all() and torch.isfinite(got[0, :, 0]).all()


def test_pools_past_32_bits(dev):
    """Pools of more than 2^32 bytes: pages at both ends are written, read and moved."""
    page, Hkv, dh = 64, 32, 128
    pages = (5 << 30) // (page * Hkv * dh * 2)
    assert pages * page * Hkv * dh > 1 << 31
    kp, vp = (torch.zeros((pages, page, Hkv, dh), dtype=BF, device=dev) for _ in range(2))
    g = torch.Generator().manual_seed(1)
    P, R, H = 100, 20, 32
    c = Case(2, (P,), (R,), Hkv, dh, page, BF)
    tab = torch.tensor([[pages - 1, 0]], dtype=torch.int32)
    k, v = ((torch.randn((1, P + R, Hkv, dh), generator=g)).to(BF) for _ in range(2))
    zero, pl = i32(0).to(dev), i32(P).to(dev)
    ws = m.new_workspace(m.WS_HEADER)
    m.paged_append(k.to(dev), v.to(dev), kp, vp, tab.to(dev), zero, 0, ws=ws)
    small_k, small_v = kp[[pages - 1, 0]].cpu(), vp[[pages - 1, 0]].cpu()
    assert same(small_k.flatten(0, 1)[:P + R], k[0]) and same(small_v.flatten(0, 1)[:P + R], v[0])
    c.kp, c.vp, c.tab = small_k, small_v, torch.tensor([[0, 1]], dtype=torch.int32)
    for n in (1, R):
        q = torch.randn((1, n, H, dh), generator=g).to(BF)
        got = m.chunk_attention_paged(q.to(dev), kp, vp, tab.to(dev), pl, P)
        check(got, q, c, lambda b: ref.causal(P, n))
    new = m.commit_paged(kp, vp, tab.to(dev), pl, P, torch.tensor([[0, 19]], dtype=torch.int32).to(dev),
                         i32(1).to(dev), R, ws=ws)
    assert new.item() == P + 2 and same(kp[0, P + 1 - page], k[0, P + 19]) and status(ws) == "ok"
    assert same(vp[0, P + 1 - page], v[0, P + 19])


def test_captured_calls_share_a_workspace(dev):
    """Two shapes captured into graphs over one workspace, replayed in turn with new
    inputs, give what eager calls give."""
    a = Case(1, (700, 20), (1, 1), 2, 128, 16, BF)
    b = Case(2, (200, 310), (50, 50), 2, 128, 32, BF)
    size = m.paged_attention_workspace_size
    ws = m.new_workspace(max(size(m.BF16, 2, 1, 8, 2, 128, 700), size(m.BF16, 2, 50, 8, 2, 128, 310)))
    calls = []
    for c, R in ((a, 1), (b, 50)):
        q = c.randn(2, R, 8, 128).to(dev)
        args = c.to(dev)
        out = torch.zeros_like(q)
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            m.chunk_attention_paged(q, *args, out=out, ws=ws)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            m.chunk_attention_paged(q, *args, out=out, ws=ws)
        calls.append((c, q, args, out, graph))
    for step in range(3):
        for c, q, args, out, graph in calls:
            q.copy_(c.randn(*q.shape))
            args[0].copy_(c.randn(*c.kp.shape))
            out.zero_()
            graph.replay()
            want = m.chunk_attention_paged(q, *args)
            assert torch.equal(out, want)


def test_two_streams_at_the_same_time(dev):
    """Calls on two streams, each with its own workspace, give what they give alone."""
    c = Case(4, (3000, 100, 900), (70, 70, 70), 4, 128, 64, BF)
    q = c.randn(3, 70, 8, 128).to(dev)
    args = c.to(dev)
    want = m.chunk_attention_paged(q, *args)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [[], []]
    for _ in range(20):
        for s, o in zip(streams, outs):
            o.append(m.chunk_attention_paged(q, *args, stream=s))
    torch.cuda.synchronize()
    assert all(torch.equal(x, want) for o in outs for x in o)


# ---------------------------------------------------------- a run together ---

@pytest.mark.parametrize("dtype", [BF, F32])
def test_prompt_steps_and_logprobs_on_pages(dev, dtype):
    """Prompts enter in two pieces, then two steps of tree attention, posterior, commit
    and log probabilities of what was accepted, for a ragged batch."""
    B, H, Hkv, dh, page, R, K, V = 3, 8, 2, 64, 16, 16, 4, 512
    lengths = [150, 33, 70]
    c = Case(9, lengths, [4 * R] * B, Hkv, dh, page, dtype, R=160)
    kp, vp, tab, _, _ = c.to(dev)
    P_max = c.tab.shape[1] * page - 100
    ws = m.new_workspace(max(m.paged_attention_workspace_size(m.BF16 if dtype == BF else m.F32, B, 100, H, Hkv, dh,
                                                              P_max), 1 << 20))
    prefix = torch.zeros(B, dtype=torch.int32, device=dev)
    kept_k, kept_v = [[] for _ in range(B)], [[] for _ in range(B)]
    for at in (0, 100):
        n = [max(0, min(100, x - at)) for x in lengths]
        rows = i32(*n).to(dev)
        k, v, q = c.randn(B, 100, Hkv, dh), c.randn(B, 100, Hkv, dh), c.randn(B, 100, H, dh)
        m.paged_append(k.to(dev), v.to(dev), kp, vp, tab, prefix, P_max, n_rows=rows, ws=ws)
        out = m.chunk_attention_paged(q.to(dev), kp, vp, tab, prefix, P_max, n_rows=rows, ws=ws)
        for b in range(B):
            kept_k[b].append(k[b, :n[b]]), kept_v[b].append(v[b, :n[b]])
            P = sum(len(x) for x in kept_k[b]) - n[b]
            if n[b]:
                one = Case.__new__(Case)
                one.__dict__.update(c.__dict__, B=1, tab=c.tab[b:b + 1])
                check(out[b:b + 1], q[b:b + 1], one, lambda _: ref.causal(P, n[b]), kp=kp.cpu(), vp=vp.cpu())
        prefix = prefix + rows
    assert prefix.cpu().tolist() == lengths
    rs = np.random.RandomState(2)
    for step in range(2):
        mask, depth = cache_ops_ref.tree(B, R, rs, max_depth=K)
        parent = torch.full((B, R), -1, dtype=torch.int32)
        bits = np.unpackbits(mask.numpy().view(np.uint8), axis=-1, bitorder="little")[..., :R]
        for b in range(B):
            for i in range(1, R):
                above = [j for j in range(i) if bits[b, i, j]]
                parent[b, i] = max(above, key=lambda j: int(depth[b, j]))
        k, v, q = c.randn(B, R, Hkv, dh), c.randn(B, R, Hkv, dh), c.randn(B, R, H, dh)
        m.paged_append(k.to(dev), v.to(dev), kp, vp, tab, prefix, P_max, ws=ws)
        out = m.tree_attention_paged(q.to(dev), kp, vp, tab, prefix, P_max, mask.to(dev), ws=ws)
        P = prefix.cpu().tolist()
        check(out, q, c, lambda b: ref.tree_sees(P[b], R, mask[b]), kp=kp.cpu(), vp=vp.cpu())
        logits = c.randn(B, R, V, std=3.0)
        tokens = logits.float().argmax(-1).int()  # a node's token: mostly its parent's choice
        for b in range(B):
            for i in range(R - 1, 0, -1):
                tokens[b, i] = tokens[b, parent[b, i]] if rs.rand() < 0.8 else rs.randint(V)
        lg = logits.to(dev)
        post = m.evaluate_posterior(lg, tokens.to(dev), parent.to(dev), depth.to(dev), K, ws=ws)
        prefix = m.commit_paged(kp, vp, tab, prefix, P_max, post.path, post.accept_len, R, ws=ws)
        path, n = post.path.cpu(), post.accept_len.cpu().tolist()
        assert prefix.cpu().tolist() == [p + x + 1 for p, x in zip(P, n)]
        for b in range(B):
            nodes = path[b, :n[b] + 1].long()
            kept_k[b].append(k[b, nodes]), kept_v[b].append(v[b, nodes])
            i, r = ref.spots(c.tab, b, page, 0, P[b] + n[b] + 1)
            assert same(kp.cpu()[i, r], torch.cat(kept_k[b])) and same(vp.cpu()[i, r], torch.cat(kept_v[b]))
        # the accepted tokens' log probabilities: each judged by its parent's row
        ids = torch.full((B, R), -1, dtype=torch.int32)
        for b in range(B):
            for a, z in zip(path[b, :n[b]].tolist(), path[b, 1:n[b] + 1].tolist()):
                ids[b, a] = tokens[b, z]
        lp = m.token_logprobs(lg, ids.to(dev), 3, ws=ws)
        assert lp.top_ids.shape == (B, R, 3)
        for b in range(B):
            for a in path[b, :n[b]].tolist():
                assert lp.rank[b, a] == 0 and lp.top_ids[b, a, 0] == ids[b, a]
                assert lp.logp[b, a] == lp.top_logp[b, a, 0]
            last = int(path[b, n[b]])
            assert lp.top_ids[b, last, 0] == post.next_token[b] and lp.rank[b, last] == -1
    assert status(ws) == "ok"
