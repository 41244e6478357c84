"""Paged attention at the sizes where its kernels and their parts change: rows at the
ends of tiles, ranges and joins of every kind, many sequences, bounded waits; and the
log probabilities at every alignment of a row.  Tolerances as in test_gpu_paged and
test_gpu_logprobs."""
import math

import numpy as np
import pytest
import torch

import cache_ops_ref
import medusa_speculative_decoding_02_gb300 as m
import paged_ref as ref
import test_gpu_logprobs as tl
from medusa_speculative_decoding_02_gb300 import build as mbuild
from test_gpu_paged import BF, F32, Case, check, i32, status

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    mbuild.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    d = torch.device("cuda:0")
    torch.cuda.set_device(d)
    return d


def workspace(c, H, dtype=BF):
    return m.new_workspace(m.paged_attention_workspace_size(m.BF16 if dtype == BF else m.F32, c.B, c.R, H, c.Hkv,
                                                            c.dh, c.P_max))


@pytest.mark.parametrize("G", [1, 3, 4])
@pytest.mark.parametrize("M", [16, 17, 32, 127, 128, 129, 136, 137, 255, 256, 257, 264, 265, 384, 385, 512, 513])
def test_rows_where_tiles_change(dev, M, G):
    """Rows a KV head around the few-row kernel's limit and the tiles of 128 and 256, in a
    ragged batch whose second sequence ends somewhere inside."""
    R = -(-M // G)
    rows = (R, max(1, R - 2), min(R, 3))
    c = Case(M + G, (130, 61, 0), rows, 2, 64, 32, BF, R=R, std=1.5)
    q = c.randn(3, R, 2 * G, 64)
    ws = workspace(c, 2 * G)
    out = torch.full_like(q, 5.0).to(dev)
    m.chunk_attention_paged(q.to(dev), *c.to(dev), n_rows=i32(*rows).to(dev), out=out, ws=ws)
    check(out, q, c, lambda b: ref.causal(c.prefix[b], rows[b]))
    for b in range(3):
        assert (out[b, rows[b]:] == 5).all()
    if R <= 256:
        mask, _ = cache_ops_ref.tree(3, R, np.random.RandomState(M))
        full = Case(M, (130, 61, 0), (R,) * 3, 2, 64, 32, BF)
        got = m.tree_attention_paged(q.to(dev), *full.to(dev), mask.to(dev), ws=ws)
        check(got, q, full, lambda b: ref.tree_sees(full.prefix[b], R, mask[b]))
    assert status(ws) == "ok"


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("prefix,R,H,Hkv,dh", [
    ((20000,), 1, 2, 1, 128), ((20000,), 1, 1, 1, 64), ((9000, 100, 5000), 1, 4, 2, 64), ((3000, 2000), 3, 8, 8, 128),
    ((6000,), 40, 2, 1, 128), ((4000, 30), 70, 16, 16, 64), ((2500,), 600, 2, 1, 64)])
def test_ranges_and_their_joins(dev, dtype, prefix, R, H, Hkv, dh):
    """Few rows over long prefixes: from two ranges of keys to more than 32."""
    c = Case(sum(prefix) + R, prefix, (R,) * len(prefix), Hkv, dh, 128, dtype, std=1.5)
    q = c.randn(c.B, R, H, dh)
    ws = workspace(c, H, dtype)
    # (partial results in the workspace, but for what clusters of CTAs join)
    assert ws.numel() > m.WS_HEADER or (dtype == BF and 16 < R * H // Hkv <= 128)
    got = m.chunk_attention_paged(q.to(dev), *c.to(dev), ws=ws)
    check(got, q, c, lambda b: ref.causal(prefix[b], R))
    rows = [max(0, R - 1 - b) for b in range(c.B)]
    out = torch.full_like(q, -3.0).to(dev)
    m.chunk_attention_paged(q.to(dev), *c.to(dev), n_rows=i32(*rows).to(dev), out=out, ws=ws)
    check(out, q, c, lambda b: ref.causal(prefix[b], rows[b]))
    for b in range(c.B):
        assert (out[b, rows[b]:] == -3).all()
    assert status(ws) == "ok"


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("B,R", [(33, 1), (40, 20), (70, 2)])
def test_many_sequences(dev, dtype, B, R):
    """More sequences than ranges are dealt out to by their lengths."""
    prefix = [(b * 37) % 700 for b in range(B)]
    c = Case(B + R, prefix, (R,) * B, 1, 64, 16, dtype)
    q = c.randn(B, R, 2, 64)
    got = m.chunk_attention_paged(q.to(dev), *c.to(dev))
    check(got, q, c, lambda b: ref.causal(prefix[b], R))


@pytest.mark.parametrize("R,G", [(65, 4), (40, 2), (300, 1)])
def test_infinities_and_bad_pages_over_ranges(dev, R, G):
    """Non-finite V in the last tile, a bad page and a bad prefix at once, with the keys
    in several ranges."""
    c = Case(R, (3000, 700, 40), (R,) * 3, 1, 128, 16, BF)
    q = c.randn(3, R, G, 128)
    for b in range(3):
        for j, x in ((R // 3, math.inf), (R - 2, math.nan)):
            i, r = ref.spots(c.tab, b, 16, c.prefix[b] + j, 1)
            c.vp[i, r, 0, 7 * b] = x
    kp, vp, tab, pl, P_max = c.to(dev)
    tab[0, 50] = -9
    pl[2] = P_max + 1
    ws = workspace(c, G)
    got = m.chunk_attention_paged(q.to(dev), kp, vp, tab, pl, P_max, ws=ws)
    assert (got[2] == 0).all() and status(ws) in ("bad page", "bad prefix")
    two = Case.__new__(Case)
    two.__dict__.update(c.__dict__, B=2)

    def sees(b):
        see = ref.causal(c.prefix[b], R)
        if b == 0:
            see[:, 800:816] = False
        return see
    check(got, q, two, sees)


@pytest.mark.parametrize("R,H,Hkv,ns", [(65, 2, 2, True), (200, 4, 1, True), (512, 2, 2, False)])
def test_waits_that_run_out(dev, R, H, Hkv, ns):
    """With no polls every wait fails at once: the status says so, the rows are zeros, and
    the same call on the same buffers is right afterwards."""
    c = Case(R, (900 if ns else 0, 30), (R, R), Hkv, 128, 64, BF)
    q = c.randn(2, R, H, 128)
    args = c.to(dev)
    ws = workspace(c, H)
    budget = m.wait_budget()
    try:
        m.set_wait_budget(0)
        out = torch.full_like(q, 9.0).to(dev)
        m.chunk_attention_paged(q.to(dev), *args, out=out, ws=ws)
        torch.cuda.synchronize()
    finally:
        m.set_wait_budget(budget)
    assert status(ws) == "timeout" and (out == 0).all()
    m.clear_device_status(ws)
    m.chunk_attention_paged(q.to(dev), *args, out=out, ws=ws)
    assert status(ws) == "ok"
    check(out, q, c, lambda b: ref.causal(c.prefix[b], R))


def test_one_page_and_shared_pages(dev):
    """A pool of a single page, and two sequences that share the pages of their prefix."""
    c = Case(1, (5,), (9,), 1, 64, 16, BF)
    kp, vp = c.kp[c.tab[0, :1].long()].contiguous(), c.vp[c.tab[0, :1].long()].contiguous()
    q = c.randn(1, 9, 2, 64)
    one = Case.__new__(Case)
    one.__dict__.update(c.__dict__, kp=kp, vp=vp, tab=torch.zeros((1, 1), dtype=torch.int32))
    for n in (1, 9):
        got = m.chunk_attention_paged(q[:, :n].contiguous().to(dev), kp.to(dev), vp.to(dev), one.tab.to(dev),
                                      i32(5).to(dev), 5)
        check(got, q[:, :n], one, lambda b: ref.causal(5, n))
    c = Case(2, (64, 64), (30, 30), 2, 128, 16, BF)
    c.tab[1, :4] = c.tab[0, :4]
    q = c.randn(2, 30, 4, 128)
    got = m.chunk_attention_paged(q.to(dev), *c.to(dev))
    check(got, q, c, lambda b: ref.causal(64, 30))


# -------------------------------------------------------- log probabilities ---

@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("V", [1, 2, 7, 8, 9, 15, 16, 17, 31, 4101, 16389])
def test_logprobs_at_every_alignment(dev, dtype, V):
    """Rows that begin and end anywhere in a 16-byte block; every place of the token."""
    g = torch.Generator().manual_seed(V)
    wide = (torch.randn((9, V + 13), generator=g) * 3).to(dtype)
    top = min(V, 6)
    for first in range(0, 9, 1 if V < 40 else 3):
        x = wide[:, first:first + V]
        tokens = torch.randint(0, V, (9,), generator=g, dtype=torch.int32)
        tokens[0], tokens[1] = 0, V - 1
        tl.check(m.token_logprobs(wide.to(dev)[:, first:first + V], tokens.to(dev), top), x, tokens, top, 1.0)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("N", [75, 76, 152, 153, 304, 305, 608, 609, 1400])
def test_logprobs_where_clusters_change(dev, dtype, N):
    """Rows shared by four CTAs, by two, a CTA each, several a CTA."""
    g = torch.Generator().manual_seed(N)
    V = 33000
    x = tl.rows(g, N, V, dtype)
    x[N // 2] = x[N // 2, 0]   # ties: too many candidates
    x[N - 1, 3:] = -math.inf   # fewer possible tokens than alternatives
    tokens = torch.randint(0, V, (N,), generator=g, dtype=torch.int32)
    out = m.token_logprobs(x.to(dev), tokens.to(dev), 9, temperature=1.1)
    keep = [0, 1, N // 2 - 1, N // 2, N - 2, N - 1] + list(range(3, N - 3, 97))
    pick = m.TokenLogprobs(out.logp[keep], out.entropy[keep], out.rank[keep], out.top_ids[keep], out.top_logp[keep])
    tl.check(pick, x[keep], tokens[keep], 9, 1.1)


def test_logprobs_of_peaked_and_flat_rows(dev):
    """Large maxima that come late, early, in every chunk; one thread with many of the best."""
    V = 70000
    x = torch.full((6, V), -20.0)
    x[0, 69999] = 300.0
    x[1, 0] = 300.0
    x[2] = torch.arange(V).float() / 100
    x[3, ::1024] = torch.arange(69).float() / 8 + 2      # the same thread in every chunk
    x[4, 128 * 8 * torch.arange(60)] = 5.0
    x[5] = torch.linspace(-4, 4, V).flip(0)
    for dtype in (BF, F32):
        y = x.to(dtype)
        tokens = torch.tensor([5, 5, 69990, 2048, 1024, 69999], dtype=torch.int32)
        tl.check(m.token_logprobs(y.to(dev), tokens.to(dev), 16), y, tokens, 16, 1.0)
        big = y.repeat(120, 1)
        out = m.token_logprobs(big.to(dev), tokens.repeat(120).to(dev), 16)
        pick = slice(714, 720)
        tl.check(m.TokenLogprobs(out.logp[pick], out.entropy[pick], out.rank[pick], out.top_ids[pick],
                                 out.top_logp[pick]), y, tokens, 16, 1.0)


@pytest.mark.parametrize("R,G,dh", [(65, 2, 64), (33, 4, 128)])
def test_ranges_of_long_sequences(dev, R, G, dh):
    """A wave of CTAs without ranges, some of whose sequences are long: those are shared
    out, the others written without a join; some rows, a sequence or a prefix are missing."""
    prefix = [8500, 3, 0, 500, 700, 60, 4100, 128, 1, 256] + [20] * 22
    rows = [R, R, R - 5, 0, 1, R, R, R, R, R // 2] + [R] * 22
    c = Case(R, prefix, rows, 4, dh, 64, BF, R=R, std=1.5)
    q = c.randn(c.B, R, 4 * G, dh)
    ws = workspace(c, 4 * G)
    assert ws.numel() > m.WS_HEADER  # there are partial results
    out = torch.full_like(q, 7.0).to(dev)
    args = c.to(dev)
    for _ in range(2):  # (the second time over the first one's partial results)
        m.chunk_attention_paged(q.to(dev), *args, n_rows=i32(*rows).to(dev), out=out, ws=ws)
        check(out, q, c, lambda b: ref.causal(prefix[b], rows[b]))
        for b in range(c.B):
            assert (out[b, rows[b]:] == 7).all()
    assert status(ws) == "ok"
    args[3][5] = -1
    out.fill_(7.0)
    m.chunk_attention_paged(q.to(dev), *args, n_rows=i32(*rows).to(dev), out=out, ws=ws)
    assert (out[5] == 0).all() and status(ws) == "bad prefix"
    five = rows[:5] + [0] + rows[6:]
    check(out, q, c, lambda b: ref.causal(prefix[b], five[b]))


@pytest.mark.parametrize("P,R,H,Hkv,dh,B", [
    (200, 17, 2, 2, 128, 1), (300, 33, 3, 1, 64, 1), (600, 65, 8, 8, 64, 1), (1000, 128, 1, 1, 128, 1),
    (1500, 20, 32, 8, 128, 1), (1024, 65, 32, 32, 128, 1), (2048, 65, 40, 40, 128, 1), (5000, 65, 40, 40, 64, 1),
    (1300, 60, 6, 3, 128, 5), (700, 18, 16, 16, 64, 2)])
def test_ranges_in_clusters(dev, P, R, H, Hkv, dh, B):
    """Few rows, whose ranges a cluster of CTAs joins: whole, empty and masked ranges, rows and
    sequences that are missing, bad pages and prefixes, non-finite V, waits that run out."""
    prefix, rows = ([P, 0, P // 2, 3, P - 1][:B], [R, R, R - 1, 0, 1][:B])
    c = Case(P + R, prefix, rows, Hkv, dh, 16, BF, R=R, std=1.5)
    q = c.randn(B, R, H, dh)
    # (V that the last row alone sees)
    i, r = ref.spots(c.tab, 0, 16, P + R - 1, 1)
    c.vp[i, r, 0, 3] = math.inf
    ws = m.new_workspace(m.paged_attention_workspace_size(m.BF16, B, R, H, Hkv, dh, P))
    out = torch.full_like(q, 7.0).to(dev)
    args, n = c.to(dev), i32(*rows).to(dev)

    def call(expect="ok"):
        m.chunk_attention_paged(q.to(dev), *args, n_rows=n, out=out, ws=ws)
        assert status(ws) == expect
        m.clear_device_status(ws)
    for _ in range(2):
        call()
        check(out, q, c, lambda b: ref.causal(prefix[b], rows[b]))
        for b in range(B):
            assert (out[b, rows[b]:] == 7).all()
    # a page in the middle that is not there
    at = P // 32
    args[2][0, at] = c.pages
    call("bad page")

    def sees(b):
        see = ref.causal(prefix[b], rows[b])
        if b == 0:
            see[:, 16 * at:16 * at + 16] = False
        return see
    check(out, q, c, sees)
    # no page is there
    args[2][0] = -1
    call("bad page")
    assert (out[0] == 0).all()
    args[2].copy_(c.tab)
    args[3][0] = P + 1
    call("bad prefix")
    assert (out[0] == 0).all()
    args[3][0] = P
    budget = m.wait_budget()
    try:
        m.set_wait_budget(0)
        call("timeout")
    finally:
        m.set_wait_budget(budget)
    for b in range(B):
        assert (out[b, :rows[b]] == 0).all()
    call()
    check(out, q, c, lambda b: ref.causal(prefix[b], rows[b]))
    # n_rows: none, and the tree of the same rows
    n.zero_()
    out.fill_(7.0)
    call()
    assert (out == 7).all()
    if B == 1:
        mask, _ = cache_ops_ref.tree(1, R, np.random.RandomState(R))
        got = m.tree_attention_paged(q.to(dev), *args, mask.to(dev), ws=ws)
        check(got, q, c, lambda b: ref.tree_sees(P, R, mask[b]))


@pytest.mark.parametrize("R,H,Hkv,dh,prefix", [
    (1, 4, 4, 128, (300, 0)), (2, 2, 1, 64, (75, 700)), (3, 1, 1, 128, (1000,)), (5, 6, 2, 128, (129, 64, 1)),
    (16, 3, 3, 64, (500,)), (17, 2, 2, 128, (257, 31)), (33, 8, 8, 64, (2000, 2100)), (64, 6, 3, 128, (1500, 0)),
    (70, 20, 10, 64, (700,)), (129, 8, 8, 128, (900,))])
def test_fp32_tiles(dev, R, H, Hkv, dh, prefix):
    """fp32: tiles of 1 to 64 rows, with bad pages, masks and V that few rows see."""
    B = len(prefix)
    rows = [max(1, R - b) for b in range(B)]
    c = Case(R + H, prefix, rows, Hkv, dh, 16, F32, R=R, std=1.5)
    q = c.randn(B, R, H, dh)
    for b in range(B):  # seen by the last row alone
        i, r = ref.spots(c.tab, b, 16, prefix[b] + rows[b] - 1, 1)
        c.vp[i, r, 0, 5] = -math.inf
    ws = workspace(c, H, F32)
    out = torch.full_like(q, 7.0).to(dev)
    args, n = c.to(dev), i32(*rows).to(dev)
    m.chunk_attention_paged(q.to(dev), *args, n_rows=n, out=out, ws=ws)
    check(out, q, c, lambda b: ref.causal(prefix[b], rows[b]))
    assert status(ws) == "ok"
    at = prefix[0] // 32
    args[2][0, at] = -5
    m.chunk_attention_paged(q.to(dev), *args, n_rows=n, out=out, ws=ws)

    def sees(b):
        see = ref.causal(prefix[b], rows[b])
        if b == 0:
            see[:, 16 * at:16 * at + 16] = False
        return see
    check(out, q, c, sees)
    for b in range(B):
        assert (out[b, rows[b]:] == 7).all()
    assert status(ws) == "bad page"
    m.clear_device_status(ws)
    args[2].copy_(c.tab)
    mask, _ = cache_ops_ref.tree(B, R, np.random.RandomState(R))
    full = Case(R + H, prefix, [R] * B, Hkv, dh, 16, F32, std=1.5)
    got = m.tree_attention_paged(q.to(dev), *full.to(dev), mask.to(dev), ws=ws)
    check(got, q, full, lambda b: ref.tree_sees(prefix[b], R, mask[b]))
    assert status(ws) == "ok"


def test_clusters_captured_and_on_two_streams(dev):
    """Calls whose ranges clusters join: a captured call replayed on new inputs, next to
    another such call on another stream."""
    a, b = Case(5, (900,), (40,), 4, 128, 32, BF), Case(6, (1500,), (60,), 8, 64, 64, BF)
    q = [c.randn(3, c.R, 2 * c.Hkv, c.dh) for c in (a, b)]
    args = [c.to(dev) for c in (a, b)]
    ws = [m.new_workspace(m.paged_attention_workspace_size(m.BF16, 1, c.R, 2 * c.Hkv, c.Hkv, c.dh, c.P_max))
          for c in (a, b)]
    assert [w.numel() for w in ws] == [m.WS_HEADER] * 2  # no partial results
    src = [x[:1].to(dev) for x in q]
    out = [torch.zeros_like(x) for x in src]
    side = torch.cuda.Stream()

    def issue(i, stream=None):
        m.chunk_attention_paged(src[i], *args[i], out=out[i], ws=ws[i], stream=stream)
    graph = m.StepGraph(lambda: issue(0))
    for k in range(3):
        for i in range(2):
            src[i].copy_(q[i][k:k + 1])
        torch.cuda.synchronize()
        for _ in range(5):
            graph.replay()
            issue(1, side)
        torch.cuda.synchronize()
        for i, c in enumerate((a, b)):
            check(out[i], q[i][k:k + 1], c, lambda _: ref.causal(c.prefix[0], c.R))
            assert status(ws[i]) == "ok"


@pytest.mark.parametrize("B,R,H,Hkv,dh,P", [
    (20, 20, 8, 8, 128, 300), (31, 65, 10, 5, 64, 200), (52, 33, 9, 3, 128, 90), (20, 17, 16, 8, 64, 8000),
    (40, 128, 5, 5, 64, 130), (153, 18, 2, 1, 128, 60)])
def test_more_tiles_than_one_wave(dev, B, R, H, Hkv, dh, P):
    """One tile a KV head and more of those than SMs: two heads a CTA (a last one alone),
    rows and sequences that are missing, bad pages, masks, non-finite V, waits that run out."""
    prefix = [P] + [(37 * b) % (P if P < 400 else 150) for b in range(1, B)]
    rows = [R, 0, 1] + [max(1, R - b % 7) for b in range(3, B)]
    c = Case(P + R, prefix, rows, Hkv, dh, 16, BF, R=R, std=1.5)
    q = c.randn(B, R, H, dh)
    for h in range(Hkv):  # (what the last row of a sequence alone sees)
        i, r = ref.spots(c.tab, 3 + h, 16, prefix[3 + h] + rows[3 + h] - 1, 1)
        c.vp[i, r, h, 3 * h] = math.nan if h % 2 else math.inf
    ws = workspace(c, H)
    out = torch.full_like(q, 7.0).to(dev)
    args, n = c.to(dev), i32(*rows).to(dev)

    def call(expect="ok"):
        m.chunk_attention_paged(q.to(dev), *args, n_rows=n, out=out, ws=ws)
        assert status(ws) == expect
        m.clear_device_status(ws)
    call()
    check(out, q, c, lambda b: ref.causal(prefix[b], rows[b]))
    for b in range(B):
        assert (out[b, rows[b]:] == 7).all()
    at = P // 32
    args[2][0, at] = c.pages
    call("bad page")

    def sees(b):
        see = ref.causal(prefix[b], rows[b])
        if b == 0:
            see[:, 16 * at:16 * at + 16] = False
        return see
    check(out, q, c, sees)
    args[2].copy_(c.tab)
    budget = m.wait_budget()
    try:
        m.set_wait_budget(0)
        call("timeout")
    finally:
        m.set_wait_budget(budget)
    for b in range(B):
        assert (out[b, :rows[b]] == 0).all()
    args[3][2] = P + 1
    call("bad prefix")
    assert (out[2, :1] == 0).all()
    args[3][2] = prefix[2]
    call()
    check(out, q, c, lambda b: ref.causal(prefix[b], rows[b]))
    mask, _ = cache_ops_ref.tree(B, R, np.random.RandomState(R))
    full = Case(P + R, prefix, [R] * B, Hkv, dh, 16, BF, std=1.5)
    got = m.tree_attention_paged(q.to(dev), *full.to(dev), mask.to(dev), ws=ws)
    check(got, q, full, lambda b: ref.tree_sees(prefix[b], R, mask[b]))
