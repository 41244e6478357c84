"""Log probabilities of given tokens on the GPU against 64 bits.

Tolerances, u = 2^-24, c = log2(e) / T (itself off by 2 u): the distance t = (x - max) c
of a logit in base 2 is off by 4 u |t|.  S = sum 2^t: a weight is off by the
exponential's 2^-22 = 4 u and by ln2 * 4 u |t|, sums of V terms by at most
(V / 512 + 64) u (chains of V / 512 to a thread, trees after them; a chain may start a
few times over, each start another product), so a relative
    s = u (4 + 3 E1 + V / 512 + 64),  E1 = sum p |t|.
ln p = ln2 (t - log2 S): off by 4 u |t| ln2, by s, by 2 steps of log2 S <= 24 (96 u) and by two
roundings of its own.  entropy = ln2 (log2 S - A / S), A = sum 2^t t: as ln S, and A / S by
its terms' own 4 u |t| (1 + ln2 |t|) and twice s: E2 = sum p t^2.  Orders and ranks
are equal.
"""
import math

import numpy as np
import pytest
import torch

import medusa_speculative_decoding_02_gb300 as m
import paged_ref as ref
from medusa_speculative_decoding_02_gb300 import build as mbuild

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -24


@pytest.fixture(scope="module")
def dev():
    mbuild.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    d = torch.device("cuda:0")
    torch.cuda.set_device(d)
    return d


def check(out, x, tokens, top, temp):
    N, V = x.shape
    r = ref.logprobs(x.double().numpy(), tokens.numpy().astype(np.int64), top, temp)
    s = U * (4 + 3 * r["E1"] + V / 512 + 64)
    x64 = x.double().numpy()

    def near(got, want, d):
        with np.errstate(invalid="ignore", over="ignore"):
            # a value past the range of fp32 rounds to infinity
            want = np.where(np.isinf(want.astype(np.float32)), want.astype(np.float32), want)
            tol = 4 * U * d + (s if want.ndim == 1 else s[:, None]) + 96 * U + 3 * U * np.abs(want)
            ok = (got == want) | (np.abs(got - want) <= tol)
        assert ok.all(), (got[~ok][:4], want[~ok][:4])

    top_x = x64.max(1)
    near(out.logp.double().cpu().numpy(), r["logp"],
         np.abs(np.take_along_axis(x64, tokens.numpy().astype(np.int64)[:, None], 1)[:, 0] - top_x) / temp)
    assert (out.rank.cpu().numpy() == r["rank"]).all()
    assert (out.top_ids.cpu().numpy() == r["ids"]).all()
    near(out.top_logp.double().cpu().numpy(), r["top_logp"],
         np.abs(np.take_along_axis(x64, r["ids"], 1) - top_x[:, None]) / temp)
    tol = U * (4 * (r["E1"] + r["E2"]) + 96) + s * (1 + 2 * r["E1"]) + 3 * U * r["entropy"]
    err = np.abs(out.entropy.double().cpu().numpy() - r["entropy"])
    assert (err <= tol).all(), (err / tol).max()


def rows(g, N, V, dtype, std=2.0):
    x = torch.randn((N, V), generator=g) * std
    x[:, torch.randint(0, V, (4,), generator=g)] += 9.0
    return x.to(dtype)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("N,V,top,temp", [
    (1, 1, 1, 1.0), (1, 2, 0, 0.5), (3, 7, 7, 1.0), (2, 16, 16, 2.0), (5, 100, 5, 1.0), (1, 32000, 5, 1.0),
    (65, 32000, 16, 0.7), (3, 50257, 1, 1.0), (2, 128001, 16, 1.3), (7, 4099, 10, 1.0), (300, 515, 3, 1.0),
    (2, 262147, 4, 1.0), (17, 8193, 0, 0.9)])
def test_logprobs(dev, dtype, N, V, top, temp):
    g = torch.Generator().manual_seed(N + V + top)
    x = rows(g, N, V, dtype)
    tokens = torch.randint(0, V, (N,), generator=g, dtype=torch.int32)
    tokens[0] = int(x[0].float().argmax())
    if N > 1:
        tokens[1] = int(x[1].float().argmin())
    ws = m.new_workspace(m.WS_HEADER)
    out = m.token_logprobs(x.to(dev), tokens.to(dev), top, temperature=temp, ws=ws)
    check(out, x, tokens, top, temp)
    assert m.read_device_status(ws) == 0


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("V", [33, 5000, 32000, 70001])
def test_ties_and_orders(dev, dtype, V):
    """Rows of equal logits, of few values, sorted ones, and a token inside a run of ties."""
    g = torch.Generator().manual_seed(V)
    x = torch.zeros((9, V))
    x[1] = torch.randint(0, 3, (V,), generator=g).float()
    x[2] = torch.arange(V).float() / V * 20          # ascending: the best come last
    x[3] = -torch.arange(V).float() / V * 20
    x[4] = 1e-3 * torch.randn(V, generator=g)
    x[5, V // 2:] = 4.0                               # a plateau far down the row
    x[6, ::2] = -0.0                                  # -0 equals 0
    x[7] = torch.where(torch.rand(V, generator=g) < 0.001, 5.0, -3.0)
    x[8] = -3.0e38                                    # the type's lowest, about
    x = x.to(dtype)
    for at in (0, V - 1, V // 2, V // 2 + 3):
        tokens = torch.full((9,), at, dtype=torch.int32)
        out = m.token_logprobs(x.to(dev), tokens.to(dev), 16)
        check(out, x, tokens, 16, 1.0)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("V", [40, 32000, 90001])
def test_masked_vocabularies(dev, dtype, V):
    """-inf and the type's lowest value: probability zero; fewer tokens than alternatives."""
    g = torch.Generator().manual_seed(V)
    x = rows(g, 6, V, torch.float32)
    low = torch.finfo(dtype).min
    x[0, 5:] = -math.inf
    x[1, 7:] = low
    x[2] = low
    x[3, torch.rand(V, generator=g) < 0.9] = -math.inf
    x[4, : V - 1] = -math.inf                          # one token is possible: entropy 0
    x[5, ::3] = low
    x = x.to(dtype)
    for at in (0, 6, V - 1):
        tokens = torch.full((6,), at, dtype=torch.int32)
        out = m.token_logprobs(x.to(dev), tokens.to(dev), 12, temperature=0.8)
        check(out, x, tokens, 12, 0.8)
    assert out.entropy[4] == 0


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("V", [20, 32000])
def test_rows_that_are_not_numbers(dev, dtype, V):
    g = torch.Generator().manual_seed(V)
    x = rows(g, 5, V, torch.float32)
    x[0] = -math.inf                                   # nothing is possible
    x[1, 3] = math.nan
    x[2, V - 2] = math.inf
    x[3] = math.nan
    x = x.to(dtype)
    tokens = torch.tensor([4, 4, V - 2, 4, 4], dtype=torch.int32)
    ws = m.new_workspace(m.WS_HEADER)
    out = m.token_logprobs(x.to(dev), tokens.to(dev), 6, ws=ws)
    assert out.logp[0] == -math.inf and out.entropy[0] == 0 and out.rank[0] == 4
    assert out.top_ids[0].tolist() == list(range(6)) and (out.top_logp[0] == -math.inf).all()
    for r in (1, 2, 3):
        assert out.logp[r].isnan() and out.entropy[r].isnan() and out.top_logp[r].isnan().all()
    keep = [i for i in range(V) if i != 3]
    order = sorted(keep, key=lambda i: (-float(x[1, i]), i))
    assert out.top_ids[1].tolist() == order[:6] and out.rank[1] == order.index(4)
    assert out.rank[2] == 0 and out.top_ids[2, 0] == V - 2
    assert out.rank[3] == -1 and (out.top_ids[3] == -1).all()
    check(m.TokenLogprobs(out.logp[4:], out.entropy[4:], out.rank[4:], out.top_ids[4:], out.top_logp[4:]), x[4:],
          tokens[4:], 6, 1.0)
    # the token is the row's NaN; no token; ids outside the vocabulary
    tokens = torch.tensor([-1, 3, -1, 4, V], dtype=torch.int32)
    out = m.token_logprobs(x.to(dev), tokens.to(dev), 0, ws=ws)
    assert m.DEVICE_STATUS[m.read_device_status(ws)] == "bad token"
    assert out.rank.tolist() == [-1, -1, -1, -1, -1]
    assert out.logp[0] == 0 and out.logp[2] == 0 and out.logp[4] == 0 and out.logp[1].isnan()
    assert torch.isfinite(out.entropy[4])


@pytest.mark.parametrize("dtype", [BF, F32])
def test_strides_shapes_and_large_logits(dev, dtype):
    g = torch.Generator().manual_seed(5)
    for V, step in ((1001, 1001), (1001, 1003), (1000, 1304), (37, 64)):
        wide = rows(g, 12, step, dtype)
        x = wide[:, :V]
        tokens = torch.randint(0, V, (12,), generator=g, dtype=torch.int32)
        out = m.token_logprobs(wide.to(dev)[:, :V], tokens.to(dev), 4)
        check(out, x, tokens, 4, 1.0)
        got = m.token_logprobs(wide.to(dev).view(3, 4, step)[..., :V], tokens.view(3, 4).to(dev), 4)
        assert got.logp.shape == (3, 4) and got.top_ids.shape == (3, 4, 4)
        assert torch.equal(got.logp.flatten(), out.logp) and torch.equal(got.top_ids.flatten(0, 1), out.top_ids)
    x = (rows(g, 3, 2000, F32) * 1e4).to(dtype)
    tokens = torch.tensor([1, 2, 3], dtype=torch.int32)
    for temp in (1e-3, 1.0, 1e4):
        check(m.token_logprobs(x.to(dev), tokens.to(dev), 5, temperature=temp), x, tokens, 5, temp)


def test_captured_and_on_two_streams(dev):
    g = torch.Generator().manual_seed(8)
    x = rows(g, 33, 32000, BF).to(dev)
    tokens = torch.randint(0, 32000, (33,), generator=g, dtype=torch.int32).to(dev)
    want = m.token_logprobs(x, tokens, 7)
    ws = m.new_workspace(m.WS_HEADER)
    out = m.token_logprobs(x, tokens, 7, ws=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m.token_logprobs(x, tokens, 7, out=out, ws=ws)
    for t in (out.logp, out.rank, out.top_ids):
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [m.token_logprobs(x, tokens, 7, stream=s) for _ in range(10) for s in streams]
    torch.cuda.synchronize()
    for o in got + [out]:
        for name in ("logp", "entropy", "rank", "top_ids", "top_logp"):
            assert torch.equal(getattr(o, name), getattr(want, name)), name


def test_ranks_calibrate_a_static_tree(dev):
    """How often the true token has rank i under a head's logits is the table that
    build_tree_static takes."""
    g = torch.Generator().manual_seed(11)
    N, V, K, S = 400, 256, 3, 4
    log_a = torch.empty((K, S))
    for k in range(K):
        x = rows(g, N, V, BF)
        order = torch.sort(x.float(), dim=1, descending=True, stable=True).indices
        true = order.gather(1, torch.randint(0, 6 + 4 * k, (N, 1), generator=g))[:, 0].int()
        rank = m.token_logprobs(x.to(dev), true.to(dev)).rank.cpu()
        assert (order.gather(1, rank.long()[:, None])[:, 0] == true).all()
        for i in range(S):
            log_a[k, i] = math.log(max(float((rank == i).float().mean()), 1e-6))
    ids = torch.arange(K * S, dtype=torch.int32).view(1, K, S).to(dev)
    t = m.build_tree_static(torch.zeros(1, dtype=torch.int32, device=dev), ids, log_a.to(dev), [S] * K, 12)
    assert t.depth[0].max() >= 1 and (t.tokens >= 0).all()
