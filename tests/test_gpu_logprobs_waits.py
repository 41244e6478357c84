"""Waits of the log probabilities that run out, on the GPU, without a hung or faulted GPU: with
the wait budget at 0 every wait for logits gives up at once."""
import pytest
import torch

import medusa_speculative_decoding_02_gb300 as m
from test_gpu_logprobs import BF, F32, check, dev, rows  # noqa: F401

pytestmark = pytest.mark.gpu


def status(ws):
    return m.DEVICE_STATUS[m.read_device_status(ws)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("N,V,top", [(1, 32000, 5), (3, 50257, 0), (65, 32000, 16), (200, 8200, 3), (1400, 8193, 4),
                                     (2000, 515, 10)])
def test_waits_that_run_out(dev, dtype, N, V, top):
    """The status says so, no row is answered from what was not read, and the same call on the
    same buffers is right afterwards."""
    g = torch.Generator().manual_seed(N)
    x = rows(g, N, V, dtype)
    x[N // 2, 4:] = -float("inf")                      # a row for the plain passes
    tokens = torch.randint(0, V, (N,), generator=g, dtype=torch.int32)
    tokens[N // 2] = 1
    if N > 60:
        tokens[7] = -1
    xd, td = x.to(dev), tokens.to(dev)
    want = m.token_logprobs(xd, td, top)
    ws = m.new_workspace(m.WS_HEADER)
    out = m.token_logprobs(xd, td, top, ws=ws)
    torch.cuda.synchronize()
    budget = m.wait_budget()
    try:
        m.set_wait_budget(0)
        for t in (out.logp, out.entropy, out.rank, out.top_ids, out.top_logp):
            t.fill_(3)
        m.token_logprobs(xd, td, top, out=out, ws=ws)
        torch.cuda.synchronize()
    finally:
        m.set_wait_budget(budget)
    assert status(ws) == "timeout"
    for t in (out.logp, out.entropy, out.top_logp):
        assert t.isnan().all()
    for t in (out.rank, out.top_ids):
        assert (t == -1).all()
    m.clear_device_status(ws)
    m.token_logprobs(xd, td, top, out=out, ws=ws)
    assert status(ws) == "ok"
    for name in ("logp", "entropy", "rank", "top_ids", "top_logp"):
        assert torch.equal(getattr(out, name), getattr(want, name)), name
    some = slice(0, 3)
    check(m.TokenLogprobs(*(getattr(out, n)[some] for n in ("logp", "entropy", "rank", "top_ids", "top_logp"))),
          x[some], tokens[some].clamp(min=0), top, 1.0)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_rows_that_wait_for_nothing(dev, dtype):
    """Rows shorter than a 16-byte block are read without a wait."""
    g = torch.Generator().manual_seed(1)
    x = rows(g, 9, 3, dtype)
    tokens = torch.randint(0, 3, (9,), generator=g, dtype=torch.int32)
    ws = m.new_workspace(m.WS_HEADER)
    budget = m.wait_budget()
    try:
        m.set_wait_budget(0)
        out = m.token_logprobs(x.to(dev), tokens.to(dev), 2, ws=ws)
        torch.cuda.synchronize()
    finally:
        m.set_wait_budget(budget)
    assert status(ws) == "ok"
    check(out, x, tokens, 2, 1.0)


def test_rows_by_passes_are_waited_for(dev):
    """Where every row takes plain passes, milliseconds each, the copies of later rows wait for
    them: longer than the budget of a wait in which nothing goes on."""
    N, V, top = 3100, 128256, 10
    x = torch.full((N, V), -float("inf"), dtype=BF, device=dev)
    x[:, :4] = torch.randn((N, 4), device=dev).to(BF)
    tokens = torch.randint(0, 4, (N,), device=dev).int()
    ws = m.new_workspace(m.WS_HEADER)
    budget = m.wait_budget()
    try:
        m.set_wait_budget(10000)
        out = m.token_logprobs(x, tokens, top, ws=ws)
        torch.cuda.synchronize()
    finally:
        m.set_wait_budget(budget)
    assert status(ws) == "ok"
    some = slice(N - 3, N)
    check(m.TokenLogprobs(*(getattr(out, n)[some] for n in ("logp", "entropy", "rank", "top_ids", "top_logp"))),
          x[some].cpu(), tokens[some].cpu(), top, 1.0)
    assert (out.top_ids[:, 4:] == torch.arange(4, top, device=dev)).all()
