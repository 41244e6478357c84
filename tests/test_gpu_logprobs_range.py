"""Log probabilities at the ends of what the call takes, on the GPU, against 64 bits.

Tolerances are those of test_gpu_logprobs.
"""
import math

import pytest
import torch

import medusa_speculative_decoding_02_gb300 as m
from test_gpu_logprobs import BF, F32, check, dev, rows  # noqa: F401

pytestmark = pytest.mark.gpu

# A CTA shares a row with others at a few rows and takes whole rows at many: the same rows
# are given once, and again and again.
REPEATS = (1, 90)


def check_repeated(dev, x, tokens, top, temp):
    n = x.shape[0]
    for reps in REPEATS:
        out = m.token_logprobs(x.to(dev).repeat(reps, 1), tokens.to(dev).repeat(reps), top, temperature=temp)
        each = [t.unflatten(0, (reps, n)) for t in (out.logp, out.entropy, out.rank, out.top_ids, out.top_logp)]
        for t in each:
            assert torch.equal(t.nan_to_num(), t[:1].expand_as(t).nan_to_num())
        last = m.TokenLogprobs(*(t[-1] for t in each))
        check(last, x, tokens, top, temp)
        # a logit of -inf, and no other that fp32 can answer for, has a log probability of -inf
        for lp, ids in ((last.logp[:, None].cpu(), tokens[:, None]), (last.top_logp.cpu(), last.top_ids.cpu())):
            at = x.double().gather(1, ids.long())
            far = (at - x.double().amax(1, keepdim=True)) / temp < -3.3e38
            assert (lp[at == -math.inf] == -math.inf).all() and torch.isfinite(lp[~far]).all()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("low", [-1e4, -1e9, -1e10, -1e12, -1e20, -1e28])
@pytest.mark.parametrize("temp", [0.7, 1.0])
def test_far_logits(dev, dtype, low, temp):
    """Tokens that are masked by a large negative number, in stretches and here and there: their
    weight is nothing, whatever the number; and rows of such numbers alone."""
    V = 32000
    g = torch.Generator().manual_seed(V)
    x = rows(g, 6, V, F32)
    x[0, 1000:] = low                                  # the first tokens are possible
    x[1, : V - 1000] = low                             # the last
    x[2, torch.rand(V, generator=g) < 0.999] = low
    x[3] = low                                         # equal ones
    x[4] = low * (1 + torch.rand(V, generator=g))
    x[5] = -low * (1 + torch.rand(V, generator=g))
    x = x.to(dtype)
    for at in (0, V - 1):
        check_repeated(dev, x, torch.full((6,), at, dtype=torch.int32), 5, temp)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("V", [8, 40, 1001, 32000])
@pytest.mark.parametrize("temp", [1e17, 1e19, 1e25, 1e28, 4e28, 1e29, 9e29])
def test_high_temperatures(dev, dtype, V, temp):
    """However high the temperature, -inf is a token of probability zero, and what lies behind a
    row in its last chunk is none at all."""
    g = torch.Generator().manual_seed(V)
    x = rows(g, 7, V, F32)
    x[1] = 1.0
    x[2, : V - 1] = -math.inf                          # one token is possible
    x[3, 5:] = -math.inf
    x[4, torch.rand(V, generator=g) < 0.5] = -math.inf
    x[4, 3] = 2.0
    x[5] = torch.rand(V, generator=g) * -3.0e38        # as far apart as the types reach
    x[6] = torch.rand(V, generator=g) * -4e29
    x = x.to(dtype)
    for at in (3, V - 1):
        check_repeated(dev, x, torch.full((7,), at, dtype=torch.int32), 5, temp)


@pytest.mark.parametrize("temp", [1.0, 4.0, 1e3, 1e30 * 0.999])
def test_differences_past_the_type(dev, temp):
    """fp32 logits further apart than fp32 reaches: their log probabilities are finite where the
    temperature makes them so."""
    g = torch.Generator().manual_seed(3)
    for V in (10, 5000):
        x = (torch.rand((3, V), generator=g) * 2 - 1) * 3.3e38
        x[1, 1:] = -3.3e38
        x[2, 2] = -math.inf
        for at in (1, V - 1):
            check_repeated(dev, x, torch.full((3,), at, dtype=torch.int32), 4, temp)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("V", [59599, 400_000, 3_000_001])
def test_sums_of_rows_by_passes(dev, dtype, V):
    """Rows that take plain passes (the token is impossible, or there are fewer possible ones than
    alternatives) sum as exactly as the others, however long they are."""
    g = torch.Generator().manual_seed(V)
    x = torch.randn((3, V), generator=g) * 0.3
    x[1] = torch.rand(V, generator=g) * 1e-3
    x[2] = torch.where(torch.rand(V, generator=g) < 0.5, 0.7, 0.1)
    x[:, 5] = -math.inf
    x = x.to(dtype)
    check_repeated(dev, x, torch.full((3,), 5, dtype=torch.int32), 6, 0.9)
