"""Rows that clusters of CTAs share, whose ends are read beside the whole blocks by some threads
of a warp, again and again and on two streams at the same time."""
import pytest
import torch

import medusa_speculative_decoding_02_gb300 as m
from test_gpu_logprobs import BF, F32, check, dev, rows  # noqa: F401

pytestmark = pytest.mark.gpu

NAMES = ("logp", "entropy", "rank", "top_ids", "top_logp")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("N", [3, 60])
def test_ends_of_rows_in_clusters(dev, dtype, N):
    g = torch.Generator().manual_seed(N)
    per = 16 // (2 if dtype == BF else 4)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for off in range(per):
        V = 33000 + 3 * off
        flat = rows(g, 1, off + N * V, dtype)[0]
        x = flat[off:].view(N, V)
        tokens = torch.randint(0, V, (N,), generator=g, dtype=torch.int32)
        tokens[0], tokens[1], tokens[2] = 0, V - 1, V - 2
        xd, td = flat.to(dev)[off:].view(N, V), tokens.to(dev)
        want = m.token_logprobs(xd, td, 5)
        torch.cuda.synchronize()
        got = [m.token_logprobs(xd, td, 5, stream=s) for _ in range(25) for s in streams]
        torch.cuda.synchronize()
        for o in got:
            for name in NAMES:
                assert torch.equal(getattr(o, name), getattr(want, name)), name
        check(m.TokenLogprobs(*(getattr(want, n)[:3] for n in NAMES)), x[:3], tokens[:3], 5, 1.0)
