"""The binding's checks of the calls on a cache in pages, behind that of the device (no GPU
needed)."""
import pytest
import torch

import medusa_speculative_decoding_02_gb300 as m


@pytest.fixture
def any_device(monkeypatch):
    monkeypatch.setattr(m, "_launch_on", lambda ref, stream: (-1, 0))


def test_numbers_of_dimensions(any_device):
    """Tensors with too few or too many dimensions get the binding's own error."""
    i32 = torch.int32
    pool, tab, pre = torch.zeros(4, 16, 2, 64), torch.zeros(3, 5, dtype=i32), torch.zeros(3, dtype=i32)
    path, n, q = torch.zeros(3, 5, dtype=i32), torch.zeros(3, dtype=i32), torch.zeros(3, 1, 2, 64)
    mask = torch.zeros(3, 1, 1, dtype=torch.int64)
    for bad in (pool[0], pool[None], pool[0, 0, 0]):
        for call in (lambda: m.commit_paged(bad, bad, tab, pre, 9, path, n, 5),
                     lambda: m.chunk_attention_paged(q, bad, bad, tab, pre, 9),
                     lambda: m.tree_attention_paged(q, bad, bad, tab, pre, 9, mask),
                     lambda: m.paged_append(q, q, bad, bad, tab, pre, 9)):
            with pytest.raises(ValueError, match="pools"):
                call()
    for bad in (path[0], path[None]):
        with pytest.raises(ValueError, match="path"):
            m.commit_paged(pool, pool, tab, pre, 9, bad, n, 5)
    with pytest.raises(ValueError, match="logits"):
        m.token_logprobs(torch.tensor(1.0), torch.tensor(1, dtype=i32))
