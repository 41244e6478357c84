"""Typical acceptance over vocabularies that are masked by large negative numbers, on the GPU,
against the oracle."""
import numpy as np
import pytest

import oracle
import synth
import medusa_speculative_decoding_02_gb300 as m
from test_gpu_parity import check_posterior, dev, oracle_tree_for, run_posterior  # noqa: F401

pytestmark = pytest.mark.gpu

LOWEST = float(np.finfo(np.float32).min)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("low", [-1e4, -1e9, -1e10, -1e12, -1e20, -1e30, LOWEST, -np.inf])
@pytest.mark.parametrize("temp", [1.0, 0.7])
def test_masked_stretches(dev, dtype, low, temp):
    """Whatever the number, a masked token has no weight: the entropies and the acceptance are those
    of the possible tokens."""
    cfg = synth.v7b()
    rng = np.random.default_rng(11)
    ot = oracle_tree_for(rng, cfg.s, cfg.n, 1, cfg.prefix)
    logits = synth.base_logits(cfg)
    synth.plant_chain(logits, ot["tokens"], ot["parent"], ot["depth"], 4, rng)
    keep = np.zeros(logits.shape[-1], bool)
    keep[:800] = keep[20000:20400] = True
    keep[ot["tokens"][0][:40]] = True
    logits[..., ~keep] = low
    lg = synth.cast(logits, dtype)
    gp = run_posterior(dev, lg, ot, cfg.K, m.TYPICAL, temp=temp)
    op = check_posterior(gp, lg, ot, cfg.K, m.TYPICAL, 0.09, 0.3, temp)
    assert int(op["accept_len"][0]) >= 4


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("low", [-3e9, -1e12, -1e30, LOWEST, -np.inf])
def test_rows_without_a_possible_token(dev, dtype, low):
    """Rows that are masked altogether accept nothing."""
    cfg = synth.tiny()
    ot = oracle_tree_for(np.random.default_rng(1), cfg.s, cfg.n, 1, cfg.prefix, cfg.V)
    lg = synth.cast(np.full((1, cfg.R, cfg.V), low, np.float32), dtype)
    gp = run_posterior(dev, lg, ot, cfg.K, m.TYPICAL)
    assert int(gp.accept_len[0]) == 0 and (gp.accept[0, 1:] == 0).all()
    assert int(gp.next_token[0]) == 0
