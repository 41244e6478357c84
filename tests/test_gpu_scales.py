"""Attention with scales and scores at the ends of fp32, on the GPU, against 64 bits.

Tolerances are those of test_gpu_paged.
"""
import numpy as np
import pytest
import torch

import cache_ops_ref
import medusa_speculative_decoding_02_gb300 as m
import paged_ref as ref
from test_gpu_paged import BF, F32, Case, check, dev  # noqa: F401

pytestmark = pytest.mark.gpu

SHAPES = [(1, 1, 1), (3, 4, 2), (8, 2, 1), (17, 2, 2), (65, 2, 2), (65, 4, 1), (150, 2, 1)]


def far_case(dtype, R, H, Hkv):
    """Keys and queries of about 1e18: scores of up to 2.3e38 before the scale."""
    c = Case(R + H, (200,), (R,), Hkv, 128, 16, dtype)
    u = torch.rand(c.kp.shape[:3], generator=c.g) * 2 - 1
    c.kp = (u[..., None] * 1.8e18 * torch.ones(128)).to(dtype)
    return c, torch.full((1, R, H, 128), 1e18).to(dtype)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("R,H,Hkv", SHAPES)
@pytest.mark.parametrize("scale", [4e-38, 6e-39, 1e-39, 3e-41, 1e-45])
def test_small_scales(dev, dtype, R, H, Hkv, scale):
    """A scale below the normal numbers is the scale."""
    c, q = far_case(dtype, R, H, Hkv)
    scale = float(np.float32(scale))
    got = m.chunk_attention_paged(q.to(dev), *c.to(dev), scale=scale)
    check(got, q, c, lambda b: ref.causal(200, R), scale=scale)


@pytest.mark.parametrize("R,H,Hkv", SHAPES)
def test_small_scales_in_one_piece(dev, R, H, Hkv):
    """The same over caches in one piece."""
    scale = float(np.float32(1e-39))
    c, q = far_case(BF, R, H, Hkv)
    k, v = (ref.sequence(p, c.tab, 0, 200 + R).to(BF).to(dev) for p in (c.kp, c.vp))
    mask, _ = cache_ops_ref.tree(1, R, np.random.RandomState(R))
    got = m.tree_attention_window(q.to(dev), m.cache_pointers([k], dev), m.cache_pointers([v], dev),
                                  c.to(dev)[3], 200, mask.to(dev), Hkv=Hkv, scale=scale)
    check(got, q, c, lambda b: ref.tree_sees(200, R, mask[b]), scale=scale)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("R,H,Hkv", SHAPES)
@pytest.mark.parametrize("power", [16, 24, 34, 50, 90])
def test_far_scores(dev, dtype, R, H, Hkv, power):
    """Scores so large that each row's weights are 1 for its best keys and 0 for the others: whole
    multiples of 2^power, which fp32 holds.  The row is the mean of the best keys' V."""
    c = Case(R + H, (300,), (R,), Hkv, 64, 16, dtype)
    n = 300 + R
    c.kp = torch.zeros_like(c.kp)
    c.kp[..., 0] = torch.randint(-90, 90, c.kp.shape[:3], generator=c.g).to(dtype)
    c.kp[..., 1] = torch.randint(0, 2, c.kp.shape[:3], generator=c.g).to(dtype) * 0.5
    c.vp = torch.randint(-8, 8, c.vp.shape, generator=c.g).to(dtype)
    q = torch.zeros(1, R, H, 64)
    q[..., 0] = 2.0 ** power * 3
    q[..., 1] = 2.0 ** power
    q = q.to(dtype)
    got = m.chunk_attention_paged(q.to(dev), *c.to(dev), scale=1.0).double().cpu()
    k, v = (ref.sequence(p, c.tab, 0, n) for p in (c.kp, c.vp))
    see = ref.causal(300, R)
    for h in range(H):
        g = h // (H // Hkv)
        s = (q[0, :, h].double() @ k[:, g].T).masked_fill(~see, -float("inf"))
        w = (s == s.amax(1, keepdim=True)).double()
        y = w @ v[:, g] / w.sum(1, keepdim=True)
        # Sums of V, small whole numbers, are exact.  They are multiplied by 1 / (number of best
        # keys), which is rounded to u = 2^-24 as the product is; two halves of the keys are
        # added after that, one more rounding: 3 u of A = mean |V| in all.  Then the rounding to
        # the type.
        A = w @ v[:, g].abs() / w.sum(1, keepdim=True)
        tol = torch.finfo(dtype).eps / 2 * y.abs() + 2.0 ** -22 * A
        assert ((got[0, :, h] - y).abs() <= tol).all(), (h, (got[0, :, h] - y).abs().max())
