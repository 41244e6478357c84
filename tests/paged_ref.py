"""Plain 64-bit references of the calls on a cache in pages and of the log
probabilities of tokens, from their definitions."""
import math

import numpy as np
import torch


def pool(g, pages, page, Hkv, dh, dtype, std=1.0):
    return (torch.randn((pages, page, Hkv, dh), generator=g) * std).to(dtype)


def table(g, need, spare=3):
    """Page numbers int32 [B, most] of sequences that need `need[b]` pages, shuffled
    over a pool (entries that no slot needs hold a number outside it); returns it
    and the pool's size."""
    pages = sum(need) + spare
    order = torch.randperm(pages, generator=g).tolist()
    t = torch.full((len(need), max(max(need), 1)), -77, dtype=torch.int32)
    for b, n in enumerate(need):
        t[b, :n] = torch.tensor([order.pop() for _ in range(n)], dtype=torch.int32)
    return t, pages


def spots(tab, b, page, first, count):
    """(pages, rows) of slots first .. first + count - 1 of sequence b."""
    slot = torch.arange(first, first + count)
    return tab[b].long()[slot // page], slot % page


def sequence(p, tab, b, slots):
    """The rows of the first `slots` slots of sequence b, float64 [slots, Hkv, dh]."""
    page = p.shape[1]
    i, r = spots(tab, b, page, 0, slots)
    return p[i, r].double()


def causal(P, n):
    """bool [n, P + n]"""
    return torch.arange(P + n)[None] <= P + torch.arange(n)[:, None]


def tree_sees(P, R, mask):
    """bool [R, P + R] of one tree (mask int64 [R, W])."""
    bits = np.unpackbits(mask.numpy().view(np.uint8), axis=-1, bitorder="little")[:, :R] > 0
    return torch.cat([torch.ones((R, P), dtype=torch.bool), torch.from_numpy(bits)], 1)


def attention(q, k, v, see, scale):
    """q [n,H,dh], k, v [N,Hkv,dh] float64, see bool [n,N]; returns (out, A, E): A =
    sum_j w_j |v_j| elementwise, E [n,H] = the largest sum_c |q_c k_c| * scale over a
    row's visible keys."""
    n, H, dh = q.shape
    Hkv = k.shape[1]
    out, A = torch.zeros_like(q), torch.zeros_like(q)
    E = torch.zeros((n, H), dtype=torch.float64)
    used = see.any(0)
    k, v, hide = k[used], v[used], ~see[:, used]
    if not k.shape[0]:
        return out, A, E
    safe = torch.where(torch.isfinite(v), v, torch.zeros_like(v))
    odd = (~torch.isfinite(v)).nonzero().tolist()
    for h in range(H):
        g = h // (H // Hkv)
        s = (q[:, h] @ k[:, g].T * scale).masked_fill(hide, -math.inf)
        top = s.amax(1, keepdim=True)
        w = torch.exp(s - torch.where(torch.isfinite(top), top, torch.zeros_like(top)))
        w = torch.where(hide, torch.zeros_like(w), w)
        total = w.sum(1, keepdim=True)
        w = w / torch.where(total == 0, torch.ones_like(total), total)
        o = w @ safe[:, g]
        for j, gg, c in odd:  # a key that a row does not see adds nothing to it
            if gg == g:
                o[:, c] += torch.where(hide[:, j], 0.0, w[:, j] * v[j, g, c])
        out[:, h], A[:, h] = o, w @ safe[:, g].abs()
        E[:, h] = (q[:, h].abs() @ k[:, g].abs().T * scale).masked_fill(hide, 0.0).amax(1)
    return out, A, E


def logprobs(x, tokens, top, temp):
    """x [N,V] float64 of finite logits and -inf; returns a dict with logp, entropy,
    rank, ids, top_logp, and for tolerances E1 = sum p |t|, E2 = sum p t^2, t the
    distance to the largest logit in base 2."""
    N, V = x.shape
    order = np.lexsort((np.broadcast_to(np.arange(V), x.shape), -x), axis=1)
    top_x = x.max(1, keepdims=True)
    with np.errstate(invalid="ignore", divide="ignore", over="ignore"):
        d = (x - top_x) / temp
        w = np.exp(d)
        S = w.sum(1, keepdims=True)
        lp = d - np.log(S)
        p = w / S
        part = np.where(p > 0, p * lp, 0.0)
        t = np.where(p > 0, d, 0.0) / math.log(2)
    rank = np.empty(N, np.int64)
    for i in range(N):
        rank[i] = np.flatnonzero(order[i] == tokens[i])[0]
    take = np.take_along_axis
    return dict(logp=take(lp, tokens[:, None], 1)[:, 0], entropy=-part.sum(1), rank=rank,
                ids=order[:, :top], top_logp=take(lp, order[:, :top], 1),
                E1=(p * np.abs(t)).sum(1), E2=(p * t * t).sum(1))
