"""Plain 64-bit references of the rotation, the 4-bit cache and the windowed
tree attention, from their definitions (numpy / torch float64)."""
import math

import numpy as np
import torch

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
E4M3 = np.array([m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
                 for e in range(16) for m in range(8)][:127])


def nearest_even(v, grid):
    """Index of the grid value nearest to v >= 0; a tie takes the even index."""
    up = np.clip(np.searchsorted(grid, v), 1, len(grid) - 1)
    lo, hi = v - grid[up - 1], grid[up] - v
    return np.where((lo < hi) | ((lo == hi) & (up % 2 == 1)), up - 1, up)


def quantize(x):
    """(codes 0..15, scale bytes) of x [..., dh] float64, blocks of 16."""
    b = np.asarray(x, np.float64).reshape(*x.shape[:-1], x.shape[-1] // 16, 16)
    fine = np.isfinite(b).all(-1)
    b = np.where(fine[..., None], b, 0.0)
    sb = nearest_even(np.abs(b).max(-1) / 6.0, E4M3)
    s = E4M3[sb]
    ratio = np.abs(b) / np.where(s > 0, s, 1.0)[..., None]
    c = nearest_even(ratio, E2M1) | np.where(b < 0, 8, 0)
    c = np.where((s > 0)[..., None], c, 0)
    return c.reshape(x.shape).astype(np.uint8), np.where(fine, sb, 0x7f).astype(np.uint8)


def pack_rows(x):
    """Row bytes [..., row bytes] (padding 0) of x [..., Hkv, dh]."""
    Hkv, dh = x.shape[-2:]
    c, s = quantize(x)
    c = c.reshape(*x.shape[:-2], Hkv * dh)
    s = s.reshape(*x.shape[:-2], Hkv * dh // 16)
    rows = np.concatenate([c[..., 0::2] | (c[..., 1::2] << 4), s], -1)
    pad = (-rows.shape[-1]) % 16
    return np.concatenate([rows, np.zeros((*rows.shape[:-1], pad), np.uint8)], -1)


def unpack_rows(rows, Hkv, dh):
    """Values float64 [..., Hkv, dh] of row bytes."""
    n = Hkv * dh // 2
    c = np.stack([rows[..., :n] & 15, rows[..., :n] >> 4], -1).reshape(*rows.shape[:-1], 2 * n)
    v = np.where(c & 8, -1.0, 1.0) * E2M1[c & 7]
    sb = rows[..., n:n + n // 8]
    s = np.where((sb & 127) == 127, np.nan, E4M3[np.minimum(sb & 127, 126)] * np.where(sb & 128, -1, 1))
    return (v * np.repeat(s, 16, -1)).reshape(*rows.shape[:-1], Hkv, dh)


def rope(x, pos, inv_freq, w, eps, norm, interleaved):
    """x [B,R,H,dh] float64, pos [B,R]; returns (result, magnitude), where
    magnitude is |y_a| + |y_b| of the element's pair (its own |y| past rot)."""
    x = np.asarray(x, np.float64)
    if norm:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
        if w is not None:
            x = x * np.asarray(w, np.float64)
    rot = 2 * len(inv_freq)
    t = pos.astype(np.float64)[..., None] * np.asarray(inv_freq, np.float64)
    cos, sin = np.cos(t)[:, :, None], np.sin(t)[:, :, None]
    a = slice(0, rot, 2) if interleaved else slice(0, rot // 2)
    b = slice(1, rot, 2) if interleaved else slice(rot // 2, rot)
    y, mag = x.copy(), np.abs(x)
    y[..., a], y[..., b] = x[..., a] * cos - x[..., b] * sin, x[..., a] * sin + x[..., b] * cos
    mag[..., a] = mag[..., b] = np.abs(x[..., a]) + np.abs(x[..., b])
    return y, mag


def tree(B, R, rs, max_depth=8):
    """Random canonical trees: masks uint64 [B,R,W] (as int64), depth int32."""
    W = (R + 63) // 64
    mask, depth = np.zeros((B, R, W), np.uint64), np.zeros((B, R), np.int32)
    for b in range(B):
        par, dep = [-1], [0]
        for i in range(1, R):
            p = int(rs.randint(0, i))
            while dep[p] >= max_depth:
                p = par[p]
            par.append(p)
            dep.append(dep[p] + 1)
        order = sorted(range(R), key=lambda i: (dep[i], i))
        place = {o: n for n, o in enumerate(order)}
        for n, o in enumerate(order):
            depth[b, n] = dep[o]
            if par[o] >= 0:
                mask[b, n] = mask[b, place[par[o]]]
            mask[b, n, n // 64] |= np.uint64(1) << np.uint64(n % 64)
    return torch.from_numpy(mask.view(np.int64)), torch.from_numpy(depth)


def visible(P, R, mask, depth, window, sinks):
    """bool [R, P+R] of one sequence (mask int64 [R,W], depth [R])."""
    bits = np.unpackbits(mask.numpy().view(np.uint8), axis=-1, bitorder="little")[:, :R] > 0
    d = depth.numpy().astype(np.int64)
    place = np.concatenate([np.arange(P), P + d])
    see = np.concatenate([np.ones((R, P), bool), bits], 1)
    if window:
        see &= (place[None] < sinks) | ((P + d)[:, None] - place[None] < window)
    return see


def attention(q, ks, vs, prefix, mask, depth, window, sinks, scale):
    """q [B,R,H,dh]; ks, vs lists of [slots,Hkv,dh] (float64); returns (out, A,
    E): A = sum_j w_j |v_j| / sum_j w_j elementwise, E [B,R,H] = the largest
    sum_c |q_c k_c| * scale over a row's visible keys."""
    B, R, H, dh = q.shape
    out = torch.zeros(q.shape, dtype=torch.float64)
    A, E = torch.zeros_like(out), torch.zeros((B, R, H), dtype=torch.float64)
    for b in range(B):
        P = int(prefix[b])
        see = visible(P, R, mask[b].cpu(), depth[b].cpu(), window, sinks)
        used = np.flatnonzero(see.any(0))
        if not len(used):
            continue
        hide = torch.from_numpy(~see[:, used])
        Hkv = ks[b].shape[1]
        for h in range(H):
            g = h // (H // Hkv)
            k, v = ks[b][used, g].double().cpu(), vs[b][used, g].double().cpu()
            x = q[b, :, h].double().cpu()
            s = (x @ k.T * scale).masked_fill(hide, -math.inf)
            top = s.amax(1, keepdim=True)
            w = torch.exp(s - torch.where(torch.isfinite(top), top, torch.zeros_like(top)))
            w = torch.where(hide, torch.zeros_like(w), w)
            total = w.sum(1, keepdim=True)
            w = w / torch.where(total == 0, torch.ones_like(total), total)
            # a key that a row does not see adds nothing to it, whatever it holds
            safe = torch.where(torch.isfinite(v), v, torch.zeros_like(v))
            o = w @ safe
            for j, c in (~torch.isfinite(v)).nonzero().tolist():
                o[:, c] += torch.where(hide[:, j], 0.0, w[:, j] * v[j, c])
            out[b, :, h], A[b, :, h] = o, w @ safe.abs()
            E[b, :, h] = (x.abs() @ k.abs().T * scale).masked_fill(hide, 0.0).amax(1)
    return out, A, E
