"""What is measured of the verification pass's attention block, and its plain form.

Four operators, in the order in which a decoding step calls them:

  rope          per-head RMS norms of queries and keys and the position
                rotation in one pass (``append``: the K and V rows go straight
                into their cache slots)
  kv4_append    K and V rows into a cache held in 4 bits, read back as values
  window        tree attention with a sliding window and first tokens (sinks)
                that stay visible, grouped KV heads
  kv4_attn      tree attention over the 4-bit cache, with or without a window

``run`` computes the plain form with elementary torch operations where ``own``
is false, and makes the framework's calls where it is true.  ``exact`` is the
definition in 64 bits.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------- cases ---

def listed():
    return [
        # the 7B step's 65 tree rows (64 nodes and the root), 32 heads, rotation
        # only (that model has no q/k norms), rows appended to the cache
        dict(name="rope_append_step", op="rope", B=1, R=65, H=32, Hkv=32, dh=128, rot=128,
             dtype="bf16", norm=False, inter=False, append=True, ragged=False, P=1024),
        # plain decoding: one token for each of eight sequences, grouped heads
        dict(name="rope_single", op="rope", B=8, R=1, H=32, Hkv=8, dh=128, rot=128,
             dtype="bf16", norm=True, inter=False, append=False, ragged=False, P=4000),
        # prompts of uneven length entering the cache, far positions, partial rotation
        dict(name="rope_prompt", op="rope", B=2, R=4093, H=32, Hkv=8, dh=128, rot=64,
             dtype="bf16", norm=True, inter=False, append=True, ragged=True, P=100003),
        # the step's rows into the 4-bit cache
        dict(name="kv4_append_step", op="kv4_append", B=1, R=65, Hkv=32, dh=128, dtype="bf16",
             ragged=False, P=1024),
        # prompts of uneven length into the 4-bit cache
        dict(name="kv4_append_prompt", op="kv4_append", B=4, R=4001, Hkv=8, dh=128, dtype="bf16",
             ragged=True, P=0),
        # the 7B step with a 1024-token window and four sinks
        dict(name="window_step", op="window", B=1, R=65, H=32, Hkv=32, dh=128, P=4096,
             window=1024, sinks=4, dtype="bf16"),
        # a ragged batch of eight, grouped heads, long contexts behind a 4096 window
        dict(name="window_batch", op="window", B=8, R=65, H=32, Hkv=8, dh=128, P=16384,
             window=4096, sinks=4, dtype="bf16"),
        # plain decoding of eight sequences, an odd window
        dict(name="window_single", op="window", B=8, R=1, H=32, Hkv=8, dh=128, P=20000,
             window=2047, sinks=64, dtype="bf16"),
        # the 7B step over 8192 prefix slots in 4 bits
        dict(name="kv4_attn_step", op="kv4_attn", B=1, R=65, H=32, Hkv=32, dh=128, P=8192,
             window=0, sinks=0, dtype="bf16"),
        # the ragged batch of eight 7B sequences, prefixes up to 4096
        dict(name="kv4_attn_batch", op="kv4_attn", B=8, R=65, H=32, Hkv=32, dh=128, P=4096,
             window=0, sinks=0, dtype="bf16"),
        # plain decoding of eight long sequences, grouped heads
        dict(name="kv4_attn_single", op="kv4_attn", B=8, R=1, H=32, Hkv=8, dh=128, P=32768,
             window=0, sinks=0, dtype="bf16"),
        # the small float32 step: odd prefix, window shorter than the tree is deep
        dict(name="kv4_attn_f32", op="kv4_attn", B=2, R=15, H=4, Hkv=2, dh=64, P=337,
             window=3, sinks=5, dtype="f32"),
    ]


HEADS = ((32, 32), (40, 40), (32, 8), (28, 4), (8, 8), (6, 3), (5, 1), (1, 1))


def _logint(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("rope", "kv4_append", "window", "kv4_attn"))
    H, Hkv = rng.choice(HEADS)
    dh = rng.choice((64, 128, 128))
    dtype = rng.choice(("bf16", "bf16", "bf16", "f32"))
    B = rng.randint(1, 8)
    if op == "rope":
        R = _logint(rng, 1, min(4096 // B, 40_000_000 // (B * (H + Hkv) * dh)))
        return dict(op=op, B=B, R=R, H=H, Hkv=Hkv, dh=dh, rot=rng.choice((dh, dh, dh // 2, 16)),
                    dtype=dtype, norm=rng.random() < 0.6, inter=rng.random() < 0.4,
                    append=rng.random() < 0.5, ragged=rng.random() < 0.5,
                    P=rng.choice((0, _logint(rng, 1, 200000))))
    if op == "kv4_append":
        R = _logint(rng, 1, 4096 // B)
        return dict(op=op, B=B, R=R, Hkv=Hkv, dh=dh, dtype=dtype, ragged=rng.random() < 0.5,
                    P=rng.choice((0, _logint(rng, 1, 4096))))
    R = rng.choice((1, 2, 17, 33, 64, 65, 129, rng.randint(1, 256)))
    if dtype == "f32":
        H, Hkv = rng.choice(((8, 8), (6, 3), (5, 1), (1, 1), (4, 2)))
        R, P = min(R, 65), rng.choice((0, _logint(rng, 1, 2048)))
    else:
        P = rng.choice((0, _logint(rng, 1, 16384), _logint(rng, 64, 16384)))
        if B * Hkv > 64:
            P = min(P, 4096)
        if B * H > 64:
            R = min(R, 65)
    window = _logint(rng, 1, 4096)
    sinks = rng.choice((0, 1, 4, 17, 64, 300))
    if op == "kv4_attn" and rng.random() < 0.5:
        window, sinks = 0, 0
    # no more pairs of a row and a slot than the largest listed case has
    while B * H * R * (min(P, window + sinks) if window else P) > 60_000_000:
        P //= 2
    return dict(op=op, B=B, R=R, H=H, Hkv=Hkv, dh=dh, P=P, window=window, sinks=sinks, dtype=dtype)


# ------------------------------------------------------------------ shapes ---

def _torch_dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _size(case):
    return 2 if case["dtype"] == "bf16" else 4


def _prefixes(case):
    """Prefix length of each sequence: the first the longest, the others uneven."""
    P, B = case["P"], case["B"]
    return [P - (P * b * 7) // (B * 8) for b in range(B)]


def _rows(case):
    """Rows of each sequence of a ragged call (the first has all of them)."""
    R, B = case["R"], case["B"]
    if not case["ragged"]:
        return [R] * B
    return [max(1, R - (R * b * 5) // (B * 6)) for b in range(B)]


def _row_bytes(Hkv, dh):
    return (Hkv * dh // 2 + Hkv * dh // 16 + 15) // 16 * 16


def _seen_slots(case, P):
    """Cache slots that at least one row of a sequence sees (as a root does)."""
    if case["window"] == 0:
        return P + case["R"]
    lo = max(0, P - case["window"] + 1)
    return min(case["sinks"], lo) + P - lo + case["R"]


def work(case):
    B, R, dh, es = case["B"], case["R"], case["dh"], _size(case)
    if case["op"] == "rope":
        n = sum(_rows(case)) * (case["H"] + case["Hkv"]) * dh
        v = sum(_rows(case)) * case["Hkv"] * dh if case["append"] else 0
        return {"bytes": 2 * es * (n + v) + 4 * B * R, "flops": 10 * n}
    if case["op"] == "kv4_append":
        n = 2 * sum(_rows(case)) * case["Hkv"] * dh
        # the rows in, 9/16 byte an element written and read back, the values out
        return {"bytes": n * es + n * 9 // 16 * 2 + n * es, "flops": 6 * n}
    seen = sum(_seen_slots(case, P) for P in _prefixes(case))
    kv = 2 * seen * case["Hkv"] * dh
    kv = kv * 9 // 16 if case["op"] == "kv4_attn" else kv * es
    return {"bytes": kv + 2 * B * R * case["H"] * dh * es + B * R * 8 * ((R + 63) // 64),
            "flops": 4 * dh * case["H"] * R * seen}


# ------------------------------------------------------------------ inputs ---

def _trees(case, seed):
    """Random candidate trees in canonical order: masks and depths."""
    B, R = case["B"], case["R"]
    rs = np.random.RandomState(seed % (1 << 31))
    W = (R + 63) // 64
    masks = np.zeros((B, R, W), np.uint64)
    depths = np.zeros((B, R), np.int32)
    for b in range(B):
        par, dep = [-1], [0]
        for i in range(1, R):
            # a parent at most seven levels down: the tree has up to eight heads
            p = int(rs.randint(0, i))
            while dep[p] >= 8:
                p = par[p]
            par.append(p)
            dep.append(dep[p] + 1)
        order = sorted(range(R), key=lambda i: (dep[i], i))
        place = {o: n for n, o in enumerate(order)}
        for n, o in enumerate(order):
            depths[b, n] = dep[o]
            if par[o] >= 0:
                masks[b, n] = masks[b, place[par[o]]]
            masks[b, n, n // 64] |= np.uint64(1) << np.uint64(n % 64)
    return (torch.from_numpy(masks.view(np.int64)).to(DEV), torch.from_numpy(depths).to(DEV))


def _midpoints(values):
    return [(a + b) / 2 for a, b in zip(values, values[1:])]


def _e4m3_values():
    """The finite values of the sign-less e4m3 bytes 0x00 .. 0x7e, by byte."""
    return [(b & 7) * 2.0 ** -9 if b < 8 else (8 + (b & 7)) * 2.0 ** ((b >> 3) - 10)
            for b in range(127)]


def _nearest(v, values):
    """Index of the value nearest to v (64 bits); a tie goes to the even index."""
    mid = torch.tensor(_midpoints(values), dtype=torch.float64, device=v.device)
    i = torch.bucketize(v, mid)
    tie = (v == mid[i.clamp(max=len(values) - 2)]) & (i % 2 == 1)
    return i + tie


def _pack4(x):
    """Rows [..., Hkv, dh] as bytes [..., row bytes]: two codes a byte (the lower
    element in the lower half), then one e4m3 scale for each 16 elements."""
    Hkv, dh = x.shape[-2:]
    blocks = x.double().unflatten(-1, (dh // 16, 16))
    scale = _nearest(blocks.abs().amax(-1) / 6.0, _e4m3_values())
    s = torch.tensor(_e4m3_values(), dtype=torch.float64, device=x.device)[scale]
    code = _nearest(blocks.abs() / s.clamp(min=2.0 ** -9).unsqueeze(-1), E2M1)
    code = torch.where(blocks < 0, code + 8, code)
    code = torch.where(s.unsqueeze(-1) > 0, code, torch.zeros_like(code)).flatten(-3)
    rows = torch.cat([code[..., 0::2] + 16 * code[..., 1::2], scale.flatten(-2)], -1)
    pad = _row_bytes(Hkv, dh) - rows.shape[-1]
    return torch.nn.functional.pad(rows, (0, pad)).to(torch.uint8)


def _unpack4(rows, Hkv, dh):
    """The float32 values [..., Hkv, dh] that bytes [..., row bytes] stand for."""
    values = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=rows.device)
    n = Hkv * dh // 2
    code = torch.stack([rows[..., :n] & 15, rows[..., :n] >> 4], -1).flatten(-2)
    scale = rows[..., n:n + Hkv * dh // 16].contiguous().view(torch.float8_e4m3fn).float()
    x = values[code.int()].unflatten(-1, (Hkv * dh // 16, 16)) * scale.unsqueeze(-1)
    return x.flatten(-2).unflatten(-1, (Hkv, dh))


def prepare(case, seed):
    g = torch.Generator(DEV)
    g.manual_seed(seed)
    dt = _torch_dtype(case)
    B, R, dh, Hkv = case["B"], case["R"], case["dh"], case["Hkv"]

    def normal(*shape, std=1.0):
        return (torch.randn(shape, generator=g, device=DEV) * std).to(dt)

    prefix = torch.tensor(_prefixes(case), dtype=torch.int32, device=DEV)
    st = dict(case=case, prefix=prefix, P_max=case["P"])
    if case["op"] in ("rope", "kv4_append"):
        st["n_rows"] = torch.tensor(_rows(case), dtype=torch.int32, device=DEV)
        # keys carry a few strong channels, as trained models' keys do
        strong = 1.0 + 4.0 * (torch.rand((Hkv, dh), generator=g, device=DEV) < 0.03)
        st["k"] = (torch.randn((B, R, Hkv, dh), generator=g, device=DEV) * strong).to(dt)
        st["v"] = normal(B, R, Hkv, dh)
    if case["op"] == "rope":
        H, rot = case["H"], case["rot"]
        st["q"] = normal(B, R, H, dh)
        st["qw"] = (1 + 0.2 * torch.randn(dh, generator=g, device=DEV)).to(dt)
        st["kw"] = (1 + 0.2 * torch.randn(dh, generator=g, device=DEV)).to(dt)
        st["inv_freq"] = torch.pow(10000.0, -torch.arange(0, rot, 2, device=DEV).double() / rot).float()
        depth = _trees(case, seed)[1] if R <= 256 else torch.arange(R, device=DEV, dtype=torch.int32)
        st["pos"] = (prefix[:, None] + depth.expand(B, R)).int().contiguous()
        st["q_out"] = torch.zeros_like(st["q"])
        if case["append"]:
            # the cache as a call with a short prefix sees it: a few slots before the rows
            st["P_max"] = min(case["P"], 37)
            st["prefix"] = prefix.clamp(max=st["P_max"])
            st["kc"] = normal(B, st["P_max"] + R, Hkv, dh)
            st["vc"] = normal(B, st["P_max"] + R, Hkv, dh)
        else:
            st["k_out"] = torch.zeros_like(st["k"])
    elif case["op"] == "kv4_append":
        rb = _row_bytes(Hkv, dh)
        st["kc"] = torch.zeros((B, case["P"] + R, rb), dtype=torch.uint8, device=DEV)
        st["vc"] = torch.zeros((B, case["P"] + R, rb), dtype=torch.uint8, device=DEV)
        st["k_out"], st["v_out"] = torch.zeros_like(st["k"]), torch.zeros_like(st["v"])
    else:
        st["q"] = normal(B, R, case["H"], dh, std=1.5)
        st["mask"], st["depth"] = _trees(case, seed)
        slots = case["P"] + R
        rows = []
        for name in ("kc", "vc"):
            if case["op"] == "window":
                st[name] = normal(B, slots, Hkv, dh)
                continue
            rows = torch.empty((B, slots, _row_bytes(Hkv, dh)), dtype=torch.uint8, device=DEV)
            for b in range(B):
                for at in range(0, slots, 4096):
                    x = normal(min(4096, slots - at), Hkv, dh)
                    rows[b, at:at + x.shape[0]] = _pack4(x)
            st[name] = rows
        st["out"] = torch.zeros_like(st["q"])
    if "kc" in st:  # the device arrays of cache addresses that a program keeps
        for name in ("kc", "vc"):
            st[name + "_ptrs"] = torch.tensor([c.data_ptr() for c in st[name]], dtype=torch.int64,
                                              device=DEV)
    return st


# ------------------------------------------------------------- plain forms ---

def _plain_rotate(x, w, st):
    case = st["case"]
    dh, rot = case["dh"], case["rot"]
    x = x.float()
    if case["norm"]:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * w.float()
    angle = st["pos"].double()[:, :, None, None] * st["inv_freq"].double()
    cos, sin = angle.cos().float(), angle.sin().float()
    a = x[..., :rot]
    if case["inter"]:
        lo, hi = a[..., 0::2], a[..., 1::2]
        a = torch.stack([lo * cos - hi * sin, lo * sin + hi * cos], -1).flatten(-2)
    else:
        lo, hi = a[..., :rot // 2], a[..., rot // 2:]
        a = torch.cat([lo * cos - hi * sin, lo * sin + hi * cos], -1)
    return torch.cat([a, x[..., rot:]], -1).to(st["q"].dtype)


def _plain_rope(st):
    case = st["case"]
    B, R = case["B"], case["R"]
    row = torch.arange(R, device=DEV)
    live = row[None, :] < st["n_rows"][:, None]
    q = _plain_rotate(st["q"], st["qw"], st)
    k = _plain_rotate(st["k"], st["kw"], st)
    keep = live[:, :, None, None]
    q = torch.where(keep, q, st["q_out"])
    if not case["append"]:
        return q, torch.where(keep, k, st["k_out"])
    seq = torch.arange(B, device=DEV)[:, None].expand(B, R)
    slot = st["prefix"][:, None] + row
    kc, vc = st["kc"], st["vc"]
    # a row that is not there writes its own slot's old value back
    kc[seq, slot] = torch.where(keep, k, kc[seq, slot])
    vc[seq, slot] = torch.where(keep, st["v"], vc[seq, slot])
    return q, kc, vc


def _plain_append4(st):
    case = st["case"]
    B, R = case["B"], case["R"]
    row = torch.arange(R, device=DEV)
    live = (row[None, :] < st["n_rows"][:, None])
    seq = torch.arange(B, device=DEV)[:, None].expand(B, R)
    slot = st["prefix"].long()[:, None] + row
    zero = torch.zeros_like(st["k"])
    out = []
    for x, cache in ((st["k"], st["kc"]), (st["v"], st["vc"])):
        cache[seq, slot] = torch.where(live[..., None], _pack4(x), cache[seq, slot])
        y = _unpack4(cache[seq, slot], case["Hkv"], case["dh"]).to(x.dtype)
        out.append(torch.where(live[..., None, None], y, zero))
    return out


def _plain_attention(st):
    case = st["case"]
    B, R, H, Hkv, dh = (case[n] for n in ("B", "R", "H", "Hkv", "dh"))
    G, window, sinks = H // Hkv, case["window"], case["sinks"]
    P = st["prefix"].long()[:, None]
    depth = st["depth"].long()
    # the slots that a sequence's rows may see: [B, N], and which of them are real
    if window:
        near = P - window + 1 + torch.arange(window - 1 + R, device=DEV)
        first = torch.arange(sinks, device=DEV).expand(B, sinks)
        slot = torch.cat([first, near], 1)
        lo = (P - window + 1).clamp(min=0)
        real = torch.cat([first < torch.minimum(lo, P), near >= 0], 1)
    else:
        slot = torch.arange(case["P"] + R, device=DEV).expand(B, case["P"] + R)
        real = slot < P + R
    slot = torch.where(real, slot, torch.zeros_like(slot))
    node = (slot - P).clamp(min=0, max=R - 1)
    in_tree = slot >= P
    spot = torch.where(in_tree, P + depth.gather(1, node), slot)  # position of each slot
    at = node[:, None, :].expand(B, R, -1)
    bits = st["mask"].gather(2, at >> 6) >> (at & 63) & 1
    seen = real[:, None] & (~in_tree[:, None] | (bits == 1))
    if window:
        seen &= (spot[:, None] < sinks) | ((P + depth)[:, :, None] - spot[:, None] < window)
    rows = torch.arange(B, device=DEV)[:, None]
    k, v = st["kc"][rows, slot], st["vc"][rows, slot]
    if case["op"] == "kv4_attn":
        k, v = _unpack4(k, Hkv, dh), _unpack4(v, Hkv, dh)
    k, v = k.float().transpose(1, 2), v.float().transpose(1, 2)  # [B, Hkv, N, dh]
    q = st["q"].float().unflatten(2, (Hkv, G)).permute(0, 2, 3, 1, 4)  # [B, Hkv, G, R, dh]
    x = q.reshape(B, Hkv, G * R, dh) @ k.transpose(2, 3) / math.sqrt(dh)
    x = x.unflatten(2, (G, R)).masked_fill(~seen[:, None, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    w = torch.exp(x - torch.where(top.isfinite(), top, torch.zeros_like(top)))
    total = w.sum(-1, keepdim=True)
    y = (w.flatten(2, 3) @ v).unflatten(2, (G, R)) / torch.where(total > 0, total, torch.ones_like(total))
    return y.permute(0, 3, 1, 2, 4).reshape(B, R, H, dh).to(st["q"].dtype)


# --------------------------------------------------------------------- run ---

def _own(st):
    import medusa_speculative_decoding_02_gb300 as m
    case = st["case"]
    op, B, R, Hkv, dh = (case[n] for n in ("op", "B", "R", "Hkv", "dh"))
    if "ws" not in st:  # one workspace for all calls, kept by the program
        size = m.WS_HEADER
        if op in ("window", "kv4_attn"):
            dt = m.BF16 if case["dtype"] == "bf16" else m.F32
            size = m.tree_attention_window_workspace_size(
                dt, B, R, case["H"], Hkv, dh, case["P"], case["window"], case["sinks"],
                kv4=op == "kv4_attn")
        st["ws"] = m.new_workspace(size)
    ws = st["ws"]
    if op == "rope":
        w = dict(q_weight=st["qw"], k_weight=st["kw"]) if case["norm"] else {}
        w.update(norm=case["norm"], eps=1e-6, interleaved=case["inter"])
        if case["append"]:
            m.qk_norm_rope_append(st["q"], st["k"], st["v"], st["pos"], st["inv_freq"],
                                  st["kc_ptrs"], st["vc_ptrs"], st["prefix"], st["P_max"],
                                  n_rows=st["n_rows"], out=st["q_out"], ws=ws, **w)
            return st["q_out"], st["kc"], st["vc"]
        return m.qk_norm_rope(st["q"], st["k"], st["pos"], st["inv_freq"], n_rows=st["n_rows"],
                              out=(st["q_out"], st["k_out"]), **w)
    if op == "kv4_append":
        m.kv4_append(st["k"], st["v"], st["kc_ptrs"], st["vc_ptrs"], st["prefix"], st["P_max"],
                     n_rows=st["n_rows"], ws=ws)
        return list(m.kv4_unpack(st["kc_ptrs"], st["vc_ptrs"], st["prefix"], st["P_max"], R, Hkv,
                                 dh, n_rows=st["n_rows"], out=(st["k_out"], st["v_out"]), ws=ws))
    call = m.tree_attention_window if op == "window" else m.tree_attention_kv4
    return call(st["q"], st["kc_ptrs"], st["vc_ptrs"], st["prefix"], st["P_max"], st["mask"], Hkv,
                depth=st["depth"], window=case["window"], sinks=case["sinks"], out=st["out"], ws=ws)


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    if op == "rope":
        return _plain_rope(state)
    if op == "kv4_append":
        return _plain_append4(state)
    return _plain_attention(state)


# ------------------------------------------------------------------- exact ---

def _exact_rope(st):
    case = st["case"]
    rot = case["rot"]
    out = {}
    theta = st["pos"].double().unsqueeze(-1) * st["inv_freq"].double()
    turn = torch.polar(torch.ones_like(theta), theta).unsqueeze(2)  # e^(i angle)
    for name, weight in (("q", "qw"), ("k", "kw")):
        x = st[name].double()
        if case["norm"]:
            x = x / (x.pow(2).sum(-1, keepdim=True) / case["dh"] + 1e-6).sqrt() * st[weight].double()
        if case["inter"]:
            z = torch.view_as_complex(x[..., :rot].reshape(*x.shape[:-1], rot // 2, 2)) * turn
            x[..., :rot] = torch.view_as_real(z).reshape(*x.shape[:-1], rot)
        else:
            z = torch.complex(x[..., :rot // 2], x[..., rot // 2:rot]) * turn
            x[..., :rot // 2], x[..., rot // 2:rot] = z.real, z.imag
        out[name] = x
    rows = _rows(case)
    q = torch.zeros_like(out["q"])
    for b, n in enumerate(rows):
        q[b, :n] = out["q"][b, :n]
    if not case["append"]:
        k = torch.zeros_like(out["k"])
        for b, n in enumerate(rows):
            k[b, :n] = out["k"][b, :n]
        return q, k
    kc, vc = st["kc"].double(), st["vc"].double()
    for b, n in enumerate(rows):
        P = int(st["prefix"][b])
        kc[b, P:P + n] = out["k"][b, :n]
        vc[b, P:P + n] = st["v"][b, :n].double()
    return q, kc, vc


def _exact_round4(x):
    """The values that a row's 4-bit form stands for, from the definition: the
    nearest of all candidates by distance, the even one of two equally near."""
    blocks = x.detach().cpu().double().numpy().reshape(-1, 16)
    scales = np.array(_e4m3_values())

    def near(v, grid):
        up = np.clip(np.searchsorted(grid, v), 1, len(grid) - 1)
        a, b = np.abs(v - grid[up - 1]), np.abs(grid[up] - v)
        return np.where((a < b) | ((a == b) & (up % 2 == 1)), up - 1, up)

    s = scales[near(np.abs(blocks).max(1) / 6.0, scales)]
    grid = np.array(E2M1)
    with np.errstate(divide="ignore", invalid="ignore"):
        r = np.where(s[:, None] > 0, np.abs(blocks) / s[:, None], 0.0)
    y = np.sign(blocks) * grid[near(r, grid)] * s[:, None]
    return torch.from_numpy(y.reshape(x.shape))


def _exact_values4(rows, Hkv, dh):
    """The 64-bit values of bytes, bit field by bit field."""
    def value(code):
        e, f = code >> 1 & 3, code & 1
        x = torch.where(e == 0, f * 0.5, torch.ldexp(1 + 0.5 * f, e.double() - 1))
        return torch.where(code & 8 != 0, -x, x)
    codes = rows[..., :Hkv * dh // 2].int()
    x = torch.empty((*rows.shape[:-1], Hkv * dh), dtype=torch.float64, device=rows.device)
    x[..., 0::2], x[..., 1::2] = value(codes & 15).double(), value(codes >> 4).double()
    s = rows[..., Hkv * dh // 2:Hkv * dh // 2 + Hkv * dh // 16].int()
    e, f = s >> 3 & 15, (s & 7).double()
    s = torch.where(e == 0, torch.ldexp(f, torch.full_like(f, -9)), torch.ldexp(8 + f, e.double() - 10))
    return (x * s.repeat_interleave(16, -1)).reshape(*rows.shape[:-1], Hkv, dh)


def _exact_attention(st):
    case = st["case"]
    B, R, H, Hkv, dh = (case[n] for n in ("B", "R", "H", "Hkv", "dh"))
    G, out = H // Hkv, torch.zeros((B, R, H, dh), dtype=torch.float64, device=DEV)
    bits = np.unpackbits(st["mask"].cpu().numpy().view(np.uint8), axis=-1, bitorder="little")
    for b, P in enumerate(_prefixes(case)):
        depth = st["depth"][b].cpu().numpy().astype(np.int64)
        place = np.concatenate([np.arange(P), P + depth])
        seen = np.concatenate([np.ones((R, P), bool), bits[b, :, :R] > 0], 1)
        if case["window"]:
            gap = (P + depth)[:, None] - place[None, :]
            seen &= (place[None, :] < case["sinks"]) | (gap < case["window"])
        used = np.flatnonzero(seen.any(0))
        hide = torch.from_numpy(~seen[:, used]).to(DEV)
        used = torch.from_numpy(used).to(DEV)
        for g in range(Hkv):
            if case["op"] == "window":
                k, v = st["kc"][b, used, g].double(), st["vc"][b, used, g].double()
            else:
                n, c = Hkv * dh // 2, dh // 2
                one = [torch.cat([st[x][b, used, g * c:(g + 1) * c],
                                  st[x][b, used, n + g * c // 8:n + (g + 1) * c // 8]], 1)
                       for x in ("kc", "vc")]
                k, v = (_exact_values4(x, 1, dh)[:, 0] for x in one)
            for h in range(g * G, (g + 1) * G):
                x = (st["q"][b, :, h].double() @ k.T / math.sqrt(dh)).masked_fill(hide, -math.inf)
                w = torch.softmax(x, -1)
                out[b, :, h] = w @ v
    return out


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "rope":
        return _exact_rope(st)
    if case["op"] == "kv4_append":
        out = []
        for name in ("k", "v"):
            y = _exact_round4(st[name])
            for b, n in enumerate(_rows(case)):
                y[b, n:] = 0
            out.append(y)
        return out
    return _exact_attention(st)
