"""What is measured of the calls that serve from a paged cache, and their plain form.

Five operators, in the order in which a server meets them:

  append      K and V rows into the pages of their sequences
  chunk       attention of a chunk of new tokens over the paged cache: prompts
              that enter piece by piece, and single tokens
  tree        attention of a candidate tree's rows over the paged cache
  commit      the accepted path's rows moved up behind the prefix, page by page
  logprobs    log probabilities of given tokens, with their ranks, the entropy
              of each row and its top alternatives

A pool of K (and V) is [pages, page, Hkv, dh]; slot j of sequence b lies in page
``page_table[b][j // page]`` at ``j % page``.

``run`` computes the plain form with elementary torch operations where ``own``
is false, and makes the framework's calls where it is true.  ``exact`` is the
definition in 64 bits.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"


# ------------------------------------------------------------------- cases ---

def listed():
    return [
        # the 7B step's 65 tree rows (64 nodes and the root) of eight sequences
        dict(name="append_step", op="append", B=8, R=65, Hkv=32, dh=128, page=64, dtype="bf16",
             ragged=False, P=1024),
        # prompts of uneven length entering a cache of small pages
        dict(name="append_prompt", op="append", B=4, R=4001, Hkv=8, dh=128, page=16, dtype="bf16",
             ragged=True, P=77),
        # one 7B sequence's accepted path, five heads
        dict(name="commit_step", op="commit", B=1, R=65, K=5, Hkv=32, dh=128, page=64, dtype="bf16",
             P=1024),
        # a full batch of sequences whose trees cross pages
        dict(name="commit_batch", op="commit", B=32, R=65, K=5, Hkv=32, dh=128, page=16, dtype="bf16",
             P=511),
        # plain decoding of eight long sequences, grouped heads
        dict(name="chunk_single", op="chunk", B=8, R=1, H=32, Hkv=8, dh=128, P=16384, page=64,
             dtype="bf16", ragged=False),
        # chunks of uneven length behind long prefixes, down to a single token
        dict(name="chunk_mixed", op="chunk", B=6, R=509, H=28, Hkv=4, dh=128, P=5001, page=32,
             dtype="bf16", ragged=True),
        # a long prompt in one piece
        dict(name="chunk_prompt", op="chunk", B=1, R=8192, H=32, Hkv=8, dh=128, P=0, page=128,
             dtype="bf16", ragged=False),
        # the 7B step
        dict(name="tree_step", op="tree", B=1, R=65, H=32, Hkv=32, dh=128, P=1024, page=64,
             dtype="bf16"),
        # a ragged batch of eight trees, grouped heads, prefixes up to 8192
        dict(name="tree_batch", op="tree", B=8, R=65, H=32, Hkv=8, dh=128, P=8192, page=16,
             dtype="bf16"),
        # the verification rows of one step: what a client sees of each node
        dict(name="logprobs_step", op="logprobs", N=65, V=32000, top=5, temp=1.0, dtype="bf16"),
        # a prompt's tokens scored
        dict(name="logprobs_prompt", op="logprobs", N=4093, V=32000, top=10, temp=0.7, dtype="bf16"),
        # rows of an odd vocabulary in 32 bits, no alternatives
        dict(name="logprobs_odd", op="logprobs", N=301, V=50257, top=0, temp=1.0, dtype="f32"),
    ]


HEADS = ((32, 32), (40, 40), (32, 8), (28, 4), (8, 8), (6, 3), (5, 1), (1, 1))
PAGES = (16, 32, 64, 128, 256)


def _logint(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("append", "chunk", "chunk", "tree", "commit", "logprobs"))
    dtype = rng.choice(("bf16", "bf16", "bf16", "f32"))
    if op == "logprobs":
        V = rng.choice((32000, _logint(rng, 100, 130000), _logint(rng, 100, 130000)))
        N = _logint(rng, 1, min(4096, 60_000_000 // V))
        return dict(op=op, N=N, V=V, top=rng.choice((0, 1, 5, 10, 16)), temp=rng.choice((1.0, 0.7, 1.3)),
                    dtype=dtype)
    H, Hkv = rng.choice(HEADS)
    dh = rng.choice((64, 128, 128))
    page = rng.choice(PAGES)
    P = rng.choice((0, _logint(rng, 1, 16384), _logint(rng, 64, 16384)))
    if op == "append":
        B = rng.randint(1, 16)
        return dict(op=op, B=B, R=_logint(rng, 1, 8192 // B), Hkv=Hkv, dh=dh, page=page, dtype=dtype,
                    ragged=rng.random() < 0.5, P=min(P, 2048))
    if op == "commit":
        return dict(op=op, B=rng.randint(1, 32), R=rng.choice((1, 15, 65, 129, 256)), K=rng.randint(1, 8),
                    Hkv=Hkv, dh=dh, page=page, dtype=dtype, P=min(P, 600))
    B = rng.randint(1, 8)
    if op == "tree":
        R = rng.choice((2, 17, 33, 64, 65, 129, rng.randint(1, 256)))
    else:
        R = rng.choice((1, 1, _logint(rng, 2, 600), _logint(rng, 64, 8192)))
    if dtype == "f32":
        H, Hkv = rng.choice(((8, 8), (6, 3), (5, 1), (1, 1), (4, 2)))
        R, P = min(R, 300), min(P, 2048)
    if B * Hkv > 64:
        P = min(P, 4096)
    # no more pairs of a row and a slot than the largest listed case has (fp32: a tenth)
    most = 1_000_000_000 if dtype == "bf16" else 100_000_000
    while B * H * R * (P + R // 2) > most:
        R, P = max(1, R // 2) if R > 64 else R, P // 2
    case = dict(op=op, B=B, R=R, H=H, Hkv=Hkv, dh=dh, P=P, page=page, dtype=dtype)
    if op == "chunk":
        case["ragged"] = rng.random() < 0.5
    return case


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
    """Rows of each sequence (the first has all of them, the last of a ragged call one)."""
    R, B = case["R"], case["B"]
    if not case.get("ragged"):
        return [R] * B
    return [max(1, R - (R * b) // max(1, B - 1)) for b in range(B)]


def _accepted(case, seed):
    """Accepted nodes beyond the root of each sequence."""
    rs = np.random.RandomState(seed % (1 << 31))
    return rs.randint(0, min(case["K"], case["R"] - 1) + 1, case["B"])


def work(case):
    es = _size(case)
    if case["op"] == "logprobs":
        N, V = case["N"], case["V"]
        return {"bytes": N * V * es + N * (4 + 12 + 8 * case["top"]), "flops": 6 * N * V}
    row = case["Hkv"] * case["dh"] * es
    if case["op"] == "append":
        return {"bytes": 4 * sum(_rows(case)) * row, "flops": 0}
    if case["op"] == "commit":
        # half of the deepest path of every sequence, K and V, read and written
        moved = case["B"] * (1 + min(case["K"], case["R"] - 1) / 2)
        return {"bytes": int(4 * moved * row), "flops": 0}
    B, R, H, dh = case["B"], case["R"], case["H"], case["dh"]
    rows, prefixes = _rows(case), _prefixes(case)
    kv = 2 * sum(P + n for P, n in zip(prefixes, rows)) * row
    if case["op"] == "chunk":
        pairs = sum(n * P + n * (n + 1) // 2 for P, n in zip(prefixes, rows))
        mask = 0
    else:
        pairs = sum(n * (P + n) for P, n in zip(prefixes, rows))
        mask = B * R * 8 * ((R + 63) // 64)
    return {"bytes": kv + 2 * sum(rows) * H * dh * es + mask, "flops": 4 * dh * H * pairs}


# ------------------------------------------------------------------ inputs ---

def _trees(case, seed):
    """Ancestor masks of random candidate trees, rows in order of depth."""
    B, R = case["B"], case["R"]
    rs = np.random.RandomState(seed % (1 << 31))
    masks = np.zeros((B, R, (R + 63) // 64), np.uint64)
    for b in range(B):
        parent, depth = [-1], [0]
        for i in range(1, R):
            p = int(rs.randint(0, i))
            while depth[p] >= 8:  # a level per head at most
                p = parent[p]
            parent.append(p)
            depth.append(depth[p] + 1)
        order = sorted(range(R), key=lambda i: (depth[i], i))
        place = {node: row for row, node in enumerate(order)}
        for row, node in enumerate(order):
            if parent[node] >= 0:
                masks[b, row] = masks[b, place[parent[node]]]
            masks[b, row, row // 64] |= np.uint64(1) << np.uint64(row % 64)
    return torch.from_numpy(masks.view(np.int64)).to(DEV)


def _prepare_logprobs(case, g):
    N, V, dt = case["N"], case["V"], _torch_dtype(case)
    # a model's logits: a broad bulk, a few strong candidates a row, ties from 16 bits
    x = torch.randn((N, V), generator=g, device=DEV) * 2.0
    hot = torch.randint(0, V, (N, 8), generator=g, device=DEV)
    x.scatter_add_(1, hot, torch.rand((N, 8), generator=g, device=DEV) * 16)
    # the tokens that were taken: mostly strong ones, and any
    pick = hot.gather(1, torch.randint(0, 8, (N, 1), generator=g, device=DEV))[:, 0]
    rare = torch.randint(0, V, (N,), generator=g, device=DEV)
    often = torch.rand((N,), generator=g, device=DEV) < 0.8
    return dict(case=case, logits=x.to(dt), tokens=torch.where(often, pick, rare).int())


def prepare(case, seed):
    g = torch.Generator(DEV)
    g.manual_seed(seed)
    if case["op"] == "logprobs":
        return _prepare_logprobs(case, g)
    dt = _torch_dtype(case)
    B, R, Hkv, dh, page = (case[n] for n in ("B", "R", "Hkv", "dh", "page"))
    # every sequence has the pages it needs, anywhere in a pool that holds a few more
    need = [-(-(P + R) // page) for P in _prefixes(case)]
    wide = -(-(case["P"] + R) // page)
    pages = sum(need) + 7
    place = torch.randperm(pages, generator=g, device=DEV).cpu()
    table, at = torch.zeros((B, wide), dtype=torch.int32), 0
    for b, n in enumerate(need):
        table[b, :n] = place[at:at + n]
        at += n
    st = dict(case=case, P_max=case["P"], table=table.to(DEV),
              prefix=torch.tensor(_prefixes(case), dtype=torch.int32, device=DEV),
              n_rows=torch.tensor(_rows(case), dtype=torch.int32, device=DEV))
    for name in ("kp", "vp"):
        pool = torch.empty((pages, page, Hkv, dh), dtype=dt, device=DEV)
        step = max(1, (1 << 25) // (page * Hkv * dh))
        for i in range(0, pages, step):
            part = pool[i:i + step]
            part.copy_(torch.randn(part.shape, generator=g, device=DEV))
        st[name] = pool
    if case["op"] == "append":
        # keys carry a few strong channels, as trained models' keys do
        strong = 1.0 + 4.0 * (torch.rand((Hkv, dh), generator=g, device=DEV) < 0.03)
        st["k"] = (torch.randn((B, R, Hkv, dh), generator=g, device=DEV) * strong).to(dt)
        st["v"] = torch.randn((B, R, Hkv, dh), generator=g, device=DEV).to(dt)
    elif case["op"] == "commit":
        rs = np.random.RandomState((seed + 1) % (1 << 31))
        length = _accepted(case, seed)
        path = np.full((B, case["K"] + 1), -1, np.int32)
        for b, n in enumerate(length):
            # the nodes lie behind the slots that the path moves to (a small tree: in
            # them already), so that a pass can be repeated on its own result
            beyond = np.arange(n + 1, R)
            path[b, :n + 1] = np.arange(n + 1)
            if len(beyond) >= n:
                path[b, 1:n + 1] = np.sort(rs.choice(beyond, n, replace=False))
        st["path"] = torch.from_numpy(path).to(DEV)
        st["accept_len"] = torch.from_numpy(length.astype(np.int32)).to(DEV)
        st["new_prefix"] = torch.zeros(B, dtype=torch.int32, device=DEV)
    else:
        st["q"] = (torch.randn((B, R, case["H"], dh), generator=g, device=DEV) * 1.5).to(dt)
        st["out"] = torch.zeros_like(st["q"])
        if case["op"] == "tree":
            st["mask"] = _trees(case, seed)
    return st


# ------------------------------------------------------------- plain forms ---

def _place(st, slot):
    """Page and row within it of slots [B, n]."""
    page = st["case"]["page"]
    return st["table"].long().gather(1, slot // page), slot % page


def _plain_append(st):
    B, R = st["case"]["B"], st["case"]["R"]
    row = torch.arange(R, device=DEV).expand(B, R)
    pg, at = _place(st, st["prefix"].long()[:, None] + row)
    live = row < st["n_rows"][:, None]
    pg, at = pg[live], at[live]
    st["kp"][pg, at] = st["k"][live]
    st["vp"][pg, at] = st["v"][live]
    return st["kp"], st["vp"]


def _plain_commit(st):
    K = st["case"]["K"]
    P = st["prefix"].long()[:, None]
    step = torch.arange(K + 1, device=DEV)[None]
    used = step <= st["accept_len"][:, None]
    source = _place(st, torch.where(used, P + st["path"], P))
    target = _place(st, torch.where(used, P + step, P))
    for pool in (st["kp"], st["vp"]):
        rows = pool[source[0][used], source[1][used]]
        pool[target[0][used], target[1][used]] = rows
    return st["kp"], st["vp"], st["prefix"] + st["accept_len"] + 1


def _plain_attention(st):
    case = st["case"]
    B, R, H, Hkv, dh = (case[n] for n in ("B", "R", "H", "Hkv", "dh"))
    G, N = H // Hkv, case["P"] + R
    P = st["prefix"].long()[:, None]
    slot = torch.arange(N, device=DEV).expand(B, N)
    real = slot < P + R
    pg, at = _place(st, torch.where(real, slot, torch.zeros_like(slot)))
    k = st["kp"][pg, at].float().transpose(1, 2)  # [B, Hkv, N, dh]
    v = st["vp"][pg, at].float().transpose(1, 2)
    node = (slot - P).clamp(min=0, max=R - 1)
    block = max(1, (1 << 28) // (B * H * N))  # rows at a time
    out = []
    for r0 in range(0, R, block):
        q = st["q"][:, r0:r0 + block].float()
        n = q.shape[1]
        row = torch.arange(r0, r0 + n, device=DEV)[None, :, None]
        if case["op"] == "chunk":
            seen = slot[:, None] <= P[:, :, None] + row
        else:
            spot = node[:, None, :].expand(B, n, N)
            bits = st["mask"][:, r0:r0 + n].gather(2, spot >> 6) >> (spot & 63) & 1
            seen = real[:, None] & ((slot < P)[:, None] | (bits == 1))
        q = q.unflatten(2, (Hkv, G)).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * n, dh)
        x = (q @ k.transpose(2, 3) / math.sqrt(dh)).unflatten(2, (G, n))
        x = x.masked_fill(~seen[:, None, None], -math.inf)
        w = torch.exp(x - x.amax(-1, keepdim=True))
        y = (w.flatten(2, 3) @ v).unflatten(2, (G, n)) / w.sum(-1, keepdim=True)
        out.append(y.permute(0, 3, 1, 2, 4).reshape(B, n, H, dh))
    y = torch.cat(out, 1).to(st["q"].dtype)
    live = torch.arange(R, device=DEV)[None] < st["n_rows"][:, None]
    return torch.where(live[:, :, None, None], y, st["out"])


def _order(x, top):
    """The ``top`` largest of each row, a tie to the lowest index: ids."""
    ids = []
    x = x.clone()
    for _ in range(top):
        best = x.amax(1, keepdim=True)
        first = (x == best).float().argmax(1, keepdim=True)  # the first of equal ones
        ids.append(first)
        x.scatter_(1, first, -math.inf)
    return torch.cat(ids, 1) if ids else torch.empty((x.shape[0], 0), dtype=torch.long, device=DEV)


def _plain_logprobs(st):
    case = st["case"]
    raw = st["logits"].float()
    x = raw / case["temp"]
    token = st["tokens"].long()[:, None]
    x = x - x.amax(1, keepdim=True)
    w = torch.exp(x)
    total = w.sum(1, keepdim=True)
    logp = x - torch.log(total)
    entropy = -(w / total * logp).sum(1)
    own_logit = raw.gather(1, token)
    index = torch.arange(raw.shape[1], device=DEV)
    rank = ((raw > own_logit) | ((raw == own_logit) & (index < token))).sum(1).int()
    ids = _order(raw, case["top"])
    return logp.gather(1, token)[:, 0], entropy, rank, ids.int(), logp.gather(1, ids)


# --------------------------------------------------------------------- run ---

def _own(st):
    import medusa_speculative_decoding_02_gb300 as m
    case = st["case"]
    op = case["op"]
    if "ws" not in st:  # one workspace for all calls, kept by the program
        size = m.WS_HEADER
        if op in ("chunk", "tree"):
            dt = m.BF16 if case["dtype"] == "bf16" else m.F32
            size = m.paged_attention_workspace_size(dt, case["B"], case["R"], case["H"], case["Hkv"],
                                                    case["dh"], case["P"])
        st["ws"] = m.new_workspace(size)
    ws = st["ws"]
    if op == "logprobs":
        r = m.token_logprobs(st["logits"], st["tokens"], case["top"], temperature=case["temp"], ws=ws)
        return r.logp, r.entropy, r.rank, r.top_ids, r.top_logp
    cache = (st["kp"], st["vp"], st["table"], st["prefix"])
    if op == "append":
        m.paged_append(st["k"], st["v"], *cache, st["P_max"], n_rows=st["n_rows"], ws=ws)
        return st["kp"], st["vp"]
    if op == "commit":
        new = m.commit_paged(*cache, st["P_max"], st["path"], st["accept_len"], case["R"],
                             new_prefix_len=st["new_prefix"], ws=ws)
        return st["kp"], st["vp"], new
    if op == "tree":
        return m.tree_attention_paged(st["q"], *cache, st["P_max"], st["mask"], out=st["out"], ws=ws)
    return m.chunk_attention_paged(st["q"], *cache, st["P_max"], n_rows=st["n_rows"], out=st["out"],
                                   ws=ws)


def run(state):
    if own:
        return _own(state)
    return {"append": _plain_append, "commit": _plain_commit, "logprobs": _plain_logprobs}.get(
        state["case"]["op"], _plain_attention)(state)


# ------------------------------------------------------------------- exact ---

def _sequence(st, name, b, slots):
    """Rows of the first ``slots`` slots of sequence b, in 64 bits: [slots, Hkv, dh]."""
    page = st["case"]["page"]
    used = st["table"][b, :-(-slots // page)].long()
    return st[name][used].double().flatten(0, 1)[:slots]


def _exact_attention(st):
    case = st["case"]
    B, R, H, Hkv, dh = (case[n] for n in ("B", "R", "H", "Hkv", "dh"))
    rows, out = _rows(case), st["out"].double()
    for b, P in enumerate(_prefixes(case)):
        n = rows[b]
        k, v = (_sequence(st, name, b, P + n) for name in ("kp", "vp"))
        for r0 in range(0, n, 1024):
            r1 = min(n, r0 + 1024)
            if case["op"] == "chunk":
                end = P + r1
                hide = torch.ones((r1 - r0, end), dtype=torch.bool, device=DEV).triu(P + r0 + 1)
            else:
                end = P + n
                words = st["mask"][b, r0:r1].cpu().numpy().view(np.uint8)
                bits = np.unpackbits(words, axis=-1, bitorder="little")[:, :n] > 0
                see = np.concatenate([np.ones((r1 - r0, P), bool), bits], 1)
                hide = torch.from_numpy(~see).to(DEV)
            for h in range(H):
                g = h * Hkv // H
                x = st["q"][b, r0:r1, h].double() @ k[:end, g].T / math.sqrt(dh)
                out[b, r0:r1, h] = torch.softmax(x.masked_fill_(hide, -math.inf), -1) @ v[:end, g]
    return out


def _exact_logprobs(st):
    case = st["case"]
    N, V, top = case["N"], case["V"], case["top"]
    logp, entropy = (torch.empty(N, dtype=torch.float64, device=DEV) for _ in range(2))
    rank = torch.empty(N, dtype=torch.int32, device=DEV)
    ids = torch.empty((N, top), dtype=torch.int32, device=DEV)
    top_logp = torch.empty((N, top), dtype=torch.float64, device=DEV)
    for i in range(0, N, 256):
        x = st["logits"][i:i + 256].double()
        n = x.shape[0]
        order = torch.sort(x, dim=1, descending=True, stable=True).indices  # ties: lowest index first
        lp = torch.log_softmax(x / case["temp"], 1)
        token = st["tokens"][i:i + 256].long()
        each = torch.arange(n, device=DEV)
        logp[i:i + n] = lp[each, token]
        entropy[i:i + n] = -torch.special.xlogy(lp.exp(), lp.exp()).sum(1)
        rank[i:i + n] = (order == token[:, None]).int().argmax(1).int()
        ids[i:i + n] = order[:, :top].int()
        top_logp[i:i + n] = lp.gather(1, order[:, :top])
    return logp, entropy, rank, ids, top_logp


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "logprobs":
        return _exact_logprobs(st)
    if case["op"] in ("chunk", "tree"):
        return _exact_attention(st)
    kp, vp = st["kp"].double(), st["vp"].double()
    new = []
    for b, P in enumerate(_prefixes(case)):
        spots = [divmod(P + i, case["page"]) for i in range(case["R"])]
        spots = [(int(p), o) for p, o in zip(st["table"][b].cpu()[[p for p, _ in spots]], [o for _, o in spots])]
        if case["op"] == "append":
            n = _rows(case)[b]
            page, at = (torch.tensor(x, device=DEV) for x in zip(*spots[:n]))
            kp[page, at], vp[page, at] = st["k"][b, :n].double(), st["v"][b, :n].double()
            continue
        nodes = st["path"][b].tolist()[:int(st["accept_len"][b]) + 1]
        for pool, old in ((kp, st["kp"]), (vp, st["vp"])):
            for i, node in enumerate(nodes):
                pool[spots[i]] = old[spots[node]].double()
        new.append(P + len(nodes))
    if case["op"] == "append":
        return kp, vp
    return kp, vp, torch.tensor(new, dtype=torch.int32, device=DEV)
