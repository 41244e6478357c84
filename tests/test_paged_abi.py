"""Refusals of the calls on a cache in pages and of the log probabilities, and the
references' own definitions: no GPU needed."""
import ctypes
import math

import numpy as np
import pytest
import torch

import medusa_speculative_decoding_02_gb300 as m
import paged_ref as ref
from medusa_speculative_decoding_02_gb300 import build as mbuild

P = ctypes.c_void_p
A, A2 = P(4096), P(8192)  # fake, 16-byte aligned device addresses: never dereferenced
ODD = P(4100)
WS = P(1 << 20)
f = ctypes.c_float


@pytest.fixture(scope="module")
def L():
    mbuild.build()
    return m.lib()


def refused(L, call, code):
    before = L.medusa_launch_count()
    rc = call()
    assert rc == code, (m.STATUS.get(rc), L.medusa_last_error())
    assert L.medusa_last_error().decode() and L.medusa_launch_count() == before


PAGES_BAD = [
    (dict(kp=None), 1), (dict(vp=None), 1), (dict(tab=None), 1), (dict(pl=None), 1), (dict(kp=ODD), 1),
    (dict(vp=ODD), 1), (dict(page=0), 1), (dict(page=8), 1), (dict(page=48), 1), (dict(page=2048), 1),
    (dict(page=-16), 1), (dict(pages=0), 1), (dict(pages=-1), 1), (dict(pages=1 << 27, page=16), 1),
    (dict(P_max=-1), 1), (dict(P_max=(1 << 29) + 1, wide=1 << 30), 1), (dict(wide=0), 1),
    (dict(wide=6), 1),  # 96 slots for P_max + R = 105
    (dict(dtype=3), 1), (dict(B=0), 1), (dict(B=65536), 1), (dict(R=0), 1), (dict(Hkv=0), 1), (dict(dh=96), 2),
    (dict(ws=None), 3), (dict(ws=P((1 << 20) + 16)), 3), (dict(ws_bytes=128), 3)]


def args(kw):
    a = dict(dtype=m.BF16, q=A, k=A, v=A, ks=1024, vs=1024, kp=A, vp=A, pages=50, page=16, tab=A, wide=7, pl=A,
             P_max=100, n=None, mask=A, B=2, R=5, H=32, Hkv=8, dh=128, K=4, path=A, al=A, npl=A2, scale=0.1, out=A,
             ws=WS, ws_bytes=1 << 30)
    a.update(kw)
    return a, (a["kp"], a["vp"], a["pages"], a["page"], a["tab"], a["wide"], a["pl"], a["P_max"])


@pytest.mark.parametrize("kw,code", PAGES_BAD + [
    (dict(k=None), 1), (dict(v=None), 1), (dict(k=ODD), 1), (dict(ks=1016), 1), (dict(vs=1028), 1),
    (dict(R=(1 << 20) + 1, wide=1 << 20), 1), (dict(Hkv=1025), 1)])
def test_append_refuses(L, kw, code):
    a, cache = args(kw)
    refused(L, lambda: L.medusa_paged_append(a["dtype"], a["k"], a["v"], a["ks"], a["vs"], *cache, a["n"], a["B"],
                                             a["R"], a["Hkv"], a["dh"], a["ws"], a["ws_bytes"], None), code)


@pytest.mark.parametrize("kw,code", PAGES_BAD + [
    (dict(path=None), 1), (dict(al=None), 1), (dict(npl=None), 1), (dict(npl=A), 1), (dict(K=9), 1), (dict(K=-1), 1),
    (dict(R=257, wide=99), 1)])
def test_commit_refuses(L, kw, code):
    a, cache = args(kw)
    refused(L, lambda: L.medusa_commit_paged(a["dtype"], *cache, a["path"], a["al"], a["B"], a["K"], a["R"], a["Hkv"],
                                             a["dh"], a["npl"], a["ws"], a["ws_bytes"], None), code)


@pytest.mark.parametrize("kw,code", PAGES_BAD + [
    (dict(q=None), 1), (dict(out=None), 1), (dict(q=ODD), 1), (dict(out=ODD), 1), (dict(H=31), 1), (dict(Hkv=64), 1),
    (dict(H=2048, Hkv=1), 1), (dict(scale=0.0), 1), (dict(scale=-1.0), 1), (dict(scale=math.inf), 1),
    (dict(scale=math.nan), 1)])
@pytest.mark.parametrize("kind", ["chunk", "tree"])
def test_attention_refuses(L, kw, code, kind):
    a, cache = args(kw)
    last = a["n"] if kind == "chunk" else a["mask"]
    fn = getattr(L, f"medusa_{kind}_attention_paged")
    refused(L, lambda: fn(a["dtype"], a["q"], *cache, last, a["B"], a["R"], a["H"], a["Hkv"], a["dh"], f(a["scale"]),
                          a["out"], a["ws"], a["ws_bytes"], None), code)


def test_attention_refuses_rows_and_masks(L):
    for kind, kw in (("chunk", dict(R=(1 << 20) + 1, wide=1 << 20)), ("tree", dict(R=257, wide=99)),
                     ("tree", dict(mask=None))):
        a, cache = args(kw)
        last = a["n"] if kind == "chunk" else a["mask"]
        fn = getattr(L, f"medusa_{kind}_attention_paged")
        refused(L, lambda: fn(a["dtype"], a["q"], *cache, last, a["B"], a["R"], a["H"], a["Hkv"], a["dh"], f(0.1),
                              a["out"], a["ws"], a["ws_bytes"], None), 1)


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=7), 1), (dict(x=None), 1), (dict(x=P(4097)), 1), (dict(x=P(4098), dtype=m.F32), 1), (dict(t=None), 1), (dict(lp=None), 1),
    (dict(en=None), 1), (dict(rk=None), 1), (dict(ids=None), 1), (dict(tl=None), 1), (dict(N=0), 1),
    (dict(N=(1 << 30) + 1), 1),
    (dict(V=0), 1), (dict(V=(1 << 24) + 1, step=1 << 25), 1), (dict(step=999), 1), (dict(step=1 << 41), 1),
    (dict(top=-1), 1), (dict(top=17), 1), (dict(V=4, top=5), 1), (dict(temp=0.0), 1), (dict(temp=-1.0), 1),
    (dict(temp=math.nan), 1), (dict(temp=math.inf), 1), (dict(temp=1e-31), 1), (dict(ws=None), 3),
    (dict(ws_bytes=255), 3), (dict(ws=P((1 << 20) + 16)), 3)])
def test_logprobs_refuse(L, kw, code):
    a = dict(dtype=m.BF16, x=A, step=1000, t=A, N=3, V=1000, top=5, temp=1.0, lp=A, en=A, rk=A, ids=A, tl=A, ws=WS,
             ws_bytes=256)
    a.update(kw)
    refused(L, lambda: L.medusa_token_logprobs(a["dtype"], a["x"], a["step"], a["t"], a["N"], a["V"], a["top"],
                                               f(a["temp"]), a["lp"], a["en"], a["rk"], a["ids"], a["tl"], a["ws"],
                                               a["ws_bytes"], None), code)


def test_workspace_sizes(L):
    size = m.paged_attention_workspace_size
    for dt in (m.BF16, m.F32):
        assert size(dt, 1, 1, 8, 8, 128, 0) == m.WS_HEADER
        assert size(dt, 1, 65, 32, 8, 128, 100000) > m.WS_HEADER
        for bad in ((dt, 0, 1, 8, 8, 128, 0), (dt, 1, 0, 8, 8, 128, 0), (dt, 1, (1 << 20) + 1, 8, 8, 128, 0),
                    (dt, 1, 1, 9, 8, 128, 0), (dt, 1, 1, 8, 8, 96, 0), (dt, 1, 1, 8, 8, 64, -1), (9, 1, 1, 8, 8, 64, 1)):
            assert size(*bad) == 0
    with pytest.raises(ValueError):
        size(m.BF16, 1, 1, 8, 8, 128, 2 ** 31)


def test_binding_refuses_before_the_library():
    pool = torch.zeros(4, 16, 2, 64)
    tab = torch.zeros(3, 5, dtype=torch.int32)
    ok = dict(k_pages=pool, v_pages=pool, page_table=tab, B=3, Hkv=2, dh=64, dtype=torch.float32, dev=-1)
    assert m._pages(**ok)[2:4] == (4, 16) and m._pages(**ok)[5] == 5
    for bad in (dict(k_pages=pool[0]), dict(k_pages=pool.bfloat16()), dict(v_pages=pool[:3]), dict(Hkv=1), dict(dh=128),
                dict(page_table=tab[:2]), dict(page_table=tab.long()), dict(page_table=tab[:, ::2]),
                dict(page_table=tab[0]), dict(v_pages=pool.transpose(1, 2)), dict(dev=0)):
        with pytest.raises(ValueError):
            m._pages(**{**ok, **bad})
    assert m._row_step(torch.zeros(3, 4, 10)[..., :7], "x") == 10
    assert m._row_step(torch.zeros(5, 10), "x") == 10 and m._row_step(torch.zeros(1, 20)[:, :9], "x") == 9
    assert m._row_step(torch.zeros(6, 1, 8, 10)[..., :3], "x") == 10
    for bad in (torch.zeros(10, 5).T, torch.zeros(3, 4, 10)[:, :2], torch.zeros(4, 10)[:, ::2]):
        with pytest.raises(ValueError):
            m._row_step(bad, "x")
    for call in (lambda: m.token_logprobs(pool, tab), lambda: m.paged_append(pool, pool, pool, pool, tab, tab, 0),
                 lambda: m.chunk_attention_paged(pool, pool, pool, tab, tab, 0)):
        with pytest.raises(ValueError):  # not on a GPU
            call()
    with pytest.raises(TypeError):
        m.token_logprobs(pool.half(), tab)


def test_references_by_hand():
    x = np.log(np.array([[1.0, 2.0, 1.0, 4.0], [0.0 + 1e-300, 1.0, 1.0, 1e-300]]))
    r = ref.logprobs(x, np.array([2, 2]), 3, 1.0)
    assert r["ids"].tolist() == [[3, 1, 0], [1, 2, 0]] and r["rank"].tolist() == [3, 1]
    assert np.allclose(r["logp"], [math.log(1 / 8), math.log(0.5)])
    assert np.allclose(r["entropy"], [0.125 * math.log(8) * 2 + 0.25 * math.log(4) + 0.5 * math.log(2), math.log(2)])
    assert ref.causal(2, 2).tolist() == [[True, True, True, False], [True] * 4]
    tab, pages = ref.table(torch.Generator().manual_seed(0), [2, 0, 3])
    assert pages == 8 and len(set(tab[tab >= 0].tolist())) == 5
    pool = torch.arange(8 * 16, dtype=torch.float64).view(8, 16, 1, 1)
    s = ref.sequence(pool, tab, 2, 40)
    assert s[17] == int(tab[2, 1]) * 16 + 1 and s.shape[0] == 40
    v = torch.tensor([[[1.0]], [[math.inf]]], dtype=torch.float64)
    out, _, _ = ref.attention(torch.zeros(2, 1, 1).double(), torch.zeros(2, 1, 1).double(), v,
                              torch.tensor([[True, False], [True, True]]), 1.0)
    assert out.flatten().tolist() == [1.0, math.inf]
