"""Refusals of the rotation, 4-bit cache and windowed attention calls, and the
4-bit reference's own definition: no GPU needed."""
import ctypes

import numpy as np
import pytest

import cache_ops_ref as ref
import medusa_speculative_decoding_02_gb300 as m
from medusa_speculative_decoding_02_gb300 import build as mbuild

P = ctypes.c_void_p
A = P(4096)          # fake, 16-byte aligned device address: never dereferenced
A2 = P(8192)
ODD = P(4100)
WS = P(1 << 20)
f = ctypes.c_float


@pytest.fixture(scope="module")
def L():
    mbuild.build()
    return m.lib()


def refused(L, rc, code):
    assert rc == code, (m.STATUS.get(rc), L.medusa_last_error())
    assert L.medusa_last_error().decode()


def _rope(L, append, **kw):
    a = dict(dtype=m.BF16, q=A, k=A, v=A, qs=4096, ks=1024, vs=1024, qw=None, kw=None, eps=1e-6, norm=1,
             pos=A, f=A, rot=128, inter=0, n=None, kc=A, vc=A, pl=A, P_max=100, B=2, R=5, H=32, Hkv=8, dh=128,
             qo=A, ko=A, ws=WS, ws_bytes=256)
    a.update(kw)
    head = (a["dtype"], a["q"], a["k"]) + ((a["v"],) if append else ()) + (a["qs"], a["ks"]) + \
        ((a["vs"],) if append else ()) + (a["qw"], a["kw"], f(a["eps"]), a["norm"], a["pos"], a["f"],
                                          a["rot"], a["inter"], a["n"])
    dims = (a["B"], a["R"], a["H"], a["Hkv"], a["dh"], a["qo"])
    if append:
        return L.medusa_qk_norm_rope_append(*head, a["kc"], a["vc"], a["pl"], a["P_max"], *dims, a["ws"],
                                            a["ws_bytes"], None)
    return L.medusa_qk_norm_rope(*head, *dims, a["ko"], None)


ROPE_BAD = [
    (dict(q=None), 1), (dict(k=None), 1), (dict(qo=None), 1), (dict(pos=None), 1), (dict(f=None), 1),
    (dict(q=ODD), 1), (dict(qo=ODD), 1), (dict(qw=ODD), 1), (dict(dtype=3), 1), (dict(B=0), 1),
    (dict(B=65536), 1), (dict(R=0), 1), (dict(R=(1 << 24) + 1), 1), (dict(B=1000, R=1 << 23), 1),
    (dict(H=30), 1), (dict(Hkv=0), 1), (dict(H=2048, Hkv=1), 1), (dict(dh=96), 2), (dict(rot=130), 1),
    (dict(rot=8), 1), (dict(rot=-16), 1), (dict(qs=4095), 1), (dict(qs=4100), 1), (dict(ks=1016), 1),
    (dict(norm=0, qw=A), 1), (dict(norm=0, kw=A), 1), (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1)]


@pytest.mark.parametrize("kw,code", ROPE_BAD + [(dict(ko=None), 1), (dict(ko=ODD), 1)])
def test_rope_rejects(L, kw, code):
    before = L.medusa_launch_count()
    refused(L, _rope(L, False, **kw), code)
    assert L.medusa_launch_count() == before


@pytest.mark.parametrize("kw,code", ROPE_BAD + [
    (dict(v=None), 1), (dict(v=ODD), 1), (dict(vs=8), 1), (dict(kc=None), 1), (dict(vc=ODD), 1),
    (dict(pl=None), 1), (dict(P_max=-1), 1), (dict(P_max=(1 << 29) + 1), 1), (dict(ws=None), 3),
    (dict(ws_bytes=128), 3), (dict(ws=P((1 << 20) + 16)), 3)])
def test_rope_append_rejects(L, kw, code):
    before = L.medusa_launch_count()
    refused(L, _rope(L, True, **kw), code)
    assert L.medusa_launch_count() == before


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=9), 1), (dict(k=None), 1), (dict(v=ODD), 1), (dict(ks=100), 1), (dict(vs=1028), 1),
    (dict(kc=None), 1), (dict(kc=ODD), 1), (dict(pl=None), 1), (dict(P_max=-2), 1), (dict(B=0), 1),
    (dict(R=0), 1), (dict(R=65536), 1), (dict(Hkv=0), 1), (dict(Hkv=1025), 1), (dict(dh=32), 2),
    (dict(ws=None), 3), (dict(ws_bytes=255), 3)])
@pytest.mark.parametrize("unpack", [False, True])
def test_kv4_rows_reject(L, kw, code, unpack):
    if unpack and set(kw) & {"ks", "vs"}:
        pytest.skip("dense outputs have no stride")
    a = dict(dtype=m.BF16, k=A, v=A, ks=1024, vs=1024, kc=A, vc=A, pl=A, P_max=9, n=None, B=1, R=4, Hkv=8,
             dh=128, ws=WS, ws_bytes=256)
    a.update(kw)
    before = L.medusa_launch_count()
    if unpack:
        rc = L.medusa_kv4_unpack(a["dtype"], a["kc"], a["vc"], a["pl"], a["P_max"], a["n"], a["B"], a["R"],
                                 a["Hkv"], a["dh"], a["k"], a["v"], a["ws"], a["ws_bytes"], None)
    else:
        rc = L.medusa_kv4_append(a["dtype"], a["k"], a["v"], a["ks"], a["vs"], a["kc"], a["vc"], a["pl"],
                                 a["P_max"], a["n"], a["B"], a["R"], a["Hkv"], a["dh"], a["ws"],
                                 a["ws_bytes"], None)
    refused(L, rc, code)
    assert L.medusa_launch_count() == before


@pytest.mark.parametrize("kw,code", [
    (dict(kc=None), 1), (dict(pl=None), 1), (dict(path=None), 1), (dict(al=None), 1), (dict(npl=A), 1),
    (dict(vc=ODD), 1), (dict(B=0), 1), (dict(K=9), 1), (dict(R=257), 1), (dict(Hkv=0), 1), (dict(dh=96), 2),
    (dict(ws_bytes=0), 3)])
def test_commit_kv4_rejects(L, kw, code):
    a = dict(kc=A, vc=A, pl=A, path=A, al=A, B=1, K=5, R=65, Hkv=32, dh=128, npl=A2, ws=WS, ws_bytes=256)
    a.update(kw)
    refused(L, L.medusa_commit_kv4(a["kc"], a["vc"], a["pl"], a["path"], a["al"], a["B"], a["K"], a["R"],
                                   a["Hkv"], a["dh"], a["npl"], a["ws"], a["ws_bytes"], None), code)


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=5), 1), (dict(q=None), 1), (dict(out=None), 1), (dict(mask=None), 1), (dict(k=None), 1),
    (dict(pl=None), 1), (dict(q=ODD), 1), (dict(out=ODD), 1), (dict(v=ODD), 1), (dict(B=0), 1),
    (dict(R=0), 1), (dict(R=257), 1), (dict(H=31), 1), (dict(Hkv=64), 1), (dict(dh=80), 2),
    (dict(P_max=-1), 1), (dict(P_max=1 << 30), 1), (dict(window=-1), 1), (dict(sinks=-1), 1),
    (dict(window=0, sinks=4), 1), (dict(depth=None), 1), (dict(scale=0.0), 1),
    (dict(scale=float("inf")), 1), (dict(ws=None), 3), (dict(ws_bytes=256), 3)])
@pytest.mark.parametrize("kind", ["window", "kv4"])
def test_attention_rejects(L, kw, code, kind):
    a = dict(dtype=m.BF16, q=A, k=A, v=A, pl=A, P_max=4096, mask=A, depth=A, window=512, sinks=4, B=1, R=65,
             H=32, Hkv=8, dh=128, scale=0.088, out=A, ws=WS, ws_bytes=1 << 30)
    a.update(kw)
    before = L.medusa_launch_count()
    rc = getattr(L, f"medusa_tree_attention_{kind}")(
        a["dtype"], a["q"], a["k"], a["v"], a["pl"], a["P_max"], a["mask"], a["depth"], a["window"],
        a["sinks"], a["B"], a["R"], a["H"], a["Hkv"], a["dh"], f(a["scale"]), a["out"], a["ws"],
        a["ws_bytes"], None)
    refused(L, rc, code)
    assert L.medusa_launch_count() == before


def test_sizes(L):
    assert m.kv4_row_bytes(32, 128) == 32 * 72 and m.kv4_row_bytes(1, 128) == 80
    assert m.kv4_row_bytes(1, 64) == 48 and m.kv4_row_bytes(3, 64) == 112
    for bad in ((0, 128), (1, 96), (-1, 64), (1025, 64)):
        assert m.kv4_row_bytes(*bad) == 0
    size = m.tree_attention_window_workspace_size
    for kv4 in (False, True):
        for dt in (m.BF16, m.F32):
            # with a window the workspace does not grow with the prefix
            near = size(dt, 8, 65, 32, 8, 128, 10000, 1024, 4, kv4)
            assert near == size(dt, 8, 65, 32, 8, 128, 1 << 29, 1024, 4, kv4) >= 256
            assert size(dt, 1, 65, 32, 8, 128, 10000, 0, 0, kv4) > 256
            for bad in ((dt, 0, 65, 32, 8, 128, 10), (dt, 1, 257, 32, 8, 128, 10), (dt, 1, 1, 30, 8, 128, 10),
                        (dt, 1, 1, 8, 8, 96, 10), (dt, 1, 1, 8, 8, 64, -1), (7, 1, 1, 8, 8, 64, 1)):
                assert size(*bad, kv4=kv4) == 0


def test_binding_refuses_before_the_library():
    import torch
    q = torch.zeros(1, 2, 4, 64)
    with pytest.raises(ValueError):  # heads not dense
        m._rows(torch.zeros(1, 2, 64, 4).transpose(2, 3), "q")
    with pytest.raises(ValueError):  # rows not evenly apart
        m._rows(torch.zeros(2, 4, 4, 64)[:, :3], "q")
    assert m._rows(torch.zeros(2, 3, 8, 64)[:, :, 2:5], "k") == 512
    assert m._rows(torch.zeros(5, 1, 8, 64)[:, :, 2:5], "k") == 512
    assert m._rows(torch.zeros(1, 1, 8, 64)[:, :, 2:5], "k") == 192
    # (a CPU tensor has device index -1: the checks run without a GPU)
    for bad in (dict(k=torch.zeros(1, 2, 4, 128)), dict(k=q.bfloat16()), dict(k=torch.zeros(1, 3, 4, 64)),
                dict(q_weight=torch.zeros(63)), dict(k_weight=torch.zeros(64).bfloat16()),
                dict(q_weight=torch.zeros(128)[::2])):
        a = dict(k=q, q_weight=None, k_weight=None, dev=-1)
        a.update(bad)
        with pytest.raises(ValueError):
            m._rope_args(q, *a.values())
    assert m._rope_args(q, q, None, torch.zeros(64), -1)[0] is None
    i32 = torch.zeros(6, dtype=torch.int32)
    assert m._vec(i32, 6, torch.int32, -1, "x") == i32.data_ptr()
    for t, n, dev in ((i32, 5, -1), (i32.long(), 6, -1), (i32, 6, 0), (i32[::2], 3, -1)):
        with pytest.raises(ValueError):
            m._vec(t, n, torch.int32, dev, "x")
    with pytest.raises(ValueError):
        m._dense(q.transpose(1, 2), (1, 4, 2, 64), torch.float32, -1, "out")
    with pytest.raises(ValueError):
        m._launch_on(q, None)
    with pytest.raises(ValueError):
        m.kv4_cache(4, 1, 100)
    with pytest.raises(TypeError):
        m.kv4_append(q.half(), q.half(), None, None, None, 0)


def test_reference_rounding():
    """The reference's grids against numbers worked out by hand."""
    assert ref.E4M3[1] == 2.0 ** -9 and ref.E4M3[8] == 2.0 ** -6 and ref.E4M3[126] == 448.0
    near = ref.nearest_even(np.array([0.25, 0.26, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 5.01, 9.0]), ref.E2M1)
    assert near.tolist() == [0, 1, 2, 2, 4, 4, 6, 6, 7, 7]
    x = np.zeros((1, 64))
    x[0, :16] = [6, -3, 0.3, 5, -5.1] + [0] * 11    # scale 1
    x[0, 16:32] = 1e9                                # scale 448, all codes 6
    x[0, 33] = np.nan
    c, s = ref.quantize(x)
    assert s.tolist() == [[56, 126, 127, 0]]
    assert c[0, :5].tolist() == [7, 13, 1, 6, 15] and (c[0, 16:32] == 7).all() and not c[0, 32:].any()
    v = ref.unpack_rows(ref.pack_rows(x[:, None]), 1, 64)
    assert v[0, 0, :5].tolist() == [6, -3, 0.5, 4, -6] and (v[0, 0, 16:32] == 2688).all()
    assert np.isnan(v[0, 0, 32:48]).all() and (v[0, 0, 48:] == 0).all()
