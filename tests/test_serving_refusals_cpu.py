"""Refusals of the serving operators: the C ABI checks its arguments on the
host before anything reaches the GPU, and the binding its tensors (CPU)."""
import ctypes

import numpy as np
import pytest

import moe_speculative_decoding_router_amd as m

P = 4096  # an aligned address that no refused call touches


@pytest.fixture(scope="module")
def lib():
    return m.lib()


def ints(*v):
    return (ctypes.c_int32 * len(v))(*v)


def cache(**kw):
    c = dict(data=P, num_pages=4, page=16, Hkv=2, D=128)
    c.update(kw)
    return m._KvCache(c["data"], c["num_pages"], c["page"], c["Hkv"], c["D"])


def rows(*off, table=P, max_pages=8, ln=P, nseq=None):
    a = ints(*off)
    r = m._KvRows(table, max_pages, ln, len(off) - 1 if nseq is None else nseq, ctypes.addressof(a) if off else None)
    r._keep = a
    return r


def append(lib, c=None, r=None, k=P, v=P, ks=256, vs=256, T=3, dtype=1, path=None, count=None, ko=None, vo=None):
    return lib.kv4_append(ctypes.byref(c or cache()), ctypes.byref(r or rows(0, 3)), k, v, ks, vs, T, dtype, path, count, ko, vo,
                          None)


def attend(lib, c=None, r=None, q=P, qs=1024, T=3, Hq=8, dtype=1, scale=1.0, parent=None, out=P, ws=P, n=1 << 40):
    return lib.kv4_attend(ctypes.byref(c or cache()), ctypes.byref(r or rows(0, 3)), q, qs, T, Hq, dtype, scale,
                          None if parent is None else ctypes.addressof(parent), out, ws, n, None)


def test_cache_bytes(lib):
    assert lib.kv4_cache_bytes(3, 64, 4, 128) == 3 * 64 * 4 * 2 * (64 + 4)
    assert lib.kv4_cache_bytes(1 << 20, 64, 8, 128) == (1 << 20) * 64 * 8 * 2 * 68
    for bad in ((0, 16, 1, 64), (1, 8, 1, 64), (1, 48, 1, 64), (1, 8192, 1, 64), (1, 16, 0, 64), (1, 16, 1, 96), (1, 16, 1, 32)):
        assert lib.kv4_cache_bytes(*bad) == 0, bad


@pytest.mark.parametrize("fn", [append, attend])
def test_cache_and_rows(lib, fn):
    for kw, rc, word in (({"c": cache(D=96)}, -2, b"D=96"), ({"c": cache(page=24)}, -1, b"page"), ({"c": cache(num_pages=0)}, -1, b"num_pages"),
                         ({"c": cache(Hkv=0)}, -1, b"Hkv"), ({"c": cache(data=None)}, -1, b"data"), ({"c": cache(data=P + 8)}, -1, b"aligned"),
                         ({"r": rows(0, 3, table=None)}, -1, b"table"), ({"r": rows(0, 3, ln=None)}, -1, b"len"),
                         ({"r": rows(0, 3, max_pages=0)}, -1, b"max_pages"), ({"r": rows(0, 3, max_pages=1 << 27)}, -1, b"max_pages"),
                         ({"r": rows(0, 2)}, -1, b"seg_off"), ({"r": rows(1, 3)}, -1, b"seg_off"), ({"r": rows(0, 2, 1, 3)}, -1, b"decrease"),
                         ({"r": rows(0, 3, nseq=0)}, -1, b"nseq"), ({"r": rows(*([0] * 65 + [3]))}, -1, b"nseq"), ({"T": 0}, -1, b"T=0"),
                         ({"dtype": 2}, -2, b"dtype")):
        assert fn(lib, **kw) == rc, kw
        assert word in lib.moe_last_error(), (kw, lib.moe_last_error())


def test_append_refusals(lib):
    for kw, word in (({"k": None}, b"k and v"), ({"v": None}, b"k and v"), ({"ks": 255}, b"k_stride"), ({"vs": 260}, b"v_stride"),
                     ({"path": P}, b"path and count"), ({"count": P}, b"path and count"), ({"ko": P}, b"k_out"),
                     ({"path": P, "count": P, "ko": P, "vo": P}, b"without path"), ({"k": P + 8}, b"aligned"),
                     ({"T": (1 << 20) + 1, "r": rows(0, (1 << 20) + 1)}, b"2^20")):
        assert append(lib, **kw) == -1, kw
        assert word in lib.moe_last_error(), (kw, lib.moe_last_error())


def test_attend_refusals(lib):
    for kw, rc, word in (({"T": 65, "r": rows(0, 65)}, -1, b"T=65"), ({"Hq": 7}, -1, b"Hq"), ({"Hq": 0}, -1, b"Hq"), ({"q": None}, -1, b"q and out"),
                         ({"out": None}, -1, b"q and out"), ({"qs": 1023}, -1, b"q_stride"), ({"scale": float("nan")}, -1, b"scale"),
                         ({"ws": None}, -1, b"workspace"), ({"ws": P + 4}, -1, b"aligned"), ({"n": 64}, -3, b"workspace"),
                         ({"parent": ints(0, 0, 1)}, -1, b"parent"), ({"parent": ints(-1, 1, 1)}, -1, b"parent"),
                         ({"parent": ints(-1, -1, 0)}, -1, b"parent"), ({"parent": ints(-1, 0, 0), "r": rows(0, 2, 3)}, -1, b"parent")):
        assert attend(lib, **kw) == rc, kw
        assert word in lib.moe_last_error(), (kw, lib.moe_last_error())
    need = lib.kv4_attend_workspace_bytes(ctypes.byref(cache()), ctypes.byref(rows(0, 3)), 3, 8, 1)
    assert need > 0 and attend(lib, n=need - 1) == -3
    assert lib.kv4_attend_workspace_bytes(ctypes.byref(cache()), ctypes.byref(rows(0, 3)), 3, 9, 1) == 0


def sample(lib, logits=P, stride=100, T=2, V=100, dtype=0, u=P, token=P, ws=P, n=1 << 40):
    return lib.sample_tokens(logits, stride, T, V, dtype, None, u, token, None, None, ws, n, None)


def accept(lib, logits=P, stride=100, T=3, V=100, dtype=0, tokens=P, off=(0, 3), parent=None, q=None, u=P, uf=None, out=P, path=P,
           count=P, ws=P, n=1 << 40):
    o = None if off is None else ints(*off)
    return lib.accept_drafts(logits, stride, T, V, dtype, None, tokens, 1 if off is None else len(off) - 1,
                             None if o is None else ctypes.addressof(o), None if parent is None else ctypes.addressof(parent), q, u, uf, out,
                             path, count, ws, n, None)


@pytest.mark.parametrize("fn", [sample, accept])
def test_logits_and_workspace(lib, fn):
    need = lib.sample_workspace_bytes(3, 100)
    assert need > 0 and lib.sample_workspace_bytes(3, 0) == 0 and lib.sample_workspace_bytes(3, (1 << 18) + 1) == 0
    for kw, rc, word in (({"logits": None}, -1, b"logits"), ({"stride": 99}, -1, b"stride"), ({"V": 0}, -1, b"V=0"),
                         ({"V": (1 << 18) + 1}, -2, b"2^18"), ({"dtype": 2}, -2, b"dtype"), ({"u": None}, -1, b"u"),
                         ({"ws": None}, -1, b"workspace"), ({"ws": P + 16}, -1, b"aligned"), ({"n": 16}, -3, b"workspace"),
                         ({"logits": P + 2}, -1, b"aligned")):
        assert fn(lib, **kw) == rc, kw
        assert word in lib.moe_last_error(), (kw, lib.moe_last_error())


def test_sample_refusals(lib):
    assert sample(lib, T=-1) == -1 and sample(lib, T=65536) == -1 and sample(lib, token=None) == -1
    assert sample(lib, T=0, logits=None, u=None, token=None, ws=None) == 0


def test_accept_refusals(lib):
    for kw, rc, word in (({"T": 0}, -1, b"T=0"), ({"T": 65, "off": (0, 65)}, -1, b"T=65"), ({"off": None}, -1, b"seg_off"),
                         ({"off": (0, 2)}, -1, b"seg_off"), ({"off": (0, 3, 2, 3)}, -1, b"decrease"), ({"parent": ints(-1, 2, 0)}, -1, b"parent"),
                         ({"tokens": None}, -1, b"tokens"), ({"out": None}, -1, b"out"), ({"path": None}, -1, b"path"), ({"count": None}, -1, b"count"),
                         ({"q": P}, -1, b"u_final"), ({"uf": P}, -1, b"u_final"),
                         ({"q": P, "uf": P, "parent": ints(-1, 0, 0)}, -2, b"chains")):
        assert accept(lib, **kw) == rc, kw
        assert word in lib.moe_last_error(), (kw, lib.moe_last_error())


def test_binding_refuses_before_the_library():
    torch = pytest.importorskip("torch")
    x, i = torch.zeros((2, 10)), torch.zeros(2, dtype=torch.int32)
    c = m.KV4Cache(data=torch.zeros(2 * 16 * 68, dtype=torch.uint8), page=16, Hkv=1, D=64)
    k = torch.zeros((2, 1, 64))
    for call in (lambda: m.sample_tokens(x, x[0]), lambda: m.sample_tokens(x.double(), x[0]), lambda: m.accept_drafts(x, i, [0, 2], x[:, 0]),
                 lambda: m.kv4_append(c, k, k, i.view(1, 2), i[:1], [0, 2]), lambda: m.kv4_attend(c, k, i.view(1, 2), i[:1], [0, 2]),
                 lambda: m.kv4_attend(c, k[0], i.view(1, 2), i[:1], [0, 2]), lambda: m.sample_tokens(x[0], x[0])):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(m.MoeError):
        m.kv4_cache(1, 24, 1, 64, device="cpu")
    assert m.kv4_cache(2, 32, 3, 128, device="cpu").num_pages == 2
    assert np.prod(m.kv4_cache(2, 32, 3, 128, device="cpu").data.shape) == m.lib().kv4_cache_bytes(2, 32, 3, 128)
