"""Refusals of the operators for prompts: the C ABI checks its arguments on the
host before anything reaches the GPU, and the binding its tensors (CPU)."""
import ctypes

import pytest

import moe_speculative_decoding_router_amd as m

P = 4096  # an aligned address that no refused call touches


@pytest.fixture(scope="module")
def lib():
    return m.lib()


def ints(*v):
    return (ctypes.c_int32 * len(v))(*v)


def address(a):
    return None if a is None else ctypes.addressof(a)


def refused(lib, fn, cases):
    for kw, rc, word in cases:
        assert fn(lib, **kw) == rc, kw
        assert word in lib.moe_last_error(), (kw, lib.moe_last_error())


def attend(lib, q=P, k=P, v=P, qs=1024, ks=256, vs=256, q_off=(0, 3), k_off=(0, 5), nseq=None, Hq=8, Hkv=2, D=128, dtype=1, scale=1.0,
           out=P, ws=P, n=1 << 40):
    a, b = (None if x is None else ints(*x) for x in (q_off, k_off))
    return lib.prompt_attend(q, k, v, qs, ks, vs, len(q_off or k_off) - 1 if nseq is None else nseq, address(a), address(b), Hq, Hkv, D, dtype,
                             scale, out, ws, n, None)


def test_prompt_attend(lib):
    nan = float("nan")
    refused(lib, attend, [
        ({"q": None}, -1, b"q and out"), ({"out": None}, -1, b"q and out"), ({"k": None}, -1, b"k and v"), ({"v": None}, -1, b"k and v"),
        ({"qs": 1023}, -1, b"q_stride"), ({"ks": 255}, -1, b"k_stride"), ({"vs": 260}, -1, b"v_stride"), ({"ks": (1 << 24) + 8}, -2, b"2^24"),
        ({"q_off": None}, -1, b"q_off"), ({"k_off": None}, -1, b"k_off"), ({"nseq": 0}, -1, b"nseq"), ({"nseq": 65}, -1, b"nseq"),
        ({"q_off": (1, 3)}, -1, b"run from 0"), ({"k_off": (0, 4, 2, 5), "q_off": (0, 1, 2, 3)}, -1, b"decrease"),
        ({"q_off": (0, (1 << 22) + 1)}, -1, b"2^22"), ({"k_off": (0, -1)}, -1, b"k_off"), ({"Hq": 7}, -1, b"Hq"), ({"Hq": 0}, -1, b"Hq"),
        ({"Hq": 16384, "qs": 1 << 22}, -1, b"Hq"), ({"Hkv": 0}, -1, b"Hkv"), ({"D": 96}, -2, b"D=96"), ({"dtype": 2}, -2, b"dtype"),
        ({"scale": nan}, -1, b"scale"), ({"q": P + 8}, -1, b"aligned"), ({"out": P + 2}, -1, b"aligned"), ({"dtype": 0, "n": 16}, -3, b"workspace"),
        ({"dtype": 0, "ws": None}, -1, b"workspace"), ({"dtype": 0, "ws": P + 16}, -1, b"aligned"),
        ({"q_off": (0, 1 << 22), "Hq": 8192, "qs": 1 << 20}, -2, b"2^23"),
        ({"k_off": (0, 1 << 22), "dtype": 0, "Hkv": 64, "Hq": 64, "qs": 8192, "ks": 8192, "vs": 8192}, -2, b"2^33")])
    off = ints(0, 3)
    size = lambda *a: lib.prompt_attend_workspace_bytes(1, address(off), address(ints(0, 5)), *a)  # noqa: E731
    assert size(8, 2, 128, 0) >= 5 * 2 * 128 * 12 and size(8, 2, 128, 1) == 0 and size(8, 3, 128, 0) == 0
    assert attend(lib, q=None, k=None, v=None, q_off=(0, 0), k_off=(0, 0), out=None, ws=None, n=0) == 0


def layer(**kw):
    base = dict(H=512, I=256, E=32, k=4, wdtype=m.MOE_BF16, Wr=P, W_gu=P, W_d=P)
    base.update(kw)
    L = m._Layer()
    for k, v in base.items():
        setattr(L, k, v)
    return L


def experts(lib, L=None, x=P, xs=512, T=100, dtype=1, idx=P, w=P, y=P, ws=P, n=1 << 50):
    return lib.moe_experts(ctypes.byref(L or layer()), x, xs, T, dtype, idx, w, y, ws, n, None)


def test_experts(lib):
    refused(lib, experts, [
        ({"x": None}, -1, b"x, topk_idx"), ({"idx": None}, -1, b"x, topk_idx"), ({"w": None}, -1, b"x, topk_idx"), ({"y": None}, -1, b"x, topk_idx"),
        ({"ws": None}, -1, b"x, topk_idx"), ({"xs": 511}, -1, b"x_stride"), ({"xs": 516}, -1, b"x_stride"), ({"T": -1}, -1, b"T=-1"),
        ({"T": (1 << 20) + 1}, -1, b"2^20"), ({"dtype": 2}, -2, b"dtype"), ({"x": P + 8}, -1, b"aligned"), ({"ws": P + 16}, -1, b"aligned"),
        ({"n": 4096}, -3, b"workspace"), ({"L": layer(wdtype=0)}, -2, b"float32 weights"), ({"L": layer(H=520)}, -2, b"H=520"),
        ({"L": layer(k=33, E=64)}, -1, b"k=33"), ({"L": layer(E=513)}, -1, b"E=513"), ({"L": layer(W_d=None)}, -1, b"W_d"),
        ({"L": layer(wdtype=2)}, -1, b"s_gu"), ({"L": layer(Wsh_gu=P)}, -1, b"shared"), ({"L": layer(W_gu=P + 8)}, -1, b"weights"),
        ({"L": layer(H=16384, E=512, k=32), "T": 1 << 20, "xs": 16384}, -2, b"grid")])
    assert experts(lib, T=0, x=None, idx=None, w=None, y=None, ws=None, n=0) == 0
    need = lib.moe_experts_workspace_bytes(ctypes.byref(layer()), 100, 1)
    assert need > 0 and experts(lib, n=need - 1) == -3 and lib.moe_experts_workspace_bytes(ctypes.byref(layer(wdtype=0)), 100, 1) == 0


def route(lib, logits=P, stride=64, T=5, E=64, k=8, idx=P, w=P):
    return lib.route_tokens(logits, stride, T, E, k, idx, w, None)


def test_route_tokens(lib):
    refused(lib, route, [({"logits": None}, -1, b"logits"), ({"idx": None}, -1, b"topk_idx"), ({"w": None}, -1, b"topk_w"), ({"stride": 63}, -1, b"stride"),
                         ({"T": -1}, -1, b"T=-1"), ({"E": 0}, -1, b"E=0"), ({"E": 513, "stride": 513}, -1, b"E=513"), ({"k": 0}, -1, b"k=0"),
                         ({"k": 33}, -1, b"k=33"), ({"k": 5, "E": 4}, -1, b"k=5")])
    assert route(lib, T=0, logits=None, idx=None, w=None) == 0


def cache(**kw):
    c = dict(data=P, num_pages=4, page=16, Hkv=2, D=128)
    c.update(kw)
    return m._KvCache(c["data"], c["num_pages"], c["page"], c["Hkv"], c["D"])


def rows(*off, table=P, max_pages=8, start=P):
    a = ints(*off)
    r = m._KvRows(table, max_pages, start, len(off) - 1, ctypes.addressof(a))
    r._keep = a
    return r


def read(lib, c=None, r=None, k=P, v=P, T=3, dtype=1):
    return lib.kv4_read(ctypes.byref(c or cache()), ctypes.byref(r or rows(0, 3)), k, v, T, dtype, None)


def copy(lib, c=None, pairs=P, n=3):
    return lib.kv4_copy_pages(ctypes.byref(c or cache()), pairs, n, None)


def test_read_and_copy(lib):
    bad = [({"c": cache(D=96)}, -2, b"D=96"), ({"c": cache(page=24)}, -1, b"page"), ({"c": cache(num_pages=0)}, -1, b"num_pages"),
           ({"c": cache(Hkv=0)}, -1, b"Hkv"), ({"c": cache(data=None)}, -1, b"data"), ({"c": cache(data=P + 8)}, -1, b"aligned")]
    refused(lib, read, bad + [({"k": None}, -1, b"k and v"), ({"v": P + 8}, -1, b"aligned"), ({"T": 4}, -1, b"seg_off"), ({"T": -1}, -1, b"T=-1"),
                              ({"T": (1 << 22) + 1}, -1, b"2^22"), ({"dtype": 2}, -2, b"dtype"), ({"r": rows(0, 3, table=None)}, -1, b"table"),
                              ({"c": cache(Hkv=1024), "r": rows(0, 1 << 22), "T": 1 << 22}, -2, b"2^28"),
                              ({"r": rows(0, 3, start=None)}, -1, b"len"), ({"r": rows(0, 3, max_pages=0)}, -1, b"max_pages")])
    refused(lib, copy, bad + [({"pairs": None}, -1, b"pairs"), ({"n": -1}, -1, b"n=-1"), ({"n": (1 << 24) + 1}, -1, b"2^24")])
    assert read(lib, r=rows(0, 0), T=0, k=None, v=None) == 0 and copy(lib, n=0, pairs=None) == 0


def pool(**kw):
    p = dict(refs=P, table=P, num_pages=100, page=16, nseq=4, max_pages=8)
    p.update(kw)
    return m._KvPool(p["refs"], p["table"], p["num_pages"], p["page"], p["nseq"], p["max_pages"])


def reserve(lib, p=None, a=P, b=P, n=3, ok=P):
    return lib.kv4_reserve(ctypes.byref(p or pool()), a, b, n, ok, None)


def fork(lib, p=None, a=P, b=P, n=3, ok=P, rows_=P, pairs=P):
    return lib.kv4_fork(ctypes.byref(p or pool()), a, b, rows_, n, pairs, ok, None)


def release(lib, p=None, a=P, b=P, n=3):
    return lib.kv4_release(ctypes.byref(p or pool()), a, b, n, None)


def compact(lib, p=None, moves=5, pairs=P, ws=P, size=1 << 40):
    return lib.kv4_compact(ctypes.byref(p or pool()), moves, pairs, ws, size, None)


def test_pages(lib):
    bad = [({"p": pool(refs=None)}, -1, b"refs"), ({"p": pool(table=None)}, -1, b"table"), ({"p": pool(num_pages=0)}, -1, b"num_pages"),
           ({"p": pool(num_pages=(1 << 24) + 1)}, -1, b"2^24"), ({"p": pool(page=8)}, -1, b"page"), ({"p": pool(page=48)}, -1, b"page"),
           ({"p": pool(nseq=0)}, -1, b"nseq"), ({"p": pool(nseq=(1 << 16) + 1)}, -1, b"nseq"), ({"p": pool(max_pages=0)}, -1, b"max_pages"),
           ({"p": pool(max_pages=1 << 27)}, -1, b"max_pages"), ({"p": pool(nseq=1 << 16, max_pages=1 << 15)}, -1, b"2^30"),
           ({"p": pool(refs=P + 2)}, -1, b"aligned")]
    lists = [({"a": None}, -1, b"non-NULL"), ({"b": None}, -1, b"non-NULL"), ({"n": 65}, -1, b"n=65"), ({"n": -1}, -1, b"n=-1")]
    refused(lib, reserve, bad + lists + [({"ok": None}, -1, b"ok")])
    refused(lib, fork, bad + lists + [({"ok": None}, -1, b"ok"), ({"rows_": None}, -1, b"rows"), ({"pairs": None}, -1, b"pairs")])
    refused(lib, release, bad + lists)
    refused(lib, compact, bad + [({"moves": 0}, -1, b"max_moves"), ({"moves": (1 << 24) + 1}, -1, b"max_moves"), ({"pairs": None}, -1, b"pairs"),
                                 ({"ws": None}, -1, b"workspace"), ({"ws": P + 1}, -1, b"aligned"), ({"size": 64}, -3, b"workspace")])
    assert reserve(lib, n=0, a=None) == 0 and fork(lib, n=0, a=None) == 0 and release(lib, n=0, a=None) == 0
    need = lib.kv4_compact_workspace_bytes(ctypes.byref(pool()), 5)
    assert need > 400 and compact(lib, size=need - 1) == -3 and lib.kv4_compact_workspace_bytes(ctypes.byref(pool()), 0) == 0


def test_binding_refuses_before_the_library():
    torch = pytest.importorskip("torch")
    i = torch.zeros(2, dtype=torch.int32)
    c = m.KV4Cache(data=torch.zeros(2 * 16 * 68, dtype=torch.uint8), page=16, Hkv=1, D=64)
    k, x = torch.zeros((2, 1, 64)), torch.zeros((2, 64))
    L = m.LayerWeights(H=64, I=32, E=2, k=1, wdtype="bf16", Wr=x, W_gu=x, W_d=x)
    for call in (lambda: m.prompt_attend(k, k, k, [0, 2]), lambda: m.prompt_attend(k[0], k, k, [0, 2]), lambda: m.prompt_attend(k.double(), k, k, [0, 2]),
                 lambda: m.experts(x, L, i.view(2, 1), x[:, :1]), lambda: m.route_tokens(x, 2), lambda: m.kv4_read(c, i.view(1, 2), i[:1], [0, 2]),
                 lambda: m.kv4_copy_pages(c, i.view(1, 2)), lambda: m.kv4_reserve(i, i.view(1, 2), 16, i, i),
                 lambda: m.kv4_fork(i, i.view(1, 2), 16, i, i, i), lambda: m.kv4_release(i, i.view(1, 2), 16, i, i),
                 lambda: m.kv4_compact(i, i.view(1, 2)), lambda: m.kv4_compact(i.view(1, 2), i.view(1, 2))):
        with pytest.raises(ValueError):
            call()
