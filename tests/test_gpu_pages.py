"""Rows read back from the 4-bit cache (kv4_read) and the pages' bookkeeping
(kv4_reserve, kv4_fork, kv4_release, kv4_compact, kv4_copy_pages), equal to
the oracle's: all of it is whole numbers or exact values."""
import random

import numpy as np
import pytest

from oracle import kv4 as okv
from oracle import pages as op

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import moe_speculative_decoding_router_amd as m  # noqa: E402

DEV = torch.device("cuda:0")
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def dev(a, dtype=torch.int32):
    return torch.tensor(a, dtype=dtype, device=DEV)


def random_cache(seed, P, Hkv, page, D):
    rng = np.random.default_rng(seed)
    data = rng.integers(0, 256, (P, Hkv, page // 16, 17 * D), dtype=np.uint8)
    for a in (8 * D, 33 * D // 2):  # scales that append writes: 2^-100 .. 2^125
        data[..., a:a + D // 2] = rng.integers(27, 253, data[..., a:a + D // 2].shape)
    return data


def read_ref(data, table, start, off):
    P, Hkv, tiles, w = data.shape
    page, D = tiles * 16, w // 17
    out = np.zeros((2, off[-1], Hkv, D))
    for s in range(len(off) - 1):
        for t in range(off[s], off[s + 1]):
            pos = max(start[s], 0) + t - off[s]
            if pos // page < table.shape[1] and 0 <= table[s, pos // page] < P:
                for h in range(Hkv):
                    k, v = okv.read_rows(data, np.array([table[s, pos // page]]), h, [pos])
                    out[0, t, h], out[1, t, h] = k[0], v[0]
    return out


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("page", [16, 64])
def test_read(D, dtype, page):
    off, start = [0, 1, 1, 38, 105], [0, 5, 13, 60]
    data = random_cache(D + page, 11, 2, page, D)
    rng = np.random.default_rng(5)
    table = rng.integers(-1, 12, (4, 7)).astype(np.int32)  # some outside the pool, some twice
    cache = m.KV4Cache(data=torch.from_numpy(data).to(DEV), page=page, Hkv=2, D=D)
    k, v = m.kv4_read(cache, dev(table), dev(start), off, dtype=DT[dtype])
    ref = read_ref(data, table, start, off)
    assert np.array_equal(k.double().cpu().numpy(), ref[0]) and np.array_equal(v.double().cpu().numpy(), ref[1])


def test_read_of_appended_rows_is_what_append_returned():
    g = torch.Generator(device=DEV).manual_seed(3)
    k, v = (torch.randn((301, 3, 128), generator=g, device=DEV, dtype=torch.float32) for _ in range(2))
    cache = m.kv4_cache(30, 32, 3, 128, device=DEV)
    off, table, zero = [0, 200, 301], torch.randperm(30, device=DEV).to(torch.int32).view(2, 15), dev([0, 0])
    sk, sv = m.kv4_append(cache, k, v, table, zero, off, return_stored=True)
    out = (torch.empty_like(k), torch.empty_like(v))
    rk, rv = m.kv4_read(cache, table, zero, off, out=out)
    assert rk is out[0] and torch.equal(rk, sk) and torch.equal(rv, sv)
    part = m.kv4_read(cache, table, dev([190, -4]), [0, 5, 25], dtype=torch.float32)[0]  # a negative start counts as 0
    assert torch.equal(part[:5], sk[190:195]) and torch.equal(part[5:], sk[200:220])


def test_read_of_nothing_and_past_the_table():
    cache = m.kv4_cache(4, 16, 1, 64, device=DEV)
    cache.data.zero_()
    table = dev([[0, 1]])
    k, v = m.kv4_read(cache, table, dev([0]), [0, 0])
    assert k.shape == (0, 1, 64) and v.dtype == torch.bfloat16
    cache.data.fill_(0x77)
    k, _ = m.kv4_read(cache, table, dev([30]), [0, 5], dtype=torch.float32)
    assert (k[:2] != 0).all() and (k[2:] == 0).all()
    k, _ = m.kv4_read(cache, table, dev([2 ** 31 - 1]), [0, 5], dtype=torch.float32)
    assert (k == 0).all()


def test_read_above_4_gib():
    cache = m.kv4_cache(130000, 16, 16, 128, device=DEV)  # 4.5 GB
    off, zero = [0, 20], dev([0])
    table = dev([[129999, 129990]])
    k = torch.randn((20, 16, 128), device=DEV)
    sk, sv = m.kv4_append(cache, k, k + 1, table, zero, off, return_stored=True)
    rk, rv = m.kv4_read(cache, table, zero, off, dtype=torch.float32)
    assert torch.equal(rk, sk) and torch.equal(rv, sv)
    m.kv4_copy_pages(cache, dev([[129999, 1], [129990, 129980]]))
    rk, rv = m.kv4_read(cache, dev([[1, 129980]]), zero, off, dtype=torch.float32)
    assert torch.equal(rk, sk) and torch.equal(rv, sv)


class Pool:
    """The device's pool beside the oracle's."""

    def __init__(self, P, S, W, page=16):
        self.refs, self.table, self.page = [0] * P, [[-1] * W for _ in range(S)], page
        self.drefs, self.dtable = dev(self.refs), dev(self.table)

    def same(self):
        assert self.drefs.tolist() == self.refs and self.dtable.tolist() == self.table

    def reserve(self, seq, rows):
        ok = m.kv4_reserve(self.drefs, self.dtable, self.page, dev(seq), dev(rows)).tolist()
        assert ok == op.reserve(self.refs, self.table, self.page, seq, rows)
        self.same()
        return ok

    def fork(self, src, dst, rows):
        pairs, ok = m.kv4_fork(self.drefs, self.dtable, self.page, dev(src), dev(dst), dev(rows))
        rp, ro = op.fork(self.refs, self.table, self.page, src, dst, rows)
        assert ok.tolist() == ro and pairs.tolist() == rp
        self.same()
        return ro

    def release(self, seq, keep):
        m.kv4_release(self.drefs, self.dtable, self.page, dev(seq), dev(keep))
        op.release(self.refs, self.table, self.page, seq, keep)
        self.same()

    def compact(self, moves=None):
        pairs = m.kv4_compact(self.drefs, self.dtable, moves).tolist()
        n = max(1, len(self.refs) // 2) if moves is None else moves
        ref = op.compact(self.refs, self.table, n)
        assert [tuple(p) for p in pairs] == ref
        self.same()
        return ref


def test_page_hand_cases():
    p = Pool(6, 3, 4)
    assert p.reserve([1, 0], [33, 16]) == [1, 1]
    assert p.reserve([0, 2], [64, 20]) == [0, 1]
    p.release([2], [0])
    assert p.fork([1], [2], [40]) == [1]
    p.release([0, 1], [0, 0])
    assert p.compact(3) == [(4, 2), (-1, -1), (-1, -1)]
    assert p.compact(1) == [(-1, -1)]
    p.release([2, 2], [40, 10])  # one sequence named twice
    p.reserve([], [])
    p.fork([], [], [])
    p.release([], [])


@pytest.mark.parametrize("seed", range(8))
def test_random_page_lives(seed):
    rnd = random.Random(seed)
    page = rnd.choice([16, 64, 4096])
    P, S, W = rnd.choice([1, 7, 60, 300]), rnd.randint(1, 70), rnd.choice([1, 5, 70, 200])
    p = Pool(P, S, W, page)
    for _ in range(25):
        k = rnd.randint(1, 64)
        names = [rnd.randint(-1, S) for _ in range(k)]
        rows = [rnd.choice([rnd.randint(-3, 3 * page), rnd.randint(0, W * page + page), rnd.randint(0, W) * page]) for _ in range(k)]
        what = rnd.randint(0, 4)
        if what <= 1:
            p.reserve(names, rows)
        elif what == 2:
            p.fork([rnd.randint(-1, S // 2) for _ in range(k)], [rnd.randint(S // 4, S) for _ in range(k)], rows)
        elif what == 3:
            p.release(names[:5], rows[:5])
        else:
            p.compact(rnd.choice([None, 1, 3, 40]))


def test_large_pool():
    """Pages beyond one pass of the search, the lowest ones taken."""
    P = 40000
    refs, table = torch.ones(P, dtype=torch.int32, device=DEV), torch.full((70, 300), -1, dtype=torch.int32, device=DEV)
    free = torch.cat([torch.arange(8100, 8300), torch.arange(16000, 33000, 7), torch.tensor([P - 1])])
    refs[free.to(DEV)] = 0
    ok = m.kv4_reserve(refs, table, 16, torch.arange(64, device=DEV, dtype=torch.int32), dev([16 * (3 * i) for i in range(64)]))
    need, served = [3 * i for i in range(64)], ok.tolist()
    at = 0
    for i in range(64):
        fits = need[i] <= len(free) - at
        assert served[i] == int(fits)
        if fits:
            assert table[i, :need[i]].tolist() == free[at:at + need[i]].tolist()
            at += need[i]
    assert int((refs == 0).sum()) == len(free) - at
    refs = (torch.rand(100003, device=DEV) < 0.6).to(torch.int32)
    held = torch.nonzero(refs)[:, 0]
    table = torch.full((3, 40000), -1, dtype=torch.int32, device=DEV)
    table.view(-1)[:len(held)] = held[torch.randperm(len(held), device=DEV)].to(torch.int32)
    before, U = table.clone(), len(held)
    pairs = m.kv4_compact(refs, table)
    assert (refs[:U] == 1).all() and (refs[U:] == 0).all()
    live = pairs[pairs[:, 0] >= 0].long()
    to = torch.arange(100003, device=DEV)
    to[live[:, 0]] = live[:, 1]
    assert torch.equal(table.long(), torch.where(before >= 0, to[before.long().clamp(min=0)], -1))
    assert (live[:, 0].diff() < 0).all() and (live[:, 1].diff() > 0).all() and len(live) == int((held >= U).sum())


@pytest.mark.parametrize("D,Hkv,page", [(64, 1, 16), (128, 4, 64), (256, 3, 256)])
def test_copy_pages(D, Hkv, page):
    data = random_cache(1, 20, Hkv, page, D)
    cache = m.KV4Cache(data=torch.from_numpy(data).to(DEV), page=page, Hkv=Hkv, D=D)
    m.kv4_copy_pages(cache, dev([[3, 4], [-1, 5], [6, -1], [20, 7], [8, 20], [9, 9], [3, 19], [0, 1]]))
    data[[4, 19, 1]] = data[[3, 3, 0]]
    assert np.array_equal(cache.data.cpu().numpy(), data)
    m.kv4_copy_pages(cache, torch.empty((0, 2), dtype=torch.int32, device=DEV))


def test_forked_prompt_goes_its_own_way():
    """A prompt shared by three answers, in two layers: rows appended to one are seen by it alone."""
    page, D, Hkv, n = 16, 64, 2, 37
    g = torch.Generator(device=DEV).manual_seed(1)
    pool = Pool(40, 5, 4, page)
    caches = [m.kv4_cache(40, page, Hkv, D, device=DEV) for _ in range(2)]
    rows = [torch.randn((2, n + 9, Hkv, D), generator=g, device=DEV) for _ in caches]
    pool.reserve([0], [n])
    zero = dev([0])
    stored = []
    for c, r in zip(caches, rows):
        stored.append(m.kv4_append(c, r[0, :n], r[1, :n], pool.dtable[:1], zero, [0, n], return_stored=True)[0])
    pairs, ok = m.kv4_fork(pool.drefs, pool.dtable, page, dev([0, 0, 0]), dev([1, 2, 3]), dev([n, n, 32]))
    assert ok.tolist() == [1, 1, 1] and pairs[2].tolist() == [-1, -1]
    for c in caches:
        m.kv4_copy_pages(c, pairs)
    m.kv4_reserve(pool.drefs, pool.dtable, page, dev([1]), dev([n + 9]))
    table = pool.dtable[:4].clone()
    for c, r, st in zip(caches, rows, stored):
        own = m.kv4_append(c, r[0, n:], r[1, n:], table[1:2].contiguous(), dev([n]), [0, 9], return_stored=True)[0]
        got = m.kv4_read(c, table, dev([0, 0, 0, 0]), [0, n, 2 * n + 9, 3 * n + 9, 3 * n + 41], dtype=torch.float32)[0]
        assert torch.equal(got[:n], st) and torch.equal(got[n:2 * n], st) and torch.equal(got[2 * n:2 * n + 9], own)
        assert torch.equal(got[2 * n + 9:3 * n + 9], st) and torch.equal(got[3 * n + 9:], st[:32])


def test_pages_in_a_graph():
    """Captured once, replayed on other tables, eager work in between."""
    P, page = 64, 16
    refs, table = torch.zeros(P, dtype=torch.int32, device=DEV), torch.full((4, 8), -1, dtype=torch.int32, device=DEV)
    seq, rows, src, dst = dev([0, 1]), dev([40, 100]), dev([0]), dev([2])
    cache = m.kv4_cache(P, page, 1, 64, device=DEV)
    cache.data.random_(0, 256)

    def step():
        ok = m.kv4_reserve(refs, table, page, seq, rows)
        pairs, ok2 = m.kv4_fork(refs, table, page, src, dst, rows[:1].contiguous())
        m.kv4_copy_pages(cache, pairs)
        m.kv4_release(refs, table, page, dst, dev0)
        moves = m.kv4_compact(refs, table, 8)
        m.kv4_copy_pages(cache, moves)
        return ok, pairs, ok2, moves
    dev0 = dev([16])
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for fill in (0, 1, 2):
        start = torch.zeros(P, dtype=torch.int32, device=DEV)
        start[torch.arange(0, P, fill + 2, device=DEV)] = 1
        datum = torch.randint(0, 256, cache.data.shape, dtype=torch.uint8, device=DEV)
        refs.copy_(start), table.fill_(-1), cache.data.copy_(datum)
        graph.replay()
        torch.cuda.synchronize()
        got = [x.clone() for x in (refs, table, cache.data, *out)]
        refs.copy_(start), table.fill_(-1), cache.data.copy_(datum)
        ref = [refs, table, cache.data, *step()]
        for a, b in zip(got[:2] + got[3:], ref[:2] + ref[3:]):
            assert torch.equal(a, b)
        assert torch.equal(got[2], ref[2])


def test_pages_on_another_stream():
    refs, table = torch.zeros(50, dtype=torch.int32, device=DEV), torch.full((2, 8), -1, dtype=torch.int32, device=DEV)
    s = torch.cuda.Stream()
    seq, rows = dev([0]), dev([100])
    s.wait_stream(torch.cuda.current_stream())
    ok = m.kv4_reserve(refs, table, 16, seq, rows, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert ok.tolist() == [1] and table[0].tolist() == list(range(7)) + [-1]
