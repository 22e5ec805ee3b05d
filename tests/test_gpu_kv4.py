"""The 4-bit K/V cache (kv4_append, kv4_attend) against the float64 oracle.

Append is compared byte for byte.  Attention: with q exact, scores carry the
float32 products' and sums' error, at most (D + 4) 2^-24 sum |q K| scale; a
relative error of that size enters every probability twice (through itself
and the sum), the running sums and rescalings add at most (rows + 64) 2^-24,
and float32 operands are exact to 2^-23 in three bf16 terms.  bf16 rounds the
probabilities (2^-8 / 2 relative, twice with the sum) and the result (2^-8)."""
import numpy as np
import pytest

from oracle import kv4 as okv

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import moe_speculative_decoding_router_amd as m  # noqa: E402

DEV = torch.device("cuda:0")
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def rounded(rng, shape, dtype, scale=1.0):
    """Host float64 values that the device type holds exactly, and the device tensor."""
    t = torch.from_numpy((scale * rng.normal(size=shape)).astype(np.float32)).to(DT[dtype])
    return t.double().numpy(), t.to(DEV)


def setup(seed, D, Hkv, page, lens, offsets, spare=2):
    """A table of random pages (-1 past the needed ones) over a pool of 0xff bytes."""
    rng = np.random.default_rng(seed)
    need = [max(1, -(-(max(0, x) + offsets[s + 1] - offsets[s]) // page)) for s, x in enumerate(lens)]
    pool = sum(need) + spare
    ids = rng.permutation(pool).astype(np.int32)
    table = np.full((len(lens), max(need) + 1), -1, dtype=np.int32)
    at = 0
    for s, n in enumerate(need):
        table[s, :n] = ids[at:at + n]
        at += n
    data = np.full((pool, Hkv, page // 16, 17 * D), 0xFF, dtype=np.uint8)
    return rng, table, data


def cache_of(data_dev, D, Hkv, page):
    return m.KV4Cache(data=data_dev, page=page, Hkv=Hkv, D=D)


def fill(rng, data, table, lens, D, Hkv, big=1.0):
    """Oracle-quantised rows for every position before the call."""
    for s, n in enumerate(lens):
        if n > 0:
            k, v = big * rng.normal(size=(n, Hkv, D)), rng.normal(size=(n, Hkv, D))
            okv.append(data, k, v, table[s:s + 1], [0], [0, n])


def check_attend(out, q, data, table, lens, offsets, parent, scale, dtype, only=slice(None)):
    """only: the call rows that are compared (the bound is theirs and the others')."""
    with np.errstate(over="ignore", invalid="ignore"):
        ref, bound, reach = okv.attend(data, q, table, lens, offsets, parent, scale)
    ref, bound, out = ref[only], bound[only], out[only]
    rows = max(max(0, x) for x in lens) + max(b - a for a, b in zip(offsets, offsets[1:]))
    D = q.shape[-1]
    rel = 2 * (D + 4) * 2.0 ** -24 * reach + (rows + 64) * 2.0 ** -24 + 4 * 2.0 ** -23 * (1 + reach)
    if dtype == "bf16":
        rel += 2 * 2.0 ** -8
    tol = rel * bound + (2.0 ** -8 * np.abs(ref) if dtype == "bf16" else 2.0 ** -24 * np.abs(ref))
    err = np.abs(out.double().cpu().numpy() - ref)
    assert np.isfinite(err).all()
    worst = float((err / (tol + 1e-30)).max())
    print(f"    largest error {err.max():.3g}, {worst:.3g} of the bound")
    assert worst <= 1.0
    return ref


# ---------------------------------------------------------------------------
# Append
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("page,Hkv", [(16, 1), (64, 3)])
def test_append_bytes(D, dtype, page, Hkv):
    offsets, lens = [0, 5, 5, 23, 24], [13, 7, 0, 200]
    rng, table, data = setup(D + page, D, Hkv, page, lens, offsets)
    T = offsets[-1]
    k, kd = rounded(rng, (T, Hkv, D), dtype)
    v, vd = rounded(rng, (T, Hkv, D), dtype, 30.0)
    for t, val in enumerate((0.0, 1e-38, 1e-30, 3e38, -0.25, 6.0)):      # whole blocks of one value
        kd[t, :, :32] = val
        k[t, :, :32] = kd[t, :, :32].double().cpu().numpy()
    kd[7, :, 32:43] = torch.tensor([6.0, -5, 3.5, 2.5, 1.75, 1.25, .75, .25, -.25, -0.0, 1e-3], dtype=DT[dtype])
    k[7, :, 32:] = kd[7, :, 32:].double().cpu().numpy()
    c = cache_of(dev(data), D, Hkv, page)
    stored = m.kv4_append(c, kd, vd, dev(table), dev(np.array(lens, dtype=np.int32)), offsets, return_stored=True)
    okv.append(data, k, v, table, lens, offsets)
    assert np.array_equal(c.data.cpu().numpy(), data)
    for got, x in zip(stored, (k, v)):
        assert got.dtype == DT[dtype] and np.array_equal(got.double().cpu().numpy(), okv.quantise(x)[2])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_append_every_rounding(dtype):
    """Each border between two codes, its neighbours on both sides and each
    code's own value, of both signs, under scales from the least to the largest."""
    D, page = 64, 16
    ulp = 2.0 ** (-23 if dtype == "f32" else -7)
    exps = [-100, -99, -64, -3, -1, 0, 1, 5, 60, 124, 125]
    k = np.zeros((len(exps), 1, D))
    for i, e in enumerate(exps):
        at = [6.0] + [b for c in (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)
                      for b in (c - 2.0 ** np.floor(np.log2(c)) * ulp, c, c + 2.0 ** np.floor(np.log2(c)) * ulp)]
        at += [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 1e-9, 2.0 ** -20, 0.1]
        k[i, 0, :32] = np.array(at) * 2.0 ** e
        k[i, 0, 32:] = -k[i, 0, :32]
    kd = dev(k.astype(np.float32)).to(DT[dtype])
    k = kd.double().cpu().numpy()
    vd = kd.flip(-1).contiguous()
    offsets, lens = [0, len(exps)], [1]
    _, table, data = setup(9, D, 1, page, lens, offsets)
    c = cache_of(dev(data), D, 1, page)
    stored = m.kv4_append(c, kd, vd, dev(table), dev(np.array(lens, dtype=np.int32)), offsets, return_stored=True)
    okv.append(data, k, k[..., ::-1], table, lens, offsets)
    assert np.array_equal(c.data.cpu().numpy(), data)
    assert np.array_equal(stored[0].double().cpu().numpy(), okv.quantise(k)[2])
    assert np.array_equal(stored[1].double().cpu().numpy(), okv.quantise(k[..., ::-1])[2])


def test_append_from_a_fused_projection():
    D, Hkv, page, offsets, lens = 128, 2, 32, [0, 9], [31]
    rng, table, data = setup(1, D, Hkv, page, lens, offsets)
    x, xd = rounded(rng, (9, 8 * D), "bf16")
    kd, vd = xd[:, 4 * D:6 * D].view(9, 2, D), xd[:, 6 * D:].view(9, 2, D)
    c = cache_of(dev(data), D, Hkv, page)
    assert m.kv4_append(c, kd, vd, dev(table), dev(np.array(lens, dtype=np.int32)), offsets) is None
    okv.append(data, x[:, 4 * D:6 * D].reshape(9, 2, D), x[:, 6 * D:].reshape(9, 2, D), table, lens, offsets)
    assert np.array_equal(c.data.cpu().numpy(), data)


def test_append_commit_and_bad_places():
    """Only the accepted rows, in path order; path entries, pages and positions that are none are passed over."""
    D, Hkv, page, offsets = 64, 2, 16, [0, 6, 12, 12, 20]
    lens = [14, 0, 3, 30]
    rng, table, data = setup(2, D, Hkv, page, lens, offsets)
    table[0, 1] = len(data)            # the second page of sequence 0: beyond the pool
    table[3, 2] = -7
    k, kd = rounded(rng, (20, Hkv, D), "f32")
    v, vd = rounded(rng, (20, Hkv, D), "f32")
    path = np.array([0, 2, 5, -1, -1, -1, 0, 6, -3, 1, 99, 4, 0, 1, 2, 3, 4, 5, 6, 7], dtype=np.int32)
    count = np.array([3, 6, 4, 8], dtype=np.int32)
    c = cache_of(dev(data), D, Hkv, page)
    m.kv4_append(c, kd, vd, dev(table), dev(np.array(lens, dtype=np.int32)), offsets, path=dev(path), count=dev(count))
    okv.append(data, k, v, table, lens, offsets, path, count)
    assert np.array_equal(c.data.cpu().numpy(), data)
    # lengths that are negative, at the table's end and far past it
    lens = [-5, table.shape[1] * page - 2, 0, 2 ** 31 - 1]
    m.kv4_append(c, kd, vd, dev(table), dev(np.array(lens, dtype=np.int32)), offsets)
    okv.append(data, k, v, table, lens, offsets)
    assert np.array_equal(c.data.cpu().numpy(), data)


# ---------------------------------------------------------------------------
# Attention
# ---------------------------------------------------------------------------
def tree(n, kind):
    return [-1] + [(j - 1) // 2 if kind == "binary" else 0 if kind == "star" else j - 1 for j in range(1, n)]


CASES = [
    # D, dtype, Hkv, G, page, lens, counts, tree
    (64, "bf16", 1, 1, 16, [0], [1], None),
    (128, "f32", 1, 1, 16, [0], [1], None),
    (128, "bf16", 2, 8, 16, [1, 15, 16, 17, 31], [1, 1, 1, 1, 1], None),
    (128, "f32", 2, 4, 64, [32, 33, 63, 64, 65], [2, 1, 3, 0, 4], None),
    (128, "bf16", 4, 16, 32, [100, 301, 77, 250], [5, 5, 5, 5], None),
    (128, "bf16", 1, 5, 16, [400], [15], "binary"),
    (64, "f32", 2, 3, 16, [129, 0], [15, 7], "binary"),
    (64, "bf16", 1, 7, 128, [90], [64], "star"),
    (256, "bf16", 1, 8, 16, [200, 3], [4, 9], "binary"),
    (256, "f32", 2, 2, 64, [65, 190], [3, 5], None),
    (64, "f32", 1, 64, 16, [70], [3], None),
    (128, "f32", 1, 20, 16, [500, 0, 90], [4, 0, 2], "star"),
]


@pytest.mark.parametrize("D,dtype,Hkv,G,page,lens,counts,kind", CASES)
def test_attend(D, dtype, Hkv, G, page, lens, counts, kind):
    offsets = [0] + list(np.cumsum(counts))
    offsets = [int(x) for x in offsets]
    rng, table, data = setup(D + sum(lens), D, Hkv, page, lens, offsets)
    fill(rng, data, table, lens, D, Hkv)
    T = offsets[-1]
    parent = None if kind is None else sum((tree(n, kind) for n in counts if n), [])
    k, kd = rounded(rng, (T, Hkv, D), dtype)
    v, vd = rounded(rng, (T, Hkv, D), dtype)
    q, qd = rounded(rng, (T, Hkv * G, D), dtype)
    c, td, ld = cache_of(dev(data), D, Hkv, page), dev(table), dev(np.array(lens, dtype=np.int32))
    m.kv4_append(c, kd, vd, td, ld, offsets)
    okv.append(data, k, v, table, lens, offsets)
    out = m.kv4_attend(c, qd, td, ld, offsets, parent=parent)
    check_attend(out, q, data, table, lens, offsets, parent, D ** -0.5, dtype)
    again = m.kv4_attend(c, qd, td, ld, offsets, parent=parent)
    assert torch.equal(out, again)


def any_rows(rng, data, D):
    """Every row of the pool holds codes and scales of some values."""
    data[:] = rng.integers(0, 256, data.shape, dtype=np.uint8)
    for at in (8 * D, 33 * D // 2):
        data[..., at:at + D // 2] = rng.integers(122, 128, data.shape[:-1] + (D // 2,), dtype=np.uint8)


@pytest.mark.parametrize("D,dtype,Hkv,G,lens,counts", [
    (64, "bf16", 2, 8, [300, 77], [5, 6]), (64, "bf16", 1, 8, [40, 1000], [8, 7]), (64, "f32", 2, 16, [333], [7]),
    (64, "f32", 1, 11, [0, 64], [4, 1]), (128, "bf16", 2, 8, [300, 77], [5, 6]), (128, "bf16", 1, 16, [40, 1000], [8, 7]),
    (128, "f32", 2, 16, [333, 31], [7, 1]), (256, "bf16", 1, 16, [150], [6]),
])
def test_attend_wide_table(D, dtype, Hkv, G, lens, counts):
    """Tables far wider than the sequences: row blocks of up to 64 rows."""
    offsets, page = [0] + [int(x) for x in np.cumsum(counts)], 64
    rng, table, data = setup(D + G, D, Hkv, page, lens, offsets)
    table = np.pad(table, ((0, 0), (0, 20000 - table.shape[1])), constant_values=-1)
    any_rows(rng, data, D)
    T = offsets[-1]
    parent = sum((tree(n, "binary") for n in counts), [])
    kd, vd = rounded(rng, (T, Hkv, D), dtype)[1], rounded(rng, (T, Hkv, D), dtype)[1]
    q, qd = rounded(rng, (T, Hkv * G, D), dtype)
    c, td, ld = cache_of(dev(data), D, Hkv, page), dev(table), dev(np.array(lens, dtype=np.int32))
    m.kv4_append(c, kd, vd, td, ld, offsets)
    data = c.data.cpu().numpy()
    out = m.kv4_attend(c, qd, td, ld, offsets, parent=parent)
    check_attend(out, q, data, table, lens, offsets, parent, D ** -0.5, dtype)


@pytest.mark.parametrize("D,dtype,Hkv,lens", [
    (64, "bf16", 24, [7 + 3 * s for s in range(64)]), (128, "bf16", 12, [(37 * s) % 301 for s in range(64)]),
    (128, "f32", 16, [900] + [5] * 63), (256, "bf16", 8, [(53 * s) % 211 for s in range(64)]),
    (64, "f32", 3, [2500, 1, 0, 90, 1700]), (256, "bf16", 4, [1500 + (997 * s) % 1703 for s in range(32)]),
])
def test_attend_many_sequences(D, dtype, Hkv, lens):
    """More units than workgroups, units of very different lengths, and long ones that shares do not divide."""
    offsets, page = list(range(len(lens) + 1)), 16
    rng, table, data = setup(Hkv, D, Hkv, page, lens, offsets)
    any_rows(rng, data, D)
    T = len(lens)
    kd, vd = rounded(rng, (T, Hkv, D), dtype)[1], rounded(rng, (T, Hkv, D), dtype)[1]
    q, qd = rounded(rng, (T, 2 * Hkv, D), dtype)
    c, td, ld = cache_of(dev(data), D, Hkv, page), dev(table), dev(np.array(lens, dtype=np.int32))
    m.kv4_append(c, kd, vd, td, ld, offsets)
    data = c.data.cpu().numpy()
    out = m.kv4_attend(c, qd, td, ld, offsets)
    check_attend(out, q, data, table, lens, offsets, None, D ** -0.5, dtype)


@pytest.mark.parametrize("D,dtype,n", [(128, "bf16", 3), (64, "f32", 1), (256, "bf16", 2)])
def test_attend_long_split(D, dtype, n):
    """One sequence over many workgroups; a few rows far apart hold most of the weight."""
    lens, offsets, page = [9973], [0, n], 64
    rng, table, data = setup(7, D, 1, page, lens, offsets)
    fill(rng, data, table, lens, D, 1)
    q, qd = rounded(rng, (n, 4, D), dtype)
    for p, f in ((3, 1.0), (5000, 1.1), (9972, 1.05)):    # rows along the first query
        okv.write_row(data, int(table[0, p // page]), 0, p % page, f * q[0, 0], rng.normal(size=D))
    c, td, ld = cache_of(dev(data), D, 1, page), dev(table), dev(np.array(lens, dtype=np.int32))
    k, kd = rounded(rng, (n, 1, D), dtype)
    v, vd = rounded(rng, (n, 1, D), dtype)
    m.kv4_append(c, kd, vd, td, ld, offsets)
    okv.append(data, k, v, table, lens, offsets)
    out = m.kv4_attend(c, qd, td, ld, offsets)
    check_attend(out, q, data, table, lens, offsets, None, D ** -0.5, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_attend_rising_scores(dtype):
    """Scores that rise along the cache move the running maximum at every step; large negative scale as well."""
    D, lens, offsets, page = 64, [700], [0, 2], 16
    rng, table, data = setup(11, D, 1, page, lens, offsets)
    k = np.ones((700, 1, D)) * (np.arange(700) / 100.0)[:, None, None]
    okv.append(data, k, rng.normal(size=(700, 1, D)), table, [0], [0, 700])
    c, td, ld = cache_of(dev(data), D, 1, page), dev(table), dev(np.array(lens, dtype=np.int32))
    kn, kd = rounded(rng, (2, 1, D), dtype)
    m.kv4_append(c, kd, kd, td, ld, offsets)
    okv.append(data, kn, kn, table, lens, offsets)
    q, qd = rounded(np.random.default_rng(3), (2, 2, D), dtype)
    q, qd = np.abs(q), qd.abs()
    for scale in (0.5, -1.0):
        out = m.kv4_attend(c, qd, td, ld, offsets, scale=scale)
        check_attend(out, q, data, table, lens, offsets, None, scale, dtype)


def test_attend_missing_pages_and_short_table():
    """Rows in pages outside the pool are not seen, whatever bytes lie in the pool; all missing: zeros."""
    D, Hkv, page, offsets = 128, 2, 16, [0, 2, 4, 6]
    lens = [60, 40, 20]
    rng, table, data = setup(5, D, Hkv, page, lens, offsets)
    fill(rng, data, table, lens, D, Hkv)
    data[0] = 0xFF                                    # page 0 is what a reader of no page might touch
    table[table == 0] = -1
    table[0, 1] = -1
    table[0, 2] = len(data)
    table[1, :] = 2 ** 31 - 1
    k, kd = rounded(rng, (6, Hkv, D), "bf16")
    q, qd = rounded(rng, (6, 4, D), "bf16")
    c, most = cache_of(dev(data), D, Hkv, page), 0
    for ln in (lens, [-3, 5, table.shape[1] * page + 1000], [2 ** 31 - 1, 0, table.shape[1] * page - 1]):
        td, ld = dev(table), dev(np.array(ln, dtype=np.int32))
        m.kv4_append(c, kd, kd, td, ld, offsets)
        host = c.data.cpu().numpy()
        use = np.minimum(np.maximum(ln, 0), table.shape[1] * page)
        # rows never written hold 0xff, which stands for no number: sequences that claim such rows are left out
        sound = []
        for s in range(3):
            pos = np.arange(min(int(use[s]) + 2, table.shape[1] * page))
            pid = table[s][pos // page]
            real = (pid >= 0) & (pid < len(host))
            written = host[np.where(real, pid, 0), 0, pos % page // 16, 8 * D + pos % 16] != 0xFF
            if (written | ~real).all():
                sound += [offsets[s], offsets[s] + 1]
        out = m.kv4_attend(c, qd, td, ld, offsets)
        assert (out[2:4] == 0).all() and {2, 3} <= set(sound)
        check_attend(out, q, host, table, use, offsets, None, D ** -0.5, "bf16", sound)
        most = max(most, len(sound))
    assert most == 6


def test_attend_strided_queries_and_outputs():
    D, Hkv, page, lens, offsets = 64, 1, 16, [50], [0, 3]
    rng, table, data = setup(6, D, Hkv, page, lens, offsets)
    fill(rng, data, table, [53], D, Hkv)
    x, xd = rounded(rng, (3, 6 * D), "f32")
    qd = xd[:, :4 * D].view(3, 4, D)
    c, td, ld = cache_of(dev(data), D, Hkv, page), dev(table), dev(np.array(lens, dtype=np.int32))
    out = torch.empty((3, 4, D), device=DEV)
    ws = torch.empty(1 << 25, dtype=torch.uint8, device=DEV)
    assert m.kv4_attend(c, qd, td, ld, offsets, out=out, workspace=ws) is out
    check_attend(out, x[:, :4 * D].reshape(3, 4, D), data, table, lens, offsets, None, D ** -0.5, "f32")


def test_attend_beyond_four_gib():
    """Pages whose bytes lie past 2^32."""
    D, Hkv, page, lens, offsets = 128, 1, 4096, [4000], [0, 2]
    rng = np.random.default_rng(8)
    per = Hkv * (page // 16) * 17 * D
    pool = (1 << 32) // per + 3
    data = torch.empty((pool, Hkv, page // 16, 17 * D), dtype=torch.uint8, device=DEV)
    table = np.array([[pool - 1, pool - 2]], dtype=np.int32)
    c, td = cache_of(data, D, Hkv, page), dev(table)
    k, kd = rounded(rng, (4002, Hkv, D), "f32")
    v, vd = rounded(rng, (4002, Hkv, D), "f32")
    q, qd = rounded(rng, (2, 2, D), "f32")
    m.kv4_append(c, kd[:4000], vd[:4000], td, dev(np.zeros(1, dtype=np.int32)), [0, 4000])
    ld = dev(np.array(lens, dtype=np.int32))
    m.kv4_append(c, kd[4000:], vd[4000:], td, ld, offsets)
    out = m.kv4_attend(c, qd, td, ld, offsets)
    host = np.zeros((2, Hkv, page // 16, 17 * D), dtype=np.uint8)
    okv.append(host, k[4000:], v[4000:], np.array([[1, 0]]), lens, offsets)
    got = data[pool - 2:].cpu().numpy()
    for h in range(1):
        kk, vv = okv.read_rows(got, np.array([1] * 4000), h, np.arange(4000))
        assert np.array_equal(kk, okv.quantise(k[:4000, h])[2]) and np.array_equal(vv, okv.quantise(v[:4000, h])[2])
    check_attend(out, q, got, np.array([[1, 0]]), lens, offsets, None, D ** -0.5, "f32")


def test_attend_graph_and_streams():
    """A captured append + attend replayed on new lengths, rows and queries
    equals the eager calls; two streams at once, each with its own workspace."""
    D, Hkv, page, offsets = 128, 2, 16, [0, 3, 5]
    rng, table, data = setup(9, D, Hkv, page, [300, 200], offsets)
    fill(rng, data, table, [300, 200], D, Hkv)
    c, td = cache_of(dev(data), D, Hkv, page), dev(table)
    ld = dev(np.array([100, 50], dtype=np.int32))
    _, kd = rounded(rng, (5, Hkv, D), "bf16")
    _, qd = rounded(rng, (5, 8, D), "bf16")
    out = torch.empty_like(qd)
    ws = torch.empty(1 << 25, dtype=torch.uint8, device=DEV)

    def step():
        m.kv4_append(c, kd, kd, td, ld, offsets)
        m.kv4_attend(c, qd, td, ld, offsets, out=out, workspace=ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    fresh = c.data.clone()
    for lens in ([100, 50], [295, 0], [0, 199]):
        for _ in range(2):
            ld.copy_(dev(np.array(lens, dtype=np.int32)))
            qd.mul_(0.75)
            c.data.copy_(fresh)
            g.replay()
            torch.cuda.synchronize()
            got, bytes_got = out.clone(), c.data.clone()
            c.data.copy_(fresh)
            step()
            assert torch.equal(got, out) and torch.equal(bytes_got, c.data)
    want = [m.kv4_attend(c, qd * f, td, ld, offsets) for f in (1.0, 0.5)]
    qs = [qd * f for f in (1.0, 0.5)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = []
    for _ in range(20):
        got.append([m.kv4_attend(c, x, td, ld, offsets, stream=st) for x, st in zip(qs, streams)])
    torch.cuda.synchronize()
    for pair in got:
        assert torch.equal(pair[0], want[0]) and torch.equal(pair[1], want[1])
