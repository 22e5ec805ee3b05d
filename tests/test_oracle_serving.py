"""The oracles of the serving operators (4-bit cache, sampling, acceptance)
against values worked out by hand and against what they have to preserve
(CPU)."""
import numpy as np
import pytest

from oracle import kv4 as okv
from oracle import sampling as osa


def test_quantise_by_hand():
    x = np.zeros(32)
    x[:10] = [6.0, -5.0, 3.5, 2.5, 1.75, 1.25, 0.75, 0.25, -0.25, -0.3]
    code, sc, val = okv.quantise(x)                    # amax 6: scale 1; every tie goes to the even code
    assert sc.tolist() == [127]
    assert code[:10].tolist() == [7, 14, 6, 4, 4, 2, 2, 0, 0, 9]
    assert val[:10].tolist() == [6, -4, 4, 2, 2, 1, 1, 0, 0, -0.5]
    for amax, e in ((6.1, 1), (12.0, 1), (12.1, 2), (3.0, -1), (3.01, 0), (1e-40, -100), (0.0, -100), (3e38, 125)):
        assert int(okv.quantise(np.full(32, amax))[1][0]) - 127 == e, amax
    assert okv.quantise(np.full(32, 3e38))[2][0] == 6.0 * 2.0 ** 125


@pytest.mark.parametrize("D", [64, 128, 256])
def test_layout_is_a_bijection(D):
    ko, kso, vo, vso = okv._offsets(D)
    seen = np.zeros((17 * D, 2), dtype=int)
    for i in range(16):
        for d in range(D):
            seen[ko(i, d), d % 2] += 1
            seen[vo(i, d), d % 2] += 1
        for b in range(D // 32):
            seen[kso(i, b)] += 1
            seen[vso(i, b)] += 1
    assert (seen == 1).all()


@pytest.mark.parametrize("D", [64, 256])
def test_append_then_read(D):
    rng = np.random.default_rng(D)
    data = np.full((5, 2, 2, 17 * D), 0xFF, dtype=np.uint8)
    k, v = rng.normal(size=(7, 2, D)), rng.normal(size=(7, 2, D))
    table = np.array([[3, 1], [0, 4]])
    okv.append(data, k, v, table, [30, 5], [0, 4, 7])
    for s, (pos, row) in enumerate(((np.arange(30, 34), 0), (np.arange(5, 8), 4))):
        for h in range(2):
            kk, vv = okv.read_rows(data, table[s][pos // 32], h, pos)
            assert np.array_equal(kk, okv.quantise(k[row:row + len(pos), h])[2])
            assert np.array_equal(vv, okv.quantise(v[row:row + len(pos), h])[2])
    assert (data[2] == 0xFF).all()


def test_filters_by_hand():
    x = np.log([8.0, 4.0, 2.0, 1.0, 1.0])
    kept = lambda **kw: osa.kept_weights(x, **kw)[1]                                     # noqa: E731
    assert kept() == 5 and kept(top_k=2) == 2 and kept(top_k=9) == 5 and kept(temperature=0.0, top_k=3) == 1
    assert kept(top_p=0.5) == 1 and kept(top_p=0.51) == 2 and kept(top_p=0.75) == 2 and kept(top_p=0.99) == 5
    assert kept(top_k=2, top_p=0.7) == 2 and kept(top_k=2, top_p=0.6) == 1   # 8 / 12 of the two
    assert kept(top_p=0.0) == 1 and kept(min_p=0.24) == 3 and kept(min_p=2.0) == 1
    w, _ = osa.kept_weights(x, top_k=4)
    assert w[3] > 0 and w[4] == 0                                            # the tie goes to the lower index
    assert osa.kept_weights(np.full(3, -np.inf))[1] == 0 and osa.draw(np.zeros(3), 0.5) == -1
    assert osa.kept_weights(np.array([np.nan, np.inf, 3.0]))[0].tolist() == [0, 1, 0]
    assert [osa.draw(np.ones(4), u) for u in (0.0, 0.2499, 0.25, 0.75, 0.9999)] == [0, 0, 1, 3, 3]


def test_chain_acceptance_keeps_the_target_distribution():
    """Integrated over its numbers on a fine grid, the first gained token of a
    chain has the target's distribution whatever the drafter's is."""
    p = np.array([[0.5, 0.2, 0.2, 0.1], [0.1, 0.2, 0.3, 0.4]])
    q = np.array([[0.1, 0.6, 0.2, 0.1], [0.25] * 4])
    n = 400
    got = np.zeros(4)
    for x in range(4):                                  # the draft, with probability q
        for i in range(n):
            u = (i + 0.5) / n
            if u * q[0, x] < p[0, x]:
                got[x] += q[0, x] / n
                continue
            for j in range(50):
                out, path = osa.accept_chain(p, q, [0, x], [u, 0.0], (j + 0.5) / 50)
                assert path == [0] and len(out) == 1
                got[out[0]] += q[0, x] / n / 50
    # the grid's steps: 1 / n in u, 1 / 50 in u_final times the rejected mass
    assert np.abs(got - p[0]).max() <= 1.0 / n + 0.5 / 50


def test_match_walks_the_tree():
    parent, tokens = [-1, 0, 0, 1, 1, 2], [9, 5, 6, 7, 8, 7]
    assert osa.accept_match([5, 8, 0, 0, 3, 0], tokens, parent) == ([5, 8, 3], [0, 1, 4])
    assert osa.accept_match([6, 0, 7, 0, 0, 2], tokens, parent) == ([6, 7, 2], [0, 2, 5])
    assert osa.accept_match([1, 0, 7, 0, 0, 2], tokens, parent) == ([1], [0])
    assert osa.accept_match([5, 0], [9, 5], [-1, 0]) == ([5, 0], [0, 1])
    assert osa.accept_match([-1, 0], [9, -1], [-1, 0]) == ([-1], [0])        # a row without tokens
