"""Rows of sample_tokens on which the search for the threshold is hard: tiny
spreads, few allowed tokens, long tails.  Results against the float64 oracle
(tolerances as in test_gpu_sampling)."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import moe_speculative_decoding_router_amd as m  # noqa: E402
import test_gpu_sampling as base  # noqa: E402

DEV = torch.device("cuda:0")
dev, check = base.dev, base.check


@pytest.mark.parametrize("V", [4099, 32000])
def test_values_that_lie_next_to_each_other(V):
    """Differences from 1e-37 down to subnormal ones: more tokens near the threshold than a list holds, and no
    finite number of parts between them."""
    rng = np.random.default_rng(V)
    T = 6
    x = rng.random((T, V)).astype(np.float32) * np.float32(1e-37)
    x[1] *= np.float32(1e-6)                                  # subnormal
    x[2] = 0.0
    x[2, V // 3] = np.float32(1e-45)
    x[3] = np.float32(1e-30) * np.float32(1.5) * rng.random(V).astype(np.float32)
    xd = dev(x)
    x, u = x.astype(np.float64), rng.random(T)
    check(x, xd, u, top_k=[1000] * T)
    check(x, xd, u, top_k=[V - 7] * T, top_p=[0.5] * T)
    check(x, xd, u, top_p=[0.9] * T)
    check(x, xd, u, top_p=[0.9] * T, temperature=[1e-37, 1e-43, 1e-45, 1e-30, 1e-38, 1e-37])


def fastest(x, u, **kw):
    """us of a call on the GPU: ten calls in a graph, the least of several replays."""
    ws = torch.empty(m.lib().sample_workspace_bytes(*x.shape), dtype=torch.uint8, device=DEV)
    m.sample_tokens(x, u, workspace=ws, **kw)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for _ in range(10):
            m.sample_tokens(x, u, workspace=ws, **kw)
    best = float("inf")
    for _ in range(8):
        a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        a.record()
        g.replay()
        b.record()
        torch.cuda.synchronize()
        best = min(best, a.elapsed_time(b) * 100)
    return best


def descent(T, V, u, dtype=torch.float32, top_k=None):
    """us of rows that only the descent over the whole row settles: equal values."""
    k = torch.full((T,), V // 2, dtype=torch.int32, device=DEV)
    return fastest(torch.zeros((T, V), dtype=dtype, device=DEV), u, top_k=k)


def allowed(rng, T, V, n, together):
    """Rows of which n tokens are allowed, next to each other or anywhere; the others are -inf."""
    x = np.full((T, V), -np.inf)
    for i in range(T):
        at = 1 + int(rng.integers(0, V - n)) + np.arange(n) if together else rng.permutation(V)[:n]
        x[i, at] = 2 * rng.normal(size=n)
    return x.astype(np.float32)


@pytest.mark.parametrize("V,n,together,k", [
    (32000, 30, True, 50), (32000, 30, True, 30), (32000, 20, False, 50), (32000, 1500, False, 1000), (32000, 1500, False, 1500),
    (32000, 3000, True, 800), (32000, 5000, False, 1000), (32000, 2000, True, 2047), (20000, 896, True, 896), (32768, 1, True, 2),
    (32000, 31990, True, 896),
])
def test_few_allowed_tokens(V, n, together, k):
    """Fewer of the search's groups hold a token than top_k counts, or more tokens lie above the groups' cut than a
    list holds: the row is listed or narrowed, and far from the time of a descent over the whole row."""
    rng = np.random.default_rng(n + k)
    T = 6
    x = allowed(rng, T, V, n, together)
    xd, u = dev(x), rng.random(T)
    check(x.astype(np.float64), xd, u, top_k=[k] * T)
    check(x.astype(np.float64), xd, u, top_k=[k] * T, top_p=[0.9, 0.99, 0.5, 1.0, 0.999, 0.2], temperature=[0.7] * T)
    ud = dev(u.astype(np.float32))
    own = fastest(xd, ud, top_k=torch.full((T,), k, dtype=torch.int32, device=DEV))
    all_ = descent(T, V, ud)
    print(f"    {own:.1f} us, by descent {all_:.1f}")
    assert own < 0.5 * all_


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V,k", [(200, 100), (1000, 300), (1500, 1000), (3000, 1000), (4093, 4000)])
def test_top_k_beyond_the_groups(V, k, dtype):
    """Short rows whose top_k is above the number of groups that hold a token."""
    rng = np.random.default_rng(V)
    T = 8
    x, xd = base.logits_of(rng, T, V, dtype)
    check(x, xd, rng.random(T), top_k=[k] * T)
    check(x, xd, rng.random(T), top_k=[k] * T, top_p=rng.choice([0.3, 0.9, 0.99], T), min_p=rng.choice([0.0, 0.02], T))


@pytest.mark.parametrize("V,top_p,temperature", [(32000, 0.99, 1.0), (32768, 0.995, 1.0), (32000, 0.999, 0.7), (20000, 0.999, 1.5),
                                                 (32000, 0.9999, 1.0), (32768, 0.99, 1.1)])
def test_long_tails(V, top_p, temperature):
    """A threshold in the tail, where a token's weight is far below the first's but many share the mass: rows without
    ties, so none of the 64 needs a descent."""
    rng = np.random.default_rng(int(V * top_p))
    T = 64
    x, xd = base.logits_of(rng, T, V, "f32")
    u, part = rng.random(T), slice(0, 12)
    check(x[part], xd[part], u[part], top_p=[top_p] * 12, temperature=[temperature] * 12)
    ud = dev(u.astype(np.float32))
    own = fastest(xd, ud, top_p=torch.full((T,), top_p, device=DEV), temperature=torch.full((T,), temperature, device=DEV))
    tied = fastest(torch.zeros((T, V), device=DEV), ud, top_p=torch.full((T,), top_p, device=DEV))
    print(f"    {own:.1f} us, by descent {tied:.1f}")
    assert own < 0.6 * tied


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [5003, 40009, 150001])
def test_no_filter_and_filters_that_are_off(V, dtype):
    """The same draws without filters as with ones that keep everything: tokens below 2^-46 of the first have no
    units on either path, so u = 0 takes the lowest token that has some."""
    rng = np.random.default_rng(V)
    T = 8
    x = rng.normal(size=(T, V))
    x[0, :V // 2] = -200                        # whole chunks below
    x[1, 1:] -= 60                              # all but one token
    x[2, :5000] = -31.5                         # 2^-45.4 of 1 where the first is 0: some have units, some none
    x[2, 5000:] = np.minimum(x[2, 5000:], 0)
    x[2, 0], x[2, V - 1] = -33, 0
    x[3] = np.where(np.arange(V) % 2, 3.0, -100)
    x[4] -= 2e-2 * np.arange(V)[::-1]
    xd = dev(x.astype(np.float32)).to(base.DT[dtype])
    off = dict(top_k=torch.zeros(T, dtype=torch.int32, device=DEV), top_p=torch.ones(T, device=DEV),
               min_p=torch.zeros(T, device=DEV))
    for u in (0.0, 2.0 ** -149, 2.0 ** -60, 0.3, 1 - 2.0 ** -24):
        ud = torch.full((T,), u, device=DEV)
        tok, prob, probs = m.sample_tokens(xd, ud, return_probs=True)
        for names in (["top_k"], ["top_p"], ["min_p"], list(off)):
            t, p, f = m.sample_tokens(xd, ud, return_probs=True, **{k: off[k] for k in names})
            assert torch.equal(t, tok), (u, names, t.tolist(), tok.tolist())
            # float64 sums of the chunks against integers: V 2^-46 of the sum, and a rounding to float32 each
            assert ((p - prob).abs() <= (2.0 ** -23 + V * 2.0 ** -46) * prob).all()
            assert ((f - probs).abs() <= (2.0 ** -23 + V * 2.0 ** -46) * probs + 2.0 ** -149).all()


@pytest.mark.parametrize("V", [5003, 40009])
def test_infinite_temperatures_and_filters_that_are_no_numbers(V):
    """An infinite temperature weighs all tokens alike, those an infinite distance from the first too; a temperature
    of NaN is 0, another filter of NaN is off."""
    rng = np.random.default_rng(V)
    T = 6
    big = 3.4028234663852886e38
    x = rng.normal(size=(T, V)).astype(np.float32)
    x[0, [5, V - 9]] = big, -big
    x[1, 1:] = -big
    x[2, ::2] = -big
    x[2, 1] = big
    x[3, rng.random(V) < 0.9] = -np.inf
    xd = dev(x)
    x, u = x.astype(np.float64), rng.random(T)
    inf, nan = [np.inf] * T, [np.nan] * T
    for kw in ({}, {"top_k": [V // 3] * T}, {"top_k": [50] * T}, {"top_p": [0.3] * T}, {"min_p": [0.5] * T},
               {"top_k": [V - 3] * T, "top_p": [0.9] * T, "min_p": [1.0] * T}):
        check(x, xd, u, temperature=inf, **kw)
        check(x, xd, u, temperature=nan, **kw)
    check(x, xd, u, top_p=nan)
    check(x, xd, u, min_p=nan, top_k=[40] * T)
    for kw in ({"top_k": [1500] * T}, {"top_p": [0.3] * T}, {"top_p": [0.999] * T}):    # the lowest value as a mask
        check(x, xd, u, **kw)
