"""prompt_attend against the formula in float64.

Scores are products of D terms in float32, with operands exact in bf16 or to
2^-24 in three bf16 terms (of which products below 2^-24 are left out): off by
at most (D + 12) 2^-24 sum |q k| scale; an error of that size enters every probability twice
(through itself and the sum); sums and rescalings add (keys + 64) 2^-24, the
exponential 2^-22, the second product's left-out terms 2^-22.  bf16 rounds the
probabilities (each by at most 2^-8 of it; their sum is not rounded) and the
result (2^-8 of it)."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import moe_speculative_decoding_router_amd as m  # noqa: E402

DEV = torch.device("cuda:0")
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def offsets(counts):
    off = [0]
    for n in counts:
        off.append(off[-1] + n)
    return off


def reference(q, k, v, off, koff, scale):
    """float64 out, sum p |v|, and the largest sum |q k| |scale| of a visible key."""
    T, Hq, D = q.shape
    G = Hq // k.shape[1]
    out, bound = torch.zeros((2, T, Hq, D), dtype=torch.float64, device=q.device)
    reach = 0.0
    for s in range(len(off) - 1):
        n, mk = off[s + 1] - off[s], koff[s + 1] - koff[s]
        if n == 0 or mk == 0:
            continue
        hide = torch.arange(mk, device=q.device)[None] > torch.arange(n, device=q.device)[:, None] + (mk - n)
        none = hide.all(1)
        for h in range(Hq):
            x = q[off[s]:off[s + 1], h].double()
            kk, vv = k[koff[s]:koff[s + 1], h // G].double(), v[koff[s]:koff[s + 1], h // G].double()
            a = (x @ kk.t().contiguous()) * scale
            far = (x.abs() @ kk.abs().t().contiguous()) * abs(scale)
            reach = max(reach, float(far.masked_fill(hide, 0).max()))
            a = a.masked_fill(hide, -float("inf"))
            a[none] = 0
            p = torch.softmax(a, -1)
            p[none] = 0
            out[off[s]:off[s + 1], h] = p @ vv
            bound[off[s]:off[s + 1], h] = p @ vv.abs()
    return out, bound, reach


def check(out, q, k, v, off, koff, scale):
    ref, bound, reach = reference(q, k, v, off, koff, scale)
    D, keys = q.shape[2], max(b - a for a, b in zip(koff, koff[1:]))
    u = 2.0 ** -24
    rel = 2 * (D + 12) * u * reach + (keys + 64) * u + 8 * u
    if q.dtype == torch.bfloat16:
        tol = (rel + 2.0 ** -8) * bound + 2.0 ** -8 * ref.abs()
    else:
        tol = rel * bound + u * ref.abs()
    err = (out.double() - ref).abs()
    assert out.dtype == q.dtype and torch.isfinite(out).all()
    worst = float((err / (tol + 1e-30)).max())
    print(f"    largest error {float(err.max()):.3g}, {worst:.3g} of the bound")
    assert worst <= 1.0


def inputs(seed, T, Tk, Hq, Hkv, D, dtype, fused=False):
    g = torch.Generator(device=DEV).manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g, device=DEV)  # noqa: E731
    if fused:
        x = r(T, (Hq + 2 * Hkv) * D + 64).to(DT[dtype])
        a, b = Hq * D, (Hq + Hkv) * D
        return x[:, :a].unflatten(1, (Hq, D)), x[:, a:b].unflatten(1, (Hkv, D)), x[:, b:b + Hkv * D].unflatten(1, (Hkv, D))
    return r(T, Hq, D).to(DT[dtype]), r(Tk, Hkv, D).to(DT[dtype]), r(Tk, Hkv, D).to(DT[dtype])


CASES = [  # query rows, keys, Hq, Hkv
    ([1], [1], 1, 1), ([1], [64], 2, 1), ([2, 1, 0, 3], None, 4, 2), ([31, 32, 33], None, 3, 3), ([63, 64, 65, 127], None, 2, 1),
    ([128, 129], None, 8, 2), ([300], None, 6, 2), ([1, 700, 0, 17], None, 4, 4), ([5], [2], 2, 2), ([200, 3], [70, 0], 2, 1),
    ([1], [3000], 4, 1), ([7, 130], [1000, 131], 16, 2), ([40], [4001], 7, 7), ([1, 1], [0, 5], 8, 8),
]


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n,keys,Hq,Hkv", CASES)
def test_shapes(n, keys, Hq, Hkv, dtype, D):
    off = offsets(n)
    koff = off if keys is None else offsets(keys)
    q, k, v = inputs(sum(n) + D, off[-1], koff[-1], Hq, Hkv, D, dtype)
    out = m.prompt_attend(q, k, v, off, None if keys is None else koff)
    check(out, q, k, v, off, koff, D ** -0.5)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_slices_of_a_projection_and_many_sequences(dtype, D):
    n = [(7 * i) % 61 for i in range(64)]
    off = offsets(n)
    q, k, v = inputs(D, off[-1], off[-1], 4, 2, D, dtype, fused=True)
    guard = torch.full((off[-1] + 64, 4, D), 7.0, dtype=DT[dtype], device=DEV)
    out = m.prompt_attend(q, k, v, off, scale=-0.3, out=guard[32:-32])
    check(out, q, k, v, off, off, -0.3)
    assert (guard[:32] == 7).all() and (guard[-32:] == 7).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("scale", [0.0, 1e-30, 3.0])
def test_scales(dtype, scale):
    off, koff = [0, 40, 200], [0, 140, 300]
    q, k, v = inputs(5, 200, 300, 4, 2, 64, dtype)
    check(m.prompt_attend(q, k, v, off, koff, scale=scale), q, k, v, off, koff, scale)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_rising_and_falling_scores(dtype):
    """The running maximum moves in every step, or never after the first."""
    off = [0, 300]
    for sign in (1, -1):
        q, k, v = inputs(6, 300, 300, 2, 1, 128, dtype)
        k = (k * 0.1 + sign * torch.linspace(-8, 8, 300, device=DEV)[:, None, None]).to(DT[dtype])
        q = (q * 0.1 + 1).to(DT[dtype])
        check(m.prompt_attend(q, k, v, off), q, k, v, off, off, 128 ** -0.5)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_other_sequences_values_stay_their_own(dtype):
    """NaN and infinities of one sequence, or behind the last, are not seen by another."""
    off = offsets([50, 33, 70])
    q, k, v = inputs(7, 160, 160, 2, 1, 64, dtype)
    clean = m.prompt_attend(q[:153], k[:153], v[:153], off)
    for x, bad in ((k, float("nan")), (v, float("inf"))):
        x[50:83] = bad
        x[153:] = bad
    out = m.prompt_attend(q[:153], k[:153], v[:153], off)
    assert torch.equal(out[:50], clean[:50]) and torch.equal(out[83:], clean[83:])


def test_long_piece_is_split_and_same_in_every_run():
    off, koff = [0, 130], [0, 20011]
    q, k, v = inputs(8, 130, 20011, 8, 2, 128, "bf16")
    out = m.prompt_attend(q, k, v, off, koff)
    check(out, q, k, v, off, koff, 128 ** -0.5)
    assert torch.equal(out, m.prompt_attend(q, k, v, off, koff))


def test_offsets_beyond_four_gib():
    """K and V rows more than 2^32 bytes behind their tensor's beginning."""
    T = 70000
    wide = torch.empty((T, 2, 16640), dtype=torch.bfloat16, device=DEV)  # 4.7 GB
    off = [0, T - 100, T]
    g = torch.Generator(device=DEV).manual_seed(1)
    tail = torch.randn((100, 3, 256), generator=g, device=DEV).bfloat16()
    wide[-100:, 0, :512] = tail[:, :2].reshape(100, 512)
    k, v = wide[:, 0, :256].unsqueeze(1), wide[:, 0, 256:512].unsqueeze(1)
    q = tail[:, 2:]
    out = m.prompt_attend(q, k, v, [0, 0, 100], off)
    ref = m.prompt_attend(q, tail[:, :1].contiguous(), tail[:, 1:2].contiguous(), [0, 100])
    assert torch.equal(out, ref)


def test_graph_and_streams():
    off, koff = [0, 3, 150], [0, 700, 1000]
    args = [inputs(s, 150, 1000, 4, 2, 128, "f32") for s in range(3)]
    q, k, v = (x.clone() for x in args[0])
    ws = torch.empty(m.lib().prompt_attend_workspace_bytes(2, (m._i32 * 3)(*off), (m._i32 * 3)(*koff), 4, 2, 128, 0),
                     dtype=torch.uint8, device=DEV)
    m.prompt_attend(q, k, v, off, koff, workspace=ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = m.prompt_attend(q, k, v, off, koff, workspace=ws)
    for a in args:
        for x, y in zip((q, k, v), a):
            x.copy_(y)
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone()
        s = torch.cuda.Stream()
        ref = m.prompt_attend(*a, off, koff, stream=s)
        torch.cuda.current_stream().wait_stream(s)
        assert torch.equal(got, ref)
        check(got, *a, off, koff, 128 ** -0.5)


def test_nothing():
    q, k, v = inputs(1, 4, 4, 2, 1, 64, "bf16")
    assert m.prompt_attend(q[:0], k[:0], v[:0], [0, 0]).shape == (0, 2, 64)
    assert (m.prompt_attend(q, k[:0], v[:0], [0, 4], [0, 0]) == 0).all()
