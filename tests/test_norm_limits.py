"""That the limits of tests/norms.py tell a kernel's roundings from one too few
terms or one rounding too many: the products are emulated in float64 with their
operands cut as the kernels cut them (CPU)."""
import pytest

torch = pytest.importorskip("torch")

import norms  # noqa: E402


def terms(x, n):
    """n bf16 terms of x, each the rest's nearest."""
    out = []
    for _ in range(n):
        t = x.to(torch.float32).to(torch.bfloat16).double()
        out.append(t)
        x = x - t
    return out


def product(a, b, n):
    """a @ b of n terms each, without the products below the last term's."""
    a, b = terms(a, n), terms(b, n)
    return sum(a[i] @ b[j] for i in range(n) for j in range(n - i))


def half(x):
    return x.to(torch.float32).to(torch.bfloat16).double()


def cut_off(x):
    """bf16 towards zero instead of to nearest."""
    return (x.to(torch.float32).view(torch.int32) & -65536).view(torch.float32).double()


def attention(q, k, v, n=None, last=half):
    """Causal, of one head; n terms, or bf16 operands with rounded probabilities (n 0), or neither."""
    T, m = len(q), len(k)
    s = (product(q, k.t(), n) if n else q @ k.t()) * q.shape[1] ** -0.5
    s = s.masked_fill(torch.arange(m)[None] > torch.arange(T)[:, None] + (m - T), -float("inf"))
    p = torch.exp(s - s.amax(1, keepdim=True))
    if n is None:
        return p / p.sum(1, keepdim=True) @ v
    if n:
        return product(p, v, n) / p.sum(1, keepdim=True)
    p = half(p)
    return last(p @ v / p.sum(1, keepdim=True))


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("T,keys", [(200, 200), (100, 700), (40, 4001)])
def test_attention(T, keys, D):
    g = torch.Generator().manual_seed(D + keys)
    q, k, v = (torch.randn((n, D), generator=g).double() for n in (T, keys, keys))
    ref = attention(q, k, v)
    limit = norms.attend_f32(keys)
    assert norms.off(attention(q, k, v, 3), ref) < 0.2 * limit
    assert norms.off(attention(q, k, v, 2), ref) > 1.5 * limit
    q, k, v = half(q), half(k), half(v)
    ref = attention(q, k, v)
    assert norms.off(attention(q, k, v, 0), ref) < norms.attend_bf16()
    assert norms.off(attention(q, k, v, 0, cut_off), ref) > norms.attend_bf16()


def ffn(x, gu, d, n=None):
    """An expert's output from x: n terms of the activations and hidden activations, or rounded hidden ones (n 0)."""
    cut = lambda a: a if n is None else half(a) if n == 0 else sum(terms(a, n))  # noqa: E731
    z = (x if n == 0 else cut(x)) @ gu.t()
    gate, up = z.chunk(2, 1)
    return cut(gate * torch.sigmoid(gate) * up) @ d.t()


@pytest.mark.parametrize("H,I", [(64, 64), (1152, 512), (2880, 1472), (8320, 128), (128, 8320)])
def test_experts(H, I):
    """Two experts a token, as every test of them has."""
    g = torch.Generator().manual_seed(H)
    x = torch.randn((60, H), generator=g).double()
    W = [(half(torch.randn((2 * I, H), generator=g) * H ** -0.5), half(torch.randn((H, I), generator=g) * I ** -0.5)) for _ in range(2)]
    w = torch.rand((60, 2), generator=g).double()
    total = lambda a, n, f=lambda o: o: sum(w[:, j:j + 1] * f(ffn(a, *W[j], n)) for j in range(2))  # noqa: E731
    ref = total(x, None)
    for fp8 in (False, True):
        assert norms.off(total(x, 3), ref) < 0.2 * norms.experts_f32(H, I, fp8)
        assert norms.off(total(x, 2), ref) > 1.2 * norms.experts_f32(H, I, fp8)
    x = half(x)
    ref = total(x, None)
    assert norms.off(half(total(x, 0)), ref) < norms.experts_bf16()
    assert norms.off(half(total(x, 0, half)), ref) > norms.experts_bf16()  # outputs stored as bf16 before they are added
