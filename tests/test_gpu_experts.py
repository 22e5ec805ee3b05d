"""The experts' products over many tokens (experts) against the formula in float64.

Bounds, with u = 2^-24 and b = half a step of the activations' type (2^-8 for
bf16, u for float32, whose three bf16 terms are exact to 2^-24 and 2^-24 is
left out of the products): a gate or up sum of H terms is off by (H + 8) u and
the left-out u of G = sum |x w|; an fp8 layer multiplies its sums by a ratio every
128 terms, H / 128 more roundings.  A hidden activation silu(g) u moves by |u| 1.1
dg + |silu(g)| du (|silu'| <= 1.1), by 8 u of itself for the exponential and
division, and b of itself when it is stored.  A row's output takes these through
sum |h error| |w| and its own sum's (I + 8) u; the token's sum k u and the last
rounding b."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import moe_speculative_decoding_router_amd as m  # noqa: E402

DEV = torch.device("cuda:0")
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def make_weights(g, E, rows, cols, wdtype):
    """Codes [E, rows, cols], block scales or None, and the float64 values."""
    r = torch.randn((E, rows, cols), generator=g, device=DEV)
    if wdtype == "bf16":
        w = (r * cols ** -0.5).bfloat16()
        return w, None, w.double()
    w = (12 * r).to(torch.float8_e4m3fn)
    s = torch.exp2(4 * torch.rand((E, rows // 128, cols // 128), generator=g, device=DEV) - 2) / 12 * cols ** -0.5
    s *= torch.randint(0, 2, s.shape, generator=g, device=DEV) * 2 - 1
    return w, s, w.double() * s.double().repeat_interleave(128, 1).repeat_interleave(128, 2)


class Layer:
    def __init__(self, seed, H, I, E, k, wdtype="bf16", shared=False):
        g = torch.Generator(device=DEV).manual_seed(seed)
        W, self.val = {}, {}
        for name, n in [("", E)] + ([("sh", 1)] if shared else []):
            for part, rows, cols in (("gu", 2 * I, H), ("d", H, I)):
                w, s, val = make_weights(g, n, rows, cols, wdtype)
                W[f"W{name}_{part}"], self.val[name + part] = w, val
                if s is not None:
                    W[f"s{name}_{part}"] = s
        self.H, self.I, self.E, self.k, self.wdtype, self.shared = H, I, E, k, wdtype, shared
        self.w = m.LayerWeights(H=H, I=I, E=E, k=k, wdtype=wdtype, Wr=torch.zeros((E, H), device=DEV),
                                **m.pack_layer_tensors(W, wdtype))

    def reference(self, x, idx, w):
        """float64 y and the bound of its error."""
        u, b = 2.0 ** -24, (2.0 ** -8 if x.dtype == torch.bfloat16 else 2.0 ** -24)
        more = 1 if x.dtype == torch.float32 else 0
        H, I = self.H, self.I
        extra = lambda n: (n + 8 + (n // 128 if self.wdtype == "fp8" else 0) + more) * u  # noqa: E731
        X = x.double()
        y, tol = torch.zeros_like(X), torch.zeros_like(X)

        def ffn(rows, gu, d):
            z, far = rows @ gu.t().contiguous(), rows.abs() @ gu.abs().t().contiguous()
            gate, up = z[:, :I], z[:, I:]
            silu = gate * torch.sigmoid(gate)
            dg, du = far[:, :I] * extra(H), far[:, I:] * extra(H)
            h = silu * up
            dh = 1.1 * dg * up.abs() + silu.abs() * du + 1.1 * dg * du + (8 * u + b) * h.abs()
            o = h @ d.t().contiguous()
            do = dh @ d.abs().t().contiguous() + (h.abs() + dh) @ d.abs().t().contiguous() * extra(I)
            return o, do

        jobs = [(("", e), (w.double() * (idx == e)).sum(1), (idx == e).any(1)) for e in range(self.E)]
        if self.shared:
            jobs.append((("sh", 0), torch.ones(len(x), dtype=torch.float64, device=DEV), torch.ones(len(x), dtype=torch.bool, device=DEV)))
        for (name, e), share, sel in jobs:
            rows = torch.nonzero(sel)[:, 0]
            if len(rows):
                o, do = ffn(X[rows], self.val[name + "gu"][e], self.val[name + "d"][e])
                y[rows] += share[rows, None] * o
                tol[rows] += share[rows, None].abs() * (do + (self.k + 2) * u * o.abs())
        return y, tol + b * (y.abs() + tol)

    def check(self, x, idx, w, y=None):
        y = m.experts(x, self.w, idx, w) if y is None else y
        ref, tol = self.reference(x, idx, w)
        err = (y.double() - ref).abs()
        assert y.dtype == x.dtype and torch.isfinite(y).all()
        worst = float((err / (tol + 1e-30)).max())
        print(f"    largest error {float(err.max()):.3g}, {worst:.3g} of the bound")
        assert worst <= 1.0
        return y

    def inputs(self, seed, T, dtype, skew=1.0):
        g = torch.Generator(device=DEV).manual_seed(seed)
        x = torch.randn((T, self.H), generator=g, device=DEV).to(DT[dtype])
        logits = skew * torch.randn((1, self.E), generator=g, device=DEV) + torch.randn((T, self.E), generator=g, device=DEV)
        idx, w = m.route_tokens(logits, self.k)
        return x, idx, w


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("H,I,E,k,wdtype,shared", [(64, 32, 4, 2, "bf16", False), (192, 96, 5, 1, "bf16", True), (320, 224, 8, 3, "bf16", False),
                                                  (128, 128, 4, 2, "fp8", True), (384, 256, 6, 2, "fp8", False), (640, 384, 3, 3, "fp8", True)])
@pytest.mark.parametrize("T", [1, 3, 33, 70, 300, 1100])
def test_shapes(T, H, I, E, k, wdtype, shared, dtype):
    L = Layer(H + I, H, I, E, k, wdtype, shared)
    L.check(*L.inputs(T, T, dtype))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("wdtype", ["bf16", "fp8"])
@pytest.mark.parametrize("T,E,k", [(64, 512, 32), (2000, 64, 4), (257, 1, 1), (4096, 16, 2), (5000, 3, 2)])
def test_tile_sizes(T, E, k, wdtype, dtype):
    """Few and many rows an expert (all tile sizes), one expert, many empty ones; lists of one and of several parts."""
    L = Layer(T, 256, 128, E, k, wdtype, shared=E == 64)
    L.check(*L.inputs(T, T, dtype, skew=3.0))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_odd_sizes_and_long_sums(dtype):
    L = Layer(9, 2880, 1440 + 32, 4, 2, "bf16")
    L.check(*L.inputs(1, 600, dtype))
    L = Layer(10, 1152, 2176, 4, 2, "fp8", shared=True)
    L.check(*L.inputs(2, 600, dtype))


@pytest.mark.parametrize("T", [5, 700])
def test_entries_that_name_no_expert_or_one_twice(T):
    L = Layer(11, 128, 64, 6, 4)
    x, idx, w = L.inputs(3, T, "bf16")
    idx[0] = -1
    idx[1, 2] = 6
    idx[2] = 3
    idx[3, 1], idx[4, 0] = 2 ** 31 - 1, -2 ** 31
    y = L.check(x, idx, w)
    assert (y[0] == 0).all()
    none = torch.full_like(idx, -1)
    assert (m.experts(x, L.w, none, w) == 0).all()


def test_all_tokens_to_one_expert_and_weights_of_any_sign():
    L = Layer(12, 256, 96, 40, 2)
    x, idx, w = L.inputs(4, 3000, "bf16")
    idx[:, 0], idx[:, 1] = 39, 0
    w = torch.randn(w.shape, device=DEV)
    L.check(x, idx, w)


def test_scales_of_zero_and_far_apart():
    L = Layer(13, 256, 256, 3, 2, "fp8")
    s_gu, s_d = L.w.s_gu, L.w.s_d
    s_gu[0, :, 0] = 0.0
    s_gu[1, 1, 1] = 0.0
    s_d[2] *= 2.0 ** 30
    s_d[0, :, 1] *= 2.0 ** -40
    s_d[1] = 0.0
    W = {"gu": s_gu, "d": s_d}
    g = torch.Generator(device=DEV).manual_seed(13)
    for part, rows, cols in (("gu", 512, 256), ("d", 256, 256)):
        w, s, _ = make_weights(g, 3, rows, cols, "fp8")
        L.val[part] = w.double() * W[part].double().repeat_interleave(128, 1).repeat_interleave(128, 2)
    x, idx, w = L.inputs(5, 200, "f32")
    idx[:10] = 1  # an expert without output: at most 2^-127 of each code is left of it
    y = m.experts(x, L.w, idx, w)
    assert y[:10].abs().max() < 1e-30
    L.check(x[10:], idx[10:], w[10:])


def test_strides_in_place_guards_and_repeats():
    L = Layer(14, 192, 64, 8, 2, shared=True)
    x, idx, w = L.inputs(6, 500, "bf16")
    wide = torch.full((500, 320), float("nan"), dtype=torch.bfloat16, device=DEV)
    wide[:, 64:256] = x
    ref = L.check(x, idx, w)
    assert torch.equal(m.experts(wide[:, 64:256], L.w, idx, w), ref)
    guard = torch.full((520, 192), 7.0, dtype=torch.bfloat16, device=DEV)
    m.experts(x, L.w, idx, w, out=guard[10:510])
    assert (guard[:10] == 7).all() and (guard[510:] == 7).all() and torch.equal(guard[10:510], ref)
    for _ in range(3):
        assert torch.equal(m.experts(x, L.w, idx, w), ref)
    y = x.clone()
    m.experts(y, L.w, idx, w, out=y)
    assert torch.equal(y, ref)
    one = m.experts(x[17:18], L.w, idx[17:18], w[17:18])  # a token alone: other tile sizes, the same sums' order
    assert (one.float() - ref[17:18].float()).abs().max() <= 0.02 * ref.float().abs().max()
    assert m.experts(x[:0], L.w, idx[:0], w[:0]).shape == (0, 192)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("wdtype", ["bf16", "fp8"])
@pytest.mark.parametrize("T,E", [(37, 4), (400, 8), (1500, 40)])
def test_every_call_gives_the_same_bits(T, E, wdtype, dtype):
    """Rows lie in another place of their expert's tiles in every call, in tiles filled to any part."""
    L = Layer(18, 256, 256, E, 2, wdtype, shared=True)
    x, idx, w = L.inputs(9, T, dtype)
    ref = L.check(x, idx, w)
    for _ in range(15):
        assert torch.equal(m.experts(x, L.w, idx, w), ref)
    order = torch.randperm(T, device=DEV)
    assert torch.equal(m.experts(x[order].contiguous(), L.w, idx[order].contiguous(), w[order].contiguous()), ref[order])


def test_neighbours_that_are_no_numbers():
    """A token's NaN stays its own."""
    L = Layer(15, 128, 64, 3, 1)
    x, idx, w = L.inputs(7, 300, "bf16")
    ref = m.experts(x, L.w, idx, w)
    x[100:150] = float("nan")
    y = m.experts(x, L.w, idx, w)
    keep = torch.ones(300, dtype=torch.bool)
    keep[100:150] = False
    assert torch.equal(y[keep], ref[keep])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_graph_and_streams(dtype):
    L = Layer(16, 256, 128, 8, 2, "fp8", shared=True)
    args = [L.inputs(s, 400, dtype) for s in range(3)]
    x, idx, w = (a.clone() for a in args[0])
    ws = torch.empty(int(m.lib().moe_experts_workspace_bytes(m.ctypes.byref(L.w._c()), 400, 0 if dtype == "f32" else 1)),
                     dtype=torch.uint8, device=DEV)
    m.experts(x, L.w, idx, w, workspace=ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = m.experts(x, L.w, idx, w, workspace=ws)
    for a in args:
        for p, q in zip((x, idx, w), a):
            p.copy_(q)
        graph.replay()
        torch.cuda.synchronize()
        got = y.clone()
        s = torch.cuda.Stream()
        ref = m.experts(a[0], L.w, a[1], a[2], stream=s)
        torch.cuda.current_stream().wait_stream(s)
        assert torch.equal(got, ref)
        L.check(*a, y=got)


def test_agrees_with_the_verify_layer():
    """64 tokens through both: the same choices, the same layer."""
    L = Layer(17, 512, 256, 16, 4)
    g = torch.Generator(device=DEV).manual_seed(8)
    L.w.Wr = torch.randn((16, 512), generator=g, device=DEV)
    x = torch.randn((64, 512), generator=g, device=DEV).bfloat16()
    y, aux = m.verify_layer(x.float(), L.w)
    idx, w = m.route_tokens(aux.logits, 4)
    assert torch.equal(idx, aux.topk_idx) and np.allclose(w.cpu(), aux.topk_w.cpu(), rtol=0, atol=1e-6)
    got = L.check(x, idx, w)
    rms = float(y.pow(2).mean().sqrt())
    assert float((got.float() - y).abs().max()) <= 4e-2 * rms
