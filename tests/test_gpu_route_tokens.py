"""route_tokens against a stable sort: the experts are equal, the weights
float32 (a difference, an exponential of 2 units, a sum of at most 32 terms
and a division: below 8 + 32 roundings of 2^-24)."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import moe_speculative_decoding_router_amd as m  # noqa: E402

DEV = torch.device("cuda:0")


def reference(x, k):
    x = np.asarray(x, dtype=np.float64)
    x = np.where(np.isnan(x), -np.inf, np.minimum(x, np.finfo(np.float32).max))
    idx = np.argsort(-x, axis=1, kind="stable")[:, :k]
    val = np.take_along_axis(x, idx, 1)
    with np.errstate(invalid="ignore"):
        e = np.where(val[:, :1] > -np.inf, np.exp(val - val[:, :1]), 0.0)
    e = np.nan_to_num(e)
    z = e.sum(1, keepdims=True)
    return idx, np.where(z > 0, e / np.where(z > 0, z, 1), 0.0)


def check(x, k):
    idx, w = m.route_tokens(x, k)
    ri, rw = reference(x.float().cpu().numpy(), k)
    assert np.array_equal(idx.cpu().numpy(), ri)
    # a difference of the logits is off by 2^-24 of itself, and weights that matter have differences below 88
    tol = (40 + 88) * 2.0 ** -24
    assert np.abs(w.double().cpu().numpy() - rw).max() <= tol
    return idx, w


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 2, 2), (5, 63, 32), (65, 64, 8), (67, 65, 1), (1000, 128, 8), (129, 200, 32),
                                   (300, 256, 8), (33, 257, 5), (4097, 512, 8), (3, 512, 32)])
def test_shapes(T, E, k):
    g = torch.Generator(device=DEV).manual_seed(T * E + k)
    check(2 * torch.randn((T, E), generator=g, device=DEV), k)


def test_ties_zeros_and_values_that_are_none():
    g = torch.Generator(device=DEV).manual_seed(1)
    x = torch.randint(-2, 3, (200, 130), generator=g, device=DEV).float()
    x[::2] *= -1  # zeros of both signs are equal
    check(x, 9)
    inf, nan = float("inf"), float("nan")
    rows = [[nan, 1, 2, -inf], [inf, 1, inf, 0], [-inf] * 4, [nan] * 4, [-inf, nan, -3e38, -inf], [3.4e38, inf, -inf, 3e38]]
    check(torch.tensor(rows, device=DEV), 4)


def test_strides_streams_empty_and_graph():
    g = torch.Generator(device=DEV).manual_seed(2)
    wide = torch.randn((70, 300), generator=g, device=DEV)
    check(wide[:, 17:145], 8)
    assert m.route_tokens(wide[:0], 4)[0].shape == (0, 4)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    a = m.route_tokens(wide, 6, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    b = m.route_tokens(wide, 6)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        idx, w = m.route_tokens(wide, 6)
    for seed in range(3):
        wide.copy_(torch.randn((70, 300), generator=g, device=DEV))
        graph.replay()
        torch.cuda.synchronize()
        ri, rw = m.route_tokens(wide, 6)
        assert torch.equal(idx, ri) and torch.equal(w, rw)
