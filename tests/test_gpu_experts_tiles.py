"""The experts' large product tiles (256 weight rows by 256 activation rows in
bf16, 128 by 128 in float32): every number of activation rows that they are
compiled for, partly filled tiles in both directions, an odd number of 32 k, both
weight formats.  Bounds as in test_gpu_experts.py.  Each test asserts that its
call takes the tiles that it is about (the rule is checked in test_host_plan.py)."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import moe_speculative_decoding_router_amd as m  # noqa: E402
import norms  # noqa: E402
from plan_rules import tile_rows  # noqa: E402
from test_gpu_experts import DEV, DT, Layer  # noqa: E402

LARGE = {"bf16": 256, "f32": 128}
# rows of the first experts; both sides of every 64 rows (a step of the tile), of a whole tile and of several
COUNTS = [1, 63, 64, 65, 127, 128, 129, 191, 192, 193, 255, 256, 257, 300, 320, 448, 511, 513, 0, 2]


def choices(L, counts, seed, dtype):
    """Tokens and choices that give expert e counts[e] rows, in an order of no meaning."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    pairs = torch.repeat_interleave(torch.arange(L.E, device=DEV), torch.tensor(counts, device=DEV))
    pairs = pairs[torch.randperm(len(pairs), generator=g, device=DEV)]
    T = len(pairs) // L.k
    idx = pairs[:T * L.k].view(T, L.k).to(torch.int32).contiguous()
    w = torch.rand(idx.shape, generator=g, device=DEV) - 0.3
    return torch.randn((T, L.H), generator=g, device=DEV).to(DT[dtype]), idx, w


def spread(E, k):
    """COUNTS, then as many more as make a multiple of k."""
    c = COUNTS + [40 + e % 7 for e in range(E - len(COUNTS))]
    c[-1] += -sum(c) % k
    return c


def takes(L, T, dtype, rows):
    assert tile_rows(T, L.k, L.E, L.I, dtype == "f32") == rows


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("H,I,E,k,wdtype,shared", [(320, 544, 64, 1, "bf16", False), (192, 672, 64, 2, "bf16", True), (576, 512, 64, 2, "bf16", False),
                                                   (64, 32, 128, 2, "bf16", False), (384, 512, 64, 2, "fp8", True), (640, 640, 64, 1, "fp8", False)])
def test_rows_of_every_number(H, I, E, k, wdtype, shared, dtype):
    """H and I leave the last weight tile partly filled, an odd number of 32 k (I 544, 672, 32), or one step of 64 k."""
    L = Layer(H + I, H, I, E, k, wdtype, shared)
    x, idx, w = choices(L, spread(E, k), H, dtype)
    takes(L, len(x), dtype, LARGE[dtype])
    ref = L.check(x, idx, w)
    for _ in range(5):
        assert torch.equal(m.experts(x, L.w, idx, w), ref)
    order = torch.randperm(len(x), device=DEV)
    assert torch.equal(m.experts(x[order].contiguous(), L.w, idx[order].contiguous(), w[order].contiguous()), ref[order])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("wdtype", ["bf16", "fp8"])
def test_one_expert_has_all(wdtype, dtype):
    """Many full tiles of one expert, one row in another, and the list's entries that name none."""
    I = 8192
    L = Layer(2, 128, I, 2, 2, wdtype)
    x, idx, w = choices(L, [2999, 1], 3, dtype)
    idx[::7, 0] = 2
    takes(L, len(x), dtype, LARGE[dtype])
    ref = L.check(x, idx, w)
    assert torch.equal(m.experts(x, L.w, idx, w), ref)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("wdtype", ["bf16", "fp8"])
def test_strides_and_a_graph(wdtype, dtype):
    L = Layer(5, 256, 512, 64, 2, wdtype, shared=True)
    args = [choices(L, spread(64, 2), s, dtype) for s in range(3)]
    T = len(args[0][0])
    takes(L, T, dtype, LARGE[dtype])
    wide = torch.full((T, 512), float("nan"), dtype=DT[dtype], device=DEV)
    x, idx, w = wide[:, 64:320], args[0][1].clone(), args[0][2].clone()
    x.copy_(args[0][0])
    m.experts(x, L.w, idx, w)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = m.experts(x, L.w, idx, w)
    for a in args:
        for p, q in zip((x, idx, w), a):
            p.copy_(q)
        graph.replay()
        torch.cuda.synchronize()
        got = y.clone()
        assert torch.equal(got, m.experts(a[0], L.w, a[1], a[2]))
        L.check(*a, y=got)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("H,I,E,T,large", [(8320, 128, 3, 50, False), (8320, 128, 128, 3700, True), (128, 8320, 1, 20, False), (128, 8320, 4, 150, True)])
def test_more_blocks_than_a_wave_has_lanes(H, I, E, T, large, dtype):
    """fp8 sums of 65 blocks of 128 k: a lane holds the scales of every 64th block, the second set one block alone.
    Scales differ by block, over a factor of 16 and by sign."""
    L = Layer(H + E, H, I, E, 1, "fp8")
    takes(L, T, dtype, LARGE[dtype] if large else 32)
    x, idx, w = L.inputs(T, T, dtype)
    y = L.check(x, idx, w)
    ref = L.reference(x, idx, w)[0]
    assert norms.off(y, ref) <= (norms.experts_f32(H, I, True) if dtype == "f32" else norms.experts_bf16())
    assert torch.equal(m.experts(x, L.w, idx, w), y)
