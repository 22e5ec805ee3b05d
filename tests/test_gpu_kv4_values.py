"""The 4-bit K/V cache with values that are no ordinary numbers: NaN and
infinities in rows and queries, scales next to 0."""
import numpy as np
import pytest

from oracle import kv4 as okv

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import moe_speculative_decoding_router_amd as m  # noqa: E402
import test_gpu_kv4 as base  # noqa: E402

DEV = torch.device("cuda:0")
dev, DT = base.dev, base.DT


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_append_nan_and_infinities(D, dtype):
    """NaN (of any sign and payload) is stored as 0 and does not touch its block; infinities as the largest value."""
    Hkv, page, offsets, lens = 2, 16, [0, 12], [3]
    rng, table, data = base.setup(D, D, Hkv, page, lens, offsets)
    T = offsets[-1]
    kd = base.rounded(rng, (T, Hkv, D), dtype)[1]
    vd = base.rounded(rng, (T, Hkv, D), dtype)[1]
    bits = torch.int32 if dtype == "f32" else torch.int16
    nans = [0x7FC00000, 0x7FFFFFFF, -1, 0x7F800001, 0x7FFF0000] if dtype == "f32" else [0x7FC0, 0x7FFF, -1, 0x7F81, -127]
    for x in (kd, vd):
        for i, b in enumerate(nans):                       # one a block, at every place of a lane's eight
            x.view(bits)[i, 0, [i, 8 + i, 40 + i]] = b
        x.view(bits)[5, 1, :32] = nans[0]                  # a block of nothing else
        x[6, 0, 5], x[6, 0, 33], x[7, 1, 31] = float("inf"), -float("inf"), float("inf")
        x.view(bits)[7, 1, 30] = nans[1]
        x[8] = float("nan")
        x[9] = -float("inf")
    assert torch.isnan(kd[:5]).sum() == 15
    k, v = kd.double().cpu().numpy(), vd.double().cpu().numpy()
    c = base.cache_of(dev(data), D, Hkv, page)
    stored = m.kv4_append(c, kd, vd, dev(table), dev(np.array(lens, dtype=np.int32)), offsets, return_stored=True)
    okv.append(data, k, v, table, lens, offsets)
    for got, x in zip(stored, (k, v)):
        want = okv.quantise(x)[2]
        assert np.isfinite(want).all() and (want[np.isnan(x)] == 0).all()
        assert np.array_equal(got.double().cpu().numpy(), want)
    assert np.array_equal(c.data.cpu().numpy(), data)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("lens", [[40, 3], [3000, 700]])     # whole units, and units split over workgroups
def test_attend_nan_and_infinite_queries(D, dtype, lens):
    """A query that holds NaN, of whatever sign and payload, gives NaN; it and infinite ones touch no other row."""
    Hkv, G, page, offsets = 2, 8, 16, [0, 3, 5]
    rng, table, data = base.setup(D + lens[0], D, Hkv, page, lens, offsets)
    base.any_rows(rng, data, D)
    T, parent = offsets[-1], [-1, 0, 0, -1, 0]
    kd, vd = base.rounded(rng, (T, Hkv, D), dtype)[1], base.rounded(rng, (T, Hkv, D), dtype)[1]
    q, qd = base.rounded(rng, (T, Hkv * G, D), dtype)
    c, td, ld = base.cache_of(dev(data), D, Hkv, page), dev(table), dev(np.array(lens, dtype=np.int32))
    m.kv4_append(c, kd, vd, td, ld, offsets)
    clean = m.kv4_attend(c, qd, td, ld, offsets, parent=parent)
    base.check_attend(clean, q, c.data.cpu().numpy(), table, lens, offsets, parent, D ** -0.5, dtype)
    bits = torch.int32 if dtype == "f32" else torch.int16
    nans = [0x7FC00000, 0x7FFFFFFF, -1, 0x7F800001, 0x7FFF8000, -2 ** 15] if dtype == "f32" else [0x7FC0, 0x7FFF, -1, 0x7F81, -127]
    none, odd = torch.zeros((T, Hkv * G), dtype=torch.bool), torch.zeros((T, Hkv * G), dtype=torch.bool)
    for i, b in enumerate(nans):
        t, h = i % T, (5 * i) % (Hkv * G)
        qd.view(bits)[t, h, (7 * i) % D] = b
        none[t, h] = odd[t, h] = True
    qd.view(bits)[3, 7] = -1                             # memory of 0xff
    none[3, 7] = odd[3, 7] = True
    qd[4, 9, 5], qd[0, 13, 2] = float("inf"), -float("inf")
    odd[4, 9] = odd[0, 13] = True
    for scale in (None, -0.5):
        want = clean if scale is None else m.kv4_attend(c, dev(q.astype(np.float32)).to(DT[dtype]), td, ld, offsets, parent=parent, scale=scale)
        out = m.kv4_attend(c, qd, td, ld, offsets, parent=parent, scale=scale).cpu()
        assert torch.isnan(out[none]).all(), [i for i, x in enumerate(out[none]) if not torch.isnan(x).all()]
        # the running maximum moves for all rows of a block together, so the others may round differently
        base.check_attend(out, q, c.data.cpu().numpy(), table, lens, offsets, parent, D ** -0.5 if scale is None else scale, dtype, ~odd)
        assert torch.isfinite(want).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("scale", [0.0, -0.0, 1e-33, -1e-33, 1.4e-45, 1e-38])
def test_attend_scales_next_to_zero(scale, dtype):
    """Scores are scale * q.k however small the scale and large the products are; 0 weighs all visible rows alike."""
    D, Hkv, page, lens, offsets = 64, 1, 16, [45], [0, 3]
    rng, table, data = base.setup(13, D, Hkv, page, lens, offsets)
    base.fill(rng, data, table, lens, D, Hkv, 1e16)
    kd, vd = base.rounded(rng, (3, Hkv, D), dtype, 1e16)[1], base.rounded(rng, (3, Hkv, D), dtype)[1]
    q, qd = base.rounded(rng, (3, 4, D), dtype, 1e16)
    c, td, ld = base.cache_of(dev(data), D, Hkv, page), dev(table), dev(np.array(lens, dtype=np.int32))
    m.kv4_append(c, kd, vd, td, ld, offsets)
    parent, scale = [-1, 0, 0], float(np.float32(scale))
    out = m.kv4_attend(c, qd, td, ld, offsets, parent=parent, scale=scale)
    base.check_attend(out, q, c.data.cpu().numpy(), table, lens, offsets, parent, scale, dtype)
