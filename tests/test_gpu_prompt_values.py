"""prompt_attend with values that are no ordinary numbers.

The definition's weights are exp(score - max) over their sum: a NaN among a
row's visible scores, one of +inf, or nothing but -inf make the whole row NaN.
Only rows that see no key are zeros, whatever their query and the sequence's
keys and values hold.  Rows beside them stay within the bounds of
test_gpu_prompt_attend.py."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import moe_speculative_decoding_router_amd as m  # noqa: E402
import test_gpu_prompt_attend as base  # noqa: E402

DEV, DT = base.DEV, base.DT
SPLIT = [(([0, 70], [0, 90]), False), (([0, 5, 75], [0, 1400, 2500]), True), (([0, 300], [0, 300]), False)]


def shares(off, koff, Hq, Hkv, D, dtype):
    """Whether the call's units are cut into shares: they take workspace beside the float32 terms."""
    f32 = dtype == "f32"
    need = m.lib().prompt_attend_workspace_bytes(len(off) - 1, (m._i32 * len(off))(*off), (m._i32 * len(off))(*koff), Hq, Hkv, D, 0 if f32 else 1)
    return need > ((koff[-1] * Hkv * D * 12 + 255) // 256 * 256 if f32 else 0)


def check_others(out, q, k, v, off, koff, scale, odd):
    """Rows and heads outside `odd` against the definition, with the queries of `odd` replaced by zeros."""
    calm = torch.where(odd[..., None], torch.zeros_like(q), q)
    ref, bound, reach = base.reference(calm, k, v, off, koff, scale)
    keys = max(b - a for a, b in zip(koff, koff[1:]))
    rel = 2 * (q.shape[2] + 12) * 2.0 ** -24 * reach + (keys + 72) * 2.0 ** -24
    half = 2.0 ** -8 if q.dtype == torch.bfloat16 else 2.0 ** -24
    tol = (rel + (half if q.dtype == torch.bfloat16 else 0)) * bound + half * ref.abs()
    bad = ~((out.double() - ref).abs() <= tol + 1e-30) & ~odd[..., None]
    assert not bad.any(), torch.nonzero(bad.any(-1)).tolist()[:10]


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("offs,cut", SPLIT)
def test_queries_that_are_no_numbers(offs, cut, dtype, D):
    """NaN of any sign and payload, and infinities, in a query give NaN in its row and head alone."""
    off, koff = offs
    Hq, Hkv = 4, 2
    assert shares(off, koff, Hq, Hkv, D, dtype) == cut
    q, k, v = base.inputs(D + koff[-1], off[-1], koff[-1], Hq, Hkv, D, dtype)
    bits = torch.int32 if dtype == "f32" else torch.int16
    nans = [0x7FC00000, 0x7FFFFFFF, -1, 0x7F800001, 0x7FFF8000, -2 ** 15] if dtype == "f32" else [0x7FC0, 0x7FFF, -1, 0x7F81, -127]
    odd = torch.zeros(q.shape[:2], dtype=torch.bool, device=DEV)
    for i, b in enumerate(nans):
        t, h = (13 * i + 2) % off[-1], i % Hq
        q.view(bits)[t, h, (29 * i) % D] = b
        odd[t, h] = True
    q.view(bits)[off[-1] - 1, 1] = -1  # memory of 0xff
    q[off[-1] - 3, 0, 7], q[off[-1] - 4, 2, D - 1] = float("inf"), -float("inf")
    odd[off[-1] - 1, 1] = odd[off[-1] - 3, 0] = odd[off[-1] - 4, 2] = True
    for scale in (D ** -0.5, -0.3):
        out = m.prompt_attend(q, k, v, off, koff, scale=scale)
        assert torch.isnan(out[odd]).all(), torch.nonzero(odd & ~torch.isnan(out).all(-1)).tolist()
        check_others(out, q, k, v, off, koff, scale, odd)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("offs,cut", SPLIT)
def test_scores_beyond_the_range(offs, cut, dtype):
    """Scores of +inf, or of -inf for every key, are no weights: NaN, not zeros."""
    off, koff = offs
    assert shares(off, koff, 2, 1, 128, dtype) == cut
    q, k, v = base.inputs(3, off[-1], koff[-1], 2, 1, 128, dtype)
    q[:, :, 0] = 0
    k[:, :, 0] = 1e20
    odd = torch.zeros(q.shape[:2], dtype=torch.bool, device=DEV)
    for t, h, x in ((3, 0, 1e20), (off[-1] - 1, 1, -1e20), (off[-1] - 2, 0, -3e20)):
        q[t, h, 0] = x
        odd[t, h] = True
    out = m.prompt_attend(q, k, v, off, koff)
    assert torch.isnan(out[odd]).all(), torch.nonzero(odd & ~torch.isnan(out).all(-1)).tolist()
    k[:, :, 0] = 0  # the others' score has no part of it
    check_others(out, q, k, v, off, koff, 128 ** -0.5, odd)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("offs,cut", SPLIT)
def test_visible_keys_that_are_no_numbers(offs, cut, dtype):
    """A key that holds NaN makes every row that sees it NaN, in the heads that share it."""
    off, koff = offs
    assert shares(off, koff, 4, 2, 64, dtype) == cut
    q, k, v = base.inputs(4, off[-1], koff[-1], 4, 2, 64, dtype)
    n, keys = off[-1] - off[-2], koff[-1] - koff[-2]
    at = keys - 20  # seen by the last 20 rows of the last sequence
    k[koff[-2] + at, 1, 33] = float("nan")
    out = m.prompt_attend(q, k, v, off, koff)
    sees = torch.arange(n, device=DEV) + keys - n >= at
    assert torch.isnan(out[off[-2]:][sees][:, 2:]).all()
    assert torch.isfinite(out[off[-2]:][:, :2]).all() and torch.isfinite(out[:off[-2]]).all()


@pytest.mark.parametrize("D", [64, 256])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n,keys,cut", [(200, 70, False), (40, 0, False), (1000, 900, True)])
def test_rows_that_see_no_key_are_zeros(n, keys, cut, dtype, D):
    off, koff = [0, n], [0, keys]
    assert shares(off, koff, 2, 1, D, dtype) == cut
    q, k, v = base.inputs(n, n, keys, 2, 1, D, dtype)
    clean = m.prompt_attend(q, k, v, off, koff)
    base.check(clean, q, k, v, off, koff, D ** -0.5)
    q[: n - keys] = float("nan")
    assert torch.equal(m.prompt_attend(q, k, v, off, koff)[: n - keys], torch.zeros_like(q[: n - keys]))
    q[: n - keys: 2], k[:], v[:] = float("inf"), float("nan"), float("nan")
    out = m.prompt_attend(q, k, v, off, koff)
    assert (out[: n - keys] == 0).all() and torch.isnan(out[n - keys:]).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("offs,cut", SPLIT)
def test_scores_up_to_the_limit(offs, cut, dtype):
    """Scores of 2^29 in magnitude, whose running maximum is rounded by up to 32 (log2): still a mean of the values."""
    off, koff = offs
    q, k, v = base.inputs(9, off[-1], koff[-1], 2, 1, 64, dtype)
    _, _, reach = base.reference(q, k, v, off, koff, 1.0)
    out = m.prompt_attend(q, k, v, off, koff, scale=2.0 ** 28.9 / reach)
    assert torch.isfinite(out).all() and float(out.abs().max()) <= 1.01 * float(v.abs().max())
