"""The norm of the errors of prompt_attend and experts on random inputs, beside
the bounds of single elements in their own tests: a product of the float32 forms
that is left out, or a rounding of the bf16 forms too many, shows here
(limits and their reasons in norms.py; what they tell apart in test_norm_limits.py)."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import moe_speculative_decoding_router_amd as m  # noqa: E402
import norms  # noqa: E402
import test_gpu_prompt_attend as attend  # noqa: E402
from plan_rules import tile_rows  # noqa: E402
from test_gpu_experts import Layer  # noqa: E402


def within(got, ref, limit):
    off = norms.off(got, ref)
    print(f"    {off:.3g} of the norm, limit {limit:.3g}")
    assert off <= limit


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n,keys", [([200], None), ([1, 300, 77], None), ([100], [700]), ([40], [4001]), ([3, 50], [1000, 700])])
def test_attention(n, keys, dtype, D):
    off = attend.offsets(n)
    koff = off if keys is None else attend.offsets(keys)
    q, k, v = attend.inputs(sum(n) + D, off[-1], koff[-1], 4, 2, D, dtype)
    ref = attend.reference(q, k, v, off, koff, D ** -0.5)[0]
    most = max(b - a for a, b in zip(koff, koff[1:]))
    within(m.prompt_attend(q, k, v, off, koff), ref, norms.attend_f32(most) if dtype == "f32" else norms.attend_bf16())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,H,I,E,wdtype,shared,large", [
    (300, 64, 64, 8, "bf16", False, ""), (70, 1152, 512, 8, "bf16", True, ""), (600, 2880, 1472, 4, "bf16", False, "f32"),
    (2000, 576, 544, 64, "bf16", False, "f32 bf16"), (300, 1152, 512, 6, "fp8", False, ""), (2000, 640, 512, 64, "fp8", True, "f32 bf16")])
def test_experts(T, H, I, E, wdtype, shared, large, dtype):
    assert (tile_rows(T, 2, E, I, dtype == "f32") > 32) == (dtype in large.split())  # the types that take large tiles
    L = Layer(H + I, H, I, E, 2, wdtype, shared)
    x, idx, w = L.inputs(T, T, dtype)
    ref = L.reference(x, idx, w)[0]
    within(m.experts(x, L.w, idx, w), ref, norms.experts_f32(H, I, wdtype == "fp8") if dtype == "f32" else norms.experts_bf16())
