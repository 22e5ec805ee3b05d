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
