"""accept_drafts and sample_tokens where a caller's values are none, and the
conditions that the comparisons of test_gpu_sampling rest on."""
import numpy as np
import pytest

from oracle import sampling as osa

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import moe_speculative_decoding_router_amd as m  # noqa: E402
import test_gpu_sampling as base  # noqa: E402

DEV = torch.device("cuda:0")
dev = base.dev


@pytest.mark.parametrize("V", [40, 5001, 60001])
def test_negative_draft_probabilities_accept_no_filtered_token(V):
    """A draft that the target's filter dropped (p = 0) is never accepted, whatever q holds; values of q below 0
    count as 0 and leave p for the last token."""
    rng = np.random.default_rng(V)
    n, S = 4, 3
    T, offsets = n * S, [0, n, 2 * n, 3 * n]
    x, xd = base.logits_of(rng, T, V, "f32")
    q = -rng.random((T, V)).astype(np.float32)
    q[2 * n:] = -np.inf
    tokens = np.zeros(T, dtype=np.int32)
    p = np.array([(lambda w: w / w.sum())(osa.kept_weights(x[t], 1.0, 5)[0]) for t in range(T)])
    for t in range(T - 1):
        s, j = divmod(t, n)
        kept = np.nonzero(p[t])[0]
        dropped = [i for i in rng.permutation(V)[:10] if p[t, i] == 0]
        tokens[t + 1] = kept[0] if j < s else dropped[0]     # the first draft of sequence 1 is kept, two of sequence 2
    u, uf = (0.01 + 0.99 * rng.random(T)).astype(np.float32), rng.random(S).astype(np.float32)
    out, path, count = m.accept_drafts(xd, dev(tokens), offsets, dev(u), draft_probs=dev(q), u_final=dev(uf),
                                       top_k=torch.full((T,), 5, dtype=torch.int32, device=DEV))
    assert count.tolist() == [1, 2, 3]
    res = [osa.accept_chain(p[a:b], q[a:b].astype(np.float64), tokens[a:b], u[a:b].astype(np.float64), float(uf[s]))
           for s, (a, b) in enumerate(zip(offsets, offsets[1:]))]
    base.compare((out, path, count), base.expect(res, offsets, T))
