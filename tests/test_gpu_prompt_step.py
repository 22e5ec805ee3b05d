"""The operators for prompts together, as a server uses them: prompts enter a
pool of pages, a second piece of one is attended behind the rows that stand
already, the experts of its tokens are chosen and computed, the prompt is
forked, the forks decode on their own, conversations end and the pool is
compacted.  Each result is compared with what plain operations make of the
cache's stored values."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import moe_speculative_decoding_router_amd as m  # noqa: E402

DEV = torch.device("cuda:0")


def i32(*v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def attention(q, k, v, off, koff):
    """float64 causal attention of packed sequences."""
    out = torch.zeros(q.shape, dtype=torch.float64, device=DEV)
    G = q.shape[1] // k.shape[1]
    for s in range(len(off) - 1):
        n, mk = off[s + 1] - off[s], koff[s + 1] - koff[s]
        hide = torch.arange(mk, device=DEV)[None] > torch.arange(n, device=DEV)[:, None] + (mk - n)
        for h in range(q.shape[1]):
            a = q[off[s]:off[s + 1], h].double() @ k[koff[s]:koff[s + 1], h // G].double().t().contiguous() * q.shape[2] ** -0.5
            out[off[s]:off[s + 1], h] = torch.softmax(a.masked_fill(hide, -float("inf")), -1) @ v[koff[s]:koff[s + 1], h // G].double()
    return out


def close(got, ref, tol):
    assert torch.isfinite(got.double()).all()
    assert float((got.double() - ref.double()).norm() / ref.double().norm()) <= tol


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_prompts_forks_and_compaction(dtype):
    # roundings of q k v and probabilities: 2^-8 each in bf16 at most, over the norm; float32 far below 1e-5
    tol = 2.0 ** -7 if dtype == torch.bfloat16 else 1e-5
    g = torch.Generator(device=DEV).manual_seed(4)
    page, Hq, Hkv, D, P, W = 16, 8, 2, 64, 120, 16
    refs, table = torch.zeros(P, dtype=torch.int32, device=DEV), torch.full((6, W), -1, dtype=torch.int32, device=DEV)
    cache = m.kv4_cache(P, page, Hkv, D, device=DEV)
    rnd = lambda *s: torch.randn(s, generator=g, device=DEV).to(dtype)  # noqa: E731

    # two prompts at once, of 37 and 70 rows, in sequences 3 and 0
    n = [37, 70]
    off = [0, 37, 107]
    assert m.kv4_reserve(refs, table, page, i32(3, 0), i32(*n)).tolist() == [1, 1]
    qkv = rnd(107, (Hq + 2 * Hkv) * D)
    q, k, v = (qkv[:, a * D:b * D].unflatten(1, (b - a, D)) for a, b in ((0, Hq), (Hq, Hq + Hkv), (Hq + Hkv, Hq + 2 * Hkv)))
    both = table[[3, 0]].contiguous()
    sk, sv = m.kv4_append(cache, k, v, both, i32(0, 0), off, return_stored=True)
    close(m.prompt_attend(q, sk, sv, off), attention(q, sk, sv, off, off), tol)

    # the next piece of the second prompt: 100 rows behind its 70
    assert m.kv4_reserve(refs, table, page, i32(0), i32(170)).tolist() == [1]
    q2, k2, v2 = rnd(100, Hq, D), rnd(100, Hkv, D), rnd(100, Hkv, D)
    sk2, sv2 = m.kv4_append(cache, k2, v2, table[:1], i32(70), [0, 100], return_stored=True)
    ak, av = m.kv4_read(cache, table[:1], i32(0), [0, 170], dtype=dtype)
    assert torch.equal(ak, torch.cat([sk[37:], sk2])) and torch.equal(av, torch.cat([sv[37:], sv2]))
    close(m.prompt_attend(q2, ak, av, [0, 100], [0, 170]), attention(q2, ak, av, [0, 100], [0, 170]), tol)

    # the experts of the piece's tokens, against the verify layer 20 tokens at a time
    H, I, E, K = 256, 128, 12, 3
    W_gu, W_d = ((0.05 * torch.randn(s, generator=g, device=DEV)).bfloat16() for s in ((E, 2 * I, H), (E, H, I)))
    Wr = torch.randn((E, H), generator=g, device=DEV)
    L = m.LayerWeights(H=H, I=I, E=E, k=K, wdtype="bf16", Wr=Wr, **m.pack_layer_tensors({"W_gu": W_gu, "W_d": W_d}, "bf16"))
    x = rnd(100, H)
    parts = [m.verify_layer(x[a:a + 20].float(), L) for a in range(0, 100, 20)]
    idx, w = m.route_tokens(torch.cat([p[1].logits.view(20, E) for p in parts]), K)
    assert torch.equal(idx.flatten(), torch.cat([p[1].topk_idx.flatten() for p in parts]))
    # the verify layer takes activations and hidden activations as bf16 above 8 tokens
    close(m.experts(x, L, idx, w), torch.cat([p[0] for p in parts]), 2.0 ** -7)

    # two answers to the second prompt; each decodes rows of its own
    pairs, ok = m.kv4_fork(refs, table, page, i32(0, 0), i32(1, 2), i32(170, 170))
    assert ok.tolist() == [1, 1] and (pairs[:, 0] == table[0, 10]).all()
    m.kv4_copy_pages(cache, pairs)
    assert m.kv4_reserve(refs, table, page, i32(1, 2), i32(175, 175)).tolist() == [1, 1]
    q3, k3, v3 = rnd(10, Hq, D), rnd(10, Hkv, D), rnd(10, Hkv, D)
    forks = table[1:3].contiguous()
    sk3, sv3 = m.kv4_append(cache, k3, v3, forks, i32(170, 170), [0, 5, 10], return_stored=True)
    fk, fv = torch.cat([ak, sk3[:5], ak, sk3[5:]]), torch.cat([av, sv3[:5], av, sv3[5:]])
    ref = attention(q3, fk, fv, [0, 5, 10], [0, 175, 350])
    before = m.kv4_attend(cache, q3, forks, i32(170, 170), [0, 5, 10])
    close(before, ref, tol)
    close(m.prompt_attend(q3, fk, fv, [0, 5, 10], [0, 175, 350]), ref, tol)

    # the others end; what is left moves to the pool's front and reads the same
    m.kv4_release(refs, table, page, i32(0, 3), i32(0, 0))
    moves = m.kv4_compact(refs, table)
    m.kv4_copy_pages(cache, moves)
    used = int((refs > 0).sum())
    assert used == 10 + 2 and (refs[:used] > 0).all() and int(table.max()) == used - 1
    after = m.kv4_attend(cache, q3, table[1:3].contiguous(), i32(170, 170), [0, 5, 10])
    assert torch.equal(after, before)
    m.kv4_release(refs, table, page, i32(1, 2), i32(0, 0))
    assert (refs == 0).all() and (table == -1).all()
