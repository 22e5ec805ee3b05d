"""The serving operators together with the verify layer, as a decoding loop
uses them: append the drafts' K/V, attend with the tree mask, run the MoE
verify layer, accept, commit the accepted rows.  With temperature 0 the loop
has to give the tokens of plain decoding (one token a step, no drafts), and
its cache the bytes of that decoding's cache."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import moe_speculative_decoding_router_amd as m  # noqa: E402

DEV = torch.device("cuda:0")
H, HQ, HKV, D, V, PAGE = 256, 8, 2, 64, 997, 16


class Model:
    def __init__(self, seed):
        g = torch.Generator(device=DEV).manual_seed(seed)
        r = lambda *s: torch.randn(s, generator=g, device=DEV)  # noqa: E731
        self.emb, self.out = r(V, H), r(H, V) / 4
        self.qkv, self.o = r(H, (HQ + 2 * HKV) * D) / 16, r(HQ * D, H) / 16
        E, inter = 16, 128
        self.layer = m.LayerWeights(H=H, I=inter, E=E, k=4, wdtype="f32", Wr=r(E, H) / 16, W_gu=r(E, 2 * inter, H) / 16,
                                    W_d=r(E, H, inter) / 11)

    def step(self, cache, tokens, table, lengths, offsets, parent):
        """Logits of the call's tokens; their K/V rows are in the cache afterwards."""
        x = self.emb[tokens.long()]
        p = x @ self.qkv
        T = len(tokens)
        q, k, v = (p[:, a * D:b * D].view(T, b - a, D) for a, b in ((0, HQ), (HQ, HQ + HKV), (HQ + HKV, HQ + 2 * HKV)))
        m.kv4_append(cache, k, v, table, lengths, offsets)
        a = m.kv4_attend(cache, q, table, lengths, offsets, parent=parent)
        x = x + a.reshape(T, HQ * D) @ self.o
        y, _ = m.verify_layer(x, self.layer)
        return (x + y) @ self.out, k, v


def greedy(n):
    return torch.zeros(n, device=DEV)


def tables(nseq, pages):
    return torch.arange(nseq * pages, dtype=torch.int32, device=DEV).flip(0).view(nseq, pages).contiguous()


def test_speculative_loop_equals_plain_decoding():
    mod, S, steps = Model(1), 3, 40
    prompts = [[5, 9, 200, 31], [7], [900, 13, 44, 44, 8, 1, 2]]
    pages = 8
    table = tables(S, pages)

    def start():
        c = m.kv4_cache(S * pages, PAGE, HKV, D, device=DEV)
        c.data.fill_(0xFF)
        off = np.cumsum([0] + [len(p) for p in prompts]).tolist()
        logits, _, _ = mod.step(c, torch.tensor(sum(prompts, []), dtype=torch.int32, device=DEV), table,
                                torch.zeros(S, dtype=torch.int32, device=DEV), off, None)
        lens = torch.tensor([len(p) for p in prompts], dtype=torch.int32, device=DEV)
        last = logits[[o - 1 for o in off[1:]]]
        tok = m.sample_tokens(last.contiguous(), greedy(S), temperature=greedy(S))[0]
        assert torch.equal(tok.long(), last.argmax(1))
        return c, lens, tok

    # plain decoding
    c0, lens, tok = start()
    plain = [[int(t)] for t in tok]
    for _ in range(steps + 8):
        logits, _, _ = mod.step(c0, tok, table, lens, list(range(S + 1)), None)
        lens = lens + 1
        tok = m.sample_tokens(logits, greedy(S), temperature=greedy(S))[0]
        for s in range(S):
            plain[s].append(int(tok[s]))

    # speculative decoding with trees of drafts: node 1 and 2 under the root, 3 and 4 under 1, 5 under 2
    rng = np.random.default_rng(2)
    c1, lens, tok = start()
    spec = [[int(t)] for t in tok]
    tree, gains = [-1, 0, 0, 1, 1, 2], []
    while min(len(x) for x in spec) < steps:
        tokens, parent, offsets = [], [], [0]
        for s in range(S):
            n = int(rng.integers(1, 7))
            a = len(spec[s])                       # the right continuations, or others, in either place
            good = plain[s][a:a + 2]
            d1, d2 = (good[0], (good[0] + 1) % V) if rng.random() < 0.6 else ((good[0] + 3) % V, good[0])
            node = [spec[s][-1], d1, d2, (good[1] + 5) % V, good[1], good[1] if rng.random() < 0.7 else 0]
            tokens += node[:n]
            parent += tree[:n]
            offsets.append(offsets[-1] + n)
        T = offsets[-1]
        td = torch.tensor(tokens, dtype=torch.int32, device=DEV)
        logits, k, v = mod.step(c1, td, table, lens, offsets, parent)
        out, path, count = m.accept_drafts(logits, td, offsets, greedy(T), parent=parent, temperature=greedy(T))
        m.kv4_append(c1, k, v, table, lens, offsets, path=path, count=count)
        lens = lens + count
        gains += count.tolist()
        for s in range(S):
            spec[s] += out[offsets[s]:offsets[s] + int(count[s])].tolist()
    for s in range(S):
        assert spec[s][:steps] == plain[s][:steps], s
    assert max(gains) == 3 and min(gains) == 1
    # the committed rows are the plain decoding's, byte for byte
    for s in range(S):
        n = int(lens[s]) // 16 * 16
        for t in range(n // 16):
            pid = int(table[s, t * 16 // PAGE])
            assert torch.equal(c0.data[pid], c1.data[pid]), (s, t)


def test_drafting_and_acceptance_by_ratio():
    """Drafts sampled from a drafter's distributions, accepted against the
    target's: with the drafter equal to the target everything is accepted,
    with a drafter of other tokens nothing is."""
    mod = Model(3)
    g = torch.Generator(device=DEV).manual_seed(4)
    logits = torch.randn((5, V), generator=g, device=DEV) * 3
    u = torch.rand(5, generator=g, device=DEV)
    uf = torch.rand(1, generator=g, device=DEV)
    temp = torch.full((5,), 0.8, device=DEV)
    topk = torch.full((5,), 50, dtype=torch.int32, device=DEV)
    drawn, prob, q = m.sample_tokens(logits, u, temperature=temp, top_k=topk, return_probs=True)
    assert torch.equal(prob, q.gather(1, drawn.long()[:, None])[:, 0])
    tokens = torch.cat([drawn[:1], drawn[:4]])
    out, path, count = m.accept_drafts(logits, tokens, [0, 5], u, draft_probs=q, u_final=uf, temperature=temp, top_k=topk)
    assert int(count) == 5 and torch.equal(out[:4], drawn[:4])
    low = logits.argsort(1)[:, :1].to(torch.int32)[:, 0]     # outside the target's top 50
    q2 = torch.zeros_like(q).scatter_(1, low.long()[:, None], 1.0)
    out, path, count = m.accept_drafts(logits, torch.cat([low[:1], low[:4]]), [0, 5], u, draft_probs=q2, u_final=uf,
                                       temperature=temp, top_k=topk)
    assert int(count) == 1 and out[1:].tolist() == [-1] * 4
    del mod
