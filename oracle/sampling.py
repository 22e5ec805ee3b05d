"""Oracle for drawing and accepting draft tokens (test infrastructure only),
in float64 from the definitions in include/moe_verify.h.

The speculative step that the pages describe ([EcoSpec] section 1, [S2-MoE]
motivation) draws drafts from a drafter and keeps those that the target
accepts; the pages give no formulas.  Readings:
  R30  a chain of sampled drafts is accepted by the ratio of the two
       distributions (accept x with probability min(1, p(x) / q(x)), else
       draw from max(p - q, 0)), which leaves the target's distribution
       unchanged;
  R31  a tree (several candidates a node, chosen, not sampled) is matched
       against the target's own draw after each node, which leaves it
       unchanged for any tree.
"""
from __future__ import annotations

import numpy as np

FLT_MAX = float(np.finfo(np.float32).max)


def kept_weights(logits, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """One row: float64 weights relative to the first of the ranking, 0 where
    a filter drops the token; and the number kept."""
    x = np.asarray(logits, dtype=np.float64).copy()
    x[np.isnan(x)] = -np.inf
    x = np.minimum(x, FLT_MAX)
    order = np.lexsort((np.arange(len(x)), -x))
    order = order[x[order] > -np.inf]
    w = np.zeros(len(x))
    if len(order) == 0:
        return w, 0
    if not temperature > 0:
        w[order[0]] = 1.0
        return w, 1
    r = np.exp((x[order] - x[order[0]]) / float(temperature))
    n = len(order)
    if top_k > 0:
        n = min(n, int(top_k))
    if top_p < 1:
        mass = np.cumsum(r[:n])
        n = min(n, int(np.searchsorted(mass, top_p * mass[-1])) + 1) if top_p > 0 else 1
    if min_p > 0:
        n = min(n, int((r >= min_p).sum()))
    n = max(n, 1)
    w[order[:n]] = r[:n]
    return w, n


def draw(w, u):
    """Lowest index whose running weight exceeds u * total; -1 without weight."""
    c = np.cumsum(w)
    if c[-1] == 0:
        return -1
    return int(min(np.searchsorted(c, u * c[-1], side="right"), np.nonzero(w)[0][-1]))


def margin(w, u):
    """Distance of u * total to the nearest step of the running weight, over the total."""
    c = np.cumsum(w)
    return float(np.abs(c / c[-1] - u).min()) if c[-1] else 1.0


def accept_match(drawn, tokens, parent):
    """One sequence: drawn[j] the target's draw after row j; parent[0] = -1.
    Returns (gained tokens, path)."""
    cur, out, path = 0, [], []
    while True:
        path.append(cur)
        out.append(int(drawn[cur]))
        nxt = [j for j in range(cur + 1, len(tokens)) if parent[j] == cur and tokens[j] == drawn[cur] and drawn[cur] >= 0]
        if not nxt:
            return out, path
        cur = nxt[0]


def accept_chain(p, q, tokens, u, u_final):
    """One sequence: p [n, V] the target's distributions, q [n, V] the
    drafter's (values below 0 count as 0), tokens [n], u [n].  Returns (gained
    tokens, path)."""
    q = np.where(q < 0, 0.0, q)
    n = len(tokens)
    j = 0
    while j + 1 < n:
        x = int(tokens[j + 1])
        if not 0 <= x < p.shape[1] or not u[j] * q[j, x] < p[j, x]:
            break
        j += 1
    w = p[j]
    if j + 1 < n:
        rest = np.maximum(p[j] - q[j], 0.0)
        if rest.sum() > 0:
            w = rest
    return [int(t) for t in tokens[1:j + 1]] + [draw(w, u_final)], list(range(j + 1))
