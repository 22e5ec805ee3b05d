"""Oracle for the 4-bit K/V cache (test infrastructure only): quantisation,
page layout and tree attention in float64, from the definitions in
include/moe_verify.h.

[EcoSpec] = review of "Less Experts, Faster Decoding": the drafts verified in
one step form a tree and a token attends to its own path (tree-attention
verify mask).  [S2-MoE] component 3: draft writes to the K/V cache are
tentative; the accepted tokens' K/V is committed.
"""
from __future__ import annotations

import numpy as np

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def quantise(x):
    """x [..., D] -> (codes uint8 [..., D], scale bytes uint8 [..., D / 32],
    values float64 [..., D]).  NaN counts as 0."""
    x = np.asarray(x, dtype=np.float64)
    x = np.where(np.isnan(x), 0.0, x)
    b = x.reshape(*x.shape[:-1], -1, 32)
    amax = np.abs(b).max(-1)
    e = np.full(amax.shape, -100)
    for n in range(-100, 126):                       # the smallest n with amax <= 6 * 2^n
        e = np.where(amax > 6.0 * 2.0 ** n, min(n + 1, 125), e)
    y = b / 2.0 ** e[..., None]
    a = np.minimum(np.abs(y), 6.0)
    dist = np.abs(a[..., None] - E2M1)
    lo = dist.argmin(-1)                             # of two equally near codes the lower
    hi = np.minimum(lo + 1, 7)
    tie = (dist.min(-1) == np.abs(a - E2M1[hi])) & (hi != lo)
    code = np.where(tie & (lo % 2 == 1), hi, lo)     # ties to the even code
    val = np.where(y < 0, -1.0, 1.0) * E2M1[code] * 2.0 ** e[..., None]
    code = code + 8 * ((y < 0) & (code > 0))
    return code.reshape(x.shape).astype(np.uint8), (e + 127).astype(np.uint8), val.reshape(x.shape)


def _offsets(D):
    """Byte of each element and scale of a tile's row i: functions of (i, index)."""
    w = D // 32
    k = lambda i, d: i * (D // 2) + d // 2                                              # noqa: E731
    ks = lambda i, b: 8 * D + 16 * b + i                                                # noqa: E731
    v = lambda i, d: 17 * D // 2 + (64 * (i // 4) + 4 * (d // (2 * w)) + i % 4) * w + d % (2 * w) // 2  # noqa: E731
    vs = lambda i, b: 33 * D // 2 + 16 * b + i                                          # noqa: E731
    return k, ks, v, vs


def write_row(data, page_id, h, pos_in_page, krow, vrow):
    """Store one row of one head; data [num_pages, Hkv, page / 16, 17 D] uint8."""
    D = data.shape[-1] // 17
    tile, i = data[page_id, h, pos_in_page // 16], pos_in_page % 16
    ko, kso, vo, vso = _offsets(D)
    for row, at, sat in ((krow, ko, kso), (vrow, vo, vso)):
        code, sc, _ = quantise(row)
        for d in range(0, D, 2):
            assert at(i, d) == at(i, d + 1)
            tile[at(i, d)] = code[d] | (code[d + 1] << 4)
        for b in range(D // 32):
            tile[sat(i, b)] = sc[b]


def append(data, k, v, table, lengths, offsets, path=None, count=None):
    """data is updated in place; k, v [T, Hkv, D]."""
    num_pages, H, tiles, _ = data.shape
    page = tiles * 16
    for s in range(len(offsets) - 1):
        r0, n = offsets[s], offsets[s + 1] - offsets[s]
        rows = [(j, j) for j in range(n)] if path is None else [(int(path[r0 + i]), i) for i in range(min(n, int(count[s])))]
        for src, j in rows:
            if not 0 <= src < n:
                continue
            pos = max(int(lengths[s]), 0) + j
            if pos // page >= table.shape[1]:
                continue
            pid = int(table[s, pos // page])
            if not 0 <= pid < num_pages:
                continue
            for h in range(H):
                write_row(data, pid, h, pos % page, k[r0 + src, h], v[r0 + src, h])


def read_rows(data, page_ids, h, positions):
    """K and V float64 [len(positions), D] of one head; page_ids: the page of each position."""
    D = data.shape[-1] // 17
    page = data.shape[2] * 16
    ko, kso, vo, vso = _offsets(D)
    p = np.asarray(positions)
    t = data[page_ids, h, p % page // 16]
    i, r = (p % 16)[:, None], np.arange(len(p))[:, None]
    d = np.arange(D)[None]
    out = []
    for at, sat in ((ko, kso), (vo, vso)):
        code = (t[r, at(i, d)] >> (4 * (d % 2))) & 15
        sc = 2.0 ** (t[r, sat(i, d // 32)].astype(np.float64) - 127)
        out.append(np.where(code & 8, -1.0, 1.0) * E2M1[code & 7] * sc)
    return out


def attend(data, q, table, lengths, offsets, parent=None, scale=1.0):
    """Returns (out float64 [T, Hq, D], bound float64 [T, Hq, D], reach): bound
    is sum_p p |v|, reach the largest sum_d |q_d K_d| * scale of a visible
    row, both for the tests' error bounds."""
    num_pages, H, tiles, _ = data.shape
    page = tiles * 16
    T, Hq, D = q.shape
    G = Hq // H
    out, bound = np.zeros((T, Hq, D)), np.zeros((T, Hq, D))
    reach = 0.0
    for s in range(len(offsets) - 1):
        r0, n = offsets[s], offsets[s + 1] - offsets[s]
        if n == 0:
            continue
        ln = min(max(int(lengths[s]), 0), table.shape[1] * page)
        pos = np.arange(min(ln + n, table.shape[1] * page))
        pid = table[s][pos // page]
        there = (pid >= 0) & (pid < num_pages)
        sees = []
        for j in range(n):
            p = (j - 1) if parent is None else int(parent[r0 + j])
            sees.append({j} | (sees[p] if p >= 0 else set()))
        for h in range(H):
            k, v = read_rows(data, np.where(there, pid, 0), h, pos)
            for j in range(n):
                vis = there & ((pos < ln) | np.isin(pos - ln, list(sees[j])))
                if not vis.any():
                    continue
                for g in range(G):
                    x = q[r0 + j, h * G + g].astype(np.float64)
                    a = (k[vis] @ x) * scale
                    reach = max(reach, float((np.abs(k[vis]) @ np.abs(x)).max() * abs(scale)))
                    w = np.exp(a - a.max())
                    w /= w.sum()
                    out[r0 + j, h * G + g] = w @ v[vis]
                    bound[r0 + j, h * G + g] = w @ np.abs(v[vis])
    return out, bound, reach
