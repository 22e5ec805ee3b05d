"""Oracle for the cache's pages (test infrastructure only): one sequence after
the other, in plain loops, from the definitions in include/moe_verify.h.
refs and table are lists (of lists) and changed in place."""
from __future__ import annotations


def _held(p, refs):
    return 0 <= p < len(refs)


def _free(refs):
    return [p for p, n in enumerate(refs) if n <= 0]


def reserve(refs, table, page, seq, rows):
    ok = []
    for i, (s, r) in enumerate(zip(seq, rows)):
        want = -(-max(r, 0) // page)
        if not 0 <= s < len(table) or s in seq[:i] or want > len(table[0]):
            ok.append(0)
            continue
        have = 0
        while have < want and _held(table[s][have], refs):
            have += 1
        if any(_held(p, refs) for p in table[s][have:want]):  # behind a gap
            ok.append(0)
            continue
        fresh = _free(refs)[:want - have]
        ok.append(int(len(fresh) == want - have))
        if ok[-1]:
            for j, p in enumerate(fresh):
                table[s][have + j] = p
                refs[p] = 1
    return ok


def fork(refs, table, page, src, dst, rows):
    n, width = len(src), len(table[0])
    valid = [0 <= src[i] < len(table) and 0 <= dst[i] < len(table) and dst[i] not in src and dst[i] not in dst[:i]
             and -(-max(rows[i], 0) // page) <= width
             and all(_held(p, refs) for p in table[src[i]][:-(-max(rows[i], 0) // page)]) for i in range(n)]
    for i in range(n):
        if valid[i]:
            release(refs, table, page, [dst[i]], [0])
    pairs, ok = [[-1, -1] for _ in range(n)], [0] * n
    part = [-1] * n
    for i in range(n):  # what is shared is counted before any page is taken
        if valid[i]:
            full = max(rows[i], 0) // page
            for j in range(full):
                table[dst[i]][j] = table[src[i]][j]
                refs[table[src[i]][j]] += 1
            if max(rows[i], 0) % page:
                part[i] = table[src[i]][full]
    empty = []
    for i in range(n):
        if not valid[i]:
            continue
        ok[i] = 1
        if part[i] >= 0:
            free = _free(refs)
            if free:
                p = free[0]
                refs[p] = 1
                table[dst[i]][max(rows[i], 0) // page] = p
                pairs[i] = [part[i], p]
            else:
                ok[i] = 0
                empty.append(dst[i])
    for s in empty:  # after the others were served
        release(refs, table, page, [s], [0])
    return pairs, ok


def release(refs, table, page, seq, keep):
    for s, k in zip(seq, keep):
        if 0 <= s < len(table):
            for j in range(-(-max(k, 0) // page), len(table[s])):
                if _held(table[s][j], refs):
                    refs[table[s][j]] -= 1
                table[s][j] = -1


def compact(refs, table, max_moves):
    pairs = []
    while len(pairs) < max_moves:
        free = [p for p in _free(refs)]
        used = [p for p, n in enumerate(refs) if n > 0]
        taken, left = {a for a, _ in pairs}, {b for _, b in pairs}
        free = [p for p in free if p not in taken]
        used = [p for p in used if p not in left]
        if not free or not used or free[0] > used[-1]:
            break
        to, frm = free[0], used[-1]
        refs[to], refs[frm] = refs[frm], 0
        for row in table:
            for j, p in enumerate(row):
                if p == frm:
                    row[j] = to
        pairs.append((frm, to))
    return pairs + [(-1, -1)] * (max_moves - len(pairs))
