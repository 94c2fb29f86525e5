"""A pool's pages in plain Python, apart from the library: rows one after the other, by
the definition in include/hk_gemm.h."""
from __future__ import annotations


def slots(tokens, page):
    return -(-tokens // page)


def arrange(refs, table, held, keep, room, parents, page):
    """(refs, table, held, copies, missing) after the call; copies: row -> (page, its copy)."""
    R, M, P = len(table), len(table[0]), len(refs)
    parents = list(range(R)) if parents is None else parents
    bad = False
    for i in range(R):
        p = parents[i]
        if not 0 <= p < R or not 0 <= held[i] <= M * page or not 0 <= held[p] <= M * page:
            bad = True
        elif not 0 <= keep[i] <= held[p] or not keep[i] <= room[i] <= M * page:
            bad = True
        else:
            used = table[p][: slots(room[i], page)][: slots(held[p], page)] if p != i else []
            own = table[i][(keep[i] // page if p == i else 0): slots(held[i], page)]
            bad = bad or any(not 0 <= e < P for e in used + own)
    if bad:
        return refs, table, held, {}, -1
    new_refs, new_table, copies = list(refs), [list(r) for r in table], {}
    free = [p for p in range(P) if refs[p] == 0]
    taken = 0
    for i in range(R):
        p = parents[i]
        heir = p if parents[p] == p else parents.index(p)
        for s in range(slots(room[i], page)):
            theirs = table[p][s] if s < slots(held[p], page) else None
            if (s + 1) * page <= keep[i]:
                now = theirs
            elif theirs is not None and heir == i and refs[theirs] == 1 and not any(
                    parents[j] == p and j != i and keep[j] >= (s + 1) * page for j in range(R)):
                now = theirs
            else:
                now = free[taken] if taken < len(free) else None
                taken += 1
                if s * page < keep[i]:
                    copies[i] = (theirs, now)
            new_table[i][s] = now
            if now is not None:
                new_refs[now] += 1
        for s in range(slots(held[i], page)):
            new_refs[table[i][s]] -= 1
    if taken > len(free):
        return refs, table, held, {}, taken - len(free)
    return new_refs, new_table, list(room), copies, 0


def compact(refs, table, held, page):
    """(refs, table, moved)"""
    used = sum(n > 0 for n in refs)
    goes = dict(zip([p for p in range(used, len(refs)) if refs[p] > 0], [p for p in range(used) if refs[p] == 0]))
    refs, table = list(refs), [list(r) for r in table]
    moved = [goes.get(p, p) if n > 0 else -1 for p, n in enumerate(refs)]
    for a, b in goes.items():
        refs[b], refs[a] = refs[a], 0
    for row, h in zip(table, held):
        for s in range(slots(h, page)):
            row[s] = goes.get(row[s], row[s])
    return refs, table, moved


def counted(table, held, pages, page):
    """The references that the tables hold."""
    n = [0] * pages
    for row, h in zip(table, held):
        for s in range(slots(h, page)):
            n[row[s]] += 1
    return n


def random_call(rng, held, page, max_pages, tokens=None):
    """keep, room, parents of a call such as a server makes: some rows grow, end, are cut back, forked or reordered."""
    R = len(held)
    parents = list(range(R))
    kind = rng.choice(("grow", "fork", "beams", "end", "mixed"))
    if kind in ("beams", "mixed"):
        parents = [rng.randrange(R) if rng.random() < 0.7 else i for i in range(R)]
    elif kind == "fork":
        p = rng.randrange(R)
        parents = [p if held[i] == 0 or rng.random() < 0.3 else i for i in range(R)]
    keep, room = [], []
    for i in range(R):
        h = held[parents[i]]
        k = h if rng.random() < 0.7 else rng.randint(0, h)
        if kind == "end" and rng.random() < 0.5:
            k = 0
        keep.append(k)
        more = 0 if kind == "end" else rng.choice((0, 1, 1, 5, rng.randint(0, 3 * page)))
        room.append(min(k + more, max_pages * page))
    return keep, room, parents if rng.random() < 0.8 or parents != list(range(R)) else None
