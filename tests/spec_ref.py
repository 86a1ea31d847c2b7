"""Plain references in 64 bits of the speculative decoding and paged cache operators: one sequence, one row, one
entry after the other (numpy)."""

from __future__ import annotations

import numpy as np

LEAST = 2.0 ** -40


def softmax(row):
    """None for a row without a distribution."""
    row = np.asarray(row, np.float64)
    if row.size == 0 or np.isnan(row).any() or row.max() == np.inf or row.max() == -np.inf:
        return None
    e = np.exp(row - row.max())
    return e / e.sum()


def draw(weights, u):
    """(token, how far u is from another outcome)."""
    upto = np.cumsum(weights)
    at = float(u) * upto[-1]
    above = np.nonzero((upto > at) & (weights > 0))[0]
    token = int(above[0]) if above.size else int(np.nonzero(weights > 0)[0][-1])
    edges = np.unique(upto)
    edges = edges[:-1] if edges.size > 1 else edges  # the end is no border for u < 1
    return token, float(np.abs(edges - at).min() / upto[-1])


def verify(x, drafts, uniforms=None, y=None, parents=None, lengths=None):
    """x [N, D + 1, V] and y [N, D, V] float64. (tokens, accepted, path, margin [N]: how far the closest decision is
    from its border, relative)."""
    N, D = drafts.shape
    V = x.shape[2]
    tokens, accepted = np.full((N, D + 1), -1, np.int32), np.zeros(N, np.int32)
    path, margin = np.full((N, D), -1, np.int32), np.full(N, np.inf)
    for i in range(N):
        n = D if lengths is None else min(max(int(lengths[i]), 0), D)
        parent = np.arange(D) - 1 if parents is None else parents[i]
        there = [j for j in range(n) if 0 <= drafts[i, j] < V and -1 <= parent[j] < j]
        at, taken, final = -1, [], -1
        while True:
            kids = [j for j in there if parent[j] == at]
            p = softmax(x[i, at + 1])
            if p is None:
                break
            if uniforms is None:
                top = int(np.argmax(np.asarray(x[i, at + 1], np.float64) + 0.0))
                go = next((j for j in kids if drafts[i, j] == top), None)
                if go is None:
                    final = top
                    break
            else:
                u, go, r = float(uniforms[i, at + 1]), None, p
                if y is not None and kids:
                    q, d = softmax(y[i, at + 1]), drafts[i, at + 1]
                    q = np.zeros(V) if q is None else q
                    a, b = u * q[d], p[d]
                    if a != b:
                        margin[i] = min(margin[i], abs(a - b) / max(a, b))
                    if a < b:
                        go = kids[0]
                    else:
                        r = np.maximum(p - q, 0.0)
                elif kids:
                    r, low, seen = p.copy(), 0.0, set()
                    for j in kids:
                        d = int(drafts[i, j])
                        if d in seen:
                            continue
                        seen.add(d)
                        high = low + p[d]
                        if u > 0 or high > 0:
                            margin[i] = min(margin[i], abs(u - high) / max(u, high))
                        if go is None and low <= u < high:
                            go = j
                        low, r[d] = high, 0.0
                if go is None:
                    final, m = draw(r if r.sum() > LEAST else p, uniforms[i, D])
                    margin[i] = min(margin[i], m)
                    break
            taken.append(go)
            at = go
        accepted[i] = len(taken)
        tokens[i, :len(taken)] = drafts[i, taken]
        tokens[i, len(taken)] = final
        path[i, :len(taken)] = taken
    return tokens, accepted, path, margin


def pages(length, S):
    return -(-int(length) // S)


def fork(tables, lengths, parents, uses, S):
    N, K = parents.shape
    beam = np.arange(K)
    parent = np.where((parents >= 0) & (parents < K), parents, beam)
    source = (parent + K * np.arange(N)[:, None]).reshape(-1)
    old_tables, old_lengths = tables.copy(), lengths.copy()
    for r in range(N * K):
        for c in range(pages(old_lengths[r], S)):
            if 0 <= old_tables[r, c] < len(uses):
                uses[old_tables[r, c]] -= 1
    for r in range(N * K):
        held, came = pages(old_lengths[r], S), pages(old_lengths[source[r]], S)
        if source[r] != r:
            tables[r, :held] = -1
            tables[r, :came] = old_tables[source[r], :came]
        lengths[r] = old_lengths[source[r]]
        for c in range(came):
            if 0 <= tables[r, c] < len(uses):
                uses[tables[r, c]] += 1


def resize(tables, lengths, new, uses, S, caches=None):
    """caches: arrays [P, S, ...]."""
    C, P = tables.shape[1], len(uses)
    old = lengths.copy()
    ok = [0 <= old[r] <= C * S and 0 <= new[r] <= C * S for r in range(len(old))]
    for r in range(len(old)):
        if ok[r] and new[r] < old[r]:
            for c in range(pages(new[r], S), pages(old[r], S)):
                if 0 <= tables[r, c] < P:
                    uses[tables[r, c]] -= 1
                tables[r, c] = -1
            lengths[r] = new[r]
    free = [p for p in range(P) if uses[p] == 0]
    # who writes into which page, and whether others use it that do not
    growers = [r for r in range(len(old)) if ok[r] and new[r] > old[r]]
    tail = {r: int(tables[r, pages(old[r], S) - 1]) for r in growers if old[r] % S}
    tail = {r: t for r, t in tail.items() if 0 <= t < P}
    left = uses.copy()
    for t in tail.values():
        left[t] -= 1
    for r in growers:
        t = tail.get(r)
        keeps = t is not None and left[t] <= 0 and r == max(q for q in tail if tail[q] == t)
        copies = t is not None and not keeps
        need = pages(new[r], S) - pages(old[r], S) + copies
        if need > len(free) or (copies and caches is None):
            break
        if copies:
            page = free.pop(0)
            uses[t] -= 1
            uses[page] = 1
            tables[r, pages(old[r], S) - 1] = page
            for c in caches:
                c[page, :old[r] % S] = c[t, :old[r] % S]
        for c in range(pages(old[r], S), pages(new[r], S)):
            page = free.pop(0)
            uses[page] = 1
            tables[r, c] = page
        lengths[r] = new[r]


def compact(caches, tables, starts, path, counts):
    """caches: arrays [P, S, ...]."""
    N, D = path.shape
    P, S = caches[0].shape[:2]
    for i in range(N):
        before = -1
        for j in range(min(max(int(counts[i]), 0), D)):
            at, start = int(path[i, j]), int(starts[i])
            if at <= before or start < 0 or start + at >= tables.shape[1] * S:
                break
            before = at
            f, t = start + at, start + j
            a, b = tables[i, f // S], tables[i, t // S]
            if 0 <= a < P and 0 <= b < P:
                for c in caches:
                    c[b, t % S] = c[a, f % S]
