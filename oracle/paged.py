"""Plain definitions of the paged-cache, shared-prefix attention and sampling
calls (numpy fp64 and Python loops) -- TEST INFRASTRUCTURE ONLY, as the rest of
this package.  include/dflv.h states what each computes."""
from __future__ import annotations

import math

import numpy as np

DEV_TOPOLOGY, DEV_CAPACITY, DEV_PATH, DEV_PAGE, DEV_SAMPLE = 1, 2, 4, 16, 32


def tables_grow(n_past, n_new, n_held, free_list, n_free, table, page, N_max):
    """Returns (n_held, n_free, table, slots, status).  The pool has as many pages
    as free_list has places."""
    B, width = table.shape
    n_held, table = n_held.copy(), table.copy()
    slots = np.full((B, N_max), -1, np.int32)
    status, asked, taken = 0, 0, 0
    for b in range(B):
        past, new, held = int(n_past[b]), int(n_new[b]), int(n_held[b])
        need = -(-(past + new) // page)
        if past < 0 or not 0 <= new <= N_max or not 0 <= held <= width or need > width:
            status |= DEV_CAPACITY
            continue
        more = max(0, need - held)
        asked += more
        if more and asked > n_free:
            status |= DEV_CAPACITY
            continue
        for t in range(held, held + more):
            table[b, t] = free_list[n_free - 1 - taken]
            if not 0 <= table[b, t] < len(free_list):
                status |= DEV_PAGE
            taken += 1
        n_held[b] = held + more
        for i in range(new):
            t = past + i
            if 0 <= table[b, t // page] < len(free_list):
                slots[b, i] = table[b, t // page] * page + t % page
            else:
                status |= DEV_PAGE
    return n_held, n_free - taken, table, slots, status


def tables_release(keep_len, n_held, free_list, n_free, table, page):
    """Returns (n_held, free_list, n_free, status)."""
    B, width = table.shape
    n_held, free_list = n_held.copy(), free_list.copy()
    status, back = 0, []
    for b in range(B):
        keep, held = -(-int(keep_len[b]) // page), int(n_held[b])
        if keep_len[b] < 0 or not 0 <= held <= width or keep > held:
            status |= DEV_CAPACITY
            continue
        back += [(b, t) for t in range(keep, held)]
    if n_free + len(back) > len(free_list):
        return n_held, free_list, n_free, status | DEV_CAPACITY
    for r, (b, t) in enumerate(back):
        free_list[n_free + len(back) - 1 - r] = table[b, t]
        n_held[b] -= 1
        if not 0 <= table[b, t] < len(free_list):
            status |= DEV_PAGE
    return n_held, free_list, n_free + len(back), status


def paged_append(slots, k_new, v_new, k, v):
    """In place; planes [n_pages][Hkv][page][D]."""
    page = k.shape[2]
    for b in range(slots.shape[0]):
        for i in range(slots.shape[1]):
            s = int(slots[b, i])
            if 0 <= s < k.shape[0] * page:
                k[s // page, :, s % page] = k_new[b, i]
                v[s // page, :, s % page] = v_new[b, i]


def paged_commit(slots, path, path_len, planes):
    for plane in planes:
        page = plane.shape[2]
        for b in range(slots.shape[0]):
            src = [int(slots[b, path[b, m]]) for m in range(int(path_len[b]))]
            rows = [plane[s // page, :, s % page].copy() for s in src]
            for m, r in enumerate(rows):
                t = int(slots[b, m])
                plane[t // page, :, t % page] = r


def prefix_attn(prefix_table, prefix_len, table, parent, n_nodes, n_past, q, k, v, scale):
    """q [B][N][Hq][D], planes [n_pages][Hkv][page][D], all fp64.  Returns the
    output and, for the tolerance, the weighted sum of |v|; NaN at padded rows."""
    B, N, Hq, D = q.shape
    Hkv, page = k.shape[1], k.shape[2]
    G = Hq // Hkv
    out = np.full(q.shape, np.nan)
    mag = np.full(q.shape, np.nan)

    def rows(plane, tab, n):
        t = np.arange(n)
        return plane[np.asarray(tab)[t // page], :, t % page]       # [n][Hkv][D]

    for b in range(B):
        n, past = int(n_nodes[b]), int(n_past[b])
        if n == 0:
            continue
        keys = np.concatenate([rows(k, prefix_table, prefix_len), rows(k, table[b], past + n)])
        vals = np.concatenate([rows(v, prefix_table, prefix_len), rows(v, table[b], past + n)])
        for i in range(n):
            seen = list(range(prefix_len + past))
            line, a = [], i
            while a >= 0:
                line.append(prefix_len + past + a)
                a = a - 1 if parent is None else int(parent[b, a])
            seen = np.array(seen + line[::-1])
            for h in range(Hq):
                s = keys[seen, h // G] @ q[b, i, h] * scale
                p = np.exp(s - s.max())
                p /= p.sum()
                out[b, i, h] = p @ vals[seen, h // G]
                mag[b, i, h] = p @ np.abs(vals[seen, h // G])
    return out, mag


def sample_row(x, T, top_k, top_p, min_p, u):
    """(token, logp, margin, status): margin is how far, relative to the mass
    it is taken of, the nearest decision (the draw, the top-p cut, the min-p
    cut) lies from going the other way."""
    x = np.asarray(x, np.float64)
    x = np.where(np.isnan(x), -np.inf, x)
    top = x.max()
    ok = (0 <= T < math.inf and top_p >= 0 and 0 <= min_p <= 1 and 0 <= u < 1 and top > -np.inf)
    if not ok or T == 0:
        return int(np.argmax(x)) if top > -np.inf else 0, 0.0, 1.0, 0 if ok else DEV_SAMPLE
    with np.errstate(invalid="ignore", over="ignore"):
        z = np.where(x == top, 0.0, np.where(np.isinf(x), -np.inf, (x - top)) / T)
        if np.isinf(top):
            z = np.where(x == top, 0.0, -np.inf)
    w = np.exp(z)
    order = np.argsort(-x, kind="stable")
    order = order[x[order] > -np.inf]
    if 0 < top_k < len(order):
        order = order[:top_k]
    margin = 1.0
    if top_p < 1:
        mass = w[order]
        before = np.concatenate([[0.0], np.cumsum(mass)[:-1]])
        cut = top_p * mass.sum()
        n = max(1, int((before < cut).sum()))
        margin = min(margin, float(np.abs(before[1:] - cut).min() / mass.sum()) if len(before) > 1 else 1.0)
        order = order[:n]
    kept = order[w[order] >= min_p]
    if min_p > 0:
        margin = min(margin, float(np.abs(w[order] - min_p)[w[order] < 1].min()) if (w[order] < 1).any() else 1.0)
    kept = np.sort(kept)
    run = np.cumsum(w[kept])
    at = u * run[-1]
    j = int((run <= at).sum())
    edges = run[:-1]
    if len(edges):
        margin = min(margin, float(np.abs(edges - at).min() / run[-1]))
    t = int(kept[min(j, len(kept) - 1)])
    return t, float(z[t] - math.log(run[-1])), margin, 0


def accept_walk(tokens, parent, n, drawn):
    """Path of the walk over already drawn tokens."""
    path = [0]
    while True:
        c = [i for i in range(1, n) if parent[i] == path[-1] and tokens[i] == drawn[path[-1]]]
        if not c:
            return path, int(drawn[path[-1]])
        path.append(c[0])
