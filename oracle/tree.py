"""Trees of drafted tokens and the pages of a cache in plain NumPy (test
infrastructure only, written from the formulas of include/mk.h)."""
from __future__ import annotations

from fractions import Fraction

import numpy as np


def ancestors(parents):
    """For each token the sorted list of itself and its ancestors."""
    paths = []
    for i, p in enumerate(parents):
        paths.append((paths[p] if 0 <= p < i else []) + [i])
    return paths


def paged_tree(parents, cu, kv, words, rows, masks, positions):
    """mk_paged_tree over copies of masks [rows, words] (uint32) and positions."""
    masks, positions = masks.copy(), positions.copy()
    bad = False
    for r in range(len(kv)):
        a, b = int(cu[r]), int(cu[r + 1])
        if a < 0 or b < a or b > rows or a < max(cu[:r + 1]):
            bad = True
            continue
        k, here = b - a, kv[r] >= b - a
        if k > 32 * words:
            positions[a:b] = [kv[r] - k + i if here else 0 for i in range(k)]
            continue
        bad |= any(not -1 <= p < i for i, p in enumerate(parents[a:b]))
        for i, path in enumerate(ancestors([int(p) for p in parents[a:b]])):
            masks[a + i] = 0
            for j in path:
                masks[a + i, j // 32] |= np.uint32(1 << j % 32)
            positions[a + i] = kv[r] - k + len(path) - 1 if here else 0
    end = min(max(int(max(cu)), 0), rows)
    positions[end:] = 0
    return masks, positions, bad


def tree_seen(mask, new, kv, window):
    """[new, kv] truth values: which keys each row of a request sees; mask [new, words]
    (uint32), or None for a chunk of a prompt."""
    ctx = kv - new
    seen = np.zeros((new, max(kv, 0)), bool)
    for i in range(new):
        bits = [j for j in range(i + 1) if mask is None or int(mask[i, j // 32]) >> (j % 32) & 1]
        p = ctx + max(len(bits), 1) - 1
        if window:
            bits = bits[-window:]
        for j in range(max(0, p - window + 1) if window else 0, ctx):
            seen[i, j] = True
        for j in bits:
            if 0 <= ctx + j < kv:
                seen[i, ctx + j] = True
    return seen


def tree_attention(q, k_cache, v_cache, table, cu_new, kv_lens, masks, scale, window=0):
    """As oracle.paged_attention, with masks [rows, words] (uint32)."""
    rows, hq, d = q.shape
    pages, hkv, page, _ = k_cache.shape
    out, lse = np.zeros((rows, hq, d)), np.full((rows, hq), -np.inf)
    wabs, smag, vmax = np.zeros((rows, hq, d)), np.zeros((rows, hq)), np.zeros((rows, hq))
    words = masks.shape[1]
    for r in range(len(kv_lens)):
        a, b, kv = int(cu_new[r]), int(cu_new[r + 1]), int(kv_lens[r])
        if b <= a or kv <= 0:
            continue
        seen = tree_seen(masks[a:b] if b - a <= 32 * words else None, b - a, kv, window)
        key = np.flatnonzero(seen.any(0))
        if not len(key):
            continue
        seen = seen[:, key]
        ids = table[r][key // page]
        ok = (ids >= 0) & (ids < pages)
        some = seen.any(1)
        for h in range(hkv):
            k = np.where(ok[:, None], k_cache[np.where(ok, ids, 0), h, key % page], 0.0)
            v = np.where(ok[:, None], v_cache[np.where(ok, ids, 0), h, key % page], 0.0)
            for g in range(h * (hq // hkv), (h + 1) * (hq // hkv)):
                s = np.where(seen, q[a:b, g] @ k.T * scale, -np.inf)
                m = np.where(some, s.max(1), 0.0)[:, None]
                e = np.exp(s - m)
                t = np.where(some, e.sum(1), 1.0)
                e = e / t[:, None]
                out[a:b, g] = e @ v
                lse[a:b, g] = np.where(some, m[:, 0] + np.log(t), -np.inf)
                wabs[a:b, g] = e @ np.abs(v)
                smag[a:b, g] = np.where(seen, np.abs(q[a:b, g]) @ np.abs(k).T * abs(scale), 0).max(1)
                vmax[a:b, g] = np.where(some, np.abs(v).max(), 0.0)
    return out, lse, wabs, smag, vmax


def _probability(x):
    x = float(x)
    return Fraction(0) if not x > 0 else Fraction(min(x, 1.0))


def _uniform(x):
    x = float(x)
    return Fraction(0) if not x > 0 else Fraction(min(x, 1.0 - 2.0 ** -24))


def tree_verify(parents, tokens, p, q, u, u_last):
    """One request's tree in exact fractions: (path, emitted, bad); q None: tokens
    that were found."""
    k, vocab = len(parents), p.shape[1]
    bad = any(not -1 <= x < i for i, x in enumerate(parents) if i) or any(not 0 <= x < vocab for x in tokens[1:])
    row = lambda m, c: [_probability(x) for x in m[c]]  # noqa: E731
    cur, path, emitted = 0, [0], []
    left, z = row(p, 0), Fraction(1)
    draft = row(q, 0) if q is not None else None
    for i in range(1, k):
        if parents[i] != cur or not parents[i] < i:
            continue
        x = int(tokens[i])
        inside = 0 <= x < vocab
        mine = left[x] if inside else Fraction(0)
        if q is not None:
            stands = _uniform(u[i]) * (draft[x] if inside else 0) * z < mine
        else:
            stands = inside and _uniform(u[i]) * z < mine
        if stands:
            cur = i
            path.append(i)
            emitted.append(x)
            left, z = row(p, i), Fraction(1)
            draft = row(q, i) if q is not None else None
        elif q is not None:
            left = [max(a - z * b, Fraction(0)) for a, b in zip(left, draft)]
            z = sum(left)
        elif inside:
            z = max(z - left[x], Fraction(0))
            left[x] = Fraction(0)
    if sum(left) == 0:
        left = row(p, cur)
    total, want, last = sum(left), _uniform(u_last), 0
    if total == 0:
        bad = True
    else:
        run = Fraction(0)
        for last, a in enumerate(left):
            run += a
            if run > want * total:
                break
    return path, emitted + [last], bad


def paged_fork(table, lens, keep, parents, next_table, page, shared, free, n_free, copying=True):
    """mk_paged_fork over copies of next_table, shared and free; parents None: in
    place.  Returns a dict, with `bad` telling whether anything was refused."""
    table, shared, free = np.array(table, np.int64), np.array(shared, np.int64), np.array(free, np.int64)
    n, width = table.shape
    in_place = parents is None
    nxt = table.copy() if in_place else np.array(next_table, np.int64)
    up = list(range(n)) if in_place else [int(p) for p in parents]
    cap = len(free)
    bad = not 0 <= n_free <= cap
    n_free = min(max(n_free, 0), cap)
    bad |= any(not -1 <= p < n for p in up)
    up = [p if 0 <= p < n else -1 for p in up]
    held, kept = [], []
    for s in range(n):
        l = min(max(int(lens[s]), 0), width * page)
        k = l if keep is None else min(max(int(keep[s]), 0), l)
        bad |= l != lens[s] or (keep is not None and k != keep[s])
        held.append(-(-l // page))
        kept.append(k)
    is_page = lambda x: 0 <= x < len(shared)  # noqa: E731
    before = shared.copy()
    children = [up.count(s) for s in range(n)]
    own = []
    for s in range(n):
        f = kept[s] // page
        own.append(kept[s] % page > 0 and children[s] > 0 and (not is_page(table[s, f]) or before[table[s, f]] == 0))
    lets = []  # entries that let a page go, in order
    for s in range(n):
        f = kept[s] // page
        for b in range(held[s]):
            x = table[s, b]
            change = children[s] - 1 if b < f else 0 if b == f and own[s] else -1
            if not is_page(x):
                bad |= children[s] != 1 or b >= f + own[s]
                continue
            shared[x] += change
            if change < 0:
                lets.append(x)
    copies = np.tile(np.array([[-1], [-1], [0]]), (1, len(up)))
    next_lens, taken, wanted = np.zeros(len(up), np.int64), 0, 0
    for i, s in enumerate(up):
        if s < 0:
            continue
        f, part = kept[s] // page, kept[s] % page > 0
        next_lens[i] = kept[s]
        if not in_place:
            nxt[i, :f] = table[s, :f]
        if part and own[s] and up.index(s) == i:
            nxt[i, f] = table[s, f]
        elif part:
            wanted += 1
            if copying and wanted <= n_free:
                fresh = free[n_free - wanted]
                copies[:, i] = table[s, f], fresh, kept[s] % page
                nxt[i, f] = fresh
                taken += 1
            else:
                bad = True
                next_lens[i] = f * page
    gone = []
    for x in lets:
        if shared[x] < 0 and x not in gone:
            bad |= shared[x] < -1
            gone.append(x)
    shared[gone] = 0
    left = n_free - taken
    bad |= left + len(gone) > cap
    gone = gone[:max(0, cap - left)]
    free[left:left + len(gone)] = gone
    return {"table": nxt, "lens": next_lens, "copies": copies, "shared": shared, "free": free, "n_left": left + len(gone), "bad": bool(bad)}
