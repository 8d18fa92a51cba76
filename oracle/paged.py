"""Paged KV cache operators in plain NumPy, float64: a step's tables, the
append's norm and rotary positions, and attention over pages (test
infrastructure only, written from the formulas of include/mk.h)."""
from __future__ import annotations

import numpy as np


def paged_tables(ctx, new, free_pages, n_free, table, page, max_tokens):
    """The tables of mk_paged_tables; returns a dict, with `refused` telling
    whether any request was refused."""
    n, width = table.shape
    table = table.copy()
    cu, kv = np.zeros(n + 1, np.int64), np.zeros(n, np.int64)
    pos, slot = np.zeros(max_tokens, np.int64), np.full(max_tokens, -1, np.int64)
    rows = asked = taken = 0
    refused = False
    for r in range(n):
        c, a = int(ctx[r]), int(new[r])
        if c < 0 or a < 0 or c + a > width * page:
            refused = True
            cu[r + 1] = cu[r]
            continue
        held, need = -(-c // page), -(-(c + a) // page) - -(-c // page)
        first, rows, before, asked = rows, rows + a, asked, asked + need
        cu[r + 1] = min(rows, max_tokens)
        if rows > max_tokens or (need and asked > n_free):
            refused = True
            continue
        if need:
            taken = asked
        for j in range(need):
            table[r, held + j] = free_pages[n_free - 1 - before - j]
        kv[r] = c + a
        for i in range(a):
            p = c + i
            pos[first + i] = p
            slot[first + i] = int(table[r, p // page]) * page + p % page
    return {"table": table, "cu_new": cu, "kv_lens": kv, "positions": pos, "slots": slot,
            "n_left": n_free - taken, "refused": refused}


def rope_rows(x, positions, axis_of_pair, inv_freq, gain=None, eps=0.0):
    """x [T, heads, d] float64 -> RMSNorm (where a gain is given), then pairs
    (i, i + len(inv_freq)) turned by positions[axis_of_pair[i]] * inv_freq[i]."""
    x = np.array(x, np.float64)
    if gain is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * np.asarray(gain, np.float64)
    half = len(inv_freq)
    if half:
        ang = np.stack([np.asarray(positions[a], np.float64) * f
                        for a, f in zip(axis_of_pair, inv_freq)], 1)[:, None]
        a, b = x[..., :half].copy(), x[..., half:2 * half].copy()
        x[..., :half] = a * np.cos(ang) - b * np.sin(ang)
        x[..., half:2 * half] = b * np.cos(ang) + a * np.sin(ang)
    return x


def paged_attention(q, k_cache, v_cache, table, cu_new, kv_lens, scale, window=0):
    """q [rows, hq, d], caches [pages, hkv, page, d], float64.  Returns out,
    lse, and for error bounds the softmax-weighted mean of |v|, the largest
    sum_e |q_e k_e| * |scale| a row met and its largest |v| (zeros where a row
    sees no key).  Pages outside the cache count as zeros."""
    rows, hq, d = q.shape
    pages, hkv, page, _ = k_cache.shape
    out, lse = np.zeros((rows, hq, d)), np.full((rows, hq), -np.inf)
    wabs, smag, vmax = np.zeros((rows, hq, d)), np.zeros((rows, hq)), np.zeros((rows, hq))
    for r in range(len(kv_lens)):
        a, b, kv = int(cu_new[r]), int(cu_new[r + 1]), int(kv_lens[r])
        if b <= a or kv <= 0:
            continue
        lo = max(0, kv - (b - a) - window + 1) if window else 0
        key = np.arange(lo, kv)
        ids = np.array([int(table[r, j // page]) for j in key])
        ok = (ids >= 0) & (ids < pages)
        p = np.arange(kv - (b - a), kv)[:, None]
        seen = (key <= p) & ((key > p - window) if window else True)
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
