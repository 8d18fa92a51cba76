"""The paged-cache operators on the GPU against oracle/paged.py (float64).

Tolerances (u = half a step of the cache's type, torch.finfo(t).eps / 2):

* tables: whole numbers, equal.
* append: each output is rounded once (u relative; 2^-25 absolute in fp16's
  subnormals); in fp32 the norm's sum of d squares, rsqrt and two products
  ((d + 8) steps of 2^-24) and the angle (2^-21 of sine and cosine) act on the
  length of the turned pair: u |x| + (2^-20 + (d + 8) 2^-24) |pair| + 2^-24.
  v is copied: equal.
* attention, A = softmax-weighted mean of |v|, n keys: the output's rounding
  u |o|, the weights' rounding u A, scores summed in fp32 (d products of
  2^-22 relative to sum |q k| scale =: ds, twice, for numerator and sum), the
  sums over the keys (n / 8 + 64) 2^-23 A, and weights below the type's normal
  range, 2^-25 |v| each in fp16:
      u (|o| + A) 1.01 + A (2 ds + (n / 8 + 64) 2^-23) [+ n 2^-25 vmax + 2^-24]
  lse: ds + (n / 8 + 64) 2^-23 + 2^-20 |lse|.
"""
import subprocess
import sys

import numpy as np
import pytest
import torch

import oracle
from tile_level_overlap_gb300 import build, mk, synth

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    build.build()
    mk.lib()


@pytest.fixture(scope="module")
def workspace():
    # whatever it holds must not matter
    return torch.full((mk.MK_PAGED_WORKSPACE_BYTES // 4,), float("nan"), device=DEV)


def ints(v):
    return torch.as_tensor(np.asarray(v, dtype=np.int64)).to(torch.int32).to(DEV)


def f64(t):
    return t.detach().double().cpu().numpy()


# ---------------------------------------------------------------- tables

def run_tables(ctx, new, page, width, max_tokens, pool, n_free=None, cap=None, seed=0):
    rng = np.random.default_rng(seed)
    n = len(ctx)
    ids = rng.permutation(pool)
    table, at = np.full((n, width), -7), 0
    for r, c in enumerate(ctx):
        for j in range(min(width, max(0, -(-c // page)))):
            table[r, j] = ids[at % pool]
            at += 1
    free = ids[at:] if at < pool else ids[:0]
    n_free = len(free) if n_free is None else n_free
    b = mk.PagedBatch(ints(table), ints(np.full(n + 1, 99)), ints(np.full(n, 99)), ints(np.full(max_tokens, 99)),
                      ints(np.full(max_tokens, 99)), page_size=page, max_new=max([1, *new]))
    left, status = ints([123]), ints([0])
    guard = free.copy()
    f = ints(free)
    b.build(ints(ctx), ints(new), f, ints([n_free]), left, status=status)
    want = oracle.paged_tables(ctx, new, free, n_free, table, page, max_tokens)
    for k in ("block_table", "cu_new", "kv_lens", "positions", "slots"):
        assert np.array_equal(getattr(b, k).cpu().numpy(), want["table" if k == "block_table" else k]), k
    assert left.item() == want["n_left"] and np.array_equal(f.cpu().numpy(), guard)
    assert status.item() == (mk.MK_ERR_BOUNDS if want["refused"] else 0)
    return want


@pytest.mark.parametrize("n,page,lo,hi,new_hi,pad", [
    (1, 16, 0, 0, 1, 0), (1, 256, 255, 255, 2, 3), (2, 32, 0, 100, 1, 0), (31, 16, 0, 65, 33, 7),
    (32, 64, 63, 65, 3, 1), (33, 128, 0, 700, 0, 5), (513, 16, 0, 40, 18, 0), (1023, 32, 0, 300, 1, 100),
    (4096, 16, 0, 20, 4, 13), (4095, 256, 0, 2000, 2, 0), (3, 16, 0, 9, 70000, 11), (700, 16, 0, 0, 300, 0)])
def test_tables_match_the_oracle(n, page, lo, hi, new_hi, pad):
    rng = np.random.default_rng(n + page)
    ctx, new = rng.integers(lo, hi + 1, n), rng.integers(0, new_hi + 1, n)
    width = int(max(-(-(ctx + new) // page))) + 2
    pool = int((-(-(ctx + new) // page)).sum()) + 5
    want = run_tables(ctx, new, page, width, int(new.sum()) + pad, pool, seed=n)
    assert not want["refused"] and want["n_left"] == 5


def test_tables_take_the_last_free_page():
    want = run_tables([15, 16], [2, 16], 16, 3, 18, 4, seed=3)
    assert want["n_left"] == 0 and not want["refused"]


@pytest.mark.parametrize("ctx,new,kw", [
    ([5, 16, 3, 20], [1, 1, 1, 30], dict(n_free=1)),           # the pages suffice for the first request that needs one
    ([16, 3, 16], [1, 2, 1], dict(n_free=0)),                  # none left: who needs none is served
    ([0, -1, 4], [2, 1, 2], {}), ([0, 1, 4], [2, -3, 2], {}),  # negative lengths
    ([0, 60, 4], [2, 5, 2], dict(width=4)),                    # over the table's width
    ([0, 2 ** 31 - 1, 4], [2, 2 ** 31 - 1, 2], {}),            # a sum past 31 bits
    ([0, 1, 4], [5, 6, 7], dict(max_tokens=12)),               # the third one's rows do not fit
    ([0, 1, 4], [5, 6, 7], dict(max_tokens=0)),
])
def test_refused_requests(ctx, new, kw):
    kw = {"width": 8, "max_tokens": 64, **kw}
    want = run_tables(ctx, new, 16, kw["width"], kw["max_tokens"], 40, n_free=kw.get("n_free"))
    assert want["refused"]


def test_free_count_outside_the_list_is_clamped_and_latched():
    for n_free, left in ((-5, 0), (9, 3)):
        b = mk.PagedBatch(ints([[-1] * 4]), ints([0, 0]), ints([0]), ints([0] * 4), ints([0] * 4), page_size=16, max_new=4)
        out, status = ints([77]), ints([0])
        b.build(ints([0]), ints([0]), ints([1, 2, 3]), ints([n_free]), out, status=status)
        assert out.item() == left and status.item() == mk.MK_ERR_BOUNDS


def test_pages_no_cache_has_give_a_refused_slot():
    b = mk.PagedBatch(ints([[-1] * 4, [-1] * 4]), ints([0] * 3), ints([0] * 2), ints([0] * 3), ints([0] * 3), page_size=16, max_new=4)
    b.build(ints([0, 0]), ints([1, 2]), ints([(1 << 28) + 3, -4]), ints([2]), ints([0]))
    assert b.slots.tolist() == [2 ** 31 - 1] * 3


# ---------------------------------------------------------------- append

def slots_and_caches(t, hkv, page, d, typ, layout, rng):
    pages = -(-t // page) + 2
    slots = (rng.permutation(pages)[:, None] * page + np.arange(page)).reshape(-1)
    slots = rng.permutation(slots)[:t]
    g = torch.Generator().manual_seed(int(rng.integers(1 << 30)))
    if layout == "hp":     # [pages][heads][tokens][d]
        kv = torch.randn(2, pages, hkv, page, d, generator=g).to(typ).to(DEV)
        k, v = kv[0], kv[1]
    elif layout == "ph":   # [pages][tokens][heads][d]
        kv = torch.randn(2, pages, page, hkv, d, generator=g).to(typ).to(DEV)
        k, v = kv[0].transpose(1, 2), kv[1].transpose(1, 2)
    else:                  # keys and values of a page together, padded rows
        kv = torch.randn(pages, 2, hkv, page, d + 8, generator=g).to(typ).to(DEV)
        k, v = kv[:, 0, :, :, :d], kv[:, 1, :, :, :d]
    return slots, k, v, kv


@pytest.mark.parametrize("t,hq,hkv,d,rot,axes,norm,packed,page,layout,typ", [
    (1, 32, 8, 128, 128, 1, True, True, 16, "hp", "bf16"), (1, 1, 1, 64, 64, 1, False, False, 256, "ph", "fp16"),
    (37, 32, 8, 128, 128, 3, True, True, 32, "ph", "bf16"), (70, 7, 1, 64, 32, 2, True, False, 64, "pad", "fp16"),
    (129, 4, 2, 64, 64, 4, False, True, 128, "pad", "bf16"), (300, 12, 4, 128, 64, 1, False, False, 16, "hp", "fp16"),
    (33, 5, 5, 128, 16, 1, True, True, 16, "hp", "bf16"), (33, 6, 3, 128, 96, 3, True, False, 32, "pad", "bf16"),
    (65, 8, 8, 64, 48, 1, False, True, 16, "ph", "fp16"), (20, 40, 8, 128, 0, 1, True, True, 16, "hp", "bf16"),
    # many tokens: rings of 32, 16 and 8 rows that go round, rows that the ring does not take
    (2500, 32, 8, 128, 128, 3, True, True, 64, "hp", "bf16"), (9000, 2, 1, 64, 64, 1, False, False, 16, "ph", "fp16"),
    (1999, 6, 3, 64, 32, 2, True, False, 32, "pad", "bf16"), (3001, 64, 16, 128, 128, 1, True, True, 16, "hp", "fp16"),
    (400, 96, 16, 128, 64, 4, True, False, 16, "ph", "bf16"), (305, 4, 4, 128, 0, 1, False, True, 256, "hp", "bf16")])
def test_append_matches_the_oracle(t, hq, hkv, d, rot, axes, norm, packed, page, layout, typ):
    rng = np.random.default_rng(t * 7 + hq)
    typ = TYPES[typ]
    g = torch.Generator().manual_seed(t)
    rows = torch.randn(t, hq + 2 * hkv, d, generator=g).to(typ).to(DEV)
    parts = rows[:, :hq], rows[:, hq:hq + hkv], rows[:, hq + hkv:]
    q, k, v = parts if packed else (p.contiguous() for p in parts)
    slots, kc, vc, whole = slots_and_caches(t, hkv, page, d, typ, layout, rng)
    slots[rng.random(t) < 0.15] = -1  # left out
    positions = rng.integers(0, 1 << 20, (axes, t))
    positions[0, 0], positions[-1, -1] = 2 ** 31 - 1, -5
    of = [int(i) for i in rng.integers(0, axes, rot // 2)]
    if of:
        of[0] = axes - 1
    theta = 1e6
    rope = mk.Rope(d, theta=theta, rotary_dim=rot, axis_of_pair=of if axes > 1 else None) if rot else None
    gains = [(1 + 0.1 * torch.randn(d, generator=g)).to(typ).to(DEV) if norm else None for _ in range(2)]
    q_out = torch.full((t, hq, d), 3.0, dtype=typ, device=DEV)
    before, cache = whole.clone(), mk.PagedCache(kc, vc, n_q_heads=hq)
    cache.append(q, k, v, ints(slots), ints(positions if axes > 1 else positions[0]) if rot else None, rope, q_out=q_out,
                 q_norm=gains[0], k_norm=gains[1], eps=1e-6)
    assert cache.status() == 0
    inv = [theta ** (-2.0 * i / rot) for i in range(rot // 2)]
    live = slots >= 0
    u = torch.finfo(typ).eps / 2

    def check(got, x, gain):
        want = oracle.rope_rows(f64(x), positions, of if axes > 1 else [0] * (rot // 2), inv, None if gain is None else f64(gain), 1e-6)
        pair = np.abs(want).copy()
        h = rot // 2
        pair[..., :h] = pair[..., h:rot] = np.hypot(want[..., :h], want[..., h:rot])
        tol = u * np.abs(want) + (2.0 ** -20 + (d + 8) * 2.0 ** -24) * pair + 2.0 ** -24
        err = np.abs(got - want)[live]
        assert (err <= tol[live]).all(), (err - tol[live]).max()

    check(f64(q_out), q, gains[0])
    assert (q_out[torch.as_tensor(~live).to(DEV)] == 3.0).all()
    at = torch.as_tensor(np.where(live, slots, 0)).to(DEV)
    check(f64(kc[at // page, :, at % page]), k, gains[1])
    sel = torch.as_tensor(live).to(DEV)
    assert torch.equal(vc[at // page, :, at % page][sel], v[sel])
    # everything else of the caches (padding included) is as it was
    kc[at[sel] // page, :, at[sel] % page] = 0
    vc[at[sel] // page, :, at[sel] % page] = 0
    now = whole.clone()
    whole.copy_(before)
    kc[at[sel] // page, :, at[sel] % page] = 0
    vc[at[sel] // page, :, at[sel] % page] = 0
    assert torch.equal(now, whole)


@pytest.mark.parametrize("slots_of", [lambda rng, t: np.full(t, -1), lambda rng, t: np.where(rng.random(t) < 0.5, -1, 2 ** 31 - 1)])
def test_append_of_left_out_and_refused_tokens_writes_nothing(slots_of):
    for t in (40, 3000):
        g = torch.Generator().manual_seed(t)
        q, k, v = (torch.randn(t, h, 64, generator=g).to(torch.float16).to(DEV) for h in (4, 2, 2))
        kc, vc = (torch.full((9, 2, 16, 64), 2.0, dtype=torch.float16, device=DEV) for _ in range(2))
        cache, out, slots = mk.PagedCache(kc, vc, n_q_heads=4), torch.full_like(q, 4.0), slots_of(np.random.default_rng(t), t)
        cache.append(q, k, v, ints(slots), ints(np.arange(t)), mk.Rope(64), q_out=out)
        assert cache.status() == (mk.MK_ERR_BOUNDS if (slots > 0).any() else 0)
        assert (out == 4).all() and (kc == 2).all() and (vc == 2).all()


def test_append_in_place_and_far_slots_refused():
    typ = torch.bfloat16
    g = torch.Generator().manual_seed(5)
    q, k, v = (torch.randn(6, h, 128, generator=g).to(typ).to(DEV) for h in (4, 2, 2))
    kc, vc = (torch.zeros(3, 2, 16, 128, dtype=typ, device=DEV) for _ in range(2))
    rope, pos = mk.Rope(128), ints(np.arange(6))
    other, cache = torch.empty_like(q), mk.PagedCache(kc, vc, n_q_heads=4)
    slots = ints([47, 3, 48, 2 ** 31 - 1, -1, 0])
    cache.append(q, k, v, slots, pos, rope, q_out=other)
    assert cache.status() == mk.MK_ERR_BOUNDS
    cache.reset()
    assert cache.status() == 0
    mine = q.clone()
    cache.append(mine, k, v, ints([47, 3, -1, -1, -1, 0]), pos, rope)
    assert cache.status() == 0
    keep = torch.tensor([0, 1, 5], device=DEV)
    assert torch.equal(mine[keep], other[keep]) and torch.equal(mine[2:5], q[2:5])
    assert int((kc.abs().sum(-1) > 0).sum()) == 6
    cache.append(q[:0], k[:0], v[:0], slots[:0], pos[:0], rope, q_out=other[:0])


# ---------------------------------------------------------------- attention

def make_attention(ctx, new, hq, hkv, d, page, typ, layout="hp", seed=0, pad=0, garbage=float("nan"), scale=1.0):
    """Pages in random order; whatever no request holds is `garbage`, the tails
    of last pages and unused table entries among it."""
    rng = np.random.default_rng(seed)
    g = torch.Generator().manual_seed(seed)
    n, kv = len(ctx), [c + a for c, a in zip(ctx, new)]
    need = [-(-x // page) for x in kv]
    width, pages = max(1, max(need)) + 2, sum(need) + 3
    ids = rng.permutation(pages)
    table, at = rng.integers(-9, 1 << 30, (n, width)), 0
    for r in range(n):
        table[r, :need[r]] = ids[at:at + need[r]]
        at += need[r]
    _, k, v, whole = slots_and_caches(pages * page - 2 * page, hkv, page, d, typ, layout, rng)
    keep_k, keep_v = k.clone(), v.clone()
    whole.fill_(garbage)
    for r in range(n):
        for j in range(need[r]):
            p, m = int(table[r, j]), min(page, kv[r] - j * page)
            k[p, :, :m], v[p, :, :m] = keep_k[p, :, :m], keep_v[p, :, :m]
    rows = sum(new) + pad
    cu = np.concatenate([[0], np.cumsum(new)])
    q = (scale * torch.randn(rows, hq, d, generator=g)).to(typ).to(DEV)
    return dict(q=q, k=k, v=v, table=table, cu=cu, kv=np.array(kv), page=page, max_new=max([1, *new]))


def check_attention(s, window=0, scale=0.0, workspace=None, refused_rows=(), status=0, max_new=None, out_pad=0):
    q, typ, d, hq = s["q"], s["q"].dtype, s["q"].shape[2], s["q"].shape[1]
    rows, total = q.shape[0], int(s["cu"][-1])
    store = torch.full((rows, hq * d + out_pad), 5.0, dtype=typ, device=DEV)
    out = store[:, :hq * d].view(rows, hq, d)
    lse = torch.full((rows, hq), 5.0, device=DEV)
    batch = mk.PagedBatch(ints(s["table"]), ints(s["cu"]), ints(s["kv"]), page_size=s["page"], max_new=max_new or s["max_new"])
    cache = mk.PagedCache(s["k"], s["v"], n_q_heads=hq, workspace=workspace)
    cache.attention(q, batch, out, lse=lse, window=window, scale=scale)
    assert cache.status() == status
    again, lse2 = torch.full_like(out, 7.0), torch.full_like(lse, 7.0)
    cache.attention(q, batch, again, lse=lse2, window=window, scale=scale)
    bare = torch.full_like(out, 7.0)
    cache.attention(q, batch, bare, window=window, scale=scale)
    k, v = f64(s["k"]), f64(s["v"])
    ref, rlse, wabs, smag, vmax = oracle.paged_attention(f64(q), k, v, s["table"], s["cu"], s["kv"], scale or d ** -0.5, window)
    live = np.arange(rows) < total
    live[list(refused_rows)] = False
    u = torch.finfo(typ).eps / 2
    keys = np.minimum(s["kv"].max(), (window + s["max_new"]) if window else 1 << 40)
    ds, sums = d * 2.0 ** -22 * smag, (keys / 8 + 64) * 2.0 ** -23
    tol = u * 1.01 * (np.abs(ref) + wabs) + wabs * (2 * ds[..., None] + sums)
    if typ == torch.float16:
        tol = tol + keys * 2.0 ** -25 * vmax[..., None] + 2.0 ** -24
    got, glse = f64(out), f64(lse)
    assert np.isfinite(got[live]).all()
    err = (np.abs(got - ref) - tol)[live]
    assert err.size == 0 or err.max() <= 0, err.max()
    none = np.isneginf(rlse) & live[:, None]
    assert np.isneginf(glse[none]).all() and (got[none] == 0).all()
    some = ~np.isneginf(rlse) & live[:, None]
    assert (np.abs(glse[some] - rlse[some]) <= (ds + sums)[some] + 2.0 ** -20 * np.abs(rlse[some])).all()
    # rows of no request are as they were, equal calls give equal bits, lse is optional
    assert (got[~live] == 5).all() and (glse[~live] == 5).all() and (store[:, hq * d:] == 5).all()
    sel = torch.as_tensor(live).to(DEV)
    assert torch.equal(out[sel], again[sel]) and torch.equal(lse[sel], lse2[sel]) and torch.equal(out[sel], bare[sel])
    return out, lse


ATT = [
    # ctx, new, hq, hkv, d, page, window, layout, type
    ([0], [1], 32, 8, 128, 16, 0, "hp", "bf16"),                         # the first token of all
    ([0, 0, 5], [1, 0, 0], 4, 2, 64, 16, 0, "hp", "fp16"),               # requests that rest
    ([4095], [1], 32, 8, 128, 16, 0, "ph", "bf16"),
    ([1, 15, 16, 17, 31, 63, 64, 65, 127, 128], [1] * 10, 8, 2, 128, 16, 0, "hp", "bf16"),
    ([1, 15, 16, 17, 31, 63, 64, 65, 127, 128], [1] * 10, 8, 2, 64, 32, 0, "ph", "fp16"),
    ([255, 256, 257, 700], [1] * 4, 6, 2, 128, 256, 0, "pad", "bf16"),
    ([300, 0, 77, 1000], [4, 2, 1, 3], 8, 8, 128, 16, 0, "hp", "fp16"),   # drafted tokens, one head each
    ([300, 0, 77, 1000], [4, 2, 1, 3], 16, 2, 64, 64, 0, "pad", "bf16"),
    ([513, 40], [5, 3], 7, 1, 128, 32, 0, "hp", "bf16"),                 # 7 query heads per kv head
    ([513, 40], [2, 1], 15, 1, 64, 16, 0, "hp", "fp16"),
    ([100, 2], [1, 1], 64, 1, 128, 16, 0, "hp", "bf16"),                 # 64 query heads on one kv head
    ([900, 20, 3], [1, 4, 3], 8, 2, 128, 16, 100, "hp", "bf16"),         # windows
    ([900, 20, 3], [1, 4, 3], 8, 2, 64, 32, 1, "ph", "fp16"),
    ([2000, 640], [1, 1], 32, 8, 128, 64, 512, "hp", "bf16"),
    ([0], [128], 4, 4, 128, 16, 0, "hp", "bf16"),                        # chunks
    ([0], [257], 8, 2, 64, 16, 0, "ph", "fp16"),
    ([0, 129, 640], [33, 65, 200], 8, 2, 128, 16, 0, "hp", "bf16"),
    ([0, 129, 640], [33, 65, 200], 8, 2, 64, 128, 0, "pad", "bf16"),
    ([1000, 3, 0, 50], [1, 90, 0, 300], 16, 4, 128, 32, 0, "hp", "fp16"),  # decode and chunks in one call
    ([500], [300], 3, 1, 128, 16, 0, "hp", "bf16"),                      # 3, 5, 6, 7 query heads per kv head
    ([500], [130], 5, 1, 64, 16, 0, "hp", "bf16"),
    ([10], [200], 12, 2, 128, 64, 0, "ph", "bf16"),
    ([77], [140], 14, 2, 128, 256, 0, "hp", "fp16"),
    ([77, 9], [40, 40], 64, 1, 64, 16, 0, "hp", "bf16"),
    ([700, 20], [150, 200], 8, 2, 128, 16, 64, "hp", "bf16"),            # windows shorter and longer than a tile
    ([700, 20], [150, 200], 8, 2, 64, 32, 1, "hp", "fp16"),
    ([3000, 0, 130], [100, 513, 1], 4, 1, 128, 64, 333, "hp", "bf16"),
    ([0], [1500], 4, 1, 128, 16, 0, "hp", "bf16"),
    ([5000], [260], 4, 1, 64, 16, 0, "hp", "bf16"),
    # many blocks per SM: the load rings go round
    ([30000, 17, 21111, 25000], [1, 1, 1, 1], 16, 16, 128, 64, 0, "hp", "bf16"),
    ([30000, 17, 21111, 25000], [4, 1, 3, 2], 32, 8, 64, 16, 0, "hp", "fp16"),
    ([30000, 17, 21111], [4, 8, 3], 32, 8, 128, 16, 0, "ph", "bf16"),
    ([9000], [2000], 8, 8, 64, 16, 0, "hp", "bf16"),
    ([6000, 30, 999], [1111, 1300, 1], 8, 4, 128, 32, 0, "ph", "fp16"),
    ([6000, 30], [1111, 1300], 14, 2, 128, 64, 1500, "hp", "bf16"),
]


@pytest.mark.parametrize("case", range(len(ATT)))
def test_attention_matches_the_oracle(case, workspace):
    ctx, new, hq, hkv, d, page, window, layout, typ = ATT[case]
    s = make_attention(ctx, new, hq, hkv, d, page, TYPES[typ], layout, seed=case, pad=case % 3)
    check_attention(s, window, workspace=workspace, out_pad=8 * (case % 2))


@pytest.mark.parametrize("new", [[1, 2, 1], [70, 2, 41]])
def test_rows_without_keys_give_zero(new, workspace):
    s = make_attention([40, 10, 0], new, 8, 2, 128, 16, torch.bfloat16, seed=3)
    for kv in ([0, 1, 0], [41, 1, 1], [0, 0, 0]):
        s["kv"] = np.minimum(np.array(kv), s["kv"])
        check_attention(s, workspace=workspace)


@pytest.mark.parametrize("new,typ", [([1, 3], "bf16"), ([130, 3], "bf16"), ([1, 40], "fp16")])
def test_peaked_and_flat_softmax(new, typ, workspace):
    for scale in (8.0, 0.0):
        s = make_attention([600, 200], new, 8, 2, 64, 16, TYPES[typ], seed=11, scale=scale)
        check_attention(s, workspace=workspace)
    s = make_attention([600, 200], new, 8, 2, 128, 16, TYPES[typ], seed=12)
    check_attention(s, workspace=workspace, scale=1.7)
    check_attention(s, workspace=workspace, scale=-0.1)


def test_growing_scores_move_the_maximum(workspace):
    # keys along q, longer and longer: every block brings a new maximum
    for new in ([1], [64]):
        s = make_attention([900], new, 4, 1, 128, 16, torch.bfloat16, seed=5)
        s["q"].fill_(0.5)
        for j in range(int(s["kv"][0])):
            s["k"][int(s["table"][0, j // 16]), 0, j % 16] = j / 64.0
        check_attention(s, workspace=workspace)
        for j in range(int(s["kv"][0])):
            s["k"][int(s["table"][0, j // 16]), 0, j % 16] = -j / 64.0
        check_attention(s, workspace=workspace)


@pytest.mark.parametrize("new", [[1, 2], [90, 130]])
def test_bad_pages_count_as_zeros(new, workspace):
    s = make_attention([300, 200], new, 8, 2, 128, 16, torch.bfloat16, seed=8)
    s["table"][0, 3], s["table"][1, 7], s["table"][1, 0] = -1, s["k"].shape[0], 2 ** 31 - 1
    check_attention(s, workspace=workspace, status=mk.MK_ERR_BOUNDS)


def test_pages_before_the_window_are_not_looked_at(workspace):
    for new in ([1, 2], [80, 2]):
        s = make_attention([3000, 700], new, 8, 2, 128, 16, torch.bfloat16, seed=9)
        for r in range(2):
            first = max(0, int(s["kv"][r]) - new[r] - 200 + 1)
            for j in range(first // 16):
                s["k"][int(s["table"][r, j])] = float("nan")
                s["v"][int(s["table"][r, j])] = float("inf")
            s["table"][r, :first // 16] = -1
        check_attention(s, window=200, workspace=workspace)


@pytest.mark.parametrize("new", [[1, 1, 1], [50, 50, 50]])
def test_bad_lengths_are_latched(new, workspace):
    s = make_attention([100, 100, 100], new, 8, 2, 64, 16, torch.bfloat16, seed=13)
    width = s["table"].shape[1] * 16
    t = dict(s, kv=s["kv"].copy())
    t["kv"][1] = -3   # as no keys
    check_attention(t, workspace=workspace, status=mk.MK_ERR_BOUNDS)
    # past the table: the rows stand at their positions, the keys past it are absent
    t = dict(s, kv=s["kv"].copy(), table=s["table"].copy())
    t["table"][1] = t["table"][0, 0]
    t["k"] = torch.nan_to_num(t["k"])
    t["v"] = torch.nan_to_num(t["v"])
    t["kv"][1] = width + 40
    q, typ = t["q"], t["q"].dtype
    out, lse = torch.zeros_like(q), torch.zeros(q.shape[:2], device=DEV)
    cache = mk.PagedCache(t["k"], t["v"], n_q_heads=8, workspace=workspace)
    cache.attention(q, mk.PagedBatch(ints(t["table"]), ints(t["cu"]), ints(t["kv"]), page_size=16, max_new=max(new)), out, lse=lse)
    assert cache.status() == mk.MK_ERR_BOUNDS and torch.isfinite(out.float()).all()
    # more new tokens than max_new: left as they were
    if new[0] > 1:
        t = dict(s, kv=s["kv"].copy(), cu=np.array([0, 50, 110, 150]))
        check_attention(t, workspace=workspace, status=mk.MK_ERR_BOUNDS, max_new=50, refused_rows=range(50, 110))
    # offsets that fall, or pass the rows
    t = dict(s, cu=np.array([0, new[0], new[0] - 1, sum(new)]))
    out.fill_(5)
    cache.reset()
    cache.attention(q, mk.PagedBatch(ints(t["table"]), ints(t["cu"]), ints(t["kv"]), page_size=16, max_new=max(new)), out, lse=lse)
    assert cache.status() == mk.MK_ERR_BOUNDS
    t = dict(s, cu=np.array([0, new[0], 2 * new[0], sum(new) + 1]))
    cache.reset()
    cache.attention(q, mk.PagedBatch(ints(t["table"]), ints(t["cu"]), ints(t["kv"]), page_size=16, max_new=max(new) + 1), out, lse=lse)
    assert cache.status() == mk.MK_ERR_BOUNDS


def test_keys_past_32_bit_offsets(workspace):
    # a cache of over 2^31 elements per tensor: pages near its end
    pages, page, d = 4200, 256, 128
    kv = torch.zeros(2, pages, 16, page, d, dtype=torch.bfloat16, device=DEV)
    assert kv[0].numel() > 2 ** 31
    g = torch.Generator(device=DEV).manual_seed(2)
    use = [pages - 1, 3, pages - 2]
    for p in use:
        kv[:, p] = torch.randn(2, 16, page, d, generator=g, device=DEV).to(torch.bfloat16)
    table = np.array([use])
    for new in (1, 70):
        q = torch.randn(new, 16, d, generator=g, device=DEV).to(torch.bfloat16)
        out = torch.empty_like(q)
        cache = mk.PagedCache(kv[0], kv[1], n_q_heads=16, workspace=workspace)
        cache.attention(q, mk.PagedBatch(ints(table), ints([0, new]), ints([700]), page_size=page, max_new=new), out)
        small = kv[:, use].contiguous()
        out2 = torch.empty_like(q)
        mk.PagedCache(small[0], small[1], n_q_heads=16, workspace=workspace).attention(
            q, mk.PagedBatch(ints([[0, 1, 2]]), ints([0, new]), ints([700]), page_size=page, max_new=new), out2)
        assert torch.equal(out, out2) and cache.status() == 0
        ref = oracle.paged_attention(f64(q), f64(small[0]), f64(small[1]), np.array([[0, 1, 2]]), [0, new], [700], d ** -0.5)[0]
        assert np.abs(f64(out) - ref).max() <= 2 ** -7 * np.abs(ref).max() + 2 ** -8 * 4  # u (|o| + A), A <= 4
    kc = kv[0]
    rope = mk.Rope(d)
    qkv = torch.randn(2, 48, d, generator=g, device=DEV).to(torch.bfloat16)
    cache.append(qkv[:, :16], qkv[:, 16:32], qkv[:, 32:], ints([(pages - 1) * page + 255, 5]), ints([0, 0]), rope)
    assert torch.equal(kc[pages - 1, :, 255], qkv[0, 16:32]) and torch.equal(kv[1, 0, :, 5], qkv[1, 32:])


def test_requests_that_share_pages(workspace):
    # one prefix in the tables of all, also twice in one of them
    s = make_attention([400, 400, 400], [1, 2, 40], 8, 2, 128, 16, torch.bfloat16, seed=17)
    s["table"][1, :20] = s["table"][0, :20]
    s["table"][2, :20] = s["table"][0, :20]
    s["table"][2, 21] = s["table"][2, 20]
    check_attention(s, workspace=workspace)


def test_many_requests(workspace):
    rng = np.random.default_rng(4)
    for n, hi in ((4096, 40), (1000, 300)):
        ctx, new = rng.integers(0, hi, n).tolist(), rng.integers(0, 3, n).tolist()
        check_attention(make_attention(ctx, new, 2, 1, 64, 16, torch.bfloat16, seed=n), workspace=workspace)


# ---------------------------------------------------------------- streams, graphs, the whole step

def test_on_another_stream_and_in_graphs(workspace):
    s = make_attention([300, 0, 900], [1, 70, 2], 8, 2, 128, 16, torch.bfloat16, seed=21, garbage=0.0)
    want, wlse = check_attention(s, workspace=workspace)
    cache = mk.PagedCache(s["k"], s["v"], n_q_heads=8, workspace=workspace)
    batch = mk.PagedBatch(ints(s["table"]), ints(s["cu"]), ints(s["kv"]), page_size=16, max_new=70)
    side = torch.cuda.Stream()
    out, lse = torch.zeros_like(s["q"]), torch.zeros_like(wlse)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        cache.attention(s["q"], batch, out, lse=lse)
    side.synchronize()
    assert torch.equal(out, want) and torch.equal(lse, wlse)
    cache.attention(s["q"], batch, out.zero_(), stream=torch.cuda.current_stream())
    assert torch.equal(out, want)
    # two graphs with a workspace each, replayed at once on two streams, with lengths that change in place
    graphs, outs = [], []
    for _ in range(2):
        c = mk.PagedCache(s["k"], s["v"], n_q_heads=8, workspace=torch.empty(mk.MK_PAGED_WORKSPACE_BYTES, dtype=torch.uint8, device=DEV))
        o, gr = torch.zeros_like(s["q"]), torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(gr):
            c.attention(s["q"], batch, o)
        graphs.append((gr, c))
        outs.append(o)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        for st, (gr, _) in zip(streams, graphs):
            with torch.cuda.stream(st):
                gr.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want) and torch.equal(outs[1], want)
    t = dict(s, kv=np.array([17, 70, 400]))
    batch.kv_lens.copy_(ints(t["kv"]))
    torch.cuda.synchronize()
    graphs[0][0].replay()
    torch.cuda.synchronize()
    want2, _ = check_attention(t, workspace=workspace)
    assert torch.equal(outs[0], want2)


def test_the_workspace_is_of_the_calls_stream():
    """Memory that the current stream has given back, and may still be using, is
    not handed to a first call on another stream."""
    s = make_attention([40, 0], [1, 3], 4, 2, 64, 16, torch.bfloat16)
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    given_back = torch.empty(mk.MK_PAGED_WORKSPACE_BYTES, dtype=torch.uint8, device="cuda")
    at = given_back.data_ptr()
    del given_back
    cache = mk.PagedCache(s["k"], s["v"], 4)
    with torch.cuda.stream(other):
        out = torch.empty_like(s["q"])
    batch = mk.PagedBatch(ints(s["table"]), ints(s["cu"]), ints(s["kv"]), page_size=16, max_new=3)
    other.wait_stream(torch.cuda.current_stream())
    cache.attention(s["q"], batch, out, stream=other)
    assert cache.workspace.data_ptr() != at
    torch.cuda.synchronize()
    want = torch.empty_like(s["q"])
    cache.attention(s["q"], batch, want)
    assert torch.equal(out, want) and cache.status() == 0


@pytest.mark.parametrize("new", [[1, 2], [70, 2]])
def test_a_nan_stays_with_its_row(new, workspace):
    s = make_attention([300, 200], new, 8, 2, 128, 16, torch.bfloat16, seed=30, garbage=0.0)
    batch = mk.PagedBatch(ints(s["table"]), ints(s["cu"]), ints(s["kv"]), page_size=16, max_new=max(new))
    cache = mk.PagedCache(s["k"], s["v"], n_q_heads=8, workspace=workspace)
    outs = []
    for spoil in (False, True):
        q = s["q"].clone()
        if spoil:
            q[0, 3, 5] = float("nan")
        out, lse = torch.zeros_like(q), torch.zeros(q.shape[:2], device=DEV)
        cache.attention(q, batch, out, lse=lse)
        outs.append((out, lse))
    (a, la), (b, lb) = outs
    assert torch.isnan(b[0, 3]).all() and torch.isnan(lb[0, 3])
    b[0, 3], lb[0, 3] = a[0, 3], la[0, 3]
    assert torch.equal(a, b) and torch.equal(la, lb)


FIRST_IN_CAPTURE = """
import sys, torch
sys.path.insert(0, %r)
from tile_level_overlap_gb300 import mk
dev = "cuda:0"
i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)
k, v = (torch.randn(40, 2, 16, 64, device=dev).to(torch.bfloat16) for _ in range(2))
cache = mk.PagedCache(k, v, n_q_heads=4, workspace=torch.empty(mk.MK_PAGED_WORKSPACE_BYTES, dtype=torch.uint8, device=dev))
t = 400
q, kn, vn = (torch.randn(t, h, 64, device=dev).to(torch.bfloat16) for h in (4, 2, 2))
batch = mk.PagedBatch(i32([[-1] * 30, [-1] * 30]), i32([0] * 3), i32([0] * 2), i32([0] * t), i32([0] * t), page_size=16, max_new=399)
ctx, new, free, n_free, left = i32([0, 0]), i32([399, 1]), i32(list(range(40))), i32([40]), i32([0])
out, qo, rope = torch.zeros_like(q), torch.zeros_like(q), mk.Rope(64)
def step():
    batch.build(ctx, new, free, n_free, left)
    cache.append(q, kn, vn, batch.slots, batch.positions, rope, q_out=qo)
    cache.attention(qo, batch, out)
g = torch.cuda.CUDAGraph()
torch.cuda.synchronize()
with torch.cuda.graph(g):
    step()
g.replay()
torch.cuda.synchronize()
got = out.clone()
bare = mk.PagedCache(k, v, n_q_heads=4)
with torch.cuda.graph(torch.cuda.CUDAGraph()):
    try:
        bare.attention(qo, batch, out)
        print("accepted")
    except ValueError:
        pass
out.zero_()
step()
torch.cuda.synchronize()
assert torch.equal(got, out) and cache.status() == 0 and got.abs().sum() > 0
print("same")
"""


def test_the_first_calls_of_a_process_in_a_capture():
    r = subprocess.run([sys.executable, "-c", FIRST_IN_CAPTURE % build.ROOT], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.split() == ["same"], r.stdout + r.stderr


def test_python_refusals():
    s = make_attention([300], [2], 8, 2, 128, 16, torch.bfloat16, seed=1, garbage=0.0)
    q, k, v = s["q"], s["k"], s["v"]
    batch = mk.PagedBatch(ints(s["table"]), ints(s["cu"]), ints(s["kv"]), page_size=16, max_new=2)
    cache, out = mk.PagedCache(k, v, n_q_heads=8), torch.empty_like(q)
    bad = [lambda: cache.attention(q.float(), batch, out), lambda: cache.attention(q.half(), batch, out),
           lambda: cache.attention(q.cpu(), batch, out), lambda: cache.attention(q, batch, out[:1]),
           lambda: cache.attention(q[:, :4], batch, out), lambda: cache.attention(q.transpose(0, 1), batch, out),
           lambda: cache.attention(q, batch, out, lse=torch.empty(2, 7, device=DEV)),
           lambda: cache.attention(q, batch, out, lse=torch.empty(2, 8, device=DEV, dtype=torch.float64)),
           lambda: mk.PagedCache(k, v.float(), n_q_heads=8), lambda: mk.PagedCache(k, v[:, :1], n_q_heads=8),
           lambda: mk.PagedCache(k.cpu(), v.cpu(), n_q_heads=8),
           lambda: mk.PagedCache(k, v, n_q_heads=8, workspace=torch.empty(100, device=DEV)),
           lambda: mk.PagedBatch(ints(s["table"]), ints([0]), ints(s["kv"]), page_size=16, max_new=2),
           lambda: mk.PagedBatch(ints(s["table"]).long(), ints(s["cu"]), ints(s["kv"]), page_size=16, max_new=2),
           lambda: batch.build(ints([1]), ints([1]), ints([1]), ints([1]), ints([1])),
           lambda: cache.append(q, q[:, :2], q[:, :2], ints([0, 1]), None, mk.Rope(128)),
           lambda: cache.append(q, q[:, :2], q[:, :2], ints([0, 1]), ints([0]), mk.Rope(128)),
           lambda: cache.append(q, q[:, :2], q[:, :2], ints([0]), ints([0, 1]), mk.Rope(128))]
    for i, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
            print("accepted", i)
    with pytest.raises(mk.MkError):
        cache.attention(q, batch, q)
    with pytest.raises(mk.MkError):
        cache.attention(q, batch, out, window=-1)


@pytest.mark.parametrize("d,hq,hkv,typ,page,axes", [(128, 8, 2, "bf16", 16, 1), (64, 6, 2, "fp16", 32, 3)])
def test_a_serving_run(d, hq, hkv, typ, page, axes, workspace):
    """Prompts in chunks, then decode steps, requests that come, rest and go:
    tables, append and attention of every step on the GPU, the counts handed on
    by device copies; each step's outputs against the whole sequences."""
    typ, rng = TYPES[typ], np.random.default_rng(d)
    n, width, pool = 5, 24, 90
    kc, vc = (torch.full((pool, hkv, page, d), float("nan"), dtype=typ, device=DEV) for _ in range(2))
    cache = mk.PagedCache(kc, vc, n_q_heads=hq, workspace=workspace)
    sections = [d // 2 - 2 * (d // 8), d // 8, d // 8] if axes == 3 else [d // 2]
    rope = mk.Rope(d, theta=1e5, sections=sections)
    of = [a for a, k in enumerate(sections) for _ in range(k)]
    inv = [1e5 ** (-2.0 * i / d) for i in range(d // 2)]
    plan = [[40, 0, 100, 0, 7], [1, 150, 100, 0, 7], [1, 1, 1, 33, 0], [1, 1, 1, 1, 1], [0, 3, 1, 1, 2], [1, 1, 1, 1, 1]]
    rows = max(sum(p) for p in plan) + 3
    free, n_free, n_left = ints(rng.permutation(pool)), ints([pool]), ints([0])
    table, ctx = ints(np.full((n, width), -1)), [0] * n
    seqs = [[np.zeros((0, h, d)) for h in (hkv, hkv)] for _ in range(n)]
    batch = mk.PagedBatch(table, ints([0] * (n + 1)), ints([0] * n), ints([0] * rows), ints([0] * rows), page_size=page, max_new=150)
    used = 0
    for step, new in enumerate(plan):
        g = torch.Generator().manual_seed(step)
        total = sum(new)
        qkv = torch.randn(rows, hq + 2 * hkv, d, generator=g).to(typ).to(DEV)
        q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
        raw = f64(qkv)
        batch.build(ints(ctx), ints(new), free, n_free, n_left, status=cache._status)
        n_free.copy_(n_left)
        pos = batch.positions if axes == 1 else torch.stack([batch.positions, batch.positions // 3, batch.positions % 5])
        cache.append(q, k, v, batch.slots, pos, rope)   # q turned in place
        out, lse = torch.full((rows, hq, d), 9.0, dtype=typ, device=DEV), torch.empty(rows, hq, device=DEV)
        cache.attention(q, batch, out, lse=lse)
        assert cache.status() == 0
        assert (out[total:] == 9).all() and torch.equal(q[total:], qkv[total:, :hq])
        used += sum(-(-(c + a) // page) - -(-c // page) for c, a in zip(ctx, new))
        assert n_left.item() == pool - used
        first = 0
        u = torch.finfo(typ).eps / 2
        for r in range(n):
            rng_rows = slice(first, first + new[r])
            first += new[r]
            if not new[r]:
                continue
            p = np.arange(ctx[r], ctx[r] + new[r])
            ps = [p] if axes == 1 else [p, p // 3, p % 5]
            kr = oracle.rope_rows(raw[rng_rows, hq:hq + hkv], ps, of, inv)
            qr = f64(q[rng_rows])
            # the cache's keys, as stored, enter the check of attention; here they are checked against the formula
            ctx[r] += new[r]
            ids = table[r, :-(-ctx[r] // page)].long()
            ks, vs = (c[ids].transpose(1, 2).reshape(-1, hkv, d)[:ctx[r]] for c in (kc, vc))
            assert np.abs(f64(ks)[p] - kr).max() <= (u + 2 ** -18) * np.abs(kr).max() * 1.5
            assert np.array_equal(f64(vs)[p], raw[rng_rows, hq + hkv:])
            seqs[r] = [np.concatenate([seqs[r][0], f64(ks)[p]]), np.concatenate([seqs[r][1], f64(vs)[p]])]
            assert np.array_equal(f64(ks), seqs[r][0])  # nothing written since has changed them
            ref, rl, wabs, smag, _ = oracle.paged_attention(qr, seqs[r][0].transpose(1, 0, 2)[None], seqs[r][1].transpose(1, 0, 2)[None],
                                                            np.zeros((1, 1), int), [0, new[r]], [ctx[r]], d ** -0.5)
            tol = u * 1.01 * (np.abs(ref) + wabs) + wabs * (2 * d * 2.0 ** -22 * smag[..., None] + 100 * 2.0 ** -23) + 2.0 ** -17
            assert (np.abs(f64(out[rng_rows]) - ref) <= tol).all()


def test_the_plans_own_cache_as_pages(workspace):
    """A prompt's keys and values that mk_prefill wrote, read by the paged
    attention where they lie."""
    cfg = synth.TOY_1L.replace(ffn=512)
    d, hkv, hq, ctx, page = cfg.head_dim, cfg.n_kv_heads, cfg.n_q_heads, 256, 32
    plan = mk.Plan(cfg, synth.make_weights(cfg, device=DEV), max_batch=2, max_ctx=ctx)
    kv = synth.make_kv_cache(cfg, 2, ctx, device=DEV)
    logits = torch.empty(2, cfg.vocab, device=DEV)
    tokens = synth.make_tokens(2 * 200, cfg.vocab).view(2, 200).to(DEV)
    plan.prefill_batch(tokens, [150, 200], kv, logits)
    assert plan.status() == mk.MK_OK
    k, v = kv[0, 0], kv[0, 1]                                    # [slot][head][ctx][d]
    blocks = ctx // page
    shape, strides = (2 * hkv * blocks - (hkv - 1) * blocks, hkv, page, d), (page * d, ctx * d, d, 1)
    paged = [torch.as_strided(t, shape, strides, t.storage_offset()) for t in (k, v)]
    table = np.array([[s * hkv * blocks + j for j in range(blocks)] for s in range(2)])
    new, lens = [1, 70], [150, 200]
    q = torch.randn(71, hq, d, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).to(DEV)
    out = torch.empty_like(q)
    cache = mk.PagedCache(*paged, n_q_heads=hq, workspace=workspace)
    cache.attention(q, mk.PagedBatch(ints(table), ints([0, 1, 71]), ints(lens), page_size=page, max_new=70), out)
    assert cache.status() == 0
    for r, rows in ((0, slice(0, 1)), (1, slice(1, 71))):
        ref, _, wabs, smag, _ = oracle.paged_attention(f64(q[rows]), f64(k[r])[None], f64(v[r])[None], np.zeros((1, 1), int), [0, new[r]],
                                                       [lens[r]], d ** -0.5)
        tol = 2.0 ** -8 * 1.01 * (np.abs(ref) + wabs) + wabs * (2 * d * 2.0 ** -22 * smag[..., None] + 100 * 2.0 ** -23)
        assert (np.abs(f64(out[rows]) - ref) <= tol).all()
