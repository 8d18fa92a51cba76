"""Steps that have chunks of prompts beside trees of drafted tokens, through
verification, keep and trim.  Paths, tokens and lengths are whole numbers, equal."""
import random

import numpy as np
import pytest
import torch

import oracle
import test_gpu_paged as paged
import test_gpu_tree as trees
from tile_level_overlap_gb300 import build, mk

pytestmark = pytest.mark.gpu
DEV, TYPES = paged.DEV, paged.TYPES
ints, f64 = paged.ints, paged.f64


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    build.build()
    mk.lib()


def expected(new, kv, words, parents, tokens, p, q, u, ul, rows):
    """What verification writes, over arrays of 55."""
    cu = np.concatenate([[0], np.cumsum(new)])
    path, emitted = np.full(rows, 55), np.full(rows, 55)
    kept, lens, bad = np.zeros(len(new), int), np.array(kv), False
    for r, k in enumerate(new):
        a, b = cu[r], cu[r + 1]
        path[a:b] = emitted[a:b] = -1
        if k == 0 or kv[r] < k:
            continue
        if k > 32 * words:  # a chunk: all of it stands, its last row says what follows
            _, e, none = oracle.tree_verify([-1], [0], p[b - 1:b], None, [0.0], ul[r])
            path[a:b], emitted[b - 1], kept[r] = np.arange(k), -1 if none else e[0], k
            continue
        x, e, wrong = oracle.tree_verify(parents[a:b], tokens[a:b], p[a:b], None if q is None else q[a:b], u[a:b], ul[r])
        path[a:a + len(x)], emitted[a:a + len(e)] = x, e
        kept[r], lens[r] = len(x), kv[r] - k + len(x)
        bad |= wrong
    return path, emitted, kept, lens, bad


def make(new, words, vocab, drawn, seed):
    rng, r = np.random.default_rng(seed), random.Random(seed)
    total = sum(new)
    # (the rows of chunks have parents and tokens that are none: they are not read)
    parents = sum((trees.grow(r, k, width=4)[:k] if k <= 32 * words else [9999] * k for k in new), [])
    p = trees.rows_of(rng, total, vocab, "soft")
    q = (0.7 * p + 0.3 * trees.rows_of(rng, total, vocab, "soft")).astype(np.float32) if drawn else None
    tokens = [-7 if k > 32 * words else int(rng.integers(0, vocab)) for k in new for _ in range(k)]
    return parents, tokens, p, q, rng.random(total).astype(np.float32), rng.random(len(new)).astype(np.float32)


def verify(new, kv, words, parents, tokens, p, q, u, ul, pad=0):
    rows = sum(new) + pad
    cu = np.concatenate([[0], np.cumsum(new)])
    b = mk.PagedBatch(ints(np.zeros((len(new), 1))), ints(cu), ints(kv), page_size=16, max_new=max([1, *new]))
    more = lambda x, v: list(x) + [v] * pad  # noqa: E731
    rows_in = lambda x: None if x is None else torch.cat([torch.as_tensor(x), torch.full((pad, x.shape[1]), float("nan"))]).to(DEV)  # noqa: E731
    f32 = lambda x: torch.tensor(np.asarray(x, np.float32)).to(DEV)  # noqa: E731
    tree = mk.DraftTree(b, ints(more(parents, 3)), ints(np.zeros((rows, words))))
    outs, status = (ints([55] * rows), ints([55] * rows), ints([55] * len(new)), ints([55] * len(new))), ints([0])
    tree.verify(ints(more(tokens, 3)), rows_in(p), f32(more(u, 0.5)), f32(ul), *outs, draft_probs=rows_in(q), status=status)
    return [t.cpu().numpy() for t in outs], status.item()


@pytest.mark.parametrize("drawn", [True, False])
@pytest.mark.parametrize("new,words,vocab", [
    ([5, 33, 1, 40], 1, 50), ([33], 1, 1), ([32, 33, 0, 64, 65], 2, 1001), ([1024, 1025, 7, 2500], 32, 40), ([9, 1024, 3000], 4, 127), ([700], 2, 128256)])
def test_chunks_stand_beside_trees(new, words, vocab, drawn):
    case = make(new, words, vocab, drawn, vocab + drawn)
    kv = [k + 11 * i for i, k in enumerate(new)]
    got, status = verify(new, kv, words, *case, pad=3)
    *want, bad = expected(new, kv, words, *case, rows=sum(new) + 3)
    for name, g, w in zip(("path", "emitted", "kept", "lens"), got, want):
        assert np.array_equal(g, w), name
    assert not bad and status == 0


def test_chunks_that_were_refused_or_have_no_mass():
    new, words = [40, 3, 50, 1500, 2], 1
    parents, tokens, p, q, u, ul = make(new, words, 60, False, 4)
    p[39], p[92] = 0, float("nan")  # the last rows of the first two chunks: a prompt's middle, nothing follows
    for kv in ([40, 3, 50, 1500, 2], [0, 9, 50, 1499, 9], [100, 0, 0, 3000, 2]):
        got, status = verify(new, kv, words, parents, tokens, p, None, u, ul)
        *want, bad = expected(new, kv, words, parents, tokens, p, None, u, ul, sum(new))
        for name, g, w in zip(("path", "emitted", "kept", "lens"), got, want):
            assert np.array_equal(g, w), name
        assert not bad and status == 0


@pytest.mark.parametrize("captured", [False, True])
def test_a_step_of_trees_and_chunks(captured):
    """Tables, masks, append, attention, verification, keep and trim of two chunks and
    two trees: the chunks keep all their tokens and pages, the trees their paths."""
    hq, hkv, d, page, vocab, width, typ = 8, 2, 64, 16, 30, 90, torch.bfloat16
    ctx, new = [37, 0, 20, 64], [9, 40, 5, 1200]
    rng, n, total = random.Random(1), 4, sum(new)
    g = torch.Generator(device=DEV).manual_seed(2)
    pages = 140
    caches = [mk.PagedCache(*torch.randn(2, pages, hkv, page, d, generator=g, device=DEV).to(typ), n_q_heads=hq) for _ in range(2)]
    group = mk.PagedLayers(caches)
    free, shared = np.random.default_rng(3).permutation(pages), ints([0] * pages)
    table = np.full((n, width), -1)
    at = pages
    for r, c in enumerate(ctx):
        for b in range(-(-c // page)):
            at -= 1
            table[r, b] = free[at]
    table, free, count, left = ints(table), ints(free), ints([at]), ints([0])
    start = [t.clone() for t in (table, free, count)] + [c.k.clone() for c in caches] + [c.v.clone() for c in caches]
    b = mk.PagedBatch(table, ints([0] * 5), ints([0] * 4), ints([0] * total), ints([0] * total), page_size=page, max_new=max(new))
    up = sum((trees.grow(rng, k) if k <= 32 else [-1] * k for k in new), [])
    tree = mk.DraftTree(b, ints(up), ints(np.zeros((total, 1))))
    q, k, v = (torch.randn(total, h, d, generator=g, device=DEV).to(typ) for h in (hq, hkv, hkv))
    p = torch.softmax(torch.randn(total, vocab, generator=g, device=DEV), -1)
    tokens, u, ul = ints([rng.randrange(vocab) for _ in range(total)]), torch.rand(total, generator=g, device=DEV) * 0.02, torch.rand(n, generator=g, device=DEV)
    path, emitted, kept, after, lens = ints([9] * total), ints([9] * total), ints([9] * n), ints([9] * n), ints([9] * n)
    ctx_t, new_t, out, status = ints(ctx), ints(new), torch.empty_like(q), ints([0])

    def step():
        b.build(ctx_t, new_t, free, count, left, status=status)
        tree.build(status=status)
        for c in caches:
            c.append(q, k, v, b.slots, q_out=torch.empty_like(q))
            c.attention(q, b, out, tree=tree)
        tree.verify(tokens, p, u, ul, path, emitted, kept, after, draft_probs=p, status=status)
        group.keep(b, path)
        b.trim(b.kv_lens, after, lens, shared, free, left, count, status=status)

    step()
    if captured:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        for t, s in zip([table, free, count] + [c.k for c in caches] + [c.v for c in caches], start):
            t.copy_(s)
        for t in (path, emitted, kept, after, lens):
            t.fill_(9)
        graph.replay()
    assert status.item() == 0 and all(c.status() == 0 for c in caches)
    cu = np.concatenate([[0], np.cumsum(new)])
    want = expected(new, [c + k for c, k in zip(ctx, new)], 1, up, tokens.tolist(), f64(p), f64(p), u.tolist(), ul.tolist(), total)
    for name, t, w in zip(("path", "emitted", "kept", "lens"), (path, emitted, kept, after), want):
        assert np.array_equal(t.cpu().numpy(), w), name
    assert lens.tolist() == after.tolist() == [c + x for c, x in zip(ctx, kept.tolist())]
    assert kept[1] == 40 and kept[3] == 1200 and kept[0] > 1
    # no page leaks, none is held twice, and the cached tokens are those that stand
    ids = [table[r, :-(-x // page)].tolist() for r, x in enumerate(lens.tolist())]
    assert sorted(sum(ids, []) + free[:count.item()].tolist()) == list(range(pages)) and not shared.any()
    for c in caches:
        for r in range(n):
            rows = torch.tensor([cu[r] + x for x in path[cu[r]:cu[r] + kept[r]].tolist()], device=DEV)
            for mine, was in ((c.k, k), (c.v, v)):
                flat = mine[ids[r]].transpose(1, 2).reshape(-1, hkv, d)[ctx[r]:lens[r]]
                assert torch.equal(flat, was[rows])


def test_without_masks_every_request_is_a_tree():
    new = [40, 1]
    parents, tokens, p, _, u, ul = make(new, 2, 30, False, 8)
    trees.run_verify([parents[:40], parents[40:]], tokens, p, None, u, ul)


def test_steps_without_rows():
    """Buffers of no rows, every request rests."""
    b = mk.PagedBatch(ints(np.full((2, 3), -1)), ints([0] * 3), ints([0] * 2), ints([]), ints([]), page_size=16, max_new=4)
    status = ints([0])
    b.build(ints([5, 20]), ints([0, 0]), ints([0] * 4), ints([4]), ints([0]), status=status)
    tree = mk.DraftTree(b, ints([]), ints(np.zeros((0, 1))))
    tree.build(status=status)
    kept, lens = ints([9, 9]), ints([9, 9])
    tree.verify(ints([]), torch.zeros(0, 7, device=DEV), torch.zeros(0, device=DEV), torch.zeros(2, device=DEV), ints([]), ints([]), kept, lens, status=status)
    assert kept.tolist() == [0, 0] and lens.tolist() == [5, 20] and status.item() == 0
    q = torch.zeros(0, 4, 64, dtype=torch.bfloat16, device=DEV)
    cache = mk.PagedCache(*(torch.zeros(3, 2, 16, 64, dtype=torch.bfloat16, device=DEV) for _ in range(2)), n_q_heads=4)
    cache.attention(q, b, q.clone(), tree=tree)
    mk.PagedLayers([cache]).keep(b, ints([]))


def test_requests_that_find_no_free_page_keep_their_context():
    """The tables refuse a request when the pages run out (kv_lens 0): with its own
    lengths in their place trim leaves it as it was, and no page leaks."""
    hq, hkv, d, page, vocab, typ = 4, 2, 64, 16, 20, torch.bfloat16
    ctx, new, words = [30, 15, 47, 16], [8, 20, 33, 0], 1  # one page more, two, a chunk that needs two, none
    n, total, pages = 4, sum(new), 10
    held = [-(-c // page) for c in ctx]  # 2, 1, 3, 1: three are free
    table, at = np.full((n, 6), -1), pages
    for r in range(n):
        for b in range(held[r]):
            at -= 1
            table[r, b] = at
    table, free, count, left, shared = ints(table), ints(list(range(at)) + [-1] * (pages - at)), ints([at]), ints([0]), ints([0] * pages)
    before, status = table.clone(), ints([0])
    b = mk.PagedBatch(table, ints([0] * 5), ints([0] * 4), ints([0] * total), ints([0] * total), page_size=page, max_new=max(new))
    tree = mk.DraftTree(b, ints(sum(([i - 1 for i in range(k)] for k in new), [])), ints(np.zeros((total, words))))
    cache = mk.PagedCache(*(torch.zeros(pages, hkv, page, d, dtype=typ, device=DEV) for _ in range(2)), n_q_heads=hq)
    ctx_t, p = ints(ctx), torch.full((total, vocab), 1 / vocab, device=DEV)
    path, emitted, kept, after, lens = ints([9] * total), ints([9] * total), ints([9] * n), ints([9] * n), ints([9] * n)
    b.build(ctx_t, ints(new), free, count, left, status=status)
    assert status.item() == mk.MK_ERR_BOUNDS and b.kv_lens.tolist() == [38, 35, 0, 16]
    tree.build()
    x = torch.ones(total, hq, d, dtype=typ, device=DEV)
    cache.append(x, x[:, :hkv].contiguous(), x[:, :hkv].contiguous(), b.slots)
    cache.attention(x, b, torch.empty_like(x), tree=tree)
    tree.verify(ints([1] * total), p, torch.zeros(total, device=DEV), torch.zeros(n, device=DEV), path, emitted, kept, after)
    mk.PagedLayers([cache]).keep(b, path)
    assert kept.tolist() == [8, 20, 0, 0] and cache.status() == 0
    mine = [torch.where(kept > 0, t, ctx_t) for t in (b.kv_lens, after)]
    b.trim(*mine, lens, shared, free, left, count)
    assert lens.tolist() == [38, 35, 47, 16]
    assert torch.equal(table[2], before[2])
    ids = [table[r, :-(-c // page)].tolist() for r, c in enumerate(lens.tolist())]
    assert sorted(sum(ids, []) + free[:count.item()].tolist()) == list(range(pages)) and not shared.any()
