"""Trees of drafted tokens and shared pages: refusals of the entry points (checked
before anything is launched, so on the CPU with addresses that are never read), and
the oracle against closed forms.  No GPU needed."""
import ctypes
import random
from fractions import Fraction

import numpy as np
import pytest

import oracle
from tile_level_overlap_gb300 import build, mk

ADDR = 1 << 20  # an aligned address that no refused call reads


@pytest.fixture(scope="module")
def lib():
    build.build()
    return mk.lib()


def at(i):
    return ADDR + (i << 16)


def cache(**kw):
    f = dict(k=ADDR, v=ADDR, workspace=ADDR, status=None, page_stride=16 * 8 * 128, head_stride=16 * 128, token_stride=128,
             n_q_heads=32, n_kv_heads=8, head_dim=128, page_size=16, n_pages=100, dtype=mk.MK_BF16)
    f.update(kw)
    return mk.mk_paged_cache(*[f[n] for n, _ in mk.mk_paged_cache._fields_])


def batch(**kw):
    f = dict(block_table=at(20), cu_new=at(21), kv_lens=at(22), positions=at(23), slots=at(24), n=4, max_blocks=8, max_tokens=0, max_new=1,
             page_size=16)
    f.update(kw)
    return mk.mk_paged_batch(*[f[n] for n, _ in mk.mk_paged_batch._fields_])


BAD_BATCH = [(dict(block_table=None), 1), (dict(cu_new=None), 1), (dict(kv_lens=None), 1), (dict(n=0), 1), (dict(max_tokens=-1), 1),
             (dict(n=mk.MK_PAGED_MAX_REQUESTS + 1), 5), (dict(page_size=17), 5)]


def test_tree_refusals(lib):
    ok = dict(b=ctypes.byref(batch()), parents=at(1), masks=at(2), words=2, positions=at(3), status=None)

    def call(**kw):
        return lib.mk_paged_tree(*{**ok, **kw}.values(), None)

    assert call() == 0  # no rows: nothing is launched
    for kw, code in BAD_BATCH:
        assert call(b=ctypes.byref(batch(**kw))) == code
    for kw in (dict(b=None), dict(parents=None), dict(masks=None), dict(positions=None), dict(words=0), dict(words=-1), dict(parents=at(1) + 2),
               dict(masks=at(2) + 1), dict(status=3)):
        assert call(**kw) == 1, kw
    assert call(words=33) == 5
    big = ctypes.byref(batch(max_tokens=100))
    for kw in (dict(masks=at(1)), dict(positions=at(1) + 396), dict(positions=at(2) + 796), dict(masks=at(21)), dict(positions=at(22)),
               dict(status=at(2) + 796)):
        assert call(b=big, **kw) == 1, kw


def test_tree_attention_refusals(lib):
    ok = dict(c=ctypes.byref(cache()), b=ctypes.byref(batch()), masks=at(1), words=1, q=at(2), qs=4096, out=at(3), os=4096, lse=None, scale=0.0, window=0)

    def call(**kw):
        return lib.mk_paged_tree_attention(*{**ok, **kw}.values(), None)

    assert call() == 0
    for kw in (dict(c=None), dict(b=None), dict(masks=None), dict(masks=at(1) + 2), dict(words=0), dict(q=None), dict(out=at(2)), dict(qs=4092),
               dict(window=-1), dict(lse=2), dict(c=ctypes.byref(cache(workspace=None)))):
        assert call(**kw) == 1, kw
    assert call(words=33) == 5
    assert call(c=ctypes.byref(cache(head_dim=96))) == 5


def test_verify_refusals(lib):
    ok = dict(b=ctypes.byref(batch()), parents=at(1), tokens=at(2), p=at(3), ps=100, q=at(4), qs=100, vocab=100, u=at(5), ul=at(6), path=at(7),
              emitted=at(8), kept=at(9), lens=at(10), status=at(11))

    def call(**kw):
        return lib.mk_tree_verify(*{**ok, **kw}.values(), None)

    for kw, code in BAD_BATCH:
        assert call(b=ctypes.byref(batch(**kw))) == code
    for name in ("b", "parents", "tokens", "p", "u", "ul", "path", "emitted", "kept", "lens"):
        assert call(**{name: None}) == 1, name
    for kw in (dict(vocab=0), dict(vocab=-5), dict(ps=99), dict(qs=99), dict(tokens=at(2) + 1), dict(q=at(4) + 2), dict(status=at(11) + 3),
               dict(kept=at(9) + 2)):
        assert call(**kw) == 1, kw
    assert call(vocab=(1 << 24) + 1, ps=1 << 25, qs=1 << 25) == 5
    assert call(ps=1 << 38) == 5 and call(qs=1 << 38) == 5
    big = ctypes.byref(batch(max_tokens=10))
    for kw in (dict(path=at(8)), dict(path=at(8) + 36), dict(kept=at(10) + 12), dict(emitted=at(1)), dict(lens=at(22)), dict(path=at(3) + 3960),
               dict(path=at(4) + 3600), dict(emitted=at(5)), dict(kept=at(6)), dict(status=at(7)), dict(lens=at(21))):
        assert call(b=big, **kw) == 1, kw


def fork_args(**kw):
    f = dict(table=at(1), n=4, lens=at(2), keep=None, parents=at(3), next=at(4), next_lens=at(5), m=6, width=8, page=16, copies=at(6), shared=at(7),
             n_pages=100, free=at(8), cap=100, n_free=at(9), n_left=at(10), status=None)
    f.update(kw)
    return f


def test_fork_refusals(lib):
    def call(**kw):
        return lib.mk_paged_fork(*fork_args(**kw).values(), None)

    for name in ("table", "lens", "next", "next_lens", "shared", "free", "n_free", "n_left"):
        assert call(**{name: None}) == 1, name
    for kw in (dict(n=0), dict(m=0), dict(width=0), dict(n_pages=0), dict(cap=-1), dict(lens=at(2) + 2), dict(status=at(11) + 1),
               dict(parents=None), dict(parents=None, m=4), dict(parents=None, next=at(1)), dict(next=at(1)), dict(next_lens=at(2)),
               dict(keep=at(5)), dict(copies=at(3)), dict(shared=at(8)), dict(n_left=at(8) + 8), dict(status=at(7) + 4), dict(free=at(9)),
               dict(copies=at(4) + 188), dict(n_left=at(2))):
        assert call(**kw) == 1, kw
    for kw in (dict(page=8), dict(page=48), dict(n=4097), dict(m=4097), dict(width=1 << 27), dict(m=4096, width=1 << 20)):
        assert call(**kw) == 5, kw


def test_layers_refusals(lib):
    rows = (ctypes.c_void_p * 3)(ADDR, 2 * ADDR, 3 * ADDR)

    def copy(c=None, ks=rows, vs=rows, n=3, copies=at(1), m=0):
        return lib.mk_paged_copy(ctypes.byref(c or cache()), ks, vs, n, copies, m, None)

    def keep(c=None, ks=rows, vs=rows, n=3, b=None, path=at(1)):
        return lib.mk_paged_keep(ctypes.byref(c or cache()), ks, vs, n, ctypes.byref(b or batch()), path, None)

    assert copy() == 0 and keep() == 0  # nothing to move: nothing is launched
    for f in (copy, keep):
        for c, code in ((cache(k=None), 1), (cache(page_stride=100), 1), (cache(head_dim=96), 5), (cache(page_size=8), 5), (cache(dtype=2), 1)):
            assert f(c) == code
        assert f(ks=None) == 1 and f(vs=None) == 1 and f(n=0) == 1 and f(n=129) == 5
        for row in ((ADDR, None, ADDR), (ADDR, ADDR + 8, ADDR)):
            bad = (ctypes.c_void_p * 3)(*row)
            assert f(ks=bad) == 1 and f(vs=bad) == 1
    assert copy(copies=None) == 1 and copy(copies=at(1) + 2) == 1 and copy(m=-1) == 1 and copy(m=4097) == 5
    assert keep(path=None) == 1 and keep(path=at(1) + 1) == 1
    for kw, code in BAD_BATCH:
        assert keep(b=batch(**kw)) == code
    assert keep(b=batch(page_size=32)) == 1
    assert keep(b=batch(max_tokens=5, slots=None)) == 1 and keep(b=batch(max_tokens=5, slots=ADDR + 2)) == 1


# ---------------------------------------------------------------- the oracle

def outcomes(parents, p, q, steps):
    """Distribution of the first emitted token of a tree whose root's children are
    drawn from q (or, q None, are the tokens 0, 1, ..): every draw of tokens with its
    probability, every uniform number in the middle of one of `steps` cells."""
    vocab, drawn = p.shape[1], len(parents) - 1
    found = np.zeros(vocab)
    cells = (np.arange(steps) + 0.5) / steps
    for code in range(vocab ** drawn if q is not None else 1):
        tokens = [0] + [code // vocab ** i % vocab if q is not None else i for i in range(drawn)]
        weight = np.prod([q[0, t] for t in tokens[1:]]) if q is not None else 1.0
        for uc in range(steps ** drawn):
            u = [0.0] + [cells[uc // steps ** i % steps] for i in range(drawn)]
            for ul in cells:
                _, emitted, _ = oracle.tree_verify(parents, tokens, p, q, u, ul)
                found[emitted[0]] += weight / steps ** (drawn + 1)
    return found


@pytest.mark.parametrize("drawn", [True, False])
def test_oracle_emits_the_targets_distribution(drawn):
    # two children of the root; all probabilities are multiples of 1/4 of what they are
    # compared with, so that cells of 1/12 of the uniform numbers are exact
    p = np.tile([[0.5, 0.25, 0.25]], (3, 1))
    q = np.tile([[0.25, 0.5, 0.25]], (3, 1)) if drawn else None
    got = outcomes([-1, 0, 0], p, q, 12)
    assert np.abs(got - p[0]).max() < 1e-12


def test_oracle_follows_the_tree():
    p = np.eye(5)[[3, 1, 4, 0, 2]]
    parents, tokens = [-1, 0, 0, 2, 2, 3], [9, 1, 3, 0, 4, 0]
    # greedy: the target wants 3 (row 2), there 4 (row 4), there 2
    assert oracle.tree_verify(parents, tokens, p[[0, 1, 2, 3, 4, 0]], None, [0.9] * 6, 0.5) == ([0, 2, 4], [3, 4, 2], False)
    assert oracle.tree_verify([-1], [0], p[:1], None, [0.0], 0.999) == ([0], [3], False)


def test_oracle_masks_and_forks():
    masks, pos, bad = oracle.paged_tree([-1, 0, 0, 1, 3], [0, 5], [12], 1, 6, np.zeros((6, 1), np.uint32), np.full(6, 9))
    assert masks[:5, 0].tolist() == [1, 3, 5, 0b1011, 0b11011] and pos.tolist() == [7, 8, 8, 9, 10, 0] and not bad
    seen = oracle.tree_seen(masks[:5], 5, 8, 2)
    assert seen[4].tolist() == [False] * 6 + [True] * 2 and seen[2].tolist() == [False, False, False, True, False, True, False, False]
    # a prompt of 20 tokens in pages of 16 goes on three times, another ends
    got = oracle.paged_fork([[7, 3], [5, -1]], [20, 9], None, [0, 0, -1, 0], np.full((4, 2), -2), 16, np.zeros(9), [0, 1, 2, 0], 3)
    assert got["table"].tolist() == [[7, 3], [7, 2], [-2, -2], [7, 1]] and got["lens"].tolist() == [20, 20, 0, 20]
    assert got["copies"].tolist() == [[-1, 3, -1, 3], [-1, 2, -1, 1], [0, 4, 0, 4]]
    assert got["shared"].tolist() == [0] * 7 + [2, 0] and got["free"].tolist() == [0, 5, 2, 0] and got["n_left"] == 2 and not got["bad"]


def test_oracle_conserves_pages():
    rng = random.Random(4)
    for _ in range(200):
        n, page, width = rng.randint(1, 5), 16, 4
        lens = [rng.randint(0, 60) for _ in range(n)]
        pool = list(range(40))
        rng.shuffle(pool)
        table, shared = [[-1] * width for _ in range(n)], [0] * 40
        for s in range(n):
            for b in range(-(-lens[s] // page)):
                if s and rng.random() < 0.3 and b < lens[s - 1] // page and b < lens[s] // page:
                    table[s][b] = table[s - 1][b]
                    shared[table[s][b]] += 1
                else:
                    table[s][b] = pool.pop()
        in_place = rng.random() < 0.4
        m = n if in_place else rng.randint(1, 7)
        parents = None if in_place else [rng.randint(-1, n - 1) for _ in range(m)]
        keep = [rng.randint(0, x) for x in lens]
        got = oracle.paged_fork(table, lens, keep, parents, np.full((m, width), -1), page, shared, pool + [0] * (40 - len(pool)), len(pool))
        holders = {}
        for i in range(m):
            for b in range(-(-int(got["lens"][i]) // page)):
                holders[int(got["table"][i, b])] = holders.get(int(got["table"][i, b]), 0) + 1
        free = got["free"][:got["n_left"]].tolist()
        assert len(set(free)) == len(free) and not set(free) & set(holders) and len(free) + len(holders) == 40
        assert all(got["shared"][x] == holders.get(x, 1) - 1 for x in range(40))
        for i in range(m):  # the page that the next token goes to has one holder
            if got["lens"][i] % page:
                assert holders[int(got["table"][i, got["lens"][i] // page])] == 1
