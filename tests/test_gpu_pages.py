"""Shared, copied and given-back pages on the GPU against oracle/tree.py: whole
numbers and moved bits, all equal."""
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


def batch_of(table, page, n=None):
    n = table.shape[0] if n is None else n
    return mk.PagedBatch(table, ints([0] * (n + 1)), ints([0] * n), page_size=page, max_new=1)


def run_fork(table, lens, keep, parents, m, page, shared, free, n_free, copying=True, same_word=False, width=None):
    table = np.array(table)
    n, width = table.shape
    start = np.full((m, width), -5)
    t, s, f, nf = ints(table), ints(shared), ints(free), ints([n_free])
    lens_t, keep_t = ints(lens), None if keep is None else ints(keep)
    next_lens, left, status = ints([77] * m), ints([77]), ints([0])
    copies = ints(np.full((3, m), 77)) if copying else None
    out = nf if same_word else left
    b = batch_of(t, page)
    if parents is None:
        b.trim(lens_t, lens_t if keep is None else keep_t, next_lens, s, f, nf, out, copies=copies, status=status)
        got_table = t
    else:
        got_table = ints(start)
        batch_of(got_table, page).fork(b, ints(parents), lens_t, next_lens, copies, s, f, nf, out, keep=keep_t, status=status)
    want = oracle.paged_fork(table, lens, keep, parents, start, page, shared, free, n_free, copying)
    got = {"table": got_table, "lens": next_lens, "shared": s, "free": f}
    if copying:
        got["copies"] = copies
    for k, v in got.items():
        assert np.array_equal(v.cpu().numpy(), want[k]), k
    assert out.item() == want["n_left"] and status.item() == (mk.MK_ERR_BOUNDS if want["bad"] else 0)
    return want


def make_pool(rng, n, page, width, most, spare, share):
    lens = [rng.randint(0, most) for _ in range(n)]
    need = sum(-(-x // page) for x in lens)
    pages = need + spare
    pool = list(range(pages))
    rng.shuffle(pool)
    table, shared = np.full((n, width), -9), np.zeros(pages, int)
    for s in range(n):
        for b in range(-(-lens[s] // page)):
            o = rng.randrange(max(1, s)) if s else 0
            if s and rng.random() < share and b < min(lens[o], lens[s]) // page and table[o, b] not in table[s]:
                table[s, b] = table[o, b]
                shared[table[s, b]] += 1
            else:
                table[s, b] = pool.pop()
    return table, lens, shared, pool + [-3] * (pages - len(pool)), len(pool)


@pytest.mark.parametrize("n,m,page,most,share,cut", [
    (1, 1, 16, 40, 0, False), (1, 8, 16, 100, 0, False), (5, 5, 32, 200, 0.5, True), (16, 16, 16, 300, 0.8, False), (33, 70, 64, 500, 0.3, True),
    (300, 100, 16, 90, 0.5, True), (3, 40, 128, 9000, 0.2, False), (40, 3, 16, 5000, 0.7, True), (4096, 4096, 16, 40, 0.5, True), (1000, 4096, 32, 200, 0.3, False),
    (4, 2, 256, 60000, 0.5, True)])
@pytest.mark.parametrize("same_word", [False, True])
def test_forks_match_the_oracle(n, m, page, most, share, cut, same_word):
    rng = random.Random(n * 31 + m)
    width = -(-most // page) + 2
    table, lens, shared, free, n_free = make_pool(rng, n, page, width, most, m + 9, share)
    keep = [rng.choice([0, x, rng.randint(0, x), x // page * page]) for x in lens] if cut else None
    parents = [rng.randint(-1 if rng.random() < 0.2 else 0, n - 1) for _ in range(m)]
    want = run_fork(table, lens, keep, parents, m, page, shared, free, n_free, same_word=same_word)
    assert not want["bad"]


@pytest.mark.parametrize("n,page,most,share", [(1, 16, 100, 0), (7, 16, 300, 0), (64, 32, 700, 0.6), (500, 16, 200, 0.4), (4096, 16, 60, 0.5), (3, 16, 30000, 0.5), (2, 256, 70000, 0.9)])
@pytest.mark.parametrize("copying", [False, True])
def test_trims_match_the_oracle(n, page, most, share, copying):
    rng = random.Random(n + most)
    width = -(-most // page) + 1
    table, lens, shared, free, n_free = make_pool(rng, n, page, width, most, n + 3, share)
    keep = [rng.choice([0, x, max(0, x - rng.randint(0, 20)), rng.randint(0, x)]) for x in lens]
    run_fork(table, lens, keep, None, n, page, shared, free, n_free, copying=copying)
    run_fork(table, lens, [0] * n, None, n, page, shared, free, n_free, copying=copying, same_word=True)  # all end
    run_fork(table, lens, None, None, n, page, shared, free, n_free, copying=copying)                     # nothing changes


def test_forks_when_pages_run_out():
    rng = random.Random(8)
    table, lens, shared, free, n_free = make_pool(rng, 6, 16, 8, 100, 30, 0.4)
    parents = [rng.randrange(6) for _ in range(20)]
    for have in (0, 1, 3, 30):
        run_fork(table, lens, None, parents, 20, 16, shared, free, min(have, n_free))
    assert run_fork(table, lens, None, parents, 20, 16, shared, free, 1)["bad"]


def test_bad_arguments_of_forks():
    table, lens, shared, free, n_free = make_pool(random.Random(3), 5, 16, 6, 80, 10, 0.0)
    ok = dict(lens=lens, keep=None, parents=[0, 1, 1, 4, -1], shared=shared, n_free=n_free)

    def call(parents="p", **kw):
        a = {**ok, **kw}
        parents = a["parents"] if parents == "p" else parents
        return run_fork(table if "table" not in kw else kw["table"], a["lens"], a["keep"], parents, 5, 16, a["shared"], free, a["n_free"])["bad"]

    assert not call()
    assert call(parents=[0, 5, -2, 2 ** 31 - 1, 1])
    assert call(lens=[-1] + lens[1:]) and call(lens=[97] + lens[1:], shared=np.ones(len(shared), int))
    assert call(keep=[-4] + lens[1:]) and call(keep=[lens[0] + 1] + lens[1:]) and call(None, keep=[lens[0] + 1] + lens[1:])
    assert call(n_free=-3) and call(n_free=len(free) + 4, parents=[0, 1, 2, 3, 4])
    bad = table.copy()
    for s in range(5):
        if lens[s] > 16:
            bad[s, 0] = -1 if s % 2 else len(shared)
    assert call(parents=[0, 0, 1, 2, 3], table=bad) and call(None, table=bad, keep=[0] * 5)


def test_a_free_list_that_overflows():
    table, lens = [[0, 1, 2], [3, 4, -1]], [48, 20]
    got = run_fork(table, lens, [0, 0], None, 2, 16, [0] * 5, [7, 7, 7], 1)
    assert got["bad"] and got["n_left"] == 3 and got["free"].tolist() == [7, 0, 1]


# ---------------------------------------------------------------- copies, kept tokens

def make_layers(n, pages, hkv, page, d, typ, layout, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    if layout == "hp":
        kv = torch.randn(n, 2, pages, hkv, page, d, generator=g, device=DEV).to(typ)
        views = [(x[0], x[1]) for x in kv]
    elif layout == "ph":
        kv = torch.randn(n, 2, pages, page, hkv, d, generator=g, device=DEV).to(typ)
        views = [(x[0].transpose(1, 2), x[1].transpose(1, 2)) for x in kv]
    else:
        kv = torch.randn(n, pages, 2, hkv, page, d + 8, generator=g, device=DEV).to(typ)
        views = [(x[:, 0, :, :, :d], x[:, 1, :, :, :d]) for x in kv]
    return kv, views, mk.PagedLayers([mk.PagedCache(k, v, n_q_heads=hkv) for k, v in views])


LAYERS = [(1, 1, 16, 64, "hp", "bf16"), (3, 8, 16, 128, "hp", "bf16"), (32, 8, 64, 128, "hp", "fp16"), (2, 3, 32, 64, "ph", "bf16"), (2, 5, 256, 128, "pad", "fp16"),
          (128, 1, 16, 64, "hp", "bf16"), (2, 130, 16, 128, "ph", "bf16")]


@pytest.mark.parametrize("n,hkv,page,d,layout,typ", LAYERS)
def test_copies_move_the_bits_of_the_first_tokens(n, hkv, page, d, layout, typ):
    rng = np.random.default_rng(n + page)
    pages = 30
    kv, views, layers = make_layers(n, pages, hkv, page, d, TYPES[typ], layout, n)
    kv.view(torch.int16)[..., 0] = 0x7fc1  # NaN with a payload
    ids = rng.permutation(pages)
    copies = np.array([[ids[0], -1, ids[1], ids[0], ids[2], ids[3], -1], [ids[10], ids[11], ids[12], ids[13], ids[14], ids[15], -1], [1, 5, page, page - 1, 0, page // 2 + 1, 0]])
    want = kv.clone()
    keys = [(w[0], w[1]) if layout == "hp" else (w[0].transpose(1, 2), w[1].transpose(1, 2)) if layout == "ph" else (w[:, 0, :, :, :d], w[:, 1, :, :, :d]) for w in want]
    for k, v in keys:
        for a, b, t in copies.T:
            if a >= 0:
                k[b, :, :t], v[b, :, :t] = k[a, :, :t].clone(), v[a, :, :t].clone()
    layers.copy(ints(copies))
    assert torch.equal(kv.view(torch.int16), want.view(torch.int16)) and layers.caches[0].status() == 0
    layers.copy(ints(np.zeros((3, 0))))


def test_copies_out_of_range_are_latched():
    kv, _, layers = make_layers(2, 4, 2, 16, 64, torch.bfloat16, "hp", 1)
    for pair, left in (([4, 0, 3], True), ([-2, 0, 3], True), ([1, 4, 3], True), ([1, -1, 3], True), ([1, 2, -1], True), ([1, 2, 17], False)):
        want = kv.clone()
        if not left:
            want[:, :, 2] = want[:, :, 1]
        layers.copy(ints(np.array(pair)[:, None]))
        assert torch.equal(kv, want) and layers.caches[0].status() == mk.MK_ERR_BOUNDS, pair
        layers.caches[0].reset()


@pytest.mark.parametrize("n,hkv,page,d,layout,typ", LAYERS)
def test_kept_tokens_move_together(n, hkv, page, d, layout, typ):
    rng = random.Random(n * 3 + page)
    new = [rng.choice([0, 1, 2, 9, 33, 70]) for _ in range(7)] + [40]
    pages = sum(new) // page + 3
    kv, views, layers = make_layers(n, pages, hkv, page, d, TYPES[typ], layout, n + 1)
    total, pad = sum(new), 3
    slots = rng.sample(range(pages * page), total) + [-1] * pad
    path = []
    for k in new:
        some = [0] + sorted(rng.sample(range(1, k), rng.randint(0, k - 1))) if k else []
        path += some + [-1] * (k - len(some))
    path += [2] * pad
    cu = np.concatenate([[0], np.cumsum(new)])
    want = kv.clone()
    keys = [(w[0], w[1]) if layout == "hp" else (w[0].transpose(1, 2), w[1].transpose(1, 2)) if layout == "ph" else (w[:, 0, :, :, :d], w[:, 1, :, :, :d]) for w in want]
    target = [(slots[c], slots[int(cu[r]) + path[c]]) for r in range(8) for c in range(int(cu[r]), int(cu[r + 1])) if path[c] >= 0]
    for w in keys:
        for x in w:
            old = x.clone()
            for to, of in target:
                x[to // page, :, to % page] = old[of // page, :, of % page]
    b = mk.PagedBatch(ints(np.zeros((8, 9))), ints(cu), ints(new), ints([0] * (total + pad)), ints(slots), page_size=page, max_new=max(new))
    layers.keep(b, ints(path))
    assert torch.equal(kv.view(torch.int16), want.view(torch.int16)) and layers.caches[0].status() == 0


def test_paths_that_are_none_are_latched():
    kv, _, layers = make_layers(1, 4, 2, 16, 64, torch.bfloat16, "hp", 1)

    def call(path, slots, cu, moved, status):
        want, old = kv.clone(), kv.clone()
        for of, to in moved:
            want[:, :, to // 16, :, to % 16] = old[:, :, of // 16, :, of % 16]
        b = mk.PagedBatch(ints(np.zeros((len(cu) - 1, 4))), ints(cu), ints([5] * (len(cu) - 1)), ints([0] * len(slots)), ints(slots), page_size=16, max_new=5)
        layers.keep(b, ints(path))
        assert torch.equal(kv, want) and layers.caches[0].status() == status
        layers.caches[0].reset()

    call([0, 3, -1, 9, -7], [0, 1, 2, 3, 4], [0, 5], [(3, 1)], 0)                       # what is behind the end is not read
    call([0, 2, 2, -1, -1], [0, 1, 2, 3, 4], [0, 5], [(2, 1)], mk.MK_ERR_BOUNDS)        # not increasing
    call([0, 2, 5, -1, -1], [0, 1, 2, 3, 4], [0, 5], [(2, 1)], mk.MK_ERR_BOUNDS)        # no token of the request
    call([-2, 2, 3, -1, -1], [0, 1, 2, 3, 4], [0, 5], [], mk.MK_ERR_BOUNDS)
    call([1, 3, 4, -1, -1], [9, -1, 20, 30, 64], [0, 5], [], mk.MK_ERR_BOUNDS)          # a slot of none, one past the pages
    call([0, 2, -1, 0, 1], [0, 1, 2, 3, 4], [0, 3, 2], [(2, 1)], mk.MK_ERR_BOUNDS)      # offsets that fall
    call([0, 2, -1, 0, 1], [0, 1, 2, 3, 4], [0, 3, 6], [(2, 1)], mk.MK_ERR_BOUNDS)      # or pass the rows


def test_copies_past_32_bit_offsets():
    kv = torch.zeros(2, 4200, 16, 256, 128, dtype=torch.bfloat16, device=DEV)
    assert kv[0].numel() > 2 ** 31
    kv[:, 4199] = torch.randn(2, 16, 256, 128, device=DEV).to(torch.bfloat16)
    layers = mk.PagedLayers([mk.PagedCache(kv[0], kv[1], n_q_heads=16)])
    layers.copy(ints([[4199, 4199], [3, 4198], [256, 100]]))
    assert torch.equal(kv[:, 3], kv[:, 4199]) and torch.equal(kv[:, 4198, :, :100], kv[:, 4199, :, :100]) and not kv[:, 4198, :, 100:].any()
    b = mk.PagedBatch(ints(np.zeros((1, 1))), ints([0, 2]), ints([2]), ints([0, 0]), ints([7 * 256 + 1, 4199 * 256 + 255]), page_size=256, max_new=2)
    layers.keep(b, ints([1, -1]))
    assert torch.equal(kv[:, 7, :, 1], kv[:, 4199, :, 255])


def test_python_refusals_of_pages():
    kv, views, layers = make_layers(2, 4, 2, 16, 64, torch.bfloat16, "hp", 1)
    with pytest.raises(ValueError):
        mk.PagedLayers([])
    other = mk.PagedCache(*(torch.zeros(4, 2, 32, 64, dtype=torch.bfloat16, device=DEV) for _ in range(2)), n_q_heads=2)
    with pytest.raises(ValueError):
        mk.PagedLayers([layers.caches[0], other])
    with pytest.raises(ValueError):
        mk.PagedLayers([layers.caches[0], layers.caches[1], layers.caches[0]])
    for c in (ints([1, 2, 3]), ints(np.zeros((2, 4))), ints(np.zeros((3, 4))).long(), ints(np.zeros((4, 3))).t()):
        with pytest.raises(ValueError):
            layers.copy(c)
    b = mk.PagedBatch(ints(np.zeros((1, 1))), ints([0, 2]), ints([2]), ints([0, 0]), ints([0, 1]), page_size=16, max_new=2)
    for path in (ints([0, 1, 2]), ints([0, 1]).long()):
        with pytest.raises(ValueError):
            layers.keep(b, path)
    with pytest.raises(ValueError):
        layers.keep(batch_of(ints(np.zeros((1, 1))), 16), ints([0, 1]))
    with pytest.raises(mk.MkError):
        layers.keep(mk.PagedBatch(ints(np.zeros((1, 1))), ints([0, 2]), ints([2]), ints([0, 0]), ints([0, 1]), page_size=32, max_new=2), ints([0, 1]))
    a, z = batch_of(ints(np.zeros((2, 3))), 16), batch_of(ints(np.zeros((4, 3))), 16)
    ok = dict(old=a, parents=ints([0, 1, 1, -1]), lens=ints([0, 0]), next_lens=ints([0] * 4), copies=ints(np.zeros((3, 4))), shared=ints([0] * 9), free_pages=ints([0] * 9),
              n_free=ints([0]), n_left=ints([0]))
    z.fork(**ok)
    for kw in (dict(old=z), dict(old=batch_of(ints(np.zeros((2, 4))), 16)), dict(old=batch_of(ints(np.zeros((2, 3))), 32)), dict(parents=None), dict(copies=None),
               dict(parents=ints([0, 1])), dict(lens=ints([0] * 4)), dict(next_lens=ints([0] * 2)), dict(copies=ints(np.zeros((2, 4)))), dict(n_left=ints([0, 0])),
               dict(shared=ok["shared"].long()), dict(keep=ints([0] * 4)), dict(status=ints([0] * 2))):
        with pytest.raises(ValueError):
            z.fork(**{**ok, **kw})
    with pytest.raises(mk.MkError):
        z.fork(**{**ok, "n_left": ok["shared"][:1]})


# ---------------------------------------------------------------- together

@pytest.mark.parametrize("d,hq,hkv,typ,page,captured", [(128, 8, 2, "bf16", 16, False), (64, 12, 4, "fp16", 32, True)])
def test_speculative_steps_give_what_single_steps_give(d, hq, hkv, typ, page, captured):
    """Two layers' caches through prompt, forks and speculative steps: after every step
    the cached keys and values of each request, read through its table, are those that
    appending its emitted tokens one by one gives, no page leaks, and the new tokens'
    attention is the oracle's."""
    rng, typ = random.Random(d), TYPES[typ]
    vocab, layers, width, pages, most = 50, 2, 12, 120, 9
    g = torch.Generator(device=DEV).manual_seed(d)
    emb = torch.randn(layers, vocab, hq + 2 * hkv, d, generator=g, device=DEV).to(typ)  # a token's q, k, v in each layer
    probs = torch.softmax(2 * torch.randn(vocab, vocab, generator=g, device=DEV), -1)   # the target: of the token alone
    draft = torch.softmax(probs.log() + 0.7 * torch.randn(vocab, vocab, generator=g, device=DEV), -1)
    kv = torch.zeros(layers, 2, pages, hkv, page, d, dtype=typ, device=DEV)
    work = torch.full((mk.MK_PAGED_WORKSPACE_BYTES // 4,), float("nan"), device=DEV)
    caches = [mk.PagedCache(x[0], x[1], n_q_heads=hq, workspace=work) for x in kv]
    group, rope = mk.PagedLayers(caches), mk.Rope(d)
    free, count, shared = ints(np.random.default_rng(1).permutation(pages)), ints([pages]), ints([0] * pages)
    left = ints([0])

    def checked(history, lens, table):
        held = {}
        for r, seq in enumerate(history):
            ids = table[r, :-(-len(seq) // page)].tolist()
            for x in ids:
                held[x] = held.get(x, 0) + 1
            assert int(lens[r]) == len(seq)
            if not seq:
                continue
            t = torch.tensor(seq, device=DEV)
            for l in range(layers):
                fresh = mk.PagedCache(*(torch.zeros(len(ids), hkv, page, d, dtype=typ, device=DEV) for _ in range(2)), n_q_heads=hq)
                rows = emb[l, t]
                fresh.append(rows[:, :hq].contiguous(), rows[:, hq:hq + hkv], rows[:, hq + hkv:], ints(np.arange(len(seq))), ints(np.arange(len(seq))), rope,
                             q_out=torch.empty(len(seq), hq, d, dtype=typ, device=DEV))
                for mine, want in ((kv[l, 0], fresh.k), (kv[l, 1], fresh.v)):
                    flat = lambda x, i: x[i].transpose(1, 2).reshape(-1, hkv, d)[:len(seq)]  # noqa: E731
                    assert torch.equal(flat(mine, ids), flat(want, list(range(len(ids)))))
        assert count.item() + len(held) == pages
        assert all(int(shared[x]) == held.get(x, 1) - 1 for x in range(pages))

    # prompts of two requests
    history = [[rng.randrange(vocab) for _ in range(k)] for k in (page + 5, 2 * page)]
    table = torch.full((2, width), -1, dtype=torch.int32, device=DEV)
    new = [len(h) for h in history]
    b = mk.PagedBatch(table, ints([0] * 3), ints([0] * 2), ints([0] * sum(new)), ints([0] * sum(new)), page_size=page, max_new=max(new))
    b.build(ints([0, 0]), ints(new), free, count, left)
    count.copy_(left)
    t = torch.tensor(sum(history, []), device=DEV)
    for l in range(layers):
        rows = emb[l, t]
        caches[l].append(rows[:, :hq].contiguous(), rows[:, hq:hq + hkv], rows[:, hq + hkv:], b.slots, b.positions, rope, q_out=torch.empty(len(t), hq, d, dtype=typ, device=DEV))
    lens = ints(new)
    checked(history, lens, table)
    # five answers: three of the first, two of the second
    parents = [0, 1, 0, 0, 1]
    n = len(parents)
    table, lens_n, copies = torch.full((n, width), -1, dtype=torch.int32, device=DEV), ints([0] * n), ints(np.zeros((3, n)))
    rows_most = n * most
    step = mk.PagedBatch(table, ints([0] * (n + 1)), ints([0] * n), ints([0] * rows_most), ints([0] * rows_most), page_size=page, max_new=most)
    step.fork(b, ints(parents), lens, lens_n, copies, shared, free, count, count)
    group.copy(copies)
    lens, history = lens_n, [list(history[x]) for x in parents]
    checked(history, lens, table)

    # a speculative step on fixed buffers, so that it can be captured
    up, toks = ints([0] * rows_most), ints([0] * rows_most)
    masks, u, ul = ints(np.zeros((rows_most, 1))), torch.zeros(rows_most, device=DEV), torch.zeros(n, device=DEV)
    tree = mk.DraftTree(step, up, masks)
    path, emitted, kept, after, next_lens, news = ints([0] * rows_most), ints([0] * rows_most), ints([0] * n), ints([0] * n), ints([0] * n), ints([0] * n)
    qs = [torch.zeros(rows_most, hq, d, dtype=typ, device=DEV) for _ in range(layers)]
    outs = [torch.zeros(rows_most, hq, d, dtype=typ, device=DEV) for _ in range(layers)]

    def one():
        step.build(lens, news, free, count, left)
        tree.build()
        for l in range(layers):
            rows = emb[l][toks.long()]
            caches[l].append(rows[:, :hq].contiguous(), rows[:, hq:hq + hkv], rows[:, hq + hkv:], step.slots, step.positions, rope, q_out=qs[l])
            caches[l].attention(qs[l], step, outs[l], tree=tree)
        tree.verify(toks, probs[toks.long()], u, ul, path, emitted, kept, after, draft_probs=draft[toks.long()])
        group.keep(step, path)
        step.trim(step.kv_lens, after, next_lens, shared, free, left, count)

    graph = None
    accepted = 0
    for it in range(7):
        drafts = [trees.grow(rng, rng.randint(1, most)) for _ in range(n)]
        roots = [rng.randrange(vocab) for _ in history] if it == 0 else nexts
        row_toks, cu = [], [0]
        for r in range(n):
            mine = [roots[r]]
            for p in drafts[r][1:]:
                w = draft[mine[p]].double().cpu().numpy()
                mine.append(int(np.searchsorted(np.cumsum(w) / w.sum(), rng.random())))
            row_toks += mine
            cu.append(cu[-1] + len(mine))
        k = cu[-1]
        fill = lambda dst, v: dst[:len(v)].copy_(torch.tensor(v, dtype=dst.dtype))  # noqa: E731
        fill(up, sum(drafts, []))
        fill(toks, row_toks)
        fill(u, [rng.random() for _ in range(rows_most)])
        fill(ul, [rng.random() for _ in range(n)])
        fill(news, [len(x) for x in drafts])
        before_lens = lens.tolist()
        if captured and graph is None and it == 1:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                one()
        if graph is not None:
            graph.replay()
        else:
            one()
        torch.cuda.synchronize()
        assert all(c.status() == 0 for c in caches)
        # attention: the new tokens' keys are the append's, before any moved
        for l in range(layers):
            for r in range(n):
                seq = history[r]
                masks_r = masks[cu[r]:cu[r + 1]].cpu().numpy().view(np.uint32)
                pos = [before_lens[r] + len(a) - 1 for a in oracle.ancestors(drafts[r])]
                assert step.positions[cu[r]:cu[r + 1]].tolist() == pos
                t = torch.tensor(seq + row_toks[cu[r]:cu[r + 1]], device=DEV)
                fresh = mk.PagedCache(*(torch.zeros(-(-len(t) // page), hkv, page, d, dtype=typ, device=DEV) for _ in range(2)), n_q_heads=hq)
                rows = emb[l, t]
                fresh.append(rows[:, :hq].contiguous(), rows[:, hq:hq + hkv], rows[:, hq + hkv:], ints(np.arange(len(t))), ints(list(range(len(seq))) + pos), rope,
                             q_out=torch.empty(len(t), hq, d, dtype=typ, device=DEV))
                blocks = np.arange(len(fresh.k))[None]
                ref, _, wabs, smag, vmax = oracle.tree_attention(f64(qs[l][cu[r]:cu[r + 1]]), f64(fresh.k), f64(fresh.v), blocks, [0, len(pos)], [len(t)], masks_r, d ** -0.5)
                err = np.abs(f64(outs[l][cu[r]:cu[r + 1]]) - ref)
                un = torch.finfo(typ).eps / 2
                tol = un * 1.01 * (np.abs(ref) + wabs) + wabs * (2 * d * 2.0 ** -22 * smag[..., None] + (len(t) / 8 + 64) * 2.0 ** -23) + len(t) * 2.0 ** -25 * vmax[..., None] + 2.0 ** -24
                assert (err <= tol).all()
        got_kept, got_emitted, nexts = kept.tolist(), emitted.tolist(), []
        for r in range(n):
            t = row_toks[cu[r]:cu[r + 1]]
            idx = torch.tensor(t, device=DEV)
            want_path, want, bad = oracle.tree_verify(drafts[r], t, f64(probs[idx]), f64(draft[idx]), u[cu[r]:cu[r + 1]].tolist(), ul[r].item())
            assert not bad and got_kept[r] == len(want) and got_emitted[cu[r]:cu[r] + len(want)] == want
            history[r] += [t[i] for i in want_path]
            nexts.append(want[-1])
            accepted += len(want) - 1
        lens.copy_(next_lens)
        checked(history, lens, table)
    assert accepted > 5
    # everything ends
    step.trim(lens, ints([0] * n), next_lens, shared, free, count, count)
    assert count.item() == pages and not shared.any() and sorted(free.tolist()) == list(range(pages))
