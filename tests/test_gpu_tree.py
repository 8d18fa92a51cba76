"""Trees of drafted tokens on the GPU against oracle/tree.py (float64, exact
fractions for the verification).  Attention has the tolerances of
test_gpu_paged.py; masks, positions, paths and tokens are whole numbers, equal."""
import random

import numpy as np
import pytest
import torch

import oracle
import test_gpu_paged as paged
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


@pytest.fixture(scope="module")
def workspace():
    return torch.full((mk.MK_PAGED_WORKSPACE_BYTES // 4,), float("nan"), device=DEV)


def grow(rng, nodes, chain=False, width=None):
    return [-1] + [i - 1 if chain or rng.random() < 0.5 else rng.randrange(max(0, i - (width or i)), i) for i in range(1, nodes)]


def words_of(x):
    """uint32 masks as the int32 that torch has."""
    return torch.from_numpy(np.ascontiguousarray(x).astype(np.uint32).view(np.int32)).to(DEV)


# ---------------------------------------------------------------- masks, positions

def run_tree(new, kv, parents, words, rows, cu=None):
    cu = np.concatenate([[0], np.cumsum(new)]) if cu is None else np.array(cu)
    width = max(1, -(-max(kv) // 16))
    b = mk.PagedBatch(ints(np.zeros((len(new), width))), ints(cu), ints(kv), ints(np.full(rows, 77)), ints(np.zeros(rows)), page_size=16, max_new=max([1, *new]))
    start = np.full((rows, words), 0xabcd1234, np.uint32)
    status = ints([0])
    tree = mk.DraftTree(b, ints(parents), words_of(start))
    tree.build(status=status)
    masks, pos, bad = oracle.paged_tree(parents, cu, kv, words, rows, start, np.full(rows, 77))
    assert np.array_equal(tree.masks.cpu().numpy().view(np.uint32), masks)
    assert np.array_equal(b.positions.cpu().numpy(), pos)
    assert status.item() == (mk.MK_ERR_BOUNDS if bad else 0)
    return bad


@pytest.mark.parametrize("n,lo,hi,words,chain,pad", [
    (1, 1, 1, 1, False, 0), (3, 0, 2, 1, False, 5), (7, 31, 33, 2, False, 1), (32, 16, 16, 1, False, 0), (5, 32, 32, 1, True, 0), (9, 60, 130, 5, False, 3),
    (2, 1024, 1024, 32, True, 0), (3, 900, 1024, 32, False, 9), (40, 1, 90, 2, False, 0), (600, 0, 9, 1, False, 700), (4096, 1, 2, 1, False, 3)])
def test_masks_match_the_oracle(n, lo, hi, words, chain, pad):
    rng = random.Random(n * 1000 + hi)
    new = [rng.randint(lo, hi) for _ in range(n)]
    parents = [p for k in new for p in (grow(rng, k, chain) if k else [])] + [-1] * pad
    kv = [k + rng.choice([0, 1, 500]) for k in new]
    assert not run_tree(new, kv, parents, words, sum(new) + pad)


def test_masks_of_forests_and_bad_parents():
    assert not run_tree([4, 3], [4, 10], [-1, -1, 1, -1, -1, 0, -1], 1, 7)       # several roots
    assert run_tree([4, 3], [9, 10], [-1, 1, 3, -2, -1, 5, 0], 1, 7)             # itself, a later one, none at all
    assert not run_tree([4, 3], [3, 0], [-1, 0, 1, 1, -1, 0, 0], 1, 7)           # refused by the step's tables
    assert run_tree([4, 3], [9, 10], [-1, 0, 0, 0, -1, 0, 0], 1, 7, cu=[0, 4, 2])  # offsets that fall
    assert run_tree([4, 3], [9, 10], [-1, 0, 0, 0, -1, 0, 0], 1, 7, cu=[0, 4, 9])  # or pass the rows
    assert run_tree([4, 3, 2], [9, 10, 5], [-1, 0, 0, 0, -1, 0, 0], 1, 7, cu=[0, 4, 2, 5])
    assert not run_tree([40, 3], [50, 10], [9] * 40 + [-1, 0, 0], 1, 43)         # a chunk's parents are not read


# ---------------------------------------------------------------- attention

def make_tree(ctx, new, words, hq, hkv, d, page, typ, layout="hp", seed=0, pad=0, masks=None, scale=1.0):
    s = paged.make_attention(ctx, new, hq, hkv, d, page, typ, layout, seed, pad, scale=scale)
    rng = random.Random(seed)
    m = np.random.default_rng(seed).integers(0, 1 << 32, (sum(new) + pad, words), dtype=np.uint64).astype(np.uint32)
    if masks == "trees":  # else any bits, those past the row itself among them
        for r, k in enumerate(new):
            if 0 < k <= 32 * words:
                a = int(s["cu"][r])
                m[a:a + k] = oracle.paged_tree(grow(rng, k), [0, k], [k], words, k, m[a:a + k], np.zeros(k))[0]
    elif masks == "empty":
        m[:] = 0
    s["masks"] = m
    return s


def check_tree(s, window=0, scale=0.0, workspace=None, status=0, live=None):
    q, typ, d, hq = s["q"], s["q"].dtype, s["q"].shape[2], s["q"].shape[1]
    rows, total = q.shape[0], int(s["cu"][-1])
    out, lse = torch.full_like(q, 5.0), torch.full((rows, hq), 5.0, device=DEV)
    batch = mk.PagedBatch(ints(s["table"]), ints(s["cu"]), ints(s["kv"]), page_size=s["page"], max_new=s["max_new"])
    cache = mk.PagedCache(s["k"], s["v"], n_q_heads=hq, workspace=workspace)
    tree = mk.DraftTree(batch, masks=words_of(s["masks"]))
    cache.attention(q, batch, out, lse=lse, window=window, scale=scale, tree=tree)
    assert cache.status() == status
    again = torch.full_like(out, 7.0)
    cache.attention(q, batch, again, window=window, scale=scale, tree=tree)
    ref, rlse, wabs, smag, vmax = oracle.tree_attention(f64(q), f64(s["k"]), f64(s["v"]), s["table"], s["cu"], s["kv"], s["masks"], scale or d ** -0.5, window)
    live = np.arange(rows) < total if live is None else live
    u = torch.finfo(typ).eps / 2
    keys = s["kv"].max()
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
    assert (got[~live] == 5).all() and (glse[~live] == 5).all()
    sel = torch.as_tensor(live).to(DEV)
    assert torch.equal(out[sel], again[sel])
    return out, lse


ATT = [
    # ctx, new, words, hq, hkv, d, page, window, layout, type
    ([0], [1], 1, 32, 8, 128, 16, 0, "hp", "bf16"),                        # few rows
    ([0, 0, 5], [1, 0, 0], 1, 4, 2, 64, 16, 0, "hp", "fp16"),
    ([300, 0, 77, 1000], [4, 2, 1, 3], 1, 32, 8, 128, 16, 0, "hp", "bf16"),
    ([300, 0, 77, 1000], [16, 11, 1, 9], 1, 8, 8, 64, 16, 0, "ph", "fp16"),
    ([62, 63, 64, 65, 126, 127, 128], [8] * 7, 2, 2, 1, 128, 32, 0, "hp", "bf16"),
    ([900, 20, 3, 0], [8, 4, 3, 8], 1, 4, 2, 128, 16, 100, "hp", "bf16"),  # windows
    ([900, 20, 3, 0], [16, 4, 3, 8], 1, 2, 2, 64, 32, 1, "ph", "fp16"),
    ([900, 20, 3, 0], [16, 4, 3, 8], 1, 2, 2, 64, 32, 3, "hp", "bf16"),
    ([30000, 17, 21111], [4, 1, 3], 1, 32, 8, 128, 16, 0, "ph", "bf16"),
    ([0], [32], 1, 4, 4, 128, 16, 0, "hp", "bf16"),                        # tiles
    ([500], [33], 2, 32, 8, 128, 16, 0, "hp", "bf16"),
    ([0, 1, 127, 128, 129, 640], [64] * 6, 2, 8, 2, 128, 16, 0, "hp", "bf16"),
    ([0, 1, 127, 128, 129, 640], [40, 64, 17, 1, 0, 63], 2, 8, 2, 64, 128, 0, "pad", "fp16"),
    ([1000, 95, 200], [160, 150, 90], 5, 16, 2, 128, 32, 0, "hp", "bf16"),  # several tiles of a tree
    ([1000, 95, 200], [300, 150, 90], 10, 7, 1, 64, 16, 0, "ph", "fp16"),
    ([77], [1024], 32, 2, 1, 128, 64, 0, "hp", "bf16"),                    # the largest tree
    ([700, 20, 40], [64, 50, 33], 2, 8, 2, 128, 16, 64, "hp", "bf16"),     # windows shorter and longer than the trees
    ([700, 20, 40], [200, 50, 33], 7, 8, 2, 64, 32, 5, "hp", "fp16"),
    ([700, 20, 40], [200, 150, 33], 7, 8, 2, 128, 32, 40, "hp", "bf16"),
    ([3000, 0, 130], [100, 513, 1], 4, 4, 1, 128, 64, 333, "hp", "bf16"),  # chunks of prompts beside trees
    ([1000, 3, 0, 50], [1, 90, 0, 300], 3, 16, 4, 128, 32, 0, "hp", "fp16"),
    ([30000, 17, 21111], [20, 64, 33], 2, 32, 8, 64, 16, 0, "hp", "bf16"),  # many blocks per SM
    ([9000], [64], 2, 16, 1, 128, 64, 0, "hp", "fp16"),
]


@pytest.mark.parametrize("case", range(len(ATT)))
@pytest.mark.parametrize("masks", ["trees", "any"])
def test_tree_attention_matches_the_oracle(case, masks, workspace):
    ctx, new, words, hq, hkv, d, page, window, layout, typ = ATT[case]
    s = make_tree(ctx, new, words, hq, hkv, d, page, TYPES[typ], layout, seed=case, pad=case % 3, masks=masks)
    check_tree(s, window, workspace=workspace)


@pytest.mark.parametrize("new", [[1, 2, 1], [70, 2, 41]])
def test_rows_whose_masks_are_empty(new, workspace):
    for ctx, window in (([40, 10, 0], 0), ([0, 0, 0], 0), ([40, 10, 0], 7), ([300, 200, 1], 1)):
        s = make_tree(ctx, new, 3, 8, 2, 128, 16, torch.bfloat16, seed=3, masks="empty")
        check_tree(s, window, workspace=workspace)
        s["masks"][::2, 0] = 1  # the root for every other row
        check_tree(s, window, workspace=workspace)
    s = make_tree([40, 10, 0], new, 3, 8, 2, 128, 16, torch.bfloat16, seed=3, masks="any")
    for kv in ([0, 1, 0], [41, 1, 1], [0, 0, 0]):  # fewer keys than new tokens
        s["kv"] = np.minimum(np.array(kv), s["kv"])
        check_tree(s, workspace=workspace)


@pytest.mark.parametrize("new,typ", [([1, 3], "bf16"), ([60, 3], "bf16"), ([1, 40], "fp16")])
def test_peaked_and_flat_softmax_of_trees(new, typ, workspace):
    for scale in (8.0, 0.0):
        check_tree(make_tree([600, 200], new, 2, 8, 2, 64, 16, TYPES[typ], seed=11, masks="trees", scale=scale), workspace=workspace)
    check_tree(make_tree([600, 200], new, 2, 8, 2, 128, 16, TYPES[typ], seed=12, masks="trees"), scale=-0.1, workspace=workspace)


@pytest.mark.parametrize("new", [[1, 2], [64, 50]])
def test_bad_pages_of_trees_count_as_zeros(new, workspace):
    s = make_tree([300, 200], new, 2, 8, 2, 128, 16, torch.bfloat16, seed=8, masks="trees")
    s["table"][0, 3], s["table"][1, 7], s["table"][1, 0] = -1, s["k"].shape[0], 2 ** 31 - 1
    check_tree(s, workspace=workspace, status=mk.MK_ERR_BOUNDS)


@pytest.mark.parametrize("new", [[2, 1], [64, 40]])
def test_trees_whose_lengths_pass_the_table(new, workspace):
    # the rows stand behind the table's last key: new tokens past it are absent
    s = make_tree([240, 100], new, 2, 8, 2, 64, 16, torch.bfloat16, seed=4, masks="any")
    s["table"][0] = s["table"][0, 0]
    s["k"], s["v"] = torch.nan_to_num(s["k"]), torch.nan_to_num(s["v"])
    width = s["table"].shape[1] * 16
    s["kv"][0] = width + new[0] // 2
    want = dict(s, table=np.concatenate([s["table"], np.full((2, 4), -1)], 1))
    q, hq, d = s["q"], 8, 64
    out = torch.empty_like(q)
    cache = mk.PagedCache(s["k"], s["v"], n_q_heads=hq, workspace=workspace)
    batch = mk.PagedBatch(ints(s["table"]), ints(s["cu"]), ints(s["kv"]), page_size=16, max_new=max(new))
    cache.attention(q, batch, out, tree=mk.DraftTree(batch, masks=words_of(s["masks"])))
    assert cache.status() == mk.MK_ERR_BOUNDS
    # without the tokens past the table: their bits cleared, what they stand for counts
    # in no window here
    ctx = int(want["kv"][0]) - new[0]
    m = s["masks"].copy()
    for i in range(new[0]):
        for j in range(new[0]):
            if ctx + j >= width:
                m[i, j // 32] &= ~np.uint32(1 << j % 32)
    ref, _, wabs, smag, _ = oracle.tree_attention(f64(q), f64(s["k"]), f64(s["v"]), want["table"], s["cu"], s["kv"], m, d ** -0.5)
    tol = 2.0 ** -8 * 1.01 * (np.abs(ref) + wabs) + wabs * (2 * d * 2.0 ** -22 * smag[..., None] + 200 * 2.0 ** -23)
    assert (np.abs(f64(out) - ref) <= tol).all()


@pytest.mark.parametrize("ctx,new,hq,hkv,d", [([100, 5, 1000], [4, 1, 3], 8, 2, 128), ([100, 5, 1000], [60, 1, 33], 8, 2, 64)])
@pytest.mark.parametrize("window", [0, 50])
def test_chains_are_causal(ctx, new, hq, hkv, d, window, workspace):
    s = make_tree(ctx, new, 2, hq, hkv, d, 16, torch.bfloat16, seed=6)
    for r, k in enumerate(new):
        for i in range(k):
            s["masks"][int(s["cu"][r]) + i] = [min((2 << i) - 1, 0xffffffff), max((2 << i) - 1 >> 32, 0)]
    out, lse = check_tree(s, window, workspace=workspace)
    plain, plse = paged.check_attention(s, window, workspace=workspace)
    # the same rows, the same keys in the same order of blocks
    assert (f64(lse) - f64(plse)).max() <= 2.0 ** -18 and np.abs(f64(out) - f64(plain)).max() <= 2.0 ** -6


def test_tree_attention_in_a_graph_on_another_stream(workspace):
    s = make_tree([700, 90, 0], [30, 64, 9], 2, 8, 2, 128, 16, torch.bfloat16, seed=2, masks="trees")
    want, _ = check_tree(s, workspace=workspace)
    batch = mk.PagedBatch(ints(s["table"]), ints(s["cu"]), ints(s["kv"]), page_size=16, max_new=64)
    cache, tree = mk.PagedCache(s["k"], s["v"], n_q_heads=8, workspace=workspace), mk.DraftTree(batch, masks=words_of(s["masks"]))
    out = torch.zeros_like(s["q"])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    cache.attention(s["q"], batch, out, tree=tree, stream=side)
    side.synchronize()
    assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    out.zero_()
    with torch.cuda.graph(graph):
        cache.attention(s["q"], batch, out, tree=tree)
    for _ in range(3):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


# ---------------------------------------------------------------- verification

def rows_of(rng, rows, vocab, kind):
    z = rng.normal(size=(rows, vocab)) * {"flat": 0.0, "soft": 1.0, "sharp": 4.0}.get(kind, 1.0)
    x = np.exp(z - z.max(1, keepdims=True))
    x /= x.sum(1, keepdims=True)
    if kind == "sparse":
        x[rng.random(x.shape) < 0.7] = 0
        x[:, 0] += 1e-3
        x /= x.sum(1, keepdims=True)
    if kind == "greedy":
        x = np.eye(vocab)[rng.integers(0, vocab, rows)]
    return x.astype(np.float32)


def run_verify(trees, tokens, p, q, u, ul, kv=None, pad=0, stride=0, cu=None):
    new = [len(t) for t in trees]
    n, total, vocab = len(trees), sum(new), p.shape[1]
    rows = total + pad
    cu = np.concatenate([[0], np.cumsum(new)]) if cu is None else np.array(cu)
    kv = np.array([k + 7 for k in new]) if kv is None else np.array(kv)
    parents = sum(trees, []) + [0] * pad
    b = mk.PagedBatch(ints(np.zeros((n, 1))), ints(cu), ints(kv), page_size=16, max_new=max([1, *new]))

    def wide(x):
        if x is None:
            return None
        t = torch.full((rows, vocab + stride), float("nan"), device=DEV)
        t[:total, :vocab] = torch.as_tensor(x)[:total].to(DEV)
        return t[:, :vocab]

    tree = mk.DraftTree(b, ints(parents))
    path, emitted, kept, lens, status = ints([55] * rows), ints([55] * rows), ints([55] * n), ints([55] * n), ints([0])
    f32 = lambda x: torch.tensor(np.asarray(x, np.float32)).to(DEV)  # noqa: E731
    args = (ints(list(tokens) + [3] * pad), wide(p), f32(list(u) + [0.5] * pad), f32(ul), path, emitted, kept, lens)
    tree.verify(*args, draft_probs=wide(q), status=status)
    want_path, want_emitted = np.full(rows, 55), np.full(rows, 55)
    want_kept, want_lens, bad = np.zeros(n, int), kv.copy(), False
    for r in range(n):
        a, b2 = int(cu[r]), int(cu[r + 1])
        if a < 0 or b2 < a or b2 > rows or b2 - a > mk.MK_TREE_MAX_NODES or a < max(cu[:r + 1]):
            bad = True
            continue
        want_path[a:b2] = want_emitted[a:b2] = -1
        if b2 == a or kv[r] < b2 - a:
            continue
        x, e, wrong = oracle.tree_verify(parents[a:b2], tokens[a:b2], p[a:b2], None if q is None else q[a:b2], np.asarray(u[a:b2], np.float32), np.float32(ul[r]))
        want_path[a:a + len(x)], want_emitted[a:a + len(e)] = x, e
        want_kept[r], want_lens[r] = len(x), kv[r] - (b2 - a) + len(x)
        bad |= wrong
    got = [t.cpu().numpy() for t in (path, emitted, kept, lens)]
    for name, g, w in zip(("path", "emitted", "kept", "lens"), got, (want_path, want_emitted, want_kept, want_lens)):
        assert np.array_equal(g, w), name
    assert status.item() == (mk.MK_ERR_BOUNDS if bad else 0)
    return want_kept


@pytest.mark.parametrize("vocab,stride", [(1, 0), (3, 0), (4, 0), (127, 1), (128, 0), (1001, 0), (1000, 24), (4099, 2), (20000, 0)])
@pytest.mark.parametrize("drawn", [True, False])
@pytest.mark.parametrize("kind", ["soft", "sharp", "sparse", "greedy", "flat"])
def test_verification_matches_the_oracle(vocab, stride, drawn, kind):
    rng = np.random.default_rng(vocab * 7 + drawn)
    r = random.Random(vocab)
    n = 40 if vocab < 200 else 6 if vocab < 5000 else 2
    trees = [grow(r, r.choice([1, 2, 5, 9, 33]), chain=i % 3 == 0, width=3) for i in range(n)]
    total = sum(map(len, trees))
    p = rows_of(rng, total, vocab, kind)
    q = rows_of(rng, total, vocab, "soft") if drawn else None
    if drawn and kind != "greedy":  # near the target, so that tokens stand
        q = (0.7 * p + 0.3 * q).astype(np.float32)
    tokens, at = [], 0
    for t in trees:
        for i, up in enumerate(t):
            src = (q if drawn else p)[at + max(up, 0)].astype(np.float64)
            tokens.append(int(rng.choice(vocab, p=src / src.sum())))
        at += len(t)
    kept = run_verify(trees, tokens, p, q, rng.random(total).astype(np.float32), rng.random(n).astype(np.float32), pad=int(rng.integers(0, 3)), stride=stride)
    # (a token found by chance among many stands seldom; one drawn near the target often)
    assert vocab < 3 or not drawn or kind == "greedy" or kept.max() > 1


@pytest.mark.parametrize("drawn", [True, False])
def test_siblings_of_one_token_and_uniforms_at_their_ends(drawn):
    rng = np.random.default_rng(1)
    trees = [[-1] + [0] * 8 + [3, 3, 9, 9]] * 30  # eight children of the root
    total, vocab = 13 * 30, 6
    p = rows_of(rng, total, vocab, "soft")
    q = rows_of(rng, total, vocab, "sharp") if drawn else None
    tokens = rng.integers(0, vocab, total).tolist()
    u = rng.choice([0.0, 0.3, 0.9, 1 - 2.0 ** -24], total)
    ul = rng.choice([0.0, 0.5, 1 - 2.0 ** -24], 30)
    run_verify(trees, tokens, p, q, u, ul)
    # the draft equal to the target: the first child stands whatever its number
    run_verify(trees, [int(np.argmax(x)) for x in p[np.repeat(np.arange(30) * 13, 13)]], p, p if drawn else None, np.full(total, 1 - 2.0 ** -24), ul)


def test_exact_borders_of_a_dyadic_row():
    # probabilities and uniforms in quarters: every comparison is of equal numbers
    p = np.array([[0.25, 0.0, 0.5, 0.25], [0.0, 1.0, 0.0, 0.0]], np.float32)
    for x in range(4):
        for u in (0.0, 0.25, 0.5, 0.75):
            for ul in (0.0, 0.25, 0.5, 0.75):
                for q in (None, np.array([[0.5, 0.25, 0.25, 0.0], [0.25] * 4], np.float32)):
                    run_verify([[-1, 0]], [0, x], p, q, [0.0, u], [ul])


def test_rows_that_are_no_probabilities_and_bad_arguments_of_a_row():
    nan, inf = float("nan"), float("inf")
    p = np.array([[0.5, nan, 0.25, -3.0, 0.25], [nan, -inf, 0.0, -0.0, -1e-30], [0.0, 0.0, 1.0, 0.0, 0.0], [0.1, inf, 0, 0, 0]], np.float32)
    q = np.array([[0.25, 0.25, nan, -1.0, 0.5]] * 4, np.float32)
    for q in (q, None):
        for ul in (0.0, 0.4, 0.99):
            run_verify([[-1, 0, 1, 2]], [0, 2, 1, 4], p, q, [0, 0.5, 0.5, 0.5], [ul])
            run_verify([[-1, 0, 0, 0]], [0, 1, 3, 2], p, q, [0, 0.5, 0.5, 0.9], [ul])
            run_verify([[-1, 0, 0, 5], [-1, 0], [-1]], [0, -1, 5, 2, 0, 2, 1], np.concatenate([p, p])[:7], None if q is None else np.concatenate([q, q])[:7],
                       [0, 0.5, 0.5, nan, 2.0, -1.0, 0.5], [ul, ul, ul])  # tokens outside, a later parent, uniforms outside
    run_verify([[-1, 0]], [0, 1], p[1:3], None, [0, 0.5], [0.5])          # a root's row without mass


def test_offsets_and_refused_requests_of_a_verification():
    rng = np.random.default_rng(5)
    p = rows_of(rng, 9, 50, "soft")
    tokens, u = rng.integers(0, 50, 9).tolist(), rng.random(9)
    trees = [[-1, 0, 0], [], [-1, 0, 1], [-1, 0, 1]]
    run_verify(trees, tokens, p, None, u, [0.1] * 4)
    run_verify(trees, tokens, p, None, u, [0.1] * 4, kv=[0, 5, 30, 2])     # refused by the step's tables
    run_verify(trees, tokens, p, None, u, [0.1] * 4, cu=[0, 3, 3, 2, 6])   # offsets that fall
    run_verify(trees, tokens, p, None, u, [0.1] * 4, cu=[0, 3, 3, 6, 11])  # or pass the rows


def test_a_deep_chain_and_a_wide_tree():
    rng = np.random.default_rng(9)
    vocab, k = 40, mk.MK_TREE_MAX_NODES
    p = np.tile(rows_of(rng, 1, vocab, "soft"), (k, 1))
    # everything stands
    run_verify([list(range(-1, k - 1))], rng.integers(0, vocab, k).tolist(), p, p, np.zeros(k), [0.7])
    # nothing stands
    run_verify([[-1] + [0] * (k - 1)], rng.integers(0, vocab, k).tolist(), p, None, np.full(k, 1 - 2.0 ** -24), [0.7])
    q = rows_of(rng, 1, vocab, "soft")
    run_verify([[-1] + [0] * 60], rng.integers(0, vocab, 61).tolist(), p[:61], np.tile(q, (61, 1)), np.full(61, 0.999), [0.7])
    # more than that is refused, the requests beside it are not
    run_verify([[-1, 0], [-1] + [0] * k, [-1]], [1] * (k + 4), np.tile(p[:1], (k + 4, 1)), None, np.full(k + 4, 0.5), [0.2, 0.3, 0.4])


def test_a_request_alone_and_among_others_gives_the_same():
    rng, r = np.random.default_rng(3), random.Random(3)
    vocab, trees = 32003, [grow(r, 12, width=3) for _ in range(30)]
    total = 360
    g = torch.Generator(device=DEV).manual_seed(1)
    p, q = (torch.softmax(3 * torch.randn(total, vocab, generator=g, device=DEV), -1) for _ in range(2))
    q = 0.6 * p + 0.4 * q
    up = torch.tensor([12 * i + max(x, 0) for i, t in enumerate(trees) for x in t], device=DEV)
    tokens = torch.multinomial(q[up], 1, generator=g)[:, 0].to(torch.int32)
    u, ul = torch.rand(total, generator=g, device=DEV), torch.rand(30, generator=g, device=DEV)

    def call(a, b):
        n, k = b - a, 12 * (b - a)
        x = slice(12 * a, 12 * b)
        batch = mk.PagedBatch(ints(np.zeros((n, 1))), ints(np.arange(n + 1) * 12), ints([12] * n), page_size=16, max_new=12)
        outs = [ints([9] * k), ints([9] * k), ints([9] * n), ints([9] * n)]
        mk.DraftTree(batch, ints(sum(trees[a:b], []))).verify(tokens[x].contiguous(), p[x], u[x].contiguous(), ul[a:b].contiguous(), *outs, draft_probs=q[x])
        return outs

    whole = call(0, 30)
    again = call(0, 30)
    assert all(torch.equal(a, b) for a, b in zip(whole, again)) and whole[2].max() > 3
    for i in range(30):
        for a, b in zip(call(i, i + 1), whole):
            k = len(b) // 30
            assert torch.equal(a, b[k * i:k * (i + 1)])


def test_python_refusals_of_trees():
    b = mk.PagedBatch(ints(np.zeros((2, 1))), ints([0, 3, 5]), ints([3, 4]), ints([0] * 5), ints([0] * 5), page_size=16, max_new=3)
    parents, masks = ints([-1, 0, 0, -1, 0]), ints(np.zeros((5, 1)))
    with pytest.raises(ValueError):
        mk.DraftTree(b)
    with pytest.raises(ValueError):
        mk.DraftTree(b, parents, ints([0] * 5))
    with pytest.raises(ValueError):
        mk.DraftTree(b, parents, masks.long())
    with pytest.raises(ValueError):
        mk.DraftTree(b, parents[:4], masks)
    with pytest.raises(ValueError):
        mk.DraftTree(b, masks=masks).build()
    with pytest.raises(ValueError):
        mk.DraftTree(b, parents, masks, ints([0] * 4)).build()
    with pytest.raises(mk.MkError):
        mk.DraftTree(b, parents, ints(np.zeros((5, 33)))).build()
    with pytest.raises(mk.MkError):
        mk.DraftTree(b, parents, masks, positions=parents).build()
    tree = mk.DraftTree(b, parents)
    p, f = torch.full((5, 7), 1 / 7, device=DEV), torch.zeros(5, device=DEV)
    ok = dict(tokens=ints([0] * 5), target_probs=p, uniforms=f, last_uniforms=f[:2].clone(), path=ints([0] * 5), emitted=ints([0] * 5), kept=ints([0] * 2),
              lens=ints([0] * 2))
    tree.verify(**ok)
    for kw in (dict(tokens=ints([0] * 4)), dict(tokens=ok["tokens"].long()), dict(target_probs=p.half()), dict(target_probs=p[:4]), dict(target_probs=p.t()),
               dict(draft_probs=p[:, :6]), dict(uniforms=f.double()), dict(last_uniforms=f), dict(kept=ints([0] * 5)), dict(path=ints([0] * 10)[::2]),
               dict(status=ints([0, 0]))):
        with pytest.raises(ValueError):
            tree.verify(**{**ok, **kw})
    with pytest.raises(mk.MkError):
        tree.verify(**{**ok, "path": ok["emitted"]})
    with pytest.raises(ValueError):
        mk.DraftTree(b, masks=masks).verify(**ok)
    cache = mk.PagedCache(*(torch.zeros(3, 2, 16, 64, dtype=torch.bfloat16, device=DEV) for _ in range(2)), n_q_heads=4)
    q = torch.zeros(5, 4, 64, dtype=torch.bfloat16, device=DEV)
    for t in (tree, mk.DraftTree(b, masks=masks[:4])):
        with pytest.raises(ValueError):
            cache.attention(q, b, torch.empty_like(q), tree=t)
