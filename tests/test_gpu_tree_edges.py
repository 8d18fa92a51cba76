"""Edges of the trees' operators on the GPU: both schedules of the tile kernel, calls
at once, captures, chunks and lone tokens in one step."""
import random
import subprocess
import sys
import threading

import numpy as np
import pytest
import torch

import oracle
import test_gpu_pages as pages
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


@pytest.fixture(scope="module")
def workspace():
    return torch.full((mk.MK_PAGED_WORKSPACE_BYTES // 4,), float("nan"), device=DEV)


def widen(s, to=3000):
    """The same requests in a table that could hold many more pages: no clusters."""
    t = np.full((s["table"].shape[0], to), 2 ** 30)
    t[:, :s["table"].shape[1]] = s["table"]
    return dict(s, table=t)


@pytest.mark.parametrize("case", range(9, len(trees.ATT)))
def test_runs_over_all_sms_match_the_oracle(case, workspace):
    ctx, new, words, hq, hkv, d, page, window, layout, typ = trees.ATT[case]
    s = trees.make_tree(ctx, new, words, hq, hkv, d, page, TYPES[typ], layout, seed=case, pad=case % 3, masks="trees")
    trees.check_tree(widen(s, 1 << 18 if page == 16 else 3000), window, workspace=workspace)


WIDE = [
    # heads of 64 in pairs: 1, 3, 5, 7, 8, 13 query heads a kv head; an odd number of kv heads has none
    ([700, 3, 90], [40, 33, 128], 4, 2, 2, 64, 16, 0, "hp", "bf16"), ([700, 3, 90], [40, 20, 42], 2, 6, 2, 64, 16, 0, "ph", "fp16"),
    ([700, 3, 90], [25, 20, 4], 1, 20, 4, 64, 32, 50, "hp", "bf16"), ([700, 3, 5000], [18, 17, 3], 1, 14, 2, 64, 16, 0, "pad", "bf16"),
    ([700, 3, 5000], [16, 9, 3], 1, 48, 6, 64, 64, 0, "hp", "fp16"), ([2000, 3, 90], [9, 9, 2], 1, 26, 2, 64, 16, 7, "hp", "bf16"),
    ([700, 3, 90], [32, 20, 3], 1, 12, 3, 64, 16, 0, "hp", "bf16"),
    # pairs, tiles of two halves and chunks in one step, blocks divided among SMs
    ([30000, 0, 100, 21111, 5], [20, 300, 64, 1, 32], 2, 32, 8, 64, 16, 0, "hp", "bf16"),
    ([3000, 0, 100, 211, 5], [20, 300, 64, 1, 32], 2, 32, 8, 64, 32, 400, "hp", "fp16"),
    ([30000, 0, 100, 21111, 5], [20, 300, 64, 1, 32], 2, 32, 8, 128, 16, 0, "hp", "bf16"),
    ([40000], [5], 1, 8, 2, 64, 16, 0, "hp", "bf16"), ([40000], [30], 1, 4, 1, 128, 64, 0, "hp", "fp16"),
]


@pytest.mark.parametrize("case", range(len(WIDE)))
def test_pairs_of_heads_and_divided_keys(case, workspace):
    ctx, new, words, hq, hkv, d, page, window, layout, typ = WIDE[case]
    s = trees.make_tree(ctx, new, words, hq, hkv, d, page, TYPES[typ], layout, seed=40 + case, pad=1, masks="trees")
    out, lse = trees.check_tree(widen(s), window, workspace=workspace)
    if case < 7:  # and in clusters
        again, lse2 = trees.check_tree(s, window, workspace=workspace)
        assert np.abs(f64(out) - f64(again))[:-1].max() <= 2.0 ** -6 and np.nanmax(np.abs(f64(lse) - f64(lse2))[:-1]) <= 2.0 ** -18


@pytest.mark.parametrize("n,hkv,rep,d,ctx,new", [
    # clusters of 16 down to a CTA: 1, 7, 8, 15, 16, 30, 76, 152 tiles
    (1, 1, 4, 128, 900, 32), (7, 1, 4, 128, 700, 30), (1, 8, 4, 128, 2000, 25), (15, 1, 2, 64, 400, 60), (2, 8, 8, 128, 300, 16), (5, 6, 4, 64, 500, 32),
    (38, 2, 4, 128, 200, 32), (19, 8, 4, 64, 300, 31), (1, 2, 16, 128, 1500, 8), (1, 1, 64, 128, 700, 2), (3, 2, 3, 128, 800, 42), (2, 2, 7, 64, 800, 36),
    # tiles of two halves, two tiles a head
    (1, 4, 4, 128, 600, 64), (1, 2, 5, 128, 500, 47), (1, 1, 4, 64, 900, 128), (2, 2, 2, 128, 90, 120)])
def test_clusters_of_every_size(n, hkv, rep, d, ctx, new, workspace):
    rng = random.Random(n * 100 + new)
    ctxs, news = [rng.randint(0, ctx) for _ in range(n)], [rng.randint(1, new) for _ in range(n)]
    ctxs[0], news[0] = ctx, new
    s = trees.make_tree(ctxs, news, -(-new // 32), hkv * rep, hkv, d, 16, torch.bfloat16, seed=n + new, pad=2, masks="trees")
    trees.check_tree(s, workspace=workspace)
    trees.check_tree(s, window=33, workspace=workspace)


def test_rows_out_of_order_among_trees(workspace):
    """Requests that fall, begin below an earlier offset, or have more rows than max_new
    are left alone, whichever schedule takes the others."""
    for wide in (False, True):
        for new in (3, 40):
            s = trees.make_tree([90, 300, 7, 50], [new] * 4, 2, 8, 2, 128, 16, torch.bfloat16, seed=5, masks="trees")
            for cu, served in (([0, new, 2, 2 + new, 4 * new], [0]), ([0, new, 2 * new, 4 * new, 4 * new], [0, 1, 3]), ([0, new, 2 * new, 3 * new, 4 * new + 1], [0, 1, 2])):
                t = widen(s) if wide else s
                q, out = s["q"], torch.full_like(s["q"], 5.0)
                cache = mk.PagedCache(s["k"], s["v"], n_q_heads=8, workspace=workspace)
                batch = mk.PagedBatch(ints(t["table"]), ints(cu), ints(s["kv"]), page_size=16, max_new=new)
                cache.attention(q, batch, out, tree=mk.DraftTree(batch, masks=trees.words_of(s["masks"])))
                assert cache.status() == mk.MK_ERR_BOUNDS
                live = np.zeros(4 * new, bool)
                for r in served:
                    live[cu[r]:cu[r + 1]] = True
                got = f64(out)
                assert (got[~live] == 5).all(), (wide, new, cu)
                kv = np.array([s["kv"][r] if r in served else 0 for r in range(4)])
                good = [0, new, 2 * new, 3 * new, 4 * new] if served == [0, 1, 2] else cu
                ref, _, wabs, smag, _ = oracle.tree_attention(f64(q), f64(torch.nan_to_num(s["k"])), f64(torch.nan_to_num(s["v"])), s["table"], good, kv, s["masks"], 128 ** -0.5)
                tol = 2.0 ** -8 * 1.01 * (np.abs(ref) + wabs) + wabs * (2 * 128 * 2.0 ** -22 * smag[..., None] + 200 * 2.0 ** -23)
                assert (np.abs(got - ref) <= tol)[live].all()


def test_many_small_trees(workspace):
    for d, hkv in ((128, 2), (64, 2)):
        rng = random.Random(d)
        n = 500
        ctx, new = [rng.randint(0, 200) for _ in range(n)], [rng.randint(0, 12) for _ in range(n)]
        s = trees.make_tree(ctx, new, 1, 4 * hkv, hkv, d, 16, torch.bfloat16, seed=d, masks="trees")
        trees.check_tree(s, workspace=workspace)


@pytest.mark.parametrize("new", [[3, 2], [60, 33]])
def test_a_nan_stays_with_its_row(new, workspace):
    for wide in (False, True):
        s = trees.make_tree([700, 90], new, 2, 8, 2, 128, 16, torch.bfloat16, seed=3, masks="trees")
        want, _ = trees.check_tree(widen(s) if wide else s, workspace=workspace)
        q = s["q"].clone()
        q[1, 3, 5] = float("nan")
        t = widen(s) if wide else s
        batch = mk.PagedBatch(ints(t["table"]), ints(t["cu"]), ints(t["kv"]), page_size=16, max_new=max(new))
        out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device=DEV)
        mk.PagedCache(s["k"], s["v"], n_q_heads=8, workspace=workspace).attention(q, batch, out, lse=lse, tree=mk.DraftTree(batch, masks=trees.words_of(s["masks"])))
        assert out[1, 3].isnan().all() and lse[1, 3].isnan()
        out[1, 3] = want[1, 3]
        assert torch.equal(out, want)


def test_windows_leave_pages_before_them_alone(workspace):
    for new in ([2, 3], [60, 40]):
        for wide in (False, True):
            s = trees.make_tree([3000, 700], new, 2, 8, 2, 64, 16, torch.bfloat16, seed=9, masks="trees")
            for r in range(2):
                first = max(0, int(s["kv"][r]) - new[r] - 200 + 1)  # what the root sees
                for j in range(first // 16):
                    s["k"][int(s["table"][r, j])] = float("nan")
                    s["v"][int(s["table"][r, j])] = float("inf")
                s["table"][r, :first // 16] = -1
                part = int(s["table"][r, first // 16])
                s["v"][part, :, :first % 16] = float("nan")
            t = dict(s, k=torch.nan_to_num(s["k"]), v=torch.nan_to_num(s["v"], posinf=0.0))
            ref, _, wabs, smag, _ = oracle.tree_attention(f64(s["q"]), f64(t["k"]), f64(t["v"]), s["table"], s["cu"], s["kv"], s["masks"], 64 ** -0.5, 200)
            u = widen(s) if wide else s
            batch = mk.PagedBatch(ints(u["table"]), ints(u["cu"]), ints(u["kv"]), page_size=16, max_new=max(new))
            out = torch.empty_like(s["q"])
            cache = mk.PagedCache(s["k"], s["v"], n_q_heads=8, workspace=workspace)
            cache.attention(s["q"], batch, out, window=200, tree=mk.DraftTree(batch, masks=trees.words_of(s["masks"])))
            tol = 2.0 ** -8 * 1.01 * (np.abs(ref) + wabs) + wabs * (2 * 64 * 2.0 ** -22 * smag[..., None] + 450 * 2.0 ** -23)
            assert cache.status() == 0 and (np.abs(f64(out) - ref) <= tol).all()


# ---------------------------------------------------------------- calls at once, captures

def verify_case(seed, n=12, vocab=5003):
    rng, r = np.random.default_rng(seed), random.Random(seed)
    forest = [trees.grow(r, r.choice([1, 4, 9]), width=3) for _ in range(n)]
    total = sum(map(len, forest))
    p = torch.tensor(trees.rows_of(rng, total, vocab, "sharp"), device=DEV)
    q = 0.7 * p + 0.3 * torch.tensor(trees.rows_of(rng, total, vocab, "soft"), device=DEV)
    cu = np.concatenate([[0], np.cumsum([len(t) for t in forest])])
    up = torch.tensor([int(cu[i]) + max(x, 0) for i, t in enumerate(forest) for x in t], device=DEV)
    g = torch.Generator(device=DEV).manual_seed(seed)
    tokens = torch.multinomial(q[up], 1, generator=g)[:, 0].to(torch.int32)
    batch = mk.PagedBatch(ints(np.zeros((n, 1))), ints(cu), ints(cu[1:] - cu[:-1] + 3), page_size=16, max_new=9)
    outs = [ints([0] * total), ints([0] * total), ints([0] * n), ints([0] * n)]
    return mk.DraftTree(batch, ints(sum(forest, []))), (tokens, p, torch.rand(total, generator=g, device=DEV), torch.rand(n, generator=g, device=DEV), *outs), dict(draft_probs=q), outs


def test_verifications_at_once_and_replayed():
    a, b = verify_case(1), verify_case(2)
    want = []
    for tree, args, kw, outs in (a, b):
        tree.verify(*args, **kw)
        torch.cuda.synchronize()
        want.append([o.clone() for o in outs])
        for o in outs:
            o.fill_(-9)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()

    def many(case, stream):
        for _ in range(300):
            case[0].verify(*case[1], **case[2], stream=stream)

    threads = [threading.Thread(target=many, args=x) for x in ((a, streams[0]), (b, streams[1]))]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    torch.cuda.synchronize()
    for case, w in zip((a, b), want):
        assert all(torch.equal(x, y) for x, y in zip(case[3], w))
    # a captured call takes what its inputs hold when it is replayed
    tree, args, kw, outs = a
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tree.verify(*args, **kw)
    u = args[2].clone()
    for value in (0.0, 0.999, None):
        args[2].copy_(u) if value is None else args[2].fill_(value)
        for o in outs:
            o.fill_(-9)
        graph.replay()
        torch.cuda.synchronize()
        got = [o.clone() for o in outs]
        tree.verify(*args, **kw)
        assert all(torch.equal(x, y) for x, y in zip(got, outs))
    assert all(torch.equal(x, y) for x, y in zip(got, want[0]))


FIRST_IN_CAPTURE = """
import sys
sys.path.insert(0, %r)
import torch
from tile_level_overlap_gb300 import mk
dev = "cuda:0"
i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)
k, v = (torch.randn(40, 2, 16, 64, device=dev).to(torch.bfloat16) for _ in range(2))
cache = mk.PagedCache(k, v, n_q_heads=4, workspace=torch.empty(mk.MK_PAGED_WORKSPACE_BYTES, dtype=torch.uint8, device=dev))
layers = mk.PagedLayers([cache])
t = 50
batch = mk.PagedBatch(i32([list(range(20)), list(range(20, 40))]), i32([0, 40, 50]), i32([140, 90]), i32([0] * t), i32(list(range(100, 140)) + list(range(400, 410))), page_size=16, max_new=40)
tree = mk.DraftTree(batch, i32([-1] + list(range(39)) + [-1] + [0] * 9), i32([[0, 0]] * t))
q = torch.randn(t, 4, 64, device=dev).to(torch.bfloat16)
out, out2 = torch.zeros_like(q), torch.zeros_like(q)
wide = mk.PagedBatch(i32([list(range(20)) + [0] * 5000, list(range(20, 40)) + [0] * 5000]), i32([0, 40, 50]), i32([140, 90]), page_size=16, max_new=40)
probs = torch.softmax(torch.randn(t, 1000, device=dev), -1)
u, ul, tok = torch.rand(t, device=dev), torch.rand(2, device=dev), i32([3] * t)
path, emitted, kept, lens, nxt = i32([0] * t), i32([0] * t), i32([0] * 2), i32([0] * 2), i32([0] * 2)
shared, free, n_free, left = i32([0] * 40), i32([0] * 40), i32([0]), i32([0])
held, big = i32([140, 90]), 2100
many = mk.PagedBatch(i32([[0]] * big), i32([0] * (big + 1)), i32([0] * big), page_size=16, max_new=1)
zeros, nxt2 = i32([0] * big), i32([0] * big)
copies = i32([[1, -1], [2, -1], [5, 0]])
def step():
    tree.build()
    cache.attention(q, batch, out, tree=tree)
    cache.attention(q, wide, out2, tree=tree)
    tree.verify(tok, probs, u, ul, path, emitted, kept, lens, draft_probs=probs)
    layers.keep(batch, path)
    layers.copy(copies)
    batch.trim(held, lens, nxt, shared, free, n_free, left)
    many.trim(zeros, zeros, nxt2, shared, free, n_free, left)
g = torch.cuda.CUDAGraph()
k0, v0 = k.clone(), v.clone()
torch.cuda.synchronize()
with torch.cuda.graph(g):
    step()
g.replay()
torch.cuda.synchronize()
got = [x.clone() for x in (out, out2, path, emitted, lens, nxt, free, k, v)]
for x in (out, out2, path, emitted, lens, nxt, free):
    x.zero_()
k.copy_(k0); v.copy_(v0)
step()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(got, (out, out2, path, emitted, lens, nxt, free, k, v)))
assert cache.status() == 0 and got[0].abs().sum() > 0
print("same")
"""


def test_the_first_calls_of_a_process_in_a_capture():
    r = subprocess.run([sys.executable, "-c", FIRST_IN_CAPTURE % build.ROOT], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.split() == ["same"], r.stdout + r.stderr


def test_pages_on_other_streams_and_at_once():
    rng = random.Random(4)
    jobs = []
    for i in range(2):
        table, lens, shared, free, n_free = pages.make_pool(rng, 700, 16, 8, 100, 800, 0.4)
        parents = [rng.randrange(700) for _ in range(700)]
        start = np.full((700, 8), -5)
        want = oracle.paged_fork(table, lens, None, parents, start, 16, shared, free, n_free)
        jobs.append((ints(table), ints(parents), ints(lens), ints(shared), ints(free), ints([n_free]), want, torch.cuda.Stream(), start))
    torch.cuda.synchronize()
    errors = []

    def work(table, parents, lens, shared, free, n_free, want, stream, start):
        with torch.cuda.stream(stream):
            for _ in range(50):
                t, s, f, left, nl, copies = ints(start), shared.clone(), free.clone(), ints([0]), ints([0] * 700), ints(np.zeros((3, 700)))
                pages.batch_of(t, 16).fork(pages.batch_of(table, 16), parents, lens, nl, copies, s, f, n_free, left, stream=stream)
                stream.synchronize()
                got = {"table": t, "lens": nl, "copies": copies, "shared": s, "free": f}
                if not all(np.array_equal(v.cpu().numpy(), want[k]) for k, v in got.items()) or left.item() != want["n_left"]:
                    errors.append(1)

    threads = [threading.Thread(target=work, args=j) for j in jobs]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    assert not errors


def test_steps_end_to_end_without_waiting(workspace):
    """Trees of one step behind those of another, launched without a pause: every kernel
    waits for what precedes it before it reads."""
    s = trees.make_tree([400, 90, 3, 700], [30, 9, 64, 40], 2, 8, 2, 128, 16, torch.bfloat16, seed=8, masks="trees")
    parents = [trees.grow(random.Random(i), 64) for i in range(6)]
    forests = [ints(sum((p[:k] for k in (30, 9, 64, 40)), [])) for p in parents]
    total = 143
    pos = ints([0] * total)
    batch = mk.PagedBatch(ints(s["table"]), ints(s["cu"]), ints(s["kv"]), pos, ints([0] * total), page_size=16, max_new=64)
    wide = mk.PagedBatch(ints(widen(s)["table"]), ints(s["cu"]), ints(s["kv"]), page_size=16, max_new=64)
    cache = mk.PagedCache(s["k"], s["v"], n_q_heads=8, workspace=workspace)
    up, masks = ints([0] * total), ints(np.zeros((total, 2)))
    tree = mk.DraftTree(batch, up, masks)
    outs = [[torch.empty_like(s["q"]) for _ in range(12)] for _ in range(2)]

    def run(outs, wait):
        for i in range(12):
            up.copy_(forests[i % 6])
            tree.build()
            if wait:
                torch.cuda.synchronize()
            cache.attention(s["q"], wide if i % 2 else batch, outs[i], tree=tree)
            if wait:
                torch.cuda.synchronize()

    run(outs[0], True)
    for _ in range(20):
        run(outs[1], False)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(*outs))


@pytest.mark.parametrize("ctx,new,hq,hkv,d,page,typ,wide", [
    # tiles of one half in runs: several of odd and even numbers of blocks, lone blocks among them; in clusters; tiles of two halves; pairs of heads
    ([5000, 300, 60, 0, 9000], [32, 20, 3, 1, 32], 32, 8, 128, 16, "bf16", True), ([20000] * 2 + [100] * 7, [8] * 9, 40, 5, 128, 64, "fp16", True),
    ([9000, 200, 3000], [13, 30, 2], 20, 5, 64, 16, "bf16", True), ([700] * 40, [25] * 40, 12, 3, 64, 32, "fp16", True),
    ([4096], [32], 32, 8, 128, 16, "bf16", False), ([1500, 90], [30, 32], 8, 2, 64, 16, "fp16", False), ([3000], [64], 16, 4, 128, 16, "bf16", False),
    ([5000, 300], [64, 40], 32, 8, 128, 16, "bf16", True), ([5000, 300], [30, 20], 32, 8, 64, 16, "bf16", True)])
def test_maxima_that_grow_with_every_block(ctx, new, hq, hkv, d, page, typ, wide, workspace):
    s = trees.make_tree(ctx, new, -(-max(new) // 32), hq, hkv, d, page, TYPES[typ], seed=len(ctx) + d, pad=1, masks="trees")
    # a head's scores grow by more than 2^8 a block of 128 keys, or fall with every other one
    s["q"][:, :, 0] = 8.0
    s["q"][:, 1::3, 0] = -8.0
    for r, kv in enumerate(s["kv"]):
        for j in range(-(-int(kv) // page)):
            p, m = int(s["table"][r, j]), min(page, int(kv) - j * page)
            s["k"][p, :, :m, 0] = (16.0 * (j * page // 128)) % 1024
    trees.check_tree(widen(s, 1 << 14 if page == 16 else 6000) if wide else s, workspace=workspace)


@pytest.mark.parametrize("drawn", [True, False])
def test_verification_in_batches_of_every_size(drawn):
    # clusters of 16 CTAs down to one: the requests of a batch are eight, in turn
    r, vocab, k = random.Random(8), 20011, 9
    forest = [trees.grow(r, k, width=3) for _ in range(8)]
    g = torch.Generator(device=DEV).manual_seed(2)
    p, q = (torch.softmax(3 * torch.randn(8 * k, vocab, generator=g, device=DEV), -1) for _ in range(2))
    q = 0.5 * p + 0.5 * q
    up = torch.tensor([k * i + max(x, 0) for i, t in enumerate(forest) for x in t], device=DEV)
    tokens = torch.multinomial(q[up], 1, generator=g)[:, 0].to(torch.int32)
    u, ul = torch.rand(8 * k, generator=g, device=DEV), torch.rand(8, generator=g, device=DEV)
    first = None
    for n in (8, 1, 2, 17, 19, 20, 21, 23, 25, 27, 30, 33, 40, 45, 51, 61, 70, 77, 101, 110, 152, 153, 305):
        of = torch.arange(n, device=DEV) % 8
        rows = (of[:, None] * k + torch.arange(k, device=DEV)).reshape(-1)
        batch = mk.PagedBatch(ints(np.zeros((n, 1))), ints(np.arange(n + 1) * k), ints([k] * n), page_size=16, max_new=k)
        outs = [ints([9] * (n * k)), ints([9] * (n * k)), ints([9] * n), ints([9] * n)]
        mk.DraftTree(batch, ints([x for i in range(n) for x in forest[i % 8]])).verify(
            tokens[rows], p[rows], u[rows], ul[of], *outs, draft_probs=q[rows] if drawn else None)
        outs = [x.view(n, -1) for x in outs]
        first = first or outs
        for x, y in zip(outs, first):
            assert torch.equal(x, y[of])
