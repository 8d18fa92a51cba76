"""Edges of the paged-cache operators on the GPU."""
import threading

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


# ---------------------------------------------------------------- append

def bits(t):
    return t.contiguous().view(torch.int16)


@pytest.mark.parametrize("t", [5, 700])                        # a block per token; the ring
@pytest.mark.parametrize("d,rot,typ", [(128, 0, "bf16"), (128, 32, "bf16"), (64, 48, "fp16"), (64, 0, "fp16"), (128, 96, "fp16")])
@pytest.mark.parametrize("gains", ["", "q", "k", "qk"])
def test_elements_that_do_not_turn_stay(t, d, rot, typ, gains):
    """Infinities, NaN (their payloads) and negative zeros outside the rotation:
    copied where there is no gain, x / sqrt(mean x^2 + eps) * gain where there
    is one, and nothing of them in their neighbours.  (A head with an infinity
    or a NaN has a norm that is not finite: its elements are 0 and NaN, or all
    NaN, as the formula says.)"""
    typ, hq, hkv, page = TYPES[typ], 6, 3, 16
    g = torch.Generator().manual_seed(t + d + rot)
    x = torch.randn(t, hq + 2 * hkv, d, generator=g).to(typ)
    spoil = torch.rand(t, hq + 2 * hkv, d, generator=g)
    spoil[:, :, :rot] = 1.0
    spoil[:, ::3] = 1.0                                         # every third head has finite values alone
    plain = x.clone()
    x[spoil < 0.02], x[(spoil >= 0.02) & (spoil < 0.04)] = float("inf"), -float("inf")
    x[(spoil >= 0.04) & (spoil < 0.05)] = float("nan")
    x[(spoil >= 0.05) & (spoil < 0.10)] = -0.0
    raw = bits(x).view(t, hq + 2 * hkv, d)
    raw[(spoil >= 0.10) & (spoil < 0.11)] = 0x7fc5 if typ == torch.bfloat16 else 0x7d23   # NaN with a payload
    x = raw.view(typ).to(DEV)
    gain = (1 + 0.1 * torch.randn(d, generator=g)).to(typ).to(DEV)
    qn, kn = gain if "q" in gains else None, gain if "k" in gains else None
    rope, pos = (mk.Rope(d, rotary_dim=rot), ints(np.arange(t) + 1)) if rot else (None, None)
    pages = -(-t // page)
    slots = ints(np.arange(t))

    def run(rows):
        kc, vc = (torch.zeros(pages, page, hkv, d, dtype=typ, device=DEV) for _ in range(2))
        out = torch.zeros(t, hq, d, dtype=typ, device=DEV)
        cache = mk.PagedCache(kc.transpose(1, 2), vc.transpose(1, 2), n_q_heads=hq)
        cache.append(rows[:, :hq], rows[:, hq:hq + hkv], rows[:, hq + hkv:], slots, pos, rope, q_out=out, q_norm=qn, k_norm=kn, eps=1e-6)
        assert cache.status() == 0
        flat = [c.reshape(-1, hkv, d)[:t] for c in (kc, vc)]
        return out, *flat

    got = run(x)
    clean = run(plain.to(DEV))
    parts = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
    assert torch.equal(bits(got[2]), bits(parts[2]))
    for out, ref, part, gn in zip(got[:2], clean[:2], parts, (qn, kn)):
        if gn is None:
            assert torch.equal(bits(out[..., rot:]), bits(part[..., rot:]))
            assert torch.equal(bits(out[..., :rot]), bits(ref[..., :rot]))    # pairs of finite elements
            continue
        x64 = part[..., :].double()
        want = x64 / torch.sqrt((x64 * x64).mean(-1, keepdim=True) + 1e-6) * gn.double()
        same = torch.isfinite(x64).all(-1)                      # heads whose norm is finite
        u = torch.finfo(typ).eps / 2
        o64, w = out[..., rot:].double(), want[..., rot:]
        assert torch.equal(torch.isnan(o64), torch.isnan(w))
        # one rounding, and the norm's sum of d squares, rsqrt and two products in fp32
        err = (o64 - w).abs() - (u * w.abs() + (d + 8) * 2.0 ** -24 * w.abs() + 2.0 ** -24)
        assert (err[same] <= 0).all()
        assert torch.equal(torch.signbit(out[..., rot:])[same], torch.signbit(w)[same])
        zero = w == 0
        assert (o64[zero] == 0).all()


# ---------------------------------------------------------------- attention: small weights

@pytest.mark.parametrize("new,ctx,d", [([1], [4000], 128), ([2, 1], [3000, 700], 64), ([90], [4000], 128), ([40, 3], [2000, 900], 64)])
def test_weights_far_below_the_largest_count_in_fp16(new, ctx, d, workspace):
    """Every 16th key has weight 1 and value 0, the others weight 2^-25.5, which
    fp16 does not hold, and values of about 3e4: the output is those alone.
    Tolerance, A the softmax-weighted mean of |v|: output and weights rounded
    (u |o| + u A), fp32 sums as in the other tests, and what is below fp16's
    normal range once weights are scaled by 2^7 or more: 2^-32 of a row's
    largest weight each, of at most 17 keys for each weight of 1."""
    typ, hq, hkv = torch.float16, 8, 2
    s = paged.make_attention(ctx, new, hq, hkv, d, 16, typ, seed=d + sum(new), garbage=float("nan"))
    s["q"].zero_()
    s["q"][..., 0] = 1.0
    g = torch.Generator().manual_seed(3)
    for r in range(len(ctx)):
        for j in range(-(-int(s["kv"][r]) // 16)):
            p, m = int(s["table"][r, j]), min(16, int(s["kv"][r]) - 16 * j)
            s["k"][p, :, :m] = 0
            s["k"][p, :, 0, 0] = 25.5
            s["v"][p, :, :m] = (2e4 + 2e4 * torch.rand(hkv, m, d, generator=g)).to(typ).to(DEV)
            s["v"][p, :, 0] = 0
    scale = float(np.log(2.0))
    out, lse = torch.zeros_like(s["q"]), torch.zeros(s["q"].shape[:2], device=DEV)
    cache = mk.PagedCache(s["k"], s["v"], n_q_heads=hq, workspace=workspace)
    cache.attention(s["q"], mk.PagedBatch(ints(s["table"]), ints(s["cu"]), ints(s["kv"]), page_size=16, max_new=max(new)), out, lse=lse, scale=scale)
    assert cache.status() == 0
    ref, rlse, wabs, smag, vmax = oracle.paged_attention(f64(s["q"]), f64(s["k"]), f64(s["v"]), s["table"], s["cu"], s["kv"], scale)
    u, keys = torch.finfo(typ).eps / 2, int(s["kv"].max())
    ds, sums = d * 2.0 ** -22 * smag, (keys / 8 + 64) * 2.0 ** -23
    tol = u * 1.01 * (np.abs(ref) + wabs) + wabs * (2 * ds[..., None] + sums) + 17 * 2.0 ** -32 * vmax[..., None] + 2.0 ** -24
    assert ref[..., :].max() > 4e-3 and (tol < 0.1 * np.maximum(ref, 4e-3)).all()
    assert (np.abs(f64(out) - ref) <= tol).all()
    assert (np.abs(f64(lse) - rlse) <= ds + sums + 2.0 ** -20 * np.abs(rlse)).all()


# ---------------------------------------------------------------- attention: offsets and lengths that do not fit

def attend(s, workspace, max_new, window=0):
    """out, lse (filled with 5 before the call) and the status."""
    out, lse = torch.full_like(s["q"], 5.0), torch.full(s["q"].shape[:2], 5.0, device=DEV)
    cache = mk.PagedCache(s["k"], s["v"], n_q_heads=s["q"].shape[1], workspace=workspace)
    cache.attention(s["q"], mk.PagedBatch(ints(s["table"]), ints(s["cu"]), ints(s["kv"]), page_size=s["page"], max_new=max_new), out, lse=lse, window=window)
    return f64(out), f64(lse), cache.status()


def check_rows(s, got, glse, r, row0, rows, kv, room=1 << 30):
    """Rows row0 .. row0 + rows as request r's last ones of kv tokens, keys past
    `room` absent; the tolerance of the other tests (bf16)."""
    q, d = f64(s["q"]), s["q"].shape[2]
    u, sums = 2.0 ** -8, (min(kv, room) / 8 + 64) * 2.0 ** -23
    for i in range(rows):
        seen = min(kv - rows + i + 1, room)
        ref, rl, wabs, smag, _ = oracle.paged_attention(q[row0 + i:row0 + i + 1], f64(s["k"]), f64(s["v"]), s["table"][r:r + 1], [0, 1], [seen], d ** -0.5)
        ds = d * 2.0 ** -22 * smag
        assert (np.abs(got[row0 + i] - ref[0]) <= (u * 1.01 * (np.abs(ref) + wabs) + wabs * (2 * ds[..., None] + sums))[0]).all(), (r, i)
        assert (np.abs(glse[row0 + i] - rl[0]) <= (ds + sums + 2.0 ** -20 * np.abs(rl))[0]).all(), (r, i)


@pytest.mark.parametrize("cu,served,rows", [
    ([0, 3, 2, 6], [(0, 0, 3)], 7),                              # the third begins inside the first
    ([0, 2, 2, 7], [(0, 0, 2)], 6),                              # past the rows
    ([0, 2, 1, 1, 2, 5, 5, 8], [(0, 0, 2), (4, 2, 3), (6, 5, 3)], 8),   # (the third rests, the fourth begins inside the first)
    ([0, 4, 0, 4, 0, 4, 0, 4], [(0, 0, 4)], 5),                  # a saw: the first alone
    ([0, 90, 40, 130], [(0, 0, 90)], 130),                       # the same with tiles
    ([0, 70, 0, 70, 0, 70, 70, 99], [(0, 0, 70), (6, 70, 29)], 110),
    ([-2, 3, 1, 4, 30], [(3, 4, 26)], 31),                       # (the first ends at 3)
    ([0, 30, 33, 20, 50, 50, 52], [(0, 0, 30), (1, 30, 3), (5, 50, 2)], 60),
])
def test_offsets_out_of_order(cu, served, rows, workspace):
    """Where offsets fall, requests that begin below an earlier offset are left
    out and latched, the others are answered, and rows of no answered one are as
    they were."""
    n = len(cu) - 1
    s = paged.make_attention([60 + 7 * r for r in range(n)], [100] * n, 8, 2, 64, 16, torch.bfloat16, seed=n, garbage=0.0)
    s["q"], s["cu"] = s["q"][:rows].contiguous(), np.array(cu)
    got, glse, status = attend(s, workspace, 100)
    few, flse, fstatus = attend(s, workspace, 4) if max(k for _, _, k in served) <= 4 else (None, None, None)
    assert status == mk.MK_ERR_BOUNDS and fstatus in (None, mk.MK_ERR_BOUNDS)
    for o, l in ((got, glse), (few, flse)):
        if o is None:
            continue
        left = np.ones(rows, bool)
        for r, row0, k in served:
            left[row0:row0 + k] = False
            check_rows(s, o, l, r, row0, k, int(s["kv"][r]))
        assert (o[left] == 5).all() and (l[left] == 5).all()


def test_a_long_saw_of_offsets(workspace):
    # every second request claims all rows: of 2000 the first is answered
    n, rows = 2000, 300
    one = paged.make_attention([50], [rows], 8, 2, 64, 16, torch.bfloat16, seed=2, garbage=0.0)
    table = np.full((n, one["table"].shape[1]), -1)
    table[0] = one["table"][0]
    s = dict(one, table=table, cu=np.array([0, rows] * (n // 2) + [0]), kv=np.array([50 + rows] * n))
    got, glse, status = attend(s, workspace, rows)
    want, wlse, ok = attend(one, workspace, rows)
    assert status == mk.MK_ERR_BOUNDS and ok == 0
    assert np.array_equal(got, want) and np.array_equal(glse, wlse)


@pytest.mark.parametrize("new", [2, 50])
def test_lengths_past_the_table(new, workspace):
    # rows stand at their positions, keys past the table's width are absent
    s = paged.make_attention([100, 90, 100], [new] * 3, 8, 2, 64, 16, torch.bfloat16, seed=13, garbage=0.0)
    room = s["table"].shape[1] * 16
    s["table"][1] = np.arange(s["table"].shape[1]) % s["k"].shape[0]
    for kv in (room + 1, room + new - 1, room + 40, 2 ** 31 - 1):
        t = dict(s, kv=np.array([s["kv"][0], kv, s["kv"][2]]))
        got, glse, status = attend(t, workspace, new)
        assert status == mk.MK_ERR_BOUNDS
        for r in range(3):
            check_rows(t, got, glse, r, r * new, new, int(t["kv"][r]), room)


@pytest.mark.parametrize("n", [500, 1500])
def test_many_requests_with_chunks(n, workspace):
    """Decode rows, drafted tokens and chunks of more than eight tiles among
    several requests a thread, and more of them than are kept in shared memory."""
    rng = np.random.default_rng(n)
    ctx = rng.integers(0, 40, n)
    new = rng.choice([0, 1, 1, 1, 2, 5], n)
    for r in rng.permutation(n)[:6]:
        new[r] = int(rng.integers(260, 420))      # 8 query heads on a kv head: tiles of 32 tokens
    for r in rng.permutation(n)[:30]:
        new[r] = int(rng.integers(3, 70))
    s = paged.make_attention(ctx.tolist(), new.tolist(), 8, 1, 64, 16, torch.bfloat16, seed=n, pad=2)
    paged.check_attention(s, workspace=workspace)
    paged.check_attention(s, window=33, workspace=workspace)


def test_bounds_past_32_bits(workspace):
    # a window past every position is none; its low 32 bits would be a window of 5
    s = paged.make_attention([300, 20], [2, 40], 8, 2, 64, 16, torch.bfloat16, seed=8, garbage=0.0)
    want, wlse = paged.check_attention(s, workspace=workspace)
    for max_new in (2 ** 32 + 1, 2 ** 31, 40):
        batch = mk.PagedBatch(ints(s["table"]), ints(s["cu"]), ints(s["kv"]), page_size=16, max_new=max_new)
        cache, out = mk.PagedCache(s["k"], s["v"], n_q_heads=8, workspace=workspace), torch.zeros_like(want)
        for window in (2 ** 32 + 5, 2 ** 31, 10 ** 12, 2 ** 31 - 1, 0):
            cache.attention(s["q"], batch, out.zero_(), window=window)
            assert torch.equal(out, want) and cache.status() == 0
        batch.max_new = 2 ** 32 + 1
        assert batch.max_new == 2 ** 31 - 1


# ---------------------------------------------------------------- threads

def test_tables_of_many_requests_from_two_threads():
    """Steps of different numbers of requests, all of them past 48 KB of shared memory."""
    def step(n, errors):
        b = mk.PagedBatch(ints(np.full((n, 1), -1)), ints([0] * (n + 1)), ints([0] * n), ints([0] * n), ints([0] * n), page_size=16, max_new=1)
        free, count, left = ints(np.arange(n)), ints([n]), ints([0])
        ctx, new = ints([0] * n), ints([1] * n)
        stream = torch.cuda.Stream()
        torch.cuda.synchronize()
        try:
            for _ in range(4000):
                b.build(ctx, new, free, count, left, stream=stream)
        except mk.MkError as e:
            errors.append(e)
        stream.synchronize()
        if not torch.equal(b.slots.cpu(), 16 * torch.arange(n - 1, -1, -1, dtype=torch.int32)) or left.item() != 0:
            errors.append(n)

    errors = []
    threads = [threading.Thread(target=step, args=(n, errors)) for n in (4096, 4088, 4080)]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    assert not errors


def test_a_batch_that_calls_share():
    """A call that comes between another's arguments and its launch (a second
    thread's, where the first has given up the interpreter) leaves what that one
    says of the batch as it was."""
    s = paged.make_attention([40, 20, 30], [1, 2, 1], 4, 2, 64, 16, torch.bfloat16, seed=2, garbage=0.0)
    n, rows = 3, 4
    table = ints(s["table"])
    batch = mk.PagedBatch(table, ints(s["cu"]), ints(s["kv"]), ints([0] * rows), ints([0] * rows), page_size=16, max_new=2)
    cache, out = mk.PagedCache(s["k"], s["v"], n_q_heads=4), torch.zeros_like(s["q"])
    cache.attention(s["q"], batch, out)
    want = out.clone()

    def between(name, owner, call, inner):
        real = getattr(owner, name)

        def spy(*args):
            setattr(owner, name, real)
            inner()
            return real(*args)
        setattr(owner, name, spy)
        call()
        assert getattr(owner, name) is real

    status, left = ints([0]), ints([0])
    between("_build", batch, lambda: batch.build(ints([40, 20, 30]), ints([1, 2, 1]), ints(np.arange(5)), ints([5]), left, status=status),
            lambda: cache.attention(s["q"][:1], batch, out[:1]))
    assert status.item() == 0 and batch.cu_new.tolist() == s["cu"].tolist() and batch.kv_lens.tolist() == s["kv"].tolist()
    assert cache.status() == mk.MK_ERR_BOUNDS        # of the inner call: rows past the first
    cache.reset()
    out.zero_()
    small = torch.zeros_like(out[:1])
    between("_attention", cache, lambda: cache.attention(s["q"], batch, out), lambda: cache.attention(s["q"][:1], batch, small))
    assert torch.equal(out, want) and torch.equal(small, want[:1])


def test_max_new_of_a_batch_can_be_set(workspace):
    """A decode step on a batch that was made for chunks."""
    s = paged.make_attention([300, 20, 900], [1, 1, 1], 8, 2, 128, 16, torch.bfloat16, seed=6)
    want, _ = paged.check_attention(s, workspace=workspace, max_new=1)
    batch = mk.PagedBatch(ints(s["table"]), ints(s["cu"]), ints(s["kv"]), page_size=16, max_new=512)
    cache, out = mk.PagedCache(s["k"], s["v"], n_q_heads=8, workspace=workspace), torch.zeros_like(s["q"])
    batch.max_new = 1
    cache.attention(s["q"], batch, out)
    assert batch.max_new == 1 and torch.equal(out, want) and cache.status() == 0
    two = paged.make_attention([300], [2], 8, 2, 128, 16, torch.bfloat16, seed=6)
    b2 = mk.PagedBatch(ints(two["table"]), ints(two["cu"]), ints(two["kv"]), page_size=16, max_new=2)
    c2, o2 = mk.PagedCache(two["k"], two["v"], n_q_heads=8, workspace=workspace), torch.full_like(two["q"], 5.0)
    b2.max_new = 1
    c2.attention(two["q"], b2, o2)                   # more than the bound: left as they were, latched
    assert c2.status() == mk.MK_ERR_BOUNDS and (o2 == 5).all()
    c2.reset()
    b2.max_new = 2
    c2.attention(two["q"], b2, o2)
    assert c2.status() == 0 and not (o2 == 5).any()
    b2.max_new = 0
    with pytest.raises(mk.MkError):
        c2.attention(two["q"], b2, o2)


# ---------------------------------------------------------------- streams

@pytest.mark.parametrize("given", ["stream", "current"])
def test_a_cache_dropped_while_another_stream_runs(given):
    """The workspace and the status word belong to the stream that the cache was
    made and first called on; a call still waits on another when the cache goes.
    Neither is handed out before it has run."""
    s = paged.make_attention([40, 900], [1, 3], 4, 2, 64, 16, torch.bfloat16, seed=4, garbage=0.0)
    batch = mk.PagedBatch(ints(s["table"]), ints(s["cu"]), ints(s["kv"]), page_size=16, max_new=3)
    want, out = torch.empty_like(s["q"]), torch.zeros_like(s["q"])
    k, v = s["k"].clone(), s["v"].clone()
    g = torch.Generator().manual_seed(9)
    kn, vn = (torch.randn(4, 2, 64, generator=g).to(torch.bfloat16).to(DEV) for _ in range(2))
    slots = ints([-1, -1, -1, int(s["table"][0, 0]) * 16])
    cache = mk.PagedCache(k, v, 4)
    cache.append(s["q"], kn, vn, slots)
    cache.attention(s["q"], batch, want)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    small, status = cache.workspace.data_ptr(), cache._status.data_ptr()
    with torch.cuda.stream(side):
        torch.cuda._sleep(600_000_000)                # a few tenths of a second
        if given == "current":
            cache.append(s["q"], kn, vn, slots)
            cache.attention(s["q"], batch, out)
    if given == "stream":
        cache.append(s["q"], kn, vn, slots, stream=side)
        cache.attention(s["q"], batch, out, stream=side)
    del cache
    took = [torch.empty(mk.MK_PAGED_WORKSPACE_BYTES, dtype=torch.uint8, device=DEV) for _ in range(2)]
    words = [torch.empty(1, dtype=torch.int32, device=DEV) for _ in range(64)]
    assert not side.query()
    assert small not in [t.data_ptr() for t in took] and status not in [t.data_ptr() for t in words]
    side.synchronize()
    assert torch.equal(out, want)


def test_a_workspace_made_after_other_streams_were_seen():
    # append alone on one stream, then attention on a second, then on the first
    s = paged.make_attention([40], [1], 4, 2, 64, 16, torch.bfloat16, seed=4, garbage=0.0)
    batch = mk.PagedBatch(ints(s["table"]), ints(s["cu"]), ints(s["kv"]), page_size=16, max_new=1)
    kn = torch.zeros(1, 2, 64, dtype=torch.bfloat16, device=DEV)
    first, second = torch.cuda.Stream(), torch.cuda.Stream()
    out, slots = torch.zeros_like(s["q"]), ints([-1])
    cache = mk.PagedCache(s["k"], s["v"], 4)
    torch.cuda.synchronize()
    cache.append(s["q"], kn, kn, slots, stream=first)
    cache.attention(s["q"], batch, out, stream=second)
    torch.cuda.synchronize()
    with torch.cuda.stream(first):
        torch.cuda._sleep(600_000_000)
    cache.attention(s["q"], batch, out, stream=first)
    at = cache.workspace.data_ptr()
    del cache
    with torch.cuda.stream(second):
        again = torch.empty(mk.MK_PAGED_WORKSPACE_BYTES, dtype=torch.uint8, device=DEV)
    assert not first.query() and again.data_ptr() != at
    torch.cuda.synchronize()


@pytest.mark.parametrize("d,typ", [(128, "bf16"), (64, "fp16")])
def test_steps_end_to_end_without_waiting(d, typ, workspace):
    """Steps of tables, append and attention (decode rows and chunks, lengths that
    change from step to step in the same arrays) launched behind one another, every
    launch starting before its predecessor has ended: the same bits as with a wait
    after every call."""
    typ, hq, hkv, page, n, steps, width, pool = TYPES[typ], 8, 2, 16, 6, 24, 40, 240
    rng = np.random.default_rng(d)
    plan = [[int(x) for x in rng.choice([0, 1, 1, 1, 2, 9, 17], n)] for _ in range(steps)]
    plan[0], plan[5][1], plan[11][4] = [70, 1, 33, 0, 150, 5], 120, 64
    rows = max(sum(p) for p in plan) + 2
    g = torch.Generator().manual_seed(d)
    qkv = torch.randn(steps, rows, hq + 2 * hkv, d, generator=g).to(typ).to(DEV)
    lens = [ints(np.sum(plan[:i], 0) if i else [0] * n) for i in range(steps)]
    adds = [ints(p) for p in plan]
    rope, order = mk.Rope(d), rng.permutation(pool)

    def run(wait):
        kc, vc = (torch.zeros(pool, hkv, page, d, dtype=typ, device=DEV) for _ in range(2))
        cache = mk.PagedCache(kc, vc, n_q_heads=hq, workspace=workspace)
        batch = mk.PagedBatch(ints(np.full((n, width), -1)), ints([0] * (n + 1)), ints([0] * n), ints([0] * rows), ints([0] * rows), page_size=page, max_new=150)
        free, counts = ints(order), [ints([pool])] + [ints([0]) for _ in range(steps)]
        q = qkv[:, :, :hq].clone()
        outs = torch.zeros(steps, rows, hq, d, dtype=typ, device=DEV)
        torch.cuda.synchronize()
        for i in range(steps):
            batch.build(lens[i], adds[i], free, counts[i], counts[i + 1], status=cache._status)
            if wait:
                torch.cuda.synchronize()
            cache.append(q[i], qkv[i, :, hq:hq + hkv], qkv[i, :, hq + hkv:], batch.slots, batch.positions, rope)
            if wait:
                torch.cuda.synchronize()
            cache.attention(q[i], batch, outs[i])
            if wait:
                torch.cuda.synchronize()
        assert cache.status() == 0
        return outs, kc, vc, counts[-1]

    want = run(True)
    for _ in range(5):
        assert all(torch.equal(a, b) for a, b in zip(run(False), want))
