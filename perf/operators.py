"""The operators of the paged KV cache, as a serving program calls them, with plain forms of the same sums.

* tables: block tables, slot maps, positions and offsets of a step from the requests' lengths, pages from a free list;
* append: RMSNorm of q and k where the model has it, rotary positions of one or several axes, k and v written to pages;
* attention: each request's new tokens (one, a few, a chunk of a prompt) against its pages, causal, with or without a window.

Head layouts are those of the model shapes in tile_level_overlap_gb300/synth.py (32 query heads on 8 kv heads of 128 or 64).
"""
import math
import random

import numpy as np
import torch

own = False  # False: the plain forms; True: the framework's entry points

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def listed():
    return [
        # a decode step of 32 running sequences, one new token each: pure latency, every step pays it
        {"name": "tables-decode-32", "op": "tables", "n": 32, "chunks": 0, "ctx_lo": 512, "ctx_hi": 2048, "new_lo": 1, "new_hi": 1, "page": 16, "pad": 0},
        # a busy step: a few hundred sequences, some of them with a chunk of a prompt, rows padded for a captured graph
        {"name": "tables-mixed-301", "op": "tables", "n": 301, "chunks": 44, "ctx_lo": 0, "ctx_hi": 9001, "new_lo": 17, "new_hi": 512, "page": 32, "pad": 1000},
        # admission of 64 whole prompts at once
        {"name": "tables-prompts-64", "op": "tables", "n": 64, "chunks": 64, "ctx_lo": 0, "ctx_hi": 0, "new_lo": 700, "new_hi": 4096, "page": 16, "pad": 0},
        # the decode step's new rows of a model with q/k norm (Qwen3-8B heads), q, k and v in one projection's rows
        {"name": "append-decode-32", "op": "append", "tokens": 32, "hq": 32, "hkv": 8, "d": 128, "rot": 128, "axes": 1, "norm": True, "packed": True, "page": 16, "pos": 2048, "type": "bf16"},
        # 1B-shape heads, a ragged prompt chunk in fp16 far into a long context
        {"name": "append-fp16-1999", "op": "append", "tokens": 1999, "hq": 32, "hkv": 8, "d": 64, "rot": 64, "axes": 1, "norm": False, "packed": False, "page": 32, "pos": 1000000, "type": "fp16"},
        # the tokens of a video: time, height and width each turn their own pairs
        {"name": "append-video-8190", "op": "append", "tokens": 8190, "hq": 32, "hkv": 8, "d": 128, "rot": 128, "axes": 3, "norm": True, "packed": True, "page": 64, "pos": 8192, "type": "bf16"},
        # one sequence decoding at context 4096 (the benchmark's own step): the smallest call
        {"name": "decode-1x4096", "op": "attention", "n": 1, "chunks": 0, "ctx_lo": 4096, "ctx_hi": 4096, "new_lo": 1, "new_hi": 1, "hq": 32, "hkv": 8, "d": 128, "page": 16, "window": 0, "type": "bf16"},
        # 32 sequences at ragged contexts (the batched benchmark's)
        {"name": "decode-32-ragged", "op": "attention", "n": 32, "chunks": 0, "ctx_lo": 512, "ctx_hi": 2048, "new_lo": 1, "new_hi": 1, "hq": 32, "hkv": 8, "d": 128, "page": 16, "window": 0, "type": "bf16"},
        # long documents: two sequences of about 128K keys, four drafted tokens each to verify
        {"name": "verify-2x128k", "op": "attention", "n": 2, "chunks": 2, "ctx_lo": 130000, "ctx_hi": 131072, "new_lo": 4, "new_hi": 4, "hq": 32, "hkv": 8, "d": 128, "page": 64, "window": 0, "type": "bf16"},
        # a step that mixes running sequences with chunks of prompts, 1B-shape heads, fp16, sliding window, odd lengths
        {"name": "mixed-window-fp16", "op": "attention", "n": 27, "chunks": 5, "ctx_lo": 1, "ctx_hi": 4099, "new_lo": 130, "new_hi": 517, "hq": 32, "hkv": 8, "d": 64, "page": 32, "window": 1024, "type": "fp16"},
        # chunked prefill: the next 512 or so tokens of two prompts whose first thousands are cached
        {"name": "chunk-2x512", "op": "attention", "n": 2, "chunks": 2, "ctx_lo": 4000, "ctx_hi": 12000, "new_lo": 470, "new_hi": 512, "hq": 32, "hkv": 8, "d": 128, "page": 16, "window": 0, "type": "bf16"},
        # a whole prompt of 8192 tokens: the largest call
        {"name": "prompt-8192", "op": "attention", "n": 1, "chunks": 1, "ctx_lo": 0, "ctx_hi": 0, "new_lo": 8192, "new_hi": 8192, "hq": 32, "hkv": 8, "d": 128, "page": 64, "window": 0, "type": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tables", "append", "attention", "attention"])
    page = rng.choice([16, 32, 64, 128])
    if op == "tables":
        n = _log(rng, 1, 1024)
        return {"op": op, "n": n, "chunks": rng.choice([0, n, rng.randint(0, n)]), "ctx_lo": 0, "ctx_hi": _log(rng, 1, 16384), "new_lo": 1,
                "new_hi": _log(rng, 1, max(2, min(8192, 260000 // n))), "page": page, "pad": rng.choice([0, rng.randint(0, 999)])}
    hkv = rng.choice([1, 2, 4, 8])
    d, typ = rng.choice([64, 128]), rng.choice(["bf16", "fp16"])
    if op == "append":
        rot = rng.choice([d, d, d // 2])
        return {"op": op, "tokens": _log(rng, 1, 8192), "hq": hkv * rng.choice([1, 2, 3, 4]), "hkv": hkv, "d": d, "rot": rot, "axes": rng.choice([1, 2, 3]),
                "norm": rng.random() < 0.5, "packed": rng.random() < 0.5, "page": page, "pos": _log(rng, 100, 1000000), "type": typ}
    kind = rng.choice(["decode", "few", "chunk", "mixed"])
    rep = rng.choice([1, 2, 3, 4, 5, 7, 8])
    n = _log(rng, 1, 128 if kind == "decode" else 64 if kind == "few" else 16)
    new_hi = {"decode": 1, "few": rng.randint(2, 8)}.get(kind) or _log(rng, 9, 2048)
    # n x new x keys x heads stays below what the largest listed case has
    most = max(64, min(131072 if kind == "decode" else 32768, 2 ** 31 // (n * new_hi * hkv * rep), 2 ** 30 // (n * hkv * d)))
    chunks = {"decode": 0, "mixed": rng.randint(0, n)}.get(kind, n)
    return {"op": op, "n": n, "chunks": chunks, "ctx_lo": 0, "ctx_hi": _log(rng, 16, most), "new_lo": 1 if kind == "few" else min(9, new_hi), "new_hi": new_hi,
            "hq": hkv * rep, "hkv": hkv, "d": d, "page": page, "window": rng.choice([0, 0, _log(rng, 1, 4096)]), "type": typ}


def _lengths(case):
    """Cached and new tokens of each request: the first `chunks` bring a chunk of a prompt, the others one token."""
    rng = random.Random("%(n)d %(chunks)d %(ctx_lo)d %(ctx_hi)d %(new_lo)d %(new_hi)d" % case)
    ctx = [rng.randint(case["ctx_lo"], case["ctx_hi"]) for _ in range(case["n"])]
    new = [rng.randint(case["new_lo"], case["new_hi"]) if r < case["chunks"] else 1 for r in range(case["n"])]
    return ctx, new


def _ceil(a, b):
    return -(-a // b)


def _ints(v, dtype=torch.int32):
    return torch.tensor(v, dtype=dtype, device=DEV)


def _prepare_tables(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    ctx, new = _lengths(case)
    page, n = case["page"], case["n"]
    held = [_ceil(c, page) for c in ctx]
    need = [_ceil(c + w, page) - h for c, w, h in zip(ctx, new, held)]
    width = max(h + w for h, w in zip(held, need)) + 3
    spare = 57  # pages that stay free
    pages = torch.randperm(sum(held) + sum(need) + spare, generator=g, device=DEV).to(torch.int32)
    h = _ints(held)
    col = torch.arange(width, device=DEV)
    first = torch.cumsum(h, 0) - h
    at = (first[:, None] + col).clamp(max=pages.numel() - 1)
    table = torch.where(col < h[:, None], pages[at], -1).to(torch.int32)
    total = sum(new)
    rows = total + case["pad"]
    s = {"case": case, "ctx": _ints(ctx), "new": _ints(new), "free": pages[sum(held):].contiguous(), "n_free": _ints([sum(need) + spare]), "n_left": _ints([0]),
         "table": table, "cu_new": _ints([0] * (n + 1)), "kv_lens": _ints([0] * n), "positions": _ints([0] * rows), "slots": _ints([0] * rows)}
    if own:
        from tile_level_overlap_gb300 import mk
        s["batch"] = mk.PagedBatch(s["table"], s["cu_new"], s["kv_lens"], s["positions"], s["slots"], page_size=page, max_new=max(new))
    return s


def _plain_tables(s):
    page = s["case"]["page"]
    ctx, new, table = s["ctx"].long(), s["new"].long(), s["table"]
    width, n_free, rows = table.shape[1], s["n_free"].long(), s["slots"].numel()
    good = (ctx >= 0) & (new >= 0) & (ctx + new <= width * page)
    new = torch.where(good, new, 0)
    held = (ctx + page - 1) // page
    need = torch.where(good, (ctx + new + page - 1) // page - held, 0)
    upto = torch.cumsum(need, 0)
    served = good & ((need == 0) | (upto <= n_free))
    left = n_free - torch.where(served, upto, 0).amax()
    col = torch.arange(width, device=DEV)
    j = col - held[:, None]
    at = (n_free - 1 - (upto - need)[:, None] - j).clamp(min=0, max=s["free"].numel() - 1)
    table = torch.where((j >= 0) & (j < need[:, None]) & served[:, None], s["free"][at], table)
    cu = torch.cat([torch.zeros_like(upto[:1]), torch.cumsum(new, 0)])
    kv = torch.where(served, ctx + new, 0)
    t = torch.arange(rows, device=DEV)
    r = torch.searchsorted(cu, t, right=True) - 1
    real = t < cu[-1]
    r = r.clamp(max=ctx.numel() - 1)
    pos = torch.where(real, ctx[r] + t - cu[r], 0)
    slot = torch.where(real & served[r], table[r, (pos // page).clamp(max=width - 1)].long() * page + pos % page, -1)
    i32 = torch.int32
    return {"table": table, "cu_new": cu.to(i32), "kv_lens": kv.to(i32), "positions": pos.to(i32), "slots": slot.to(i32), "n_left": left.to(i32)}


def _own_tables(s):
    s["batch"].build(s["ctx"], s["new"], s["free"], s["n_free"], s["n_left"])
    return {"table": s["table"], "cu_new": s["cu_new"], "kv_lens": s["kv_lens"], "positions": s["positions"], "slots": s["slots"], "n_left": s["n_left"]}


def _sections(case):
    """How many pairs each axis turns."""
    half, axes = case["rot"] // 2, case["axes"]
    return [half - (axes - 1) * (half // (axes + 1))] + [half // (axes + 1)] * (axes - 1)


def _axis_of_pair(case):
    return [a for a, k in enumerate(_sections(case)) for _ in range(k)]


THETA, EPS = 1000000.0, 1e-6


def _prepare_append(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    typ, t, hq, hkv, d, page = TYPES[case["type"]], case["tokens"], case["hq"], case["hkv"], case["d"], case["page"]
    normal = lambda *shape: torch.randn(shape, generator=g, device=DEV).to(typ)  # noqa: E731
    if case["packed"]:
        rows = normal(t, hq + 2 * hkv, d)
        q, k, v = rows[:, :hq], rows[:, hq:hq + hkv], rows[:, hq + hkv:]
    else:
        q, k, v = normal(t, hq, d), normal(t, hkv, d), normal(t, hkv, d)
    pages = _ceil(t, page) + 3
    slots = (torch.randperm(pages, generator=g, device=DEV)[:, None] * page + torch.arange(page, device=DEV)).reshape(-1)[:t].to(torch.int32)
    start = torch.randint(0, max(1, case["pos"] - t + 1), (case["axes"], 1), generator=g, device=DEV)
    step = torch.tensor([[1], [3], [5]], device=DEV)[:case["axes"]]  # the other axes move slower or return, as rows and columns of a picture do
    positions = (start + torch.arange(t, device=DEV) // step % max(1, case["pos"])).to(torch.int32).contiguous()
    gain = lambda: (1 + 0.02 * torch.randn(d, generator=g, device=DEV)).to(typ) if case["norm"] else None  # noqa: E731
    s = {"case": case, "q": q, "k": k, "v": v, "slots": slots, "positions": positions, "q_norm": gain(), "k_norm": gain(), "axis": _ints(_axis_of_pair(case), torch.int64),
         "k_cache": normal(pages, hkv, page, d), "v_cache": normal(pages, hkv, page, d), "q_out": torch.empty(t, hq, d, dtype=typ, device=DEV)}
    if own:
        from tile_level_overlap_gb300 import mk
        s["cache"] = mk.PagedCache(s["k_cache"], s["v_cache"], n_q_heads=hq)
        s["rope"] = mk.Rope(d, theta=THETA, rotary_dim=case["rot"], sections=_sections(case))
    return s


def _turned(x, cos, sin):
    h = cos.shape[-1]
    a, b = x[..., :h], x[..., h:2 * h]
    return torch.cat([a * cos - b * sin, b * cos + a * sin, x[..., 2 * h:]], -1)


def _plain_append(s):
    case = s["case"]
    typ, page = s["q"].dtype, case["page"]
    pair = torch.arange(case["rot"] // 2, dtype=torch.float64, device=DEV)
    angle = s["positions"].double()[s["axis"]].t() * THETA ** (-2 * pair / case["rot"])
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    q, k = s["q"].float(), s["k"].float()
    if case["norm"]:
        q = q * torch.rsqrt((q * q).mean(-1, keepdim=True) + EPS) * s["q_norm"].float()
        k = k * torch.rsqrt((k * k).mean(-1, keepdim=True) + EPS) * s["k_norm"].float()
    slot = s["slots"].long()
    s["k_cache"][slot // page, :, slot % page] = _turned(k, cos, sin).to(typ)
    s["v_cache"][slot // page, :, slot % page] = s["v"]
    return {"q": _turned(q, cos, sin).to(typ), "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _own_append(s):
    s["cache"].append(s["q"], s["k"], s["v"], s["slots"], s["positions"], s["rope"], q_out=s["q_out"], q_norm=s["q_norm"], k_norm=s["k_norm"], eps=EPS)
    return {"q": s["q_out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _exact_append(s):
    case = s["case"]
    page, half = case["page"], case["rot"] // 2
    freq = torch.tensor([THETA ** (-i / half) for i in range(half)], dtype=torch.float64, device=DEV)
    angle = torch.stack([s["positions"][a].double() * freq[i] for i, a in enumerate(_axis_of_pair(case))], 1)
    turn = torch.polar(torch.ones_like(angle), angle)[:, None]

    def rows(x, gain):
        x = x.double()
        if gain is not None:
            x = x / (x.square().sum(-1, keepdim=True) / x.shape[-1] + EPS).sqrt() * gain.double()
        z = torch.complex(x[..., :half].contiguous(), x[..., half:2 * half].contiguous()) * turn
        x = x.clone()
        x[..., :half], x[..., half:2 * half] = z.real, z.imag
        return x

    k_cache, v_cache = s["k_cache"].double(), s["v_cache"].double()
    p, o = s["slots"].long() // page, s["slots"].long() % page
    k_cache[p, :, o] = rows(s["k"], s["k_norm"])
    v_cache[p, :, o] = s["v"].double()
    return {"q": rows(s["q"], s["q_norm"]), "k_cache": k_cache, "v_cache": v_cache}


def _prepare_attention(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    typ, page, hq, hkv, d = TYPES[case["type"]], case["page"], case["hq"], case["hkv"], case["d"]
    ctx, new = _lengths(case)
    kv = [c + w for c, w in zip(ctx, new)]
    need = [_ceil(x, page) for x in kv]
    width = max(need) + 1
    pages = sum(need) + 5
    order = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
    h = _ints(need)
    col = torch.arange(width, device=DEV)
    at = ((torch.cumsum(h, 0) - h)[:, None] + col).clamp(max=pages - 1)
    total = sum(new)
    normal = lambda *shape: torch.randn(shape, generator=g, device=DEV, dtype=torch.float32).to(typ)  # noqa: E731
    cu = [0]
    for w in new:
        cu.append(cu[-1] + w)
    s = {"case": case, "q": normal(total, hq, d), "k_cache": normal(pages, hkv, page, d), "v_cache": normal(pages, hkv, page, d),
         "table": torch.where(col < h[:, None], order[at], -1).to(torch.int32).contiguous(), "cu_new": _ints(cu), "kv_lens": _ints(kv), "max_new": max(new),
         "out": torch.empty(total, hq, d, dtype=typ, device=DEV), "lse": torch.empty(total, hq, dtype=torch.float32, device=DEV)}
    if own:
        from tile_level_overlap_gb300 import mk
        s["batch"] = mk.PagedBatch(s["table"], s["cu_new"], s["kv_lens"], page_size=page, max_new=s["max_new"])
        s["cache"] = mk.PagedCache(s["k_cache"], s["v_cache"], n_q_heads=hq)
    return s


def _plain_attention(s):
    case = s["case"]
    hq, hkv, d, page, most = case["hq"], case["hkv"], case["d"], case["page"], s["max_new"]
    cu, kv = s["cu_new"].long(), s["kv_lens"].long()
    n, keys, total = kv.numel(), s["table"].shape[1] * page, s["q"].shape[0]
    at = s["table"].clamp(min=0).long()
    j = torch.arange(keys, device=DEV)
    k = s["k_cache"][at].transpose(1, 2).reshape(n, hkv, keys, d).float()
    v = s["v_cache"][at].transpose(1, 2).reshape(n, hkv, keys, d).float()
    v = torch.where((j < kv[:, None])[:, None, :, None], v, 0)
    i = torch.arange(most, device=DEV)
    q = s["q"][(cu[:-1, None] + i).clamp(max=total - 1)].float().reshape(n, most, hkv, hq // hkv, d).permute(0, 2, 3, 1, 4).reshape(n, hkv, -1, d)
    pos = (kv - cu[1:] + cu[:-1])[:, None] + i
    seen = (j <= pos[..., None]) & (j < kv[:, None, None])
    if case["window"]:
        seen = seen & (j > pos[..., None] - case["window"])
    x = (q @ k.transpose(2, 3)).mul_(d ** -0.5).reshape(n, hkv, hq // hkv, most, keys)
    x.masked_fill_(~seen[:, None, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0, top)
    x.sub_(top).exp_()
    tot = x.sum(-1, keepdim=True)
    o = (x.reshape(n, hkv, -1, keys) @ v).reshape(n, hkv, hq // hkv, most, d) / torch.where(tot > 0, tot, 1)
    lse = (top + tot.log())[..., 0]
    t = torch.arange(total, device=DEV)
    r = torch.searchsorted(cu, t, right=True) - 1
    rows = lambda y: y.movedim(3, 1)[r, t - cu[r]].flatten(1, 2)  # noqa: E731
    return {"out": rows(o).to(s["q"].dtype), "lse": rows(lse)}


def _own_attention(s):
    s["cache"].attention(s["q"], s["batch"], s["out"], lse=s["lse"], window=s["case"]["window"])
    return {"out": s["out"], "lse": s["lse"]}


def _exact_attention(s):
    case = s["case"]
    hq, hkv, page, d = case["hq"], case["hkv"], case["page"], case["d"]
    outs, lses = [], []
    cu, kv = s["cu_new"].tolist(), s["kv_lens"].tolist()
    for r, total in enumerate(kv):
        a, b = cu[r], cu[r + 1]
        pages = s["table"][r, :_ceil(total, page)].long()
        for h in range(hq):
            k = s["k_cache"][pages, h * hkv // hq].reshape(-1, d)[:total].double()
            v = s["v_cache"][pages, h * hkv // hq].reshape(-1, d)[:total].double()
            pos = torch.arange(total - (b - a), total, device=DEV)[:, None]
            key = torch.arange(total, device=DEV)
            hidden = (key > pos) | (key <= pos - (case["window"] or total + 1))
            score = (s["q"][a:b, h].double() @ k.t() / math.sqrt(d)).masked_fill(hidden, -math.inf)
            lse = torch.logsumexp(score, -1)
            outs.append(torch.exp(score - lse[:, None]) @ v)
            lses.append(lse)
    merge = lambda parts: torch.cat([torch.stack(parts[r * hq:(r + 1) * hq], 1) for r in range(len(kv))])  # noqa: E731
    return {"out": merge(outs), "lse": merge(lses)}


def prepare(case, seed):
    return {"tables": _prepare_tables, "append": _prepare_append, "attention": _prepare_attention}[case["op"]](case, seed)


def run(state):
    op = state["case"]["op"]
    if own:
        return {"tables": _own_tables, "append": _own_append, "attention": _own_attention}[op](state)
    return {"tables": _plain_tables, "append": _plain_append, "attention": _plain_attention}[op](state)


def exact(case, seed):
    if case["op"] == "tables":
        return None  # whole numbers
    s = prepare(case, seed)
    return _exact_append(s) if case["op"] == "append" else _exact_attention(s)


def work(case):
    if case["op"] == "append":
        row = (case["hq"] + 2 * case["hkv"]) * case["d"]
        turned = (case["hq"] + case["hkv"]) * case["d"]
        gains = 4 * case["d"] if case["norm"] else 0
        return {"bytes": case["tokens"] * (4 * row + 4 + 4 * case["axes"]) + gains, "flops": case["tokens"] * turned * (7 if case["norm"] else 3)}
    ctx, new = _lengths(case)
    ctx, new, page = np.array(ctx, dtype=np.int64), np.array(new, dtype=np.int64), case["page"]
    n, total = case["n"], int(new.sum())
    if case["op"] == "tables":
        taken = int((-(-(ctx + new) // page) - -(-ctx // page)).sum())
        started = int((ctx % page > 0).sum())  # requests whose next token goes to a page that they hold
        return {"bytes": 8 * n + 8 * taken + 4 * started + 4 * (2 * n + 1) + 8 * (total + case["pad"]) + 8, "flops": 4 * total}
    w = case["window"] or 1 << 40
    read = np.minimum(ctx + new, w + new - 1)  # keys that any of a request's rows sees
    seen = sum(int(np.minimum(np.arange(c + 1, c + k + 1), w).sum()) for c, k in zip(ctx.tolist(), new.tolist()))
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    tables = 4 * int((-(-(ctx + new) // page)).sum()) + 4 * (2 * n + 1)
    return {"bytes": int(read.sum()) * hkv * d * 4 + total * hq * (4 * d + 4) + tables, "flops": 4 * d * hq * seen}
