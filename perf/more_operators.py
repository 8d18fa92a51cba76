"""The operators of speculative decoding over the paged KV cache, as a serving program calls them, with plain forms of the same sums.

* tree: each drafted token's ancestors as a bit mask, and its position, from the tree's parents;
* attention: the rows of a tree over a request's pages, each seeing the cached tokens and its own ancestors;
* verify: which drafted tokens stand against the target's probabilities, and the token that follows them, from given random numbers;
* trim: the accepted path's keys and values move together in every layer, the pages behind them and those of finished requests go back to the free list;
* fork: requests that continue others share their whole pages; a page that two would write is copied in every layer.

Head layouts, vocabularies and layers are those of the model shapes in tile_level_overlap_gb300/synth.py.
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
        # a step's trees of 32 running sequences: pure latency, every step pays it
        {"name": "tree-32x16", "op": "tree", "n": 32, "lo": 16, "hi": 16, "chain": False, "words": 1, "ctx": 2048, "pad": 0},
        # a busy step: 256 sequences with trees of all sizes, rows padded for a captured graph
        {"name": "tree-256x128", "op": "tree", "n": 256, "lo": 1, "hi": 128, "chain": False, "words": 4, "ctx": 4096, "pad": 777},
        # one sequence with a tree of 32 drafted tokens over 4096 cached ones: the smallest call of a step, paid by every layer
        {"name": "attention-1x4096", "op": "attention", "n": 1, "lo": 32, "hi": 32, "chunks": 0, "chunk": 0, "words": 1, "ctx_lo": 4096, "ctx_hi": 4096, "hq": 32, "hkv": 8, "d": 128,
         "page": 16, "window": 0, "type": "bf16"},
        # 32 sequences at ragged contexts (the batched benchmark's), a tree of up to 64 drafted tokens each
        {"name": "attention-32-ragged", "op": "attention", "n": 32, "lo": 40, "hi": 64, "chunks": 0, "chunk": 0, "words": 2, "ctx_lo": 512, "ctx_hi": 2048, "hq": 32, "hkv": 8, "d": 128,
         "page": 16, "window": 0, "type": "bf16"},
        # small trees beside chunks of two prompts in one step, 1B-shape heads, fp16, sliding window, odd lengths
        {"name": "attention-mixed-fp16", "op": "attention", "n": 48, "lo": 1, "hi": 13, "chunks": 2, "chunk": 301, "words": 1, "ctx_lo": 1, "ctx_hi": 4099, "hq": 32, "hkv": 8, "d": 64,
         "page": 32, "window": 1024, "type": "fp16"},
        # one sequence, four drafted tokens in a row: the smallest verification
        {"name": "verify-1x4", "op": "verify", "n": 1, "lo": 5, "hi": 5, "chain": True, "vocab": 128256, "draft": True},
        # 32 sequences with trees of up to 32 tokens, children drawn from the draft's probabilities (Qwen3-8B vocabulary)
        {"name": "verify-32-trees", "op": "verify", "n": 32, "lo": 17, "hi": 32, "chain": False, "vocab": 151936, "draft": True},
        # 64 sequences whose drafts were looked up in their own text: no draft probabilities
        {"name": "verify-64-lookup", "op": "verify", "n": 64, "lo": 1, "hi": 9, "chain": True, "vocab": 128256, "draft": False},
        # after a verification: 32 sequences keep a path of their trees, in the 32 layers of the 8B shape
        {"name": "trim-32", "op": "trim", "n": 32, "lo": 32, "hi": 32, "ctx_lo": 128, "ctx_hi": 640, "finish": 0.0, "shared": 0, "layers": 32, "hkv": 8, "d": 128, "page": 16, "type": "bf16"},
        # 256 sequences, some of them finished, prompts shared by pairs; 16 layers of the 1B shape
        {"name": "trim-256", "op": "trim", "n": 256, "lo": 1, "hi": 61, "ctx_lo": 64, "ctx_hi": 512, "finish": 0.1, "shared": 64, "layers": 16, "hkv": 8, "d": 64, "page": 32, "type": "fp16"},
        # a step of a search with 16 beams that share most of their pages, 1B shape
        {"name": "fork-beams-16", "op": "fork", "n": 16, "m": 16, "ctx_lo": 900, "ctx_hi": 1100, "shared": 880, "layers": 16, "hkv": 8, "d": 64, "page": 16, "type": "bf16"},
        # eight prompts answered 8 times each: 64 requests from 8, 8B shape
        {"name": "fork-samples-64", "op": "fork", "n": 8, "m": 64, "ctx_lo": 500, "ctx_hi": 2048, "shared": 0, "layers": 32, "hkv": 8, "d": 128, "page": 64, "type": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tree", "attention", "attention", "verify", "trim", "fork"])
    page = rng.choice([16, 32, 64, 128])
    if op == "tree":
        hi = _log(rng, 2, 512)
        return {"op": op, "n": _log(rng, 1, min(1024, max(1, 32768 // hi))), "lo": rng.choice([1, hi]), "hi": hi, "chain": rng.random() < 0.25, "words": rng.choice([-(-hi // 32), 16]),
                "ctx": _log(rng, 1, 100000), "pad": rng.choice([0, rng.randint(0, 999)])}
    hkv = rng.choice([1, 2, 4, 8])
    d, typ = rng.choice([64, 128]), rng.choice(["bf16", "fp16"])
    if op == "attention":
        rep = rng.choice([1, 2, 3, 4, 5, 7, 8])
        hi = _log(rng, 2, 160)
        n = _log(rng, 1, min(64, 4096 // hi))
        chunks = rng.choice([0, 0, rng.randint(0, n)])
        chunk = _log(rng, 170, 600) if chunks else 0
        most = max(64, min(131072, 2 ** 31 // (n * max(hi, chunk) * hkv * rep), 2 ** 29 // (n * hkv * d)))
        return {"op": op, "n": n, "lo": rng.choice([1, hi]), "hi": hi, "chunks": chunks, "chunk": chunk, "words": -(-hi // 32), "ctx_lo": 0, "ctx_hi": _log(rng, 16, most),
                "hq": hkv * rep, "hkv": hkv, "d": d, "page": page, "window": rng.choice([0, 0, _log(rng, 1, 4096)]), "type": typ}
    if op == "verify":
        vocab = rng.choice([_log(rng, 100, 60000), 128256, 151936])
        hi = _log(rng, 2, 48)
        return {"op": op, "n": _log(rng, 1, max(1, min(128, 2 ** 27 // (vocab * hi)))), "lo": rng.choice([1, hi]), "hi": hi, "chain": rng.random() < 0.5, "vocab": vocab,
                "draft": rng.random() < 0.7}
    layers = rng.choice([1, 16, 32])
    fit = max(1, 2 ** 20 // (layers * hkv * d))  # tokens of all requests, in thousands
    n = _log(rng, 1, min(256, 1 + fit))
    ctx = _log(rng, 16, max(32, min(4096, 1000 * fit // n)))
    if op == "trim":
        return {"op": op, "n": n, "lo": 1, "hi": _log(rng, 2, 64), "ctx_lo": 1, "ctx_hi": ctx, "finish": rng.choice([0.0, 0.2, 1.0]), "shared": rng.choice([0, ctx // 2]), "layers": layers,
                "hkv": hkv, "d": d, "page": page, "type": typ}
    most = max(1, 2 ** 27 // (layers * hkv * d * page))  # copied pages stay below what the largest listed case has
    return {"op": op, "n": n, "m": min(most, rng.choice([n, max(1, n // 2), min(512, 4 * n + 3)])), "ctx_lo": 0, "ctx_hi": ctx, "shared": rng.choice([0, ctx // 2]), "layers": layers, "hkv": hkv, "d": d,
            "page": page, "type": typ}


def _ceil(a, b):
    return -(-a // b)


def _ints(v, dtype=torch.int32):
    return torch.tensor(v, dtype=dtype, device=DEV)


def _rng(case):
    """For what a case's shapes are made from, whatever the seed."""
    return random.Random(" ".join("%s" % case[k] for k in sorted(case) if k != "name"))


def _parents(rng, nodes, chain):
    """Each node's parent (the root's is -1): in a tree half of the nodes lengthen the last branch, the others start one."""
    return [-1] + [i - 1 if chain or rng.random() < 0.5 else rng.randrange(i) for i in range(1, nodes)]


def _ancestors(parents):
    """Each node's set of ancestors, itself among them, as a number's bits."""
    masks = []
    for i, p in enumerate(parents):
        masks.append((masks[p] if p >= 0 else 0) | 1 << i)
    return masks


def _starts(lens):
    cu = [0]
    for x in lens:
        cu.append(cu[-1] + x)
    return cu


# ---------------------------------------------------------------- tree

def _trees(case):
    rng = _rng(case)
    new = [rng.randint(case["lo"], case["hi"]) for _ in range(case["n"])]
    return new, [_parents(rng, k, case["chain"]) for k in new]


def _prepare_tree(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    new, trees = _trees(case)
    rows, words = sum(new) + case["pad"], case["words"]
    kv = _ints(new) + torch.randint(0, case["ctx"], (case["n"],), generator=g, device=DEV, dtype=torch.int32)
    s = {"case": case, "cu": _ints(_starts(new)), "kv": kv, "parents": _ints(sum(trees, []) + [-1] * case["pad"]), "masks": torch.zeros(rows, words, dtype=torch.int32, device=DEV),
         "positions": torch.zeros(rows, dtype=torch.int32, device=DEV), "slots": torch.zeros(rows, dtype=torch.int32, device=DEV)}
    if own:
        from tile_level_overlap_gb300 import mk
        table = torch.zeros(case["n"], _ceil(case["ctx"] + case["hi"], 16), dtype=torch.int32, device=DEV)
        s["batch"] = mk.PagedBatch(table, s["cu"], s["kv"], s["positions"], s["slots"], page_size=16, max_new=case["hi"])
        s["tree"] = mk.DraftTree(s["batch"], s["parents"], s["masks"])
    return s


def _plain_tree(s):
    case, cu = s["case"], s["cu"].long()
    rows, words, n = s["masks"].shape[0], s["masks"].shape[1], cu.numel() - 1
    t = torch.arange(rows, device=DEV)
    r = (torch.searchsorted(cu, t, right=True) - 1).clamp(max=n - 1)
    real = t < cu[-1]
    up = torch.where(real & (s["parents"] >= 0), cu[r] + s["parents"], t)  # the root's parent is itself
    own_bit = torch.zeros(rows, 32 * words, dtype=torch.bool, device=DEV)
    own_bit[t, torch.where(real, t - cu[r], 0)] = real
    seen = own_bit
    for _ in range(case["hi"].bit_length()):  # ancestors 1, 2, 4, .. steps up
        seen = seen | seen[up]
        up = up[up]
    weight = torch.ones(32, dtype=torch.int64, device=DEV) << torch.arange(32, device=DEV)
    masks = (seen.reshape(rows, words, 32) * weight).sum(-1)
    masks = torch.where(masks >= 2 ** 31, masks - 2 ** 32, masks).to(torch.int32)
    position = s["kv"].long()[r] - (cu[1:] - cu[:-1])[r] + seen.sum(-1) - 1
    return {"masks": masks, "positions": torch.where(real, position, 0).to(torch.int32)}


def _own_tree(s):
    s["tree"].build()
    return {"masks": s["masks"], "positions": s["positions"]}


# ---------------------------------------------------------------- attention

def _requests(case):
    """Cached tokens, rows and trees (None: a chunk of a prompt) of each request; chunks come first."""
    rng = _rng(case)
    ctx = [rng.randint(case["ctx_lo"], case["ctx_hi"]) for _ in range(case["n"])]
    new = [case["chunk"] - rng.randint(0, 7) if r < case["chunks"] else rng.randint(case["lo"], case["hi"]) for r in range(case["n"])]
    return ctx, new, [None if r < case["chunks"] else _ancestors(_parents(rng, k, False)) for r, k in enumerate(new)]


def _prepare_attention(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    typ, page, hq, hkv, d, words = TYPES[case["type"]], case["page"], case["hq"], case["hkv"], case["d"], case["words"]
    ctx, new, trees = _requests(case)
    kv = [c + w for c, w in zip(ctx, new)]
    need = [_ceil(x, page) for x in kv]
    width = max(need) + 1
    pages = sum(need) + 5
    order = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
    h = _ints(need)
    col = torch.arange(width, device=DEV)
    at = ((torch.cumsum(h, 0) - h)[:, None] + col).clamp(max=pages - 1)
    total = sum(new)
    rows = [m for k, tree in zip(new, trees) for m in (tree or [0] * k)]
    masks = np.array([[m >> 32 * w & 0xffffffff for w in range(words)] for m in rows], dtype=np.uint32).view(np.int32)
    normal = lambda *shape: torch.randn(shape, generator=g, device=DEV, dtype=torch.float32).to(typ)  # noqa: E731
    s = {"case": case, "q": normal(total, hq, d), "k_cache": normal(pages, hkv, page, d), "v_cache": normal(pages, hkv, page, d),
         "table": torch.where(col < h[:, None], order[at], -1).to(torch.int32).contiguous(), "cu": _ints(_starts(new)), "kv": _ints(kv), "most": max(new),
         "masks": torch.from_numpy(masks).to(DEV), "out": torch.empty(total, hq, d, dtype=typ, device=DEV), "lse": torch.empty(total, hq, dtype=torch.float32, device=DEV)}
    if own:
        from tile_level_overlap_gb300 import mk
        s["batch"] = mk.PagedBatch(s["table"], s["cu"], s["kv"], page_size=page, max_new=s["most"])
        s["tree"] = mk.DraftTree(s["batch"], None, s["masks"])
        s["cache"] = mk.PagedCache(s["k_cache"], s["v_cache"], n_q_heads=hq)
    return s


def _plain_attention(s):
    case = s["case"]
    hq, hkv, d, page, most, words = case["hq"], case["hkv"], case["d"], case["page"], s["most"], case["words"]
    cu, kv = s["cu"].long(), s["kv"].long()
    n, keys, total = kv.numel(), s["table"].shape[1] * page, s["q"].shape[0]
    new = cu[1:] - cu[:-1]
    at = s["table"].clamp(min=0).long()
    j = torch.arange(keys, device=DEV)
    k = s["k_cache"][at].transpose(1, 2).reshape(n, hkv, keys, d).float()
    v = s["v_cache"][at].transpose(1, 2).reshape(n, hkv, keys, d).float()
    v = torch.where((j < kv[:, None])[:, None, :, None], v, 0)
    i = torch.arange(most, device=DEV)
    row = (cu[:-1, None] + i).clamp(max=total - 1)
    q = s["q"][row].float().reshape(n, most, hkv, hq // hkv, d).permute(0, 2, 3, 1, 4).reshape(n, hkv, -1, d)
    ctx = (kv - new)[:, None, None]
    # the bits of a tree's rows, or of a chunk's: the row itself and those before it
    bit = torch.arange(32 * max(words, _ceil(most, 32)), device=DEV)
    held = (s["masks"][row].long()[..., (bit // 32).clamp(max=words - 1)] >> bit % 32 & 1 != 0) & (bit < 32 * words)
    bits = torch.where((new > 32 * words)[:, None, None], bit <= i[:, None], held) & (bit <= i[:, None])
    last = ctx + bits.sum(-1, keepdim=True) - 1
    seen = (j < ctx) & (j > last - case["window"] if case["window"] else j >= 0)
    if case["window"]:
        bits = bits & (bits.flip(-1).cumsum(-1).flip(-1) <= case["window"])
    node = j - ctx
    seen = seen | ((node >= 0) & (node < bit.numel()) & torch.gather(bits, 2, node.clamp(0, bit.numel() - 1).expand(n, most, keys)))
    seen = seen & (j < kv[:, None, None])
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
    s["cache"].attention(s["q"], s["batch"], s["out"], lse=s["lse"], window=s["case"]["window"], tree=s["tree"])
    return {"out": s["out"], "lse": s["lse"]}


def _exact_attention(s):
    case = s["case"]
    hq, hkv, page, d, window = case["hq"], case["hkv"], case["page"], case["d"], case["window"]
    ctxs, news, trees = _requests(case)
    outs, lses, a = [], [], 0
    for r, (ctx, new, tree) in enumerate(zip(ctxs, news, trees)):
        total, b = ctx + new, a + new
        hidden = np.zeros((new, total), dtype=bool)
        for i in range(new):
            path = [x for x in range(i + 1) if tree is None or tree[i] >> x & 1]
            hidden[i, ctx:] = True
            hidden[i, [ctx + x for x in (path[-window:] if window else path)]] = False
            if window:
                hidden[i, :max(0, min(ctx, ctx + len(path) - window))] = True
        hidden = torch.from_numpy(hidden).to(DEV)
        pages = s["table"][r, :_ceil(total, page)].long()
        for h in range(hq):
            k = s["k_cache"][pages, h * hkv // hq].reshape(-1, d)[:total].double()
            v = s["v_cache"][pages, h * hkv // hq].reshape(-1, d)[:total].double()
            score = (s["q"][a:b, h].double() @ k.t() / math.sqrt(d)).masked_fill(hidden, -math.inf)
            lse = torch.logsumexp(score, -1)
            outs.append(torch.exp(score - lse[:, None]) @ v)
            lses.append(lse)
        a = b
    merge = lambda parts: torch.cat([torch.stack(parts[r * hq:(r + 1) * hq], 1) for r in range(len(news))])  # noqa: E731
    return {"out": merge(outs), "lse": merge(lses)}


# ---------------------------------------------------------------- verify

def _prepare_verify(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    new, trees = _trees(case)
    n, rows, vocab = case["n"], sum(new), case["vocab"]
    cu = _starts(new)
    rand = lambda *shape: torch.rand(shape, generator=g, device=DEV)  # noqa: E731
    # a draft that is near the target, both as sharp as a model's
    z = torch.randn(rows, vocab, generator=g, device=DEV)
    q = torch.softmax(3 * z, -1)
    z.mul_(0.9).add_(torch.randn(rows, vocab, generator=g, device=DEV), alpha=0.43)
    p = torch.softmax(z.mul_(3), -1)
    del z
    # every node's token is drawn from its parent's row of the draft
    up = _ints([c + max(0, x) for c, tree in zip(cu, trees) for x in tree], torch.int64)
    tokens = torch.cat([(q[at] / -torch.log1p(-torch.rand(at.numel(), vocab, generator=g, device=DEV))).argmax(-1) for at in up.split(256)]).to(torch.int32)
    s = {"case": case, "cu": _ints(cu), "kv": _ints(new) + torch.randint(0, 4096, (n,), generator=g, device=DEV, dtype=torch.int32), "parents": _ints(sum(trees, [])), "tokens": tokens,
         "p": p, "q": q if case["draft"] else None, "u": rand(rows), "u_last": rand(n), "most": max(new)}
    for name, size in (("path", rows), ("emitted", rows), ("kept", n), ("lens", n)):
        s[name] = torch.zeros(size, dtype=torch.int32, device=DEV)
    if own:
        from tile_level_overlap_gb300 import mk
        table = torch.zeros(n, _ceil(4096 + case["hi"], 16), dtype=torch.int32, device=DEV)
        s["batch"] = mk.PagedBatch(table, s["cu"], s["kv"], page_size=16, max_new=s["most"])
        s["tree"] = mk.DraftTree(s["batch"], s["parents"])
    return s


def _plain_verify(s):
    cu, n, rows = s["cu"].long(), s["case"]["n"], s["parents"].numel()
    base, new = cu[:-1], cu[1:] - cu[:-1]
    r = torch.arange(n, device=DEV)
    cur, depth = torch.zeros_like(r), torch.zeros_like(r)
    path = torch.full((rows + 1,), -1, dtype=torch.int32, device=DEV)
    emitted = path.clone()
    path[base] = 0
    left = s["p"][base].double()  # what is left of the target's row at the node that stands last
    z = torch.ones(n, dtype=torch.float64, device=DEV)
    for i in range(1, s["most"]):  # a node's index is over its parent's
        t = (base + i).clamp(max=rows - 1)
        asked = (i < new) & (s["parents"][t] == cur)
        x = s["tokens"][t].long()
        mine = left[r, x]
        if s["q"] is None:
            accept = asked & (s["u"][t].double() * z < mine)
            reject = asked & ~accept
            z = torch.where(reject, z - mine, z)
            left[r, x] = torch.where(reject, 0, mine)
        else:
            drawn = s["q"][base + cur]
            accept = asked & (s["u"][t].double() * drawn[r, x].double() * z < mine)
            reject = asked & ~accept
            left = torch.where(reject[:, None], (left - z[:, None] * drawn.double()).clamp_(min=0), left)
            z = torch.where(reject, left.sum(-1), z)
        at = torch.where(accept, base + depth, rows)
        emitted[at] = x.to(torch.int32)
        depth = depth + accept
        path[torch.where(accept, base + depth, rows)] = i
        cur = torch.where(accept, i, cur)
        left = torch.where(accept[:, None], s["p"][base + cur].double(), left)
        z = torch.where(accept, 1.0, z)
    none = left.sum(-1, keepdim=True) == 0
    left = torch.where(none, s["p"][base + cur].double(), left).cumsum_(-1)
    last = (left <= s["u_last"].double()[:, None] * left[:, -1:]).sum(-1)
    emitted[base + depth] = last.to(torch.int32)
    kept = depth + 1
    return {"path": path[:rows], "emitted": emitted[:rows], "kept": kept.to(torch.int32), "lens": (s["kv"] - new + kept).to(torch.int32)}


def _own_verify(s):
    s["tree"].verify(s["tokens"], s["p"], s["u"], s["u_last"], s["path"], s["emitted"], s["kept"], s["lens"], draft_probs=s["q"])
    return {"path": s["path"], "emitted": s["emitted"], "kept": s["kept"], "lens": s["lens"]}


# ---------------------------------------------------------------- pages

def _pool(case, lens, prompts, g, more):
    """Requests' pages in random order, of which each odd request holds its neighbour's first ones (whole pages of the first `shared` tokens of
    both's prompts); `more` pages are free. Tables, free list and counts of other holders lie in one buffer, so that a pass can begin with them as they were."""
    page, n = case["page"], len(lens)
    held = [_ceil(x, page) for x in lens]
    lent = [min(prompts[r], prompts[r - 1], case["shared"]) // page if r % 2 else 0 for r in range(n)]
    width = max(held) + 2
    fresh = [h - c for h, c in zip(held, lent)]
    used = sum(fresh)
    pages = used + more
    order = torch.randperm(pages, generator=g, device=DEV)
    col = torch.arange(width, device=DEV)
    start = torch.tensor(_starts(fresh)[:-1], device=DEV)
    h, c = torch.tensor(held, device=DEV)[:, None], torch.tensor(lent, device=DEV)[:, None]
    mine = order[(start[:, None] + col - c).clamp(0, pages - 1)]
    table = torch.where(col < c, mine.roll(1, 0), mine)
    table = torch.where(col < h, table, -1)
    shared = torch.bincount(table[(col < h)], minlength=pages).sub_(1).clamp_(min=0)
    ints = torch.cat([table.flatten(), shared, order[used:], order.new_zeros(used), order.new_tensor([more])]).to(torch.int32)
    now = ints.clone()
    a, b = n * width, n * width + pages
    s = {"case": case, "before": ints, "now": now, "table": now[:a].view(n, width), "shared": now[a:b], "free": now[b:b + pages], "n_free": now[b + pages:], "n_left": _ints([0]),
         "held": _ints(lens), "pages": pages}
    kv = torch.empty(case["layers"], 2, pages, case["hkv"], page, case["d"], dtype=TYPES[case["type"]], device=DEV)
    s["kv"] = kv.normal_(generator=g)
    if own:
        from tile_level_overlap_gb300 import mk
        s["layers"] = mk.PagedLayers([mk.PagedCache(x[0], x[1], n_q_heads=case["hkv"]) for x in kv])
    return s


def _plain_hold(s, lens, keep, parents, copying):
    """Requests trimmed to `keep` tokens and continued by `parents`: what the next ones hold, which pages they copy, and the pool after it."""
    page, table, shared, free = s["case"]["page"], s["table"].long(), s["shared"].long(), s["free"]
    n, width = table.shape
    m, r = parents.numel(), torch.arange(n, device=DEV)
    n_free = s["n_free"].long()
    live = parents >= 0
    up = parents.clamp(min=0)
    i = torch.arange(m, device=DEV)
    children = torch.zeros(n, dtype=torch.int64, device=DEV).index_add_(0, up, live.long())
    first = torch.full((n,), m, dtype=torch.int64, device=DEV).scatter_reduce_(0, up, torch.where(live, i, m), "amin")
    held, whole, part = (lens + page - 1) // page, keep // page, keep % page > 0
    edge = table[r, whole.clamp(max=width - 1)]
    alone = part & (children > 0) & (shared[edge.clamp(min=0)] == 0)
    b = torch.arange(width, device=DEV)
    change = torch.where(b < whole[:, None], children[:, None] - 1, torch.where((b == whole[:, None]) & alone[:, None], 0, -1))
    change = torch.where(b < held[:, None], change, 0)
    shared.index_add_(0, table.clamp(min=0).flatten(), change.flatten())
    # pages that nobody holds, at the first place where they were let go
    entry = torch.arange(n * width, device=DEV)
    gone = (change.flatten() < 0) & (shared[table.clamp(min=0).flatten()] < 0)
    at = table.flatten()[gone]
    least = torch.full_like(shared, n * width).scatter_reduce_(0, at, entry[gone], "amin")
    back = at[least[at] == entry[gone]]
    need = live & part[up] & ~((first[up] == i) & alone[up])
    upto = need.long().cumsum(0)
    served = need & (upto <= n_free) if copying else need & False
    taken = served.sum()
    fresh = free[(n_free - upto).clamp(min=0)].long()
    lens_next = torch.where(live, torch.where(need & ~served, whole[up] * page, keep[up]), 0)
    rows = table[up]
    rows[i, whole[up].clamp(max=width - 1)] = torch.where(served, fresh, rows[i, whole[up].clamp(max=width - 1)])
    some = b < ((lens_next + page - 1) // page)[:, None]
    copies = torch.stack([torch.where(served, edge[up], -1), torch.where(served, fresh, -1), torch.where(served, keep[up] % page, 0)])
    n_left = n_free - taken
    free[(n_left + torch.arange(back.numel(), device=DEV)).clamp(max=free.numel() - 1)] = back.to(torch.int32)
    s["shared"].copy_(shared.clamp_(min=0))
    s["n_left"].copy_(n_left + back.numel())
    return rows, some, lens_next, copies


def _path(rng, parents):
    """A random node's path from the root."""
    at, path = rng.randrange(len(parents)), []
    while at >= 0:
        path.append(at)
        at = parents[at]
    return path[::-1]


def _kept(case):
    rng = _rng(case)
    ctx = [rng.randint(case["ctx_lo"], case["ctx_hi"]) for _ in range(case["n"])]
    new = [rng.randint(case["lo"], case["hi"]) for _ in range(case["n"])]
    paths = [_path(rng, _parents(rng, k, False)) for k in new]
    return ctx, new, paths, [rng.random() < case["finish"] for _ in range(case["n"])]


def _prepare_trim(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    ctx, new, paths, finished = _kept(case)
    page = case["page"]
    lens = [c + k for c, k in zip(ctx, new)]
    s = _pool(case, lens, ctx, g, 33)
    cu = torch.tensor(_starts(new), device=DEV)
    r = torch.repeat_interleave(torch.arange(case["n"], device=DEV), cu[1:] - cu[:-1])
    pos = s["held"].long()[r] - (cu[1:] - cu[:-1])[r] + torch.arange(sum(new), device=DEV) - cu[r]
    s |= {"cu": cu.to(torch.int32), "slots": (s["table"].long()[r, pos // page] * page + pos % page).to(torch.int32),
          "path": _ints(sum((p + [-1] * (k - len(p)) for p, k in zip(paths, new)), [])), "positions": pos.to(torch.int32),
          "keep": _ints([0 if f else c + len(p) for c, p, f in zip(ctx, paths, finished)]), "lens": _ints([0] * case["n"])}
    if own:
        from tile_level_overlap_gb300 import mk
        s["batch"] = mk.PagedBatch(s["table"], s["cu"], s["held"], s["positions"], s["slots"], page_size=page, max_new=max(new))
    return s


def _plain_trim(s):
    s["now"].copy_(s["before"])
    page, cu = s["case"]["page"], s["cu"].long()
    t = torch.arange(s["path"].numel(), device=DEV)
    first = cu[torch.searchsorted(cu, t, right=True) - 1]
    source = torch.where(s["path"] >= 0, s["slots"].long()[(first + s["path"]).clamp(min=0)], s["slots"].long())
    target = s["slots"].long()
    s["kv"][:, :, target // page, :, target % page] = s["kv"][:, :, source // page, :, source % page]
    r = torch.arange(s["case"]["n"], device=DEV)
    _, _, lens, _ = _plain_hold(s, s["held"].long(), s["keep"].long(), r, False)
    s["lens"].copy_(lens)
    return _trimmed(s)


def _own_trim(s):
    s["now"].copy_(s["before"])
    s["layers"].keep(s["batch"], s["path"])
    s["batch"].trim(s["held"], s["keep"], s["lens"], s["shared"], s["free"], s["n_free"], s["n_left"])
    return _trimmed(s)


def _trimmed(s):
    return {"kv": s["kv"].view(torch.int16), "lens": s["lens"], "table": s["table"], "shared": s["shared"], "free": s["free"], "n_left": s["n_left"]}


def _continued(case):
    rng = _rng(case)
    lens = [rng.randint(case["ctx_lo"], case["ctx_hi"]) for _ in range(case["n"])]
    return lens, sorted(rng.randrange(-1 if rng.random() < 0.1 else 0, case["n"]) for _ in range(case["m"]))


def _prepare_fork(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    lens, parents = _continued(case)
    s = _pool(case, lens, lens, g, case["m"] + 33)
    width, m = s["table"].shape[1], case["m"]
    s |= {"parents": _ints(parents), "next": torch.full((m, width), -1, dtype=torch.int32, device=DEV), "lens": _ints([0] * m), "copies": torch.zeros(3, m, dtype=torch.int32, device=DEV)}
    if own:
        from tile_level_overlap_gb300 import mk
        batch = lambda table, k: mk.PagedBatch(table, _ints([0] * (k + 1)), _ints([0] * k), page_size=case["page"], max_new=1)  # noqa: E731
        s["batch"], s["next_batch"] = batch(s["table"], case["n"]), batch(s["next"], m)
    return s


def _plain_fork(s):
    s["now"].copy_(s["before"])
    held = s["held"].long()
    rows, some, lens, copies = _plain_hold(s, held, held, s["parents"].long(), True)
    s["next"].copy_(torch.where(some, rows, s["next"].long()))
    s["lens"].copy_(lens)
    s["copies"].copy_(copies)
    # tokens past the copied ones stay as they are
    do = copies[0] >= 0
    source, target = torch.where(do, copies[0], 0), torch.where(do, copies[1], 0)
    token = torch.arange(s["case"]["page"], device=DEV)
    inside = (do[:, None] & (token < copies[2][:, None]))[:, None, :, None]
    moved = torch.where(inside, s["kv"][:, :, source], s["kv"][:, :, target])
    s["kv"].index_copy_(2, torch.where(do, target, target[do.long().argmax()]), torch.where(do[:, None, None, None], moved, moved[:, :, do.long().argmax()][:, :, None]))
    return _forked(s)


def _own_fork(s):
    s["now"].copy_(s["before"])
    s["next_batch"].fork(s["batch"], s["parents"], s["held"], s["lens"], s["copies"], s["shared"], s["free"], s["n_free"], s["n_left"])
    s["layers"].copy(s["copies"])
    return _forked(s)


def _forked(s):
    return {"kv": s["kv"].view(torch.int16), "next": s["next"], "lens": s["lens"], "copies": s["copies"], "shared": s["shared"], "free": s["free"], "n_left": s["n_left"]}


def prepare(case, seed):
    return {"tree": _prepare_tree, "attention": _prepare_attention, "verify": _prepare_verify, "trim": _prepare_trim, "fork": _prepare_fork}[case["op"]](case, seed)


def run(state):
    op = state["case"]["op"]
    if own:
        return {"tree": _own_tree, "attention": _own_attention, "verify": _own_verify, "trim": _own_trim, "fork": _own_fork}[op](state)
    return {"tree": _plain_tree, "attention": _plain_attention, "verify": _plain_verify, "trim": _plain_trim, "fork": _plain_fork}[op](state)


def exact(case, seed):
    # the others answer in whole numbers, or in bits that were moved
    return _exact_attention(prepare(case, seed)) if case["op"] == "attention" else None


def work(case):
    op, n = case["op"], case["n"]
    if op == "tree":
        rows = sum(_trees(case)[0])
        return {"bytes": 4 * (2 * n + 1) + 8 * rows + 4 * rows * case["words"] + 4 * case["pad"], "flops": 2 * rows}
    if op == "verify":
        # of each request at least one row of the target, and where its drafts have probabilities theirs, to draw the last token
        rows = sum(_trees(case)[0])
        return {"bytes": 4 * n * case["vocab"] * (2 if case["draft"] else 1) + 28 * rows, "flops": 3 * n * case["vocab"]}
    token = 0 if op == "attention" else 4 * case["layers"] * case["hkv"] * case["d"]  # a token's keys and values in all layers
    if op == "trim":
        _, new, paths, _ = _kept(case)
        moved = sum(a != b for p in paths for a, b in enumerate(p))
        return {"bytes": 2 * moved * token + 8 * sum(new) + 4 * (5 * n + 3), "flops": moved}
    if op == "fork":
        lens, parents = _continued(case)
        page = case["page"]
        others = [p for k, p in enumerate(parents) if p >= 0 and (k and parents[k - 1] == p)]
        copied = sum(lens[p] % page for p in others)
        entries = sum(_ceil(lens[p], page) for p in parents if p >= 0)
        return {"bytes": 2 * copied * token + 8 * entries + 4 * (n + 6 * case["m"]), "flops": entries}
    ctx, new, trees = _requests(case)
    w = case["window"] or 1 << 40
    read = seen = 0
    for c, k, tree in zip(ctx, new, trees):
        depth = [i + 1 for i in range(k)] if tree is None else [bin(m).count("1") for m in tree]
        cached = [min(c, max(0, w - x)) for x in depth]
        read += max(cached) + k
        seen += sum(a + min(x, w) for a, x in zip(cached, depth))
    hq, hkv, d, rows = case["hq"], case["hkv"], case["d"], sum(new)
    tables = 4 * sum(_ceil(c + k, case["page"]) for c, k in zip(ctx, new)) + 4 * (2 * n + 1) + 4 * case["words"] * rows
    return {"bytes": read * hkv * d * 4 + rows * hq * (4 * d + 4) + tables, "flops": 4 * d * hq * seen}
