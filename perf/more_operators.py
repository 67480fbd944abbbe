"""The operators of a serving step with drafted tokens over a 4-bit key/value cache, as cases that can be timed: attention
with a sliding window and a few first tokens, attention of a tree of drafted tokens, the pages of growing and finished
sequences, and moving the accepted tokens of a draft into place.

A case is a dict of plain values.  `run` computes it either with elementary torch operations (`own` false: the plain
form) or with the library's calls (`own` true).  Both take what `prepare` gives; the two keep the cache each in its
own layout, filled in `prepare` from the same keys and values, as a serving program has it filled before the call.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
BLOCK = 32          # values that share a scale: 32 channels of one token of one head
LIMIT = 32768.0     # larger magnitudes are stored as this


# ---------------------------------------------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------------------------------------------

def _attn(name, op, fmt, dim, heads, group, batch, rows_lo, rows_hi, len_lo, len_hi, page, window, sinks):
    """rows per sequence, tokens per sequence before those rows"""
    return {"name": name, "op": op, "fmt": fmt, "dim": dim, "heads": heads, "group": group, "batch": batch,
            "rows_lo": rows_lo, "rows_hi": rows_hi, "len_lo": len_lo, "len_hi": len_hi, "page": page,
            "window": window, "sinks": sinks}


def _pages(name, batch, rows_lo, rows_hi, len_lo, len_hi, page):
    return {"name": name, "op": "pages", "batch": batch, "rows_lo": rows_lo, "rows_hi": rows_hi, "len_lo": len_lo,
            "len_hi": len_hi, "page": page}


def _keep(name, fmt, dim, heads, batch, rows_lo, rows_hi, most, len_lo, len_hi, page, caches, ydt):
    return {"name": name, "op": "keep", "fmt": fmt, "dim": dim, "heads": heads, "batch": batch, "rows_lo": rows_lo,
            "rows_hi": rows_hi, "most": most, "len_lo": len_lo, "len_hi": len_hi, "page": page, "caches": caches,
            "ydt": ydt}


def listed():
    return [
        # one token of one stream in a decoder of 20 heads of 64 that sees its first 4 tokens and the last 224
        _attn("sinks_token", "sinks", "q4_0", 64, 20, 1, 1, 1, 1, 447, 447, 448, 224, 4),
        # endless streams of very unequal age, decoded together: grouped heads, the first 4 tokens and the last 2048
        _attn("sinks_streams", "sinks", "q4_1", 128, 8, 4, 48, 1, 1, 0, 32767, 64, 2048, 4),
        # a chunk of a long prompt, behind tokens of which most have left the window: the most arithmetic
        _attn("sinks_prompt", "sinks", "q4_0", 128, 8, 4, 1, 4096, 4096, 9001, 9001, 64, 4095, 65),
        # a small tree checked for one utterance, a few hundred tokens, 20 heads of 64: what a call costs at least
        _attn("tree_one", "tree", "q4_0", 64, 20, 1, 1, 13, 13, 211, 211, 448, 0, 0),
        # a serving batch whose requests have trees of unequal sizes over unequal contexts, grouped heads
        _attn("tree_batch", "tree", "q4_0", 128, 8, 4, 32, 7, 64, 300, 8191, 64, 0, 0),
        # wide heads, a sliding window and sinks, 25 drafted tokens a request
        _attn("tree_window", "tree", "q4_1", 256, 2, 8, 16, 25, 25, 1500, 20011, 32, 4096, 4),
        # a large tree over one long document
        _attn("tree_long", "tree", "q4_0", 128, 8, 8, 1, 127, 127, 100003, 100003, 256, 0, 0),
        # a decoding step of a serving batch: one token each, a new page now and then
        _pages("pages_decode", 96, 1, 1, 1, 8191, 64),
        # drafts of thousands of requests, small pages
        _pages("pages_drafts", 4096, 5, 64, 0, 4000, 32),
        # prompts are admitted: few requests, many rows and pages
        _pages("pages_prompts", 61, 237, 9001, 0, 0, 64),
        # one utterance's tree was verified: the accepted tokens of four layers' caches move into place
        _keep("keep_one", "q4_0", 64, 20, 1, 13, 13, 5, 211, 211, 448, 4, "f32"),
        # a large batch's, grouped heads
        _keep("keep_batch", "q4_1", 128, 8, 256, 17, 64, 12, 31, 2047, 64, 1, "bf16"),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    most = {k: max(work(c)[k] for c in listed()) for k in ("bytes", "flops")}
    while True:
        op = rng.choice(["sinks", "sinks", "tree", "tree", "pages", "keep"])
        fmt = rng.choice(["q4_0", "q4_1"])
        dim = rng.choice([64, 96, 128, 256])
        heads = rng.choice([1, 2, 4, 5, 8, 12, 20])
        page = rng.choice([32, 64, 96, 128, 256, 448])
        if op == "pages":
            batch = _log_int(rng, 1, 8192)
            lo = _log_int(rng, 1, max(1, 65536 // batch))
            before = rng.choice([0, 0, 1, 31, 1000, 4093])
            c = _pages("", batch, lo, min(max(1, 65536 // batch), lo * rng.randint(1, 4)), before,
                       before * rng.randint(1, 3), page)
        elif op == "keep":
            batch = _log_int(rng, 1, 256)
            rows = _log_int(rng, 2, 64)
            before = _log_int(rng, 1, max(1, 262144 // batch))
            c = _keep("", fmt, dim, heads, batch, max(1, rows // rng.randint(1, 4)), rows, rng.randint(1, min(16, rows)),
                      before // rng.randint(1, 3), min(8192, before), page, rng.choice([1, 2, 4]), rng.choice(["bf16", "f32"]))
            c["len_lo"] = min(c["len_lo"], c["len_hi"])
        else:
            group = rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
            batch = _log_int(rng, 1, 64)
            before = _log_int(rng, 1, 100003) - 1
            if op == "sinks":
                rows = 1 if rng.random() < 0.5 else _log_int(rng, 2, 4096)
                window, sinks = _log_int(rng, 1, 8192), rng.choice([0, 1, 4, 17, 64, 200])
            else:
                rows = _log_int(rng, 2, 200)
                window, sinks = rng.choice([(0, 0), (0, 0), (200, 4), (4096, 33), (1000, 0)])
            c = _attn("", op, fmt, dim, heads, group, batch, max(1, rows // rng.randint(1, 4)), rows,
                      before // rng.randint(1, 4), before, page, window, sinks)
        del c["name"]
        w = work(c)
        if op in ("sinks", "tree") and (_scores(c) > 1 << 30 or sum(_lengths(c)[1]) * heads * dim > 1 << 30):
            continue
        if w["bytes"] <= most["bytes"] and w["flops"] <= most["flops"]:
            return c


def _scores(c):
    """Scores that the plain form of an attention case holds at once."""
    rows, lens = _lengths(c)
    return c["batch"] * c["heads"] * c["group"] * max(rows) * (_width(c, max(rows), max(lens)) + max(rows))


def _width(c, most, longest):
    """Context tokens that the plain form takes of each sequence: the sinks and what any row's window reaches."""
    return min(longest, c["sinks"] + c["window"] + most - 1) if c["window"] else longest


def _spread(lo, hi, i, n):
    """The i-th of n values over [lo, hi]: the smallest first, the largest in the middle."""
    return hi if i == n // 2 else lo if i == 0 else lo + int((hi - lo) * ((i * 0.6180339887498949 + 0.07) % 1.0))


def _lengths(c):
    """(rows of each sequence, tokens of each sequence with those rows): a case has the same with every seed."""
    n = c["batch"]
    rows = [_spread(c["rows_lo"], c["rows_hi"], i, n) for i in range(n)]
    return rows, [_spread(c["len_lo"], c["len_hi"], (i * 3 + 1) % n, n) + r for i, r in enumerate(rows)]


def _seen_by(c, rows, tokens):
    """(tokens of a sequence that any of its rows sees, pairs of a row and a token that it sees).  For a tree as if its rows
    were one behind the other at most: a node's ancestors are counted as _tree makes them, half the rows on average."""
    before, w, s = tokens - rows, c["window"], c["sinks"]
    if c["op"] == "tree":
        near = min(before, w) if w else before
        far = min(s, before - near)
        return near + far + rows, (near + far + min(rows, 8) / 2.0) * rows
    p = np.arange(before, tokens, dtype=np.int64)
    lo = np.maximum(0, p + 1 - w)
    pairs = int((p + 1 - lo + np.minimum(s, lo)).sum())
    first = int(lo[0])
    return tokens - first + min(s, first), pairs


def _moved(c):
    """How many rows of each sequence are accepted."""
    rows = _lengths(c)[0]
    return [min(r, 1 + (i * 5 + c["most"] - 1) % c["most"]) for i, r in enumerate(rows)]


def work(case):
    rows, lens = _lengths(case)
    if case["op"] == "pages":
        new = sum(-(-t // case["page"]) - -(-(t - r) // case["page"]) for r, t in zip(rows, lens))
        # grown: a length, a new length and a row start a sequence, a page read and written, a row's position and slot; and
        # cut back: the same without rows
        return {"bytes": 2 * 16.0 * case["batch"] + 2 * 8.0 * new + 12.0 * sum(rows), "flops": 0.0}
    H, D = case["heads"], case["dim"]
    bits = 4.5 if case["fmt"] == "q4_0" else 5.0
    if case["op"] == "keep":
        n = 2 * sum(_moved(case)) * H * D * case["caches"]
        # moved in 4 bits, and read back
        return {"bytes": 3 * n * bits / 8 + n * (2 if case["ydt"] == "bf16" else 4), "flops": 0.0}
    seen = [_seen_by(case, r, t) for r, t in zip(rows, lens)]
    tokens, pairs, hq = sum(t for t, _ in seen), sum(p for _, p in seen), H * case["group"]
    return {"bytes": 2 * tokens * H * D * bits / 8 + 4.0 * sum(rows) * hq * D, "flops": 4.0 * pairs * hq * D}


# ---------------------------------------------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------------------------------------------

def _rng(seed, salt):
    g = torch.Generator(device=DEV)
    g.manual_seed((int(seed) * 1000003 + salt) % (1 << 62))
    return g


def _keys_values(n, heads, dim, seed, salt):
    """Keys and values of n tokens [n, heads, dim] in bf16: keys with a mean and a spread of their own in every channel (a
    few channels much larger), values nearer to zero."""
    g = _rng(seed, salt)
    wide = torch.exp(0.5 * torch.randn((1, heads, dim), generator=_rng(seed, 71), device=DEV))
    mean = 0.7 * torch.randn((1, heads, dim), generator=_rng(seed, 72), device=DEV)
    k = torch.randn((n, heads, dim), generator=g, device=DEV).mul_(wide).add_(mean)
    v = torch.randn((n, heads, dim), generator=g, device=DEV).mul_(0.5)
    return k.to(torch.bfloat16), v.to(torch.bfloat16)


def _type(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _start_of(rows):
    start = torch.zeros(len(rows) + 1, dtype=torch.int32)
    start[1:] = torch.cumsum(torch.tensor(rows), 0)
    return start.to(DEV)


def _int32(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def _plan(case, seed):
    """Where the tokens are: pages in a random order, some of the pool unused."""
    rows, lens = _lengths(case)
    page, batch = case["page"], case["batch"]
    per = max(1, (max(lens) + page - 1) // page)
    need = torch.tensor([(t + page - 1) // page for t in lens])
    pages = int(need.sum()) + 3
    order = torch.randperm(pages, generator=_rng(seed, 11), device=DEV).to(torch.int32)
    take = (torch.cumsum(need, 0) - need)[:, None] + torch.arange(per)
    take = torch.where(torch.arange(per) < need[:, None], take, torch.zeros_like(take))
    return {"rows": rows, "lens": lens, "pages": pages, "per": per, "table": order[take.to(DEV)].contiguous(),
            "start": _start_of(rows), "len": _int32(lens)}


def _queries(case, plan, seed):
    """Queries [rows, heads * group, dim], sharper in some heads than in others."""
    hq = case["heads"] * case["group"]
    q = torch.randn((sum(plan["rows"]), hq, case["dim"]), generator=_rng(seed, 31), device=DEV)
    q *= torch.exp(0.4 * torch.randn((1, hq, 1), generator=_rng(seed, 32), device=DEV))
    return q.to(torch.bfloat16)


def _tree(case, plan, seed):
    """Which drafted tokens a row sees: its ancestors and itself [rows, longest draft], one row of truth values each.  A
    node's parent is one of the 12 before it, or (the first few) the context's last token."""
    most = max(plan["rows"])
    r = np.random.RandomState(seed % (1 << 31))
    sees = np.zeros((sum(plan["rows"]), most), bool)
    at = 0
    for n in plan["rows"]:
        for i in range(n):
            parent = i - 1 - r.randint(0, 12)
            if parent >= 0:
                sees[at + i] = sees[at + parent]
            sees[at + i, i] = True
        at += n
    return sees


def _mask_words(sees):
    """The same as 32-bit words: bit j % 32 of word j / 32 is drafted token j."""
    n, most = sees.shape
    words = -(-most // 32)
    bits = np.zeros((n, words * 32), bool)
    bits[:, :most] = sees
    return torch.from_numpy(np.packbits(bits, axis=1, bitorder="little").view(np.int32).reshape(n, words).copy()).to(DEV)


def _paths(case, seed):
    """The accepted rows of each sequence: nodes that stay where they are, and then ones from further back (drafts are in
    the order of their levels, the likeliest node of each first)."""
    rows, counts = _lengths(case)[0], _moved(case)
    r = np.random.RandomState((seed + 17) % (1 << 31))
    path = np.zeros((len(rows), case["most"]), np.int32)
    for i, (n, c) in enumerate(zip(rows, counts)):
        far = min(n - c, r.randint(0, c + 1))
        path[i, :c - far] = np.arange(c - far)
        path[i, c - far:c] = np.sort(c + r.permutation(n - c)[:far])
    return path


def _prepare_pages(case, seed):
    """Sequences with tokens, and a free list; the lengths that they get, and how they are after that."""
    rows, lens = _lengths(case)
    before = [t - r for r, t in zip(rows, lens)]
    page, batch = case["page"], case["batch"]
    per = (max(lens) + page - 1) // page + 1
    had = torch.tensor([-(-t // page) for t in before])
    new = sum(-(-t // page) for t in lens) - int(had.sum())
    pages = int(had.sum()) + new + 5
    order = torch.randperm(pages, generator=_rng(seed, 11), device=DEV).to(torch.int32)
    j = torch.arange(per)
    take = ((torch.cumsum(had, 0) - had)[:, None] + j).to(DEV)
    has = (j < had[:, None]).to(DEV)
    table = torch.where(has, order[torch.where(has, take, torch.zeros_like(take))], torch.full_like(has, -1, dtype=torch.int32)).contiguous()
    free = pages - int(had.sum())
    pool = torch.zeros(4 + pages, dtype=torch.int32, device=DEV)   # free pages, pages lacking, two spare, the list
    pool[0] = free
    pool[4:4 + free] = order[pages - free:]
    s = {"op": "pages", "page": page, "pages": pages, "batch": batch, "per": per, "rows": sum(rows), "len": _int32(before),
         "want": _int32(lens), "back": _int32(before), "table": table, "pool": pool,
         "row_start": torch.zeros(batch + 1, dtype=torch.int32, device=DEV),
         "no_rows": torch.zeros(batch + 1, dtype=torch.int32, device=DEV),
         "pos": torch.full((sum(rows),), -1, dtype=torch.int32, device=DEV),
         "slot": torch.full((sum(rows),), -1, dtype=torch.int64, device=DEV)}
    if own:
        from block_quantized_bit_amd import wq
        s["wq"], s["desc"] = wq, wq.cache_desc("q4_0", 64, 1, page, pages)
    return s


def prepare(case, seed):
    if case["op"] == "pages":
        return _prepare_pages(case, seed)
    plan = _plan(case, seed)
    H, D, page, batch = case["heads"], case["dim"], case["page"], case["batch"]
    rows, lens = plan["rows"], plan["lens"]
    s = {"op": case["op"], "fmt": case["fmt"], "dim": D, "heads": H, "page": page, "batch": batch, "rows": sum(rows),
         "max_rows": max(rows), "max_len": max(lens), "table": plan["table"], "len": plan["len"], "start": plan["start"]}
    if own:
        from block_quantized_bit_amd import wq
        s["wq"] = wq
        s["desc"] = wq.cache_desc(case["fmt"], D, H, page, plan["pages"])
        size = wq.wq_cache_size(s["desc"])
        s["caches"] = [torch.zeros(size, dtype=torch.uint8, device=DEV) for _ in range(case.get("caches", 1))]
        s["seqs"] = wq.seqs(batch, sum(rows), plan["len"], plan["table"], row_start=None if max(rows) == 1 else plan["start"])
    else:
        nb, per_block = D // BLOCK, 1 if case["fmt"] == "q4_0" else 2
        s["caches"] = []
        for _ in range(case.get("caches", 1)):
            c = {}
            for w in ("k", "v"):
                c[w + "_codes"] = torch.zeros((plan["pages"], page, H, D // 2), dtype=torch.uint8, device=DEV)
                c[w + "_scales"] = torch.zeros((plan["pages"], page, H, nb, per_block), dtype=torch.float16, device=DEV)
            s["caches"].append(c)
    for layer, cache in enumerate(s["caches"]):          # fill the caches, a sequence at a time
        for b, t in enumerate(lens):
            k, v = _keys_values(t, H, D, seed, 100 + b + 100000 * layer)
            if own:
                whole = wq.seqs(1, t, plan["len"][b:b + 1], plan["table"][b:b + 1], row_start=_int32([0, t]))
                wq.wq_cache_write(s["desc"], whole, k, H * D, v, H * D, wq.WQ_BF16, cache)
            else:
                at = torch.arange(t, device=DEV)
                slot = plan["table"][b].long()[at // page] * page + at % page
                for w, x in (("k", k), ("v", v)):
                    codes, scales = _quantise(x.float(), case["fmt"])
                    cache[w + "_codes"].view(-1, H, D // 2)[slot] = codes
                    cache[w + "_scales"].view(-1, H, nb, per_block)[slot] = scales
    if case["op"] == "keep":
        counts = _moved(case)
        s["path"], s["count"] = torch.from_numpy(_paths(case, seed)).to(DEV), _int32(counts)
        s["kept"], s["kept_start"], s["max_kept"] = sum(counts), _start_of(counts), max(counts)
        s["ydt"] = case["ydt"]
        s["want"] = torch.zeros(batch, dtype=torch.int32, device=DEV)
        if own:
            s["k_out"] = [torch.empty((s["kept"], H, D), dtype=_type(case["ydt"]), device=DEV) for _ in s["caches"]]
            s["v_out"] = [torch.empty_like(x) for x in s["k_out"]]
            s["kept_seqs"] = wq.seqs(batch, s["kept"], s["want"], plan["table"], row_start=s["kept_start"])
    else:
        hq = H * case["group"]
        s["group"], s["window"], s["sinks"] = case["group"], case["window"], case["sinks"]
        s["width"] = _width(case, max(rows), max(lens))
        s["scale"] = D ** -0.5
        s["q"] = _queries(case, plan, seed)
        if case["op"] == "tree":
            s["tree"] = _mask_words(_tree(case, plan, seed))
        if own:
            s["y"] = torch.empty_like(s["q"])
            size_of = wq.wq_attn_tree_workspace_size if case["op"] == "tree" else wq.wq_attn_sinks_workspace_size
            n = size_of(s["desc"], s["seqs"], hq, case["window"], case["sinks"])
            s["ws"] = torch.empty(n, dtype=torch.uint8, device=DEV) if n else None
    if own:
        torch.cuda.synchronize()
    return s


# ---------------------------------------------------------------------------------------------------------------
# The plain form
# ---------------------------------------------------------------------------------------------------------------

def _quantise(x, fmt):
    """fp32 values [..., dim] -> bytes of two codes [..., dim / 2] and fp16 scales [..., dim / 32, 1 or 2]."""
    x = x.clamp(-LIMIT, LIMIT).unflatten(-1, (-1, BLOCK))
    if fmt == "q4_0":
        big = x.abs().argmax(-1, keepdim=True)        # the first of the largest
        d = (x.gather(-1, big) / -8.0).half()
        base, low, scales = 0.0, -8.0, d
    else:
        lo = x.amin(-1, keepdim=True)
        d = ((x.amax(-1, keepdim=True) - lo) / torch.full_like(lo, 15.0)).half()   # a quotient, not a product with 1/15
        m = lo.half()
        base, low, scales = m.float(), 0.0, torch.cat([d, m], -1)
    f = d.float()
    q = torch.where(f == 0, torch.zeros_like(x), torch.round((x - base) / f).clamp(low, low + 15.0)) - low
    q = torch.where(f == 0, torch.full_like(q, -low), q).to(torch.uint8).flatten(-2)
    return q[..., 0::2] | (q[..., 1::2] << 4), scales


def _values(codes, scales, fmt):
    """The fp32 values that bytes and scales stand for."""
    q = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).float().unflatten(-1, (-1, BLOCK))
    d = scales[..., 0:1].float()
    x = (q - 8.0) * d if fmt == "q4_0" else q * d + scales[..., 1:2].float()
    return x.flatten(-2)


def _at(s, token):
    """Places [batch, n] of tokens in the pool."""
    return s["table"].long().gather(1, token // s["page"]) * s["page"] + token % s["page"]


def _plain_attention(s):
    H, G, D, B, most, width = s["heads"], s["group"], s["dim"], s["batch"], s["max_rows"], s["width"]
    tree, window, sinks = s["op"] == "tree", s["window"], s["sinks"]
    first, length = s["start"][:-1].long(), s["len"].long()
    count = s["start"][1:].long() - first
    i = torch.arange(most, device=DEV)
    row = (first[:, None] + i).clamp(max=s["rows"] - 1)
    before = (length - count)[:, None]                                  # [B, 1]
    # the tokens that any row can see: the sinks and the last ones (all, without a window)
    j = torch.arange(width, device=DEV)[None]
    token = torch.where(j < sinks, j, (length[:, None] - (width - j)).clamp(min=sinks)) if window and width < s["max_len"] else j
    token = token.expand(B, width)
    fresh = torch.ones_like(token, dtype=torch.bool)
    fresh[:, 1:] = token[:, 1:] > token[:, :-1]                         # (where a sequence is short, a token comes again)
    inside = token.clamp(max=s["max_len"] - 1)
    slot = _at(s, inside)
    cache = s["caches"][0]
    nb = D // BLOCK
    k, v = (_values(cache[w + "_codes"].view(-1, H, D // 2)[slot], cache[w + "_scales"].view(-1, H, nb, cache[w + "_scales"].shape[-1])[slot],
                    s["fmt"]) for w in ("k", "v"))                      # [B, width, H, D]
    q = s["q"].float()[row].view(B, most, H, G, D)
    score = torch.matmul(q.permute(0, 2, 3, 1, 4).reshape(B, H, G * most, D), k.permute(0, 2, 3, 1).contiguous())
    score = score.view(B, H, G, most, width) * s["scale"]
    t = token[:, None]                                                  # [B, 1, width]
    if tree:
        bits = (s["tree"][row][..., None] >> torch.arange(32, device=DEV, dtype=torch.int32)) & 1
        bits = bits.flatten(-2).bool()                                  # [B, most, 32 words]
        bits &= torch.arange(bits.shape[-1], device=DEV) < count[:, None, None]
        node = (t - before[..., None]).expand(B, most, width)
        sees = (t < before[..., None]).expand(B, most, width)
        if window:
            depth = bits.sum(-1, keepdim=True)
            sees = sees & ((t >= before[..., None] + depth - window) | (t < sinks))
        drafted = (node >= 0) & (node < count[:, None, None])
        sees = sees | (drafted & bits.gather(2, node.clamp(0, bits.shape[-1] - 1)))
    else:
        pos = (before + i)[..., None]
        sees = (t <= pos) & (t < length[:, None, None]) & ((t > pos - window) | (t < sinks))
    sees = sees & fresh[:, None]
    score = score.masked_fill(~sees[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(top == -math.inf, torch.zeros_like(top), top))
    total = p.sum(-1, keepdim=True)
    p = p / torch.where(total == 0, torch.ones_like(total), total)
    y = torch.matmul(p.view(B, H, G * most, width), v.permute(0, 2, 1, 3).contiguous()).view(B, H, G, most, D)
    y = y.permute(0, 3, 1, 2, 4).reshape(B, most, H * G, D)
    return y[(i < count[:, None])].to(torch.bfloat16)


def _plain_assign(s, want, row_start, rows):
    """Lengths become `want`: pages that are no longer needed go in front of the free list, in the order of sequences and
    pages; then the new ones are taken from its front.  The list is held with its front at the end."""
    page, batch, per, table, pool = s["page"], s["batch"], s["per"], s["table"], s["pool"]
    old, new = s["len"].long(), want.long()
    has, needs = (old + page - 1) // page, ((new + page - 1) // page)
    j = torch.arange(per, device=DEV)
    gone = (j >= needs[:, None]) & (j < has[:, None]) & (table >= 0) & (table < s["pages"])
    come = (j >= has[:, None]) & (j < needs[:, None])
    rank_gone, rank_come = ((m.flatten().long().cumsum(0) - 1).view(batch, per) for m in (gone, come))
    n_gone, n_come, free = gone.sum(), come.sum(), pool[0].long()
    spare = s["pages"]                                                   # entries of no use go behind the list
    released = torch.zeros(spare + 1, dtype=torch.int32, device=DEV)
    released[torch.where(gone, rank_gone, spare)] = table
    behind = (free - 1 - (rank_come - n_gone)).clamp(min=-1)
    page_of = torch.where(rank_come < n_gone, released[rank_come.clamp(0, spare)],
                          torch.where(behind >= 0, pool[4:][behind.clamp(0, spare - 1)], -1))
    table.copy_(torch.where(come, page_of, table))
    n_list = (free + n_gone - n_come).clamp(min=0)
    place = torch.arange(spare, device=DEV)
    pool[4:] = torch.where((place >= free) & (place < n_list), released[(n_list - 1 - place + n_come).clamp(0, spare)], pool[4:])
    pool[0], pool[1] = n_list, (n_come - n_gone - free).clamp(min=0)
    grown = (new - old).clamp(min=0)
    row_start[1:] = grown.cumsum(0)
    if rows:
        r = torch.arange(rows, device=DEV)
        b = torch.searchsorted(row_start, r, right=True) - 1
        pos = old[b] + r - row_start[b]
        at = table[b, (pos // page)].long()
        s["pos"].copy_(pos)
        s["slot"].copy_(torch.where(at >= 0, at * page + pos % page, -1))
    s["len"].copy_(want)


def _plain_keep(s):
    H, D, count = s["heads"], s["dim"], s["count"].long()
    before = s["len"].long() - (s["start"][1:] - s["start"][:-1]).long()
    s["want"].copy_(before + count)
    j = torch.arange(s["max_kept"], device=DEV)
    taken = j < count[:, None]
    source, target = (_at(s, torch.where(taken, before[:, None] + x, 0)) for x in (s["path"][:, :s["max_kept"]].long(), j))
    source, target = source[taken], target[taken]
    out = []
    for cache in s["caches"]:
        for x in cache.values():
            flat = x.view(-1, *x.shape[2:])
            flat[target] = flat[source]
        for w in ("k", "v"):
            codes, scales = (cache[w + e].flatten(0, 1)[target] for e in ("_codes", "_scales"))
            out.append(_values(codes, scales, s["fmt"]).to(_type(s["ydt"])))
    return out + [s["want"]]


def run(state):
    s = state
    if s["op"] == "pages":
        # tokens are added, and taken back (as a draft that is not accepted, or requests that end)
        if own:
            wq = s["wq"]
            wq.wq_pages_assign(s["desc"], s["batch"], s["len"], s["want"], s["table"], s["per"], s["pool"], s["rows"],
                               s["row_start"], s["pos"], s["slot"])
            wq.wq_pages_assign(s["desc"], s["batch"], s["len"], s["back"], s["table"], s["per"], s["pool"], 0, s["no_rows"],
                               None, None)
        else:
            _plain_assign(s, s["want"], s["row_start"], s["rows"])
            _plain_assign(s, s["back"], s["no_rows"], 0)
        return [s["table"], s["row_start"], s["pos"], s["slot"], s["len"], s["no_rows"], s["pool"]]
    if not own:
        return _plain_keep(s) if s["op"] == "keep" else _plain_attention(s)
    wq, ld = s["wq"], s["heads"] * s["dim"]
    if s["op"] == "keep":
        ydt = wq.WQ_BF16 if s["ydt"] == "bf16" else wq.WQ_F32
        wq.wq_cache_keep(s["desc"], s["seqs"], s["path"], s["path"].shape[1], s["count"], s["caches"], s["want"])
        out = []
        for cache, k, v in zip(s["caches"], s["k_out"], s["v_out"]):
            wq.wq_cache_read(s["desc"], s["kept_seqs"], cache, k, ld, v, ld, ydt)
            out += [k, v]
        return out + [s["want"]]
    hq = s["heads"] * s["group"]
    ws = (s["ws"], 0 if s["ws"] is None else s["ws"].numel())
    if s["op"] == "tree":
        wq.wq_attn_tree(s["desc"], s["seqs"], hq, s["q"], hq * s["dim"], s["caches"][0], s["scale"], s["window"], s["sinks"],
                        s["tree"], s["tree"].shape[1], s["y"], hq * s["dim"], *ws)
    else:
        wq.wq_attn_sinks(s["desc"], s["seqs"], hq, s["q"], hq * s["dim"], s["caches"][0], s["scale"], s["window"], s["sinks"],
                         s["y"], hq * s["dim"], *ws)
    return s["y"]


# ---------------------------------------------------------------------------------------------------------------
# The definition in 64 bits
# ---------------------------------------------------------------------------------------------------------------

def _stored(x, fmt):
    """The values in 64 bits that the format stores for x [n, heads, dim].  Where the format names a rounding (a quotient
    or difference in 32 bits, a scale in 16) it is made here too; everything else is exact."""
    n, heads, dim = x.shape
    z = x.double().reshape(-1, BLOCK)
    z = torch.minimum(torch.maximum(z, torch.tensor(-LIMIT, dtype=torch.float64, device=z.device)),
                      torch.tensor(LIMIT, dtype=torch.float64, device=z.device))
    top, bottom = z.max(1).values, z.min(1).values
    if fmt == "q4_0":
        a = torch.maximum(top, -bottom)
        tie = (top == a) & (bottom == -a)
        # on a tie the earlier of the two decides
        first_top = (z == top[:, None]).double().argmax(1)
        first_bottom = (z == bottom[:, None]).double().argmax(1)
        negative = torch.where(tie, first_bottom < first_top, bottom == -a)
        big = torch.where(negative, -a, a)
        d = (big / -8).float().half().double()[:, None]
        c = torch.where(d == 0, torch.zeros_like(z), torch.round((z / d).float().double()))
        out = torch.minimum(torch.maximum(c, torch.full_like(c, -8.0)), torch.full_like(c, 7.0)) * d
    else:
        d = ((top - bottom).float().double() / 15).float().half().double()[:, None]
        m = bottom.float().half().double()[:, None]
        c = torch.where(d == 0, torch.zeros_like(z), torch.round(((z - m).float().double() / d).float().double()))
        out = torch.minimum(torch.maximum(c, torch.zeros_like(c)), torch.full_like(c, 15.0)) * d + m
    return out.reshape(n, heads, dim)


def _hidden(case, sees, r, t):
    """Which tokens [r, t] the rows of a sequence do not see; sees: a tree's rows, or None."""
    token = torch.arange(t, device=DEV)[None, :]
    before = t - r
    if sees is None:
        last = torch.arange(before, t, device=DEV)[:, None]
        far = (token <= last - case["window"]) & (token >= case["sinks"])
        return far | (token > last)
    hidden = torch.zeros((r, t), dtype=torch.bool, device=DEV)
    seen = torch.from_numpy(sees[:, :r]).to(DEV)
    hidden[:, before:] = ~seen
    if case["window"]:
        # the rows that a row sees are the nearest part of its window
        left = (case["window"] - seen.double().sum(1))[:, None]
        context = token[:, :before].double()
        hidden[:, :before] = (context < before - left) & (context >= case["sinks"])
    return hidden


def exact(case, seed):
    if case["op"] == "pages":
        return None
    plan = _plan(case, seed)
    H, D = case["heads"], case["dim"]
    if case["op"] == "keep":
        path, counts, out = _paths(case, seed), _moved(case), []
        for layer in range(case["caches"]):
            kept = {0: [], 1: []}
            for b, (r, t) in enumerate(zip(plan["rows"], plan["lens"])):
                pick = torch.from_numpy(path[b, :counts[b]].astype(np.int64) + (t - r)).to(DEV)
                for w, x in enumerate(_keys_values(t, H, D, seed, 100 + b + 100000 * layer)):
                    kept[w].append(_stored(x[pick], case["fmt"]))
            out += [torch.cat(kept[0]), torch.cat(kept[1])]
        return out + [None]
    if work(case)["flops"] > 4e12:
        return None
    G = case["group"]
    q = _queries(case, plan, seed).double()
    tree = _tree(case, plan, seed) if case["op"] == "tree" else None
    y = torch.zeros(q.shape, dtype=torch.float64, device=DEV)
    at = 0
    for b, (r, t) in enumerate(zip(plan["rows"], plan["lens"])):
        k, v = _keys_values(t, H, D, seed, 100 + b)
        hidden = _hidden(case, None if tree is None else tree[at:at + r], r, t)
        for h in range(H):
            kh, vh = _stored(k[:, h:h + 1], case["fmt"])[:, 0], _stored(v[:, h:h + 1], case["fmt"])[:, 0]
            for g in range(G):
                z = (q[at:at + r, h * G + g] @ kh.t()) / math.sqrt(D)
                z[hidden] = -math.inf
                y[at:at + r, h * G + g] = torch.nan_to_num(torch.softmax(z, 1), nan=0.0) @ vh
        at += r
    return y
