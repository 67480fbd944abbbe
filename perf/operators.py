"""The operators of a 4-bit key/value cache, as cases that can be timed: writing rows into the cache and reading them
back, and attention over it.

A case is a dict of plain values.  `run` computes it either with elementary torch operations (`own` false: the plain
form) or with the library's calls (`own` true).  Both take what `prepare` gives; the two keep the cache each in its
own layout, filled in `prepare` from the same keys and values, as a serving program has it filled before the call.
"""
import math

import torch

own = False

DEV = "cuda"
BLOCK = 32          # values that share a scale: 32 channels of one token of one head
LIMIT = 32768.0     # larger magnitudes are stored as this


# ---------------------------------------------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------------------------------------------

def _cache(name, fmt, dim, heads, batch, rows_lo, rows_hi, before, page, xdt, ydt):
    return {"name": name, "op": "cache", "fmt": fmt, "dim": dim, "heads": heads, "batch": batch, "rows_lo": rows_lo,
            "rows_hi": rows_hi, "before": before, "page": page, "xdt": xdt, "ydt": ydt}


def _attn(name, fmt, dim, heads, group, batch, rows_lo, rows_hi, len_lo, len_hi, page, causal, window):
    return {"name": name, "op": "attn", "fmt": fmt, "dim": dim, "heads": heads, "group": group, "batch": batch,
            "rows_lo": rows_lo, "rows_hi": rows_hi, "len_lo": len_lo, "len_hi": len_hi, "page": page,
            "causal": causal, "window": window}


def listed():
    return [
        # one decoded token of one utterance, in a decoder of 20 heads of 64: what a call costs at least
        _cache("cache_one_token", "q4_0", 64, 20, 1, 1, 1, 223, 448, "bf16", "bf16"),
        # one token each of many requests, at odd places of their pages
        _cache("cache_decode_batch", "q4_1", 128, 8, 96, 1, 1, 4001, 64, "bf16", "f32"),
        # the keys and values of cross-attention: 1500 frames of four utterances, as fp32 projections leave them
        _cache("cache_frames", "q4_0", 64, 20, 4, 1500, 1500, 0, 1504, "f32", "bf16"),
        # long prompts of unequal lengths, behind tokens that are there already
        _cache("cache_prompts", "q4_1", 128, 8, 7, 1237, 9001, 45, 64, "bf16", "bf16"),
        # self-attention of one utterance's token: a few hundred tokens, 20 heads of 64
        _attn("attn_self_token", "q4_0", 64, 20, 1, 1, 1, 1, 224, 224, 448, True, 0),
        # cross-attention of 16 requests' tokens over 1500 frames
        _attn("attn_cross_token", "q4_0", 64, 20, 1, 16, 1, 1, 1500, 1500, 1504, False, 0),
        # a serving batch of very unequal lengths, grouped heads
        _attn("attn_decode_ragged", "q4_1", 128, 8, 4, 61, 1, 1, 1, 8191, 64, True, 0),
        # one long document, token by token: the length has to be shared out over the chip
        _attn("attn_decode_long", "q4_0", 128, 8, 8, 1, 1, 1, 131077, 131077, 256, True, 0),
        # a full serving batch of long contexts: the most bytes
        _attn("attn_decode_full", "q4_0", 128, 8, 5, 32, 1, 1, 30011, 32768, 128, True, 0),
        # five drafted tokens a request checked at once, wide heads, a sliding window
        _attn("attn_draft_window", "q4_1", 256, 2, 8, 16, 5, 5, 4500, 20011, 32, True, 4096),
        # a chunk of a long prompt over the tokens before it: the most arithmetic
        _attn("attn_prompt_chunk", "q4_0", 128, 8, 4, 1, 2048, 2048, 18432, 18432, 64, True, 0),
        # fresh prompts of unequal lengths, heads of 96 channels
        _attn("attn_prompt_ragged", "q4_1", 96, 12, 1, 9, 3, 701, 0, 0, 96, True, 0),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    most = {k: max(work(c)[k] for c in listed()) for k in ("bytes", "flops")}
    while True:
        fmt = rng.choice(["q4_0", "q4_1"])
        dim = rng.choice([64, 96, 128, 256])
        heads = rng.choice([1, 2, 4, 5, 8, 12, 20])
        page = rng.choice([32, 64, 96, 128, 256, 448])
        if rng.random() < 0.35:
            batch = _log_int(rng, 1, 128)
            lo = _log_int(rng, 1, max(1, 32768 // batch))
            c = _cache("", fmt, dim, heads, batch, lo, min(max(1, 32768 // batch), lo * rng.randint(1, 4)),
                       rng.choice([0, 1, 17, 1000, 4093]), page, rng.choice(["bf16", "f32"]), rng.choice(["bf16", "f32"]))
        else:
            group = rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
            batch = _log_int(rng, 1, 64)
            if rng.random() < 0.6:                      # token by token, or a few drafted tokens
                rows = rng.choice([1, 1, 1, 2, 3, 5])
                lo = _log_int(rng, 1, 131072)
                c = _attn("", fmt, dim, heads, group, batch, rows, rows, lo, min(131072, lo * rng.randint(1, 3)), page,
                          True, rng.choice([0, 0, 0, 100, 4096]))
                if rng.random() < 0.25:
                    c["causal"], c["window"] = False, 0
            else:                                       # prompts, fresh or behind other tokens
                rows = _log_int(rng, 6, 2048)
                before = rng.choice([0, 0, 333, 8000])
                c = _attn("", fmt, dim, heads, group, batch, max(1, rows // rng.randint(1, 4)), rows, before, before + rng.choice([0, 0, 1, 700]), page,
                          True, rng.choice([0, 0, 0, 512]))
        del c["name"]
        w = work(c)
        padded = c["op"] == "cache" or _padded(c) <= 1 << 31
        if padded and w["bytes"] <= most["bytes"] and w["flops"] <= most["flops"]:
            return c


def _padded(c):
    """Scores of the case when every sequence is as long as the longest: what the plain form holds at once."""
    rows, lens = _lengths(c)
    return c["batch"] * c["heads"] * c["group"] * max(rows) * max(lens)


def _spread(lo, hi, i, n):
    """The i-th of n values over [lo, hi]: the smallest first, the largest in the middle."""
    return hi if i == n // 2 else lo if i == 0 else lo + int((hi - lo) * ((i * 0.6180339887498949 + 0.07) % 1.0))


def _lengths(c):
    """(rows of each sequence, tokens of each sequence with those rows): a case has the same with every seed."""
    n = c["batch"]
    rows = [_spread(c["rows_lo"], c["rows_hi"], i, n) for i in range(n)]
    if c["op"] == "cache":
        return rows, [c["before"] + r for r in rows]
    # a length is of the whole sequence where rows are few, and of the tokens before the rows where it is a prompt
    lens = [_spread(c["len_lo"], c["len_hi"], (i * 3 + 1) % n, n) for i in range(n)]
    if c["rows_hi"] > 5 and c["len_lo"] < c["rows_hi"] * 4:
        lens = [a + r for a, r in zip(lens, rows)]
    return rows, lens


def work(case):
    rows, lens = _lengths(case)
    H, D = case["heads"], case["dim"]
    bits = 4.5 if case["fmt"] == "q4_0" else 5.0
    if case["op"] == "cache":
        n = 2 * sum(rows) * H * D
        width = {"bf16": 2, "f32": 4}
        return {"bytes": n * (width[case["xdt"]] + width[case["ydt"]]) + 2 * n * bits / 8, "flops": 6.0 * n}
    G, w = case["group"], case["window"]
    tokens = pairs = 0
    for r, t in zip(rows, lens):
        if not case["causal"]:
            tokens += t
            pairs += r * t
            continue
        # row i at position t - r + i sees that many tokens and itself, at most w of them
        lo, hi = max(0, t - r) + 1, t               # tokens seen without a window, first and last row that sees any
        n = hi - lo + 1
        if n <= 0:
            continue
        if w == 0 or hi <= w:
            pairs += (lo + hi) * n // 2
            tokens += t
        else:
            short = max(0, w - lo + 1)                # rows that see fewer than w
            pairs += (lo + lo + short - 1) * short // 2 + (n - short) * w
            tokens += t - max(0, lo - w)
    return {"bytes": 2 * tokens * H * D * bits / 8 + 4.0 * sum(rows) * H * G * D, "flops": 4.0 * pairs * H * G * D}


# ---------------------------------------------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------------------------------------------

def _rng(seed, salt):
    g = torch.Generator(device=DEV)
    g.manual_seed((int(seed) * 1000003 + salt) % (1 << 62))
    return g


def _keys_values(n, heads, dim, seed, salt, dtype):
    """Keys and values of n tokens [n, heads, dim]: keys with a mean and a spread of their own in every channel (a few
    channels much larger), values nearer to zero."""
    g = _rng(seed, salt)
    wide = torch.exp(0.5 * torch.randn((1, heads, dim), generator=_rng(seed, 71), device=DEV))
    mean = 0.7 * torch.randn((1, heads, dim), generator=_rng(seed, 72), device=DEV)
    k = torch.randn((n, heads, dim), generator=g, device=DEV).mul_(wide).add_(mean)
    v = torch.randn((n, heads, dim), generator=g, device=DEV).mul_(0.5)
    return k.to(dtype), v.to(dtype)


def _type(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _plan(case, seed):
    """Where the tokens are: pages in a random order, some of the pool unused."""
    rows, lens = _lengths(case)
    page, batch = case["page"], case["batch"]
    per = (max(lens) + page - 1) // page
    need = [(t + page - 1) // page for t in lens]
    pages = sum(need) + 3
    order = torch.randperm(pages, generator=_rng(seed, 11), device=DEV).to(torch.int32)
    take = torch.zeros((batch, per), dtype=torch.int64)
    at = 0
    for b, n in enumerate(need):
        take[b, :n] = torch.arange(at, at + n)
        at += n
    table = order[take.to(DEV)].contiguous()
    start = torch.zeros(batch + 1, dtype=torch.int32)
    start[1:] = torch.cumsum(torch.tensor(rows), 0)
    return {"rows": rows, "lens": lens, "pages": pages, "per": per, "table": table, "start": start.to(DEV),
            "len": torch.tensor(lens, dtype=torch.int32, device=DEV)}


def _queries(case, plan, seed):
    """Queries [rows, heads * group, dim], sharper in some heads than in others."""
    hq = case["heads"] * case["group"]
    q = torch.randn((sum(plan["rows"]), hq, case["dim"]), generator=_rng(seed, 31), device=DEV)
    q *= torch.exp(0.4 * torch.randn((1, hq, 1), generator=_rng(seed, 32), device=DEV))
    return q.to(torch.bfloat16)


def prepare(case, seed):
    plan = _plan(case, seed)
    H, D, page = case["heads"], case["dim"], case["page"]
    rows, lens = plan["rows"], plan["lens"]
    s = {"op": case["op"], "fmt": case["fmt"], "dim": D, "heads": H, "page": page, "batch": case["batch"],
         "rows": sum(rows), "max_rows": max(rows), "table": plan["table"], "len": plan["len"], "start": plan["start"]}
    if own:
        from block_quantized_bit_amd import wq
        s["wq"] = wq
        s["desc"] = wq.cache_desc(case["fmt"], D, H, page, plan["pages"])
        s["cache"] = torch.zeros(wq.wq_cache_size(s["desc"]), dtype=torch.uint8, device=DEV)
        one = max(rows) == 1
        s["seqs"] = wq.seqs(case["batch"], sum(rows), plan["len"], plan["table"], row_start=None if one else plan["start"])
    if case["op"] == "cache":
        k, v = _keys_values(sum(rows), H, D, seed, 1, _type(case["xdt"]))
        s["k"], s["v"] = k, v
        s["xdt"], s["ydt"] = case["xdt"], case["ydt"]
        if own:
            s["k_out"] = torch.empty((sum(rows), H, D), dtype=_type(case["ydt"]), device=DEV)
            s["v_out"] = torch.empty_like(s["k_out"])
        return s
    s["group"], s["causal"], s["window"] = case["group"], case["causal"], case["window"]
    s["scale"] = case["dim"] ** -0.5
    s["q"] = _queries(case, plan, seed)
    if own:
        s["y"] = torch.empty_like(s["q"])
        n = wq.wq_attn_workspace_size(s["desc"], s["seqs"], H * case["group"])
        s["ws"] = torch.empty(n, dtype=torch.uint8, device=DEV) if n else None
    else:
        nb, per_block = D // BLOCK, 1 if case["fmt"] == "q4_0" else 2
        for w in ("k", "v"):
            s[w + "_codes"] = torch.zeros((plan["pages"], page, H, D // 2), dtype=torch.uint8, device=DEV)
            s[w + "_scales"] = torch.zeros((plan["pages"], page, H, nb, per_block), dtype=torch.float16, device=DEV)
    for b, t in enumerate(lens):                      # fill the cache, a sequence at a time
        if t == 0:
            continue
        k, v = _keys_values(t, H, D, seed, 100 + b, torch.bfloat16)
        if own:
            whole = wq.seqs(1, t, plan["len"][b:b + 1], plan["table"][b:b + 1],
                            row_start=torch.tensor([0, t], dtype=torch.int32, device=DEV))
            wq.wq_cache_write(s["desc"], whole, k, H * D, v, H * D, wq.WQ_BF16, s["cache"])
        else:
            at = torch.arange(t, device=DEV)
            slot = plan["table"][b].long()[at // page] * page + at % page
            for w, x in (("k", k), ("v", v)):
                codes, scales = _quantise(x.float(), case["fmt"])
                s[w + "_codes"].view(-1, H, D // 2)[slot] = codes
                s[w + "_scales"].view(-1, H, nb, per_block)[slot] = scales
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


def _plain_cache(s):
    out = []
    for x in (s["k"], s["v"]):
        codes, scales = _quantise(x.float(), s["fmt"])
        out.append(_values(codes, scales, s["fmt"]).to(_type(s["ydt"])))
    return out


def _plain_attention(s):
    H, G, D, B, page = s["heads"], s["group"], s["dim"], s["batch"], s["page"]
    per, most = s["table"].shape[1], s["max_rows"]
    table = s["table"].long()
    k, v = (_values(s[w + "_codes"][table], s[w + "_scales"][table], s["fmt"]).view(B, per * page, H, D) for w in ("k", "v"))
    first, length = s["start"][:-1].long(), s["len"].long()
    count = s["start"][1:].long() - first
    i = torch.arange(most, device=DEV)
    at = (first[:, None] + i).clamp(max=s["rows"] - 1)
    q = s["q"].float()[at].view(B, most, H, G, D)
    score = torch.matmul(q.permute(0, 2, 3, 1, 4).reshape(B, H, G * most, D), k.permute(0, 2, 3, 1).contiguous())
    score = score.view(B, H, G, most, per * page) * s["scale"]
    t = torch.arange(per * page, device=DEV)
    sees = (t < length[:, None])[:, None, :].expand(B, most, -1)
    if s["causal"]:
        pos = (length - count)[:, None] + i
        sees = sees & (t <= pos[..., None])
        if s["window"]:
            sees = sees & (t > pos[..., None] - s["window"])
    score = score.masked_fill(~sees[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(top == -math.inf, torch.zeros_like(top), top))
    total = p.sum(-1, keepdim=True)
    p = p / torch.where(total == 0, torch.ones_like(total), total)
    y = torch.matmul(p.view(B, H, G * most, per * page), v.permute(0, 2, 1, 3).contiguous()).view(B, H, G, most, D)
    y = y.permute(0, 3, 1, 2, 4).reshape(B, most, H * G, D)
    return y[(i < count[:, None])].to(torch.bfloat16)


def run(state):
    s = state
    if not own:
        return _plain_cache(s) if s["op"] == "cache" else _plain_attention(s)
    wq, ld = s["wq"], s["heads"] * s["dim"]
    if s["op"] == "cache":
        xdt, ydt = (wq.WQ_BF16 if s[t] == "bf16" else wq.WQ_F32 for t in ("xdt", "ydt"))
        wq.wq_cache_write(s["desc"], s["seqs"], s["k"], ld, s["v"], ld, xdt, s["cache"])
        wq.wq_cache_read(s["desc"], s["seqs"], s["cache"], s["k_out"], ld, s["v_out"], ld, ydt)
        return [s["k_out"], s["v_out"]]
    hq = s["heads"] * s["group"]
    wq.wq_attn(s["desc"], s["seqs"], hq, s["q"], hq * s["dim"], s["cache"], s["scale"], s["causal"], s["window"],
               s["y"], hq * s["dim"], s["ws"], 0 if s["ws"] is None else s["ws"].numel())
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


def exact(case, seed):
    plan = _plan(case, seed)
    H, D = case["heads"], case["dim"]
    if case["op"] == "cache":
        k, v = _keys_values(sum(plan["rows"]), H, D, seed, 1, _type(case["xdt"]))
        return [_stored(x, case["fmt"]) for x in (k, v)]
    if work(case)["flops"] > 4e12:
        return None
    G = case["group"]
    q = _queries(case, plan, seed).double()
    y = torch.zeros(q.shape, dtype=torch.float64, device=DEV)
    at = 0
    for b, (r, t) in enumerate(zip(plan["rows"], plan["lens"])):
        if t > 0:
            k, v = _keys_values(t, H, D, seed, 100 + b, torch.bfloat16)
            seen_to = torch.arange(t - r, t, device=DEV) if case["causal"] else torch.full((r,), t - 1, device=DEV)
            token = torch.arange(t, device=DEV)
            hidden = token[None, :] > seen_to[:, None]
            if case["window"]:
                hidden = hidden | (token[None, :] <= seen_to[:, None] - case["window"])
            for h in range(H):
                kh, vh = _stored(k[:, h:h + 1], case["fmt"])[:, 0], _stored(v[:, h:h + 1], case["fmt"])[:, 0]
                for g in range(G):
                    z = (q[at:at + r, h * G + g] @ kh.t()) / math.sqrt(D)
                    z[hidden] = -math.inf
                    y[at:at + r, h * G + g] = torch.nan_to_num(torch.softmax(z, 1), nan=0.0) @ vh
        at += r
    return y
