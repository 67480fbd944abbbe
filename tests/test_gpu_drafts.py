"""Pages and kept rows where a call's arrays hold what no ordinary step leaves there: the pool's own words, entries that are no
page among thousands that are given back, rows cut by the maps, lengths without pages; and the whole step, captured."""
import numpy as np
import pytest
import torch

from block_quantized_bit_amd import wq
from block_quantized_bit_amd.inputs import bf16_bits_to_f32, f32_to_bf16_bits

from cache_helpers import Q4_0, Q4_1, Case, check_attn, stored
from gpu_helpers import DEV, dev_bf16, require_gpu, say
from parts_helpers import HostPages, attend_seen, dev_words, run_seen, sees_sinks, sees_tree, trees, words
from test_gpu_pages import KEEP, DevPages, _i32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


class Pages(HostPages):
    """The rule where the maps cut rows off too: those that a sequence is left with are its last tokens (wq_seqs: row i of n is
    token len - n + i), where HostPages lists its first ones."""

    def assign(self, want, rows):
        grow = [max(max(int(w), 0) - t, 0) for w, t in zip(want, self.len)]
        start, pos, slot = super().assign(want, sum(grow))
        cut = np.minimum(start, rows)
        keep = np.concatenate([np.arange(e - n, e) for e, n in zip(start[1:], np.diff(cut))]).astype(int)
        return cut.tolist(), [pos[i] for i in keep], [slot[i] for i in keep]


@pytest.mark.parametrize("batch,rows", [(5, 300), (40, 40000), (3000, 200000), (9001, 200000)])
@pytest.mark.parametrize("word", [1, 3, 127, 2**31 - 1, -1, -2**31])
def test_a_pools_other_words_can_hold_anything(batch, rows, word):
    """A call goes by the number of free pages and the list; by one workgroup and by many."""
    say("words", batch, rows, word)
    per = 12
    h, d = Pages(32, 20000, batch, per), DevPages(32, 20000, batch, per, rows)
    rng = np.random.default_rng(batch)
    top = min(per * 32, 2 * rows // batch)
    for step in range(4):
        want = rng.integers(0, top + 1, batch) if step < 3 else np.zeros(batch, int)
        out = h.assign(want, rows)
        d.pool[1:4] = word
        d.assign(want)
        d.pool[2:4] = 0
        d.check(h, out, f"call {step}")


@pytest.mark.parametrize("maps", [False, True], ids=["no maps", "maps"])
@pytest.mark.parametrize("holes", [[], [0], [4095, 4096, 8191], "some", "all"], ids=str)
@pytest.mark.parametrize("batch,per", [(1, 9000), (3, 5000), (40, 300), (1200, 9)])
def test_thousands_of_entries_given_back(batch, per, holes, maps):
    """More than a workgroup looks at together, with entries among them that are no page, while other sequences take some of
    them; then others take the rest."""
    say("given back", batch, per, holes, maps)
    page, pages, rows = 32, batch * per + 50, 40000 if maps else 0
    h, d = Pages(page, pages, batch + 2, per), DevPages(page, pages, batch + 2, per, rows)
    rng = np.random.default_rng(per)
    full = np.array([per * page] * batch + [1, 0])
    wants = [full, np.array([0 if b % 5 else 40 for b in range(batch)] + [per * page - 3, 20]),
             np.array([int(x) for x in rng.integers(0, 2 * page * per, batch + 2)])]
    for step, want in enumerate(wants):
        if step == 1:
            at = np.arange(batch * per)
            at = at if holes == "all" else rng.permutation(at)[:batch * per // 3] if holes == "some" else np.array(holes, int)
            table = d.table.cpu().numpy()
            for k, i in enumerate(at):
                table[i // per, i % per] = h.table[i // per][i % per] = (-1, pages, -2**31)[k % 3]
            d.table.copy_(torch.from_numpy(table))
        out = h.assign(want, rows)
        d.assign(want, maps)
        d.check(h, out if maps else (out[0], None, None), f"call {step}")


def test_a_missing_page_does_not_cost_what_the_others_do():
    """One entry that is no page among 30000 that are given back: their pages are still looked at once or twice each."""
    took = []
    for hole in (False, True, False, True):
        d = DevPages(32, 30000, 1, 30000, 0)
        d.assign([960000], maps=False)
        if hole:
            d.table[0, 7] = -1
        d.want = _i32([0])
        events = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
        torch.cuda.synchronize()
        events[0].record()
        wq.wq_pages_assign(d.desc, 1, d.len, d.want, d.table, 30000, d.pool, 0, d.start)
        events[1].record()
        torch.cuda.synchronize()
        assert d.pool[:2].tolist() == [30000 - hole, 0]
        took.append(events[0].elapsed_time(events[1]))
    say("us", [round(1000 * t, 1) for t in took])
    assert min(took[1], took[3]) < 30 * min(took[0], took[2])      # (each one looked up from the start: some 2000 times)


@pytest.mark.parametrize("fmt,dim,heads,group,page", [(Q4_0, 128, 2, 4, 64), (Q4_1, 64, 3, 1, 32)], ids=["q4_0", "q4_1"])
def test_a_captured_step_with_its_last_call(orc, fmt, dim, heads, group, page):
    """The header's step, whole, as one graph: what wq_cache_keep wrote is what the lengths go back to and the next replay starts
    from, with nothing made on the host but the drafts."""
    batch, most, per, pages, ld = 4, 14, 8, 40, 5
    width, hq = heads * dim, heads * group
    rng = np.random.default_rng(dim)
    desc = wq.cache_desc(fmt, dim, heads, page, pages)
    caches = [torch.from_numpy(rng.integers(0, 256, wq.wq_cache_size(desc), dtype=np.uint8)).to(DEV) for _ in range(2)]
    zeros = lambda *s: torch.zeros(s, dtype=torch.int32, device=DEV)  # noqa: E731
    pool, length, grow, want, kept, table = zeros(4 + pages), zeros(batch), zeros(batch), zeros(batch), zeros(batch), zeros(batch, per)
    wq.wq_pages_init(pages, pool)
    rows = batch * most
    start, after, pos, slot = zeros(batch + 1), zeros(batch + 1), zeros(rows), torch.zeros(rows, dtype=torch.int64, device=DEV)
    path, count, tree = zeros(batch, ld), zeros(batch), zeros(rows, 1)
    seqs = wq.seqs(batch, rows, length, table, start)
    K, V, Q = (torch.zeros((rows, w), dtype=torch.int16, device=DEV) for w in (width, width, hq * dim))
    Y = torch.zeros_like(Q)
    n = wq.wq_attn_tree_workspace_size(desc, seqs, hq, 0, 0)
    ws = torch.empty(max(n, 16), dtype=torch.uint8, device=DEV)
    scale = dim ** -0.5

    def step():
        torch.add(length, grow, out=want)
        wq.wq_pages_assign(desc, batch, length, want, table, per, pool, rows, start, pos, slot)
        for cache in caches:
            wq.wq_cache_write(desc, seqs, K, width, V, width, wq.WQ_BF16, cache)
        wq.wq_attn_tree(desc, seqs, hq, Q, hq * dim, caches[1], scale, 0, 0, tree, 1, Y, hq * dim, ws, n)
        wq.wq_cache_keep(desc, seqs, path, ld, count, caches, kept)
        wq.wq_pages_assign(desc, batch, length, kept, table, per, pool, 0, after)

    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        step()                                                # (nothing grows: no rows)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    host_k, host_v = ([np.zeros((0, heads, dim), np.uint16) for _ in range(batch)] for _ in range(2))
    for t in range(8):
        counts = rng.integers(1, most + 1, batch)
        if t % 3 == 1:
            counts[rng.integers(0, batch)] = 0
        at = np.concatenate([[0], np.cumsum(counts)])
        m = int(at[-1])
        masks = trees(rng, counts, "tree")
        tree[:m] = dev_words(words(masks, 1, m))
        kb, vb, qb = (f32_to_bf16_bits(rng.standard_normal((rows, w), dtype=np.float32)) for w in (width, width, hq * dim))
        for x, y in ((K, kb), (V, vb), (Q, qb)):
            x.copy_(dev_bf16(y))
        paths = [np.flatnonzero(x[int(rng.integers(0, a))])[:ld] if a else np.zeros(0, int) for a, x in zip(counts, masks)]
        p = np.full((batch, ld), -1, np.int32)
        for b, x in enumerate(paths):
            p[b, :len(x)] = x
        path.copy_(torch.from_numpy(p).to(DEV))
        count.copy_(_i32([len(x) for x in paths]))
        grow.copy_(_i32(counts))
        Y.fill_(0x7BAD)
        graph.replay()
        torch.cuda.synchronize()
        assert start.cpu().tolist() == at.tolist() and after.cpu().tolist() == [0] * (batch + 1), t
        place = [(b, len(host_k[b]) + j) for b in range(batch) for j in range(counts[b])]
        assert pos.cpu().tolist()[:m] == [x for _, x in place], t

        class Now:
            pass

        now = Now()
        now.fmt, now.dim, now.heads, now.batch, now.rows = fmt, dim, heads, batch, rows
        now.lens, now.counts, now.start = [len(x) + int(a) for x, a in zip(host_k, counts)], [int(x) for x in counts], at
        now.present = lambda b: np.ones(now.lens[b], bool)  # noqa: B023
        full = [[np.concatenate([x[b], y.reshape(rows, heads, dim)[at[b]:at[b + 1]]]) for b in range(batch)]
                for x, y in ((host_k, kb), (host_v, vb))]
        ref, ab, A = attend_seen(now, orc, full[0], full[1], bf16_bits_to_f32(qb).reshape(rows, hq, dim), group, scale,
                                 sees_tree(now, masks, 1, 0, 0))
        y = Y.cpu().numpy().view(np.uint16)
        check_attn(bf16_bits_to_f32(y).reshape(rows, hq, dim)[:m], ref[:m], ab[:m], A[:m], f"step {t}")
        assert np.all(y[m:] == 0x7BAD)
        for b in range(batch):
            pick = at[b] + paths[b]
            host_k[b] = np.concatenate([host_k[b], kb.reshape(rows, heads, dim)[pick]])
            host_v[b] = np.concatenate([host_v[b], vb.reshape(rows, heads, dim)[pick]])
        lens = [len(x) for x in host_k]
        assert kept.cpu().tolist() == lens and length.cpu().tolist() == lens, t
        held = [int(x) for b in range(batch) for x in table[b, :-(-lens[b] // page)].cpu()]
        free = pool[4:4 + int(pool[0])].cpu().tolist()
        assert sorted(held + free) == list(range(pages)) and pool[1].item() == 0, t


@pytest.mark.parametrize("others", [0, 9000])
def test_pages_that_were_lacking(others):
    """Entries that got no page stay without one while their sequence goes on, and get one when it has shrunk and grows again."""
    page, per = 32, 8
    h, d = Pages(page, 4 + others, 2 + others, per), DevPages(page, 4 + others, 2 + others, per, 200 + others)

    def call(a, b):
        want = np.array([a, b] + [1] * others)
        out = h.assign(want, 200 + others)
        d.assign(want)
        d.check(h, out, f"{a} and {b}")
        slot = d.slot.cpu().tolist()[out[0][1]:out[0][2]]          # of the second sequence's rows
        return d.pool[1].item(), d.table[1].cpu().tolist()[:-(-b // page)], slot

    def first():                                              # the others take theirs
        want = np.array([0, 0] + [1] * others)
        out = h.assign(want, 200 + others)
        d.assign(want)
        d.check(h, out, "the others")

    first()
    lacking, table, slot = call(64, 96)
    assert lacking == 1 and table[2] == -1 and slot[64:] == [-1] * 32 and -1 not in slot[:64]
    lacking, table, slot = call(0, 96)                        # two pages are free again
    assert lacking == 0 and table[2] == -1 and d.pool[0].item() == 2
    lacking, table, slot = call(0, 97)                        # a page for the token that is new, none for the hole
    assert lacking == 0 and table[2] == -1 and table[3] >= 0 and len(slot) == 1 and slot[0] >= 0
    lacking, table, slot = call(0, 64)                        # back to before, and on: all are there
    assert lacking == 0 and d.pool[0].item() == 2
    lacking, table, slot = call(0, 97)
    assert lacking == 0 and min(table) >= 0 and len(slot) == 33 and min(slot) >= 0


def test_no_sequences_is_no_call():
    """With a batch of 0 nothing is written: neither row starts nor counts."""
    d = DevPages(32, 10, 3, 4, 50)
    d.assign([40, 0, 7])
    before = [x.clone() for x in (d.pool, d.len, d.table, d.start, d.pos, d.slot)]
    wq.wq_pages_assign(d.desc, 0, d.len, d.want, d.table, 4, d.pool, 50, d.start, d.pos, d.slot)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(before, (d.pool, d.len, d.table, d.start, d.pos, d.slot)))


# rows and tokens of the sequences, heads, group: single tokens, and drafts whose tiles have 16, 32, 128 and 256 columns, whole and
# (over 3001 tokens) shared out
WIDTHS = {"token": ([1, 1], [70, 33], 2, 4), "16": ([3, 70], [80, 300], 1, 4), "32": ([12] * 40, [70] * 40, 8, 4),
          "128": ([32] * 8, [150] * 8, 16, 4), "256": ([128] * 8, [140] * 8, 16, 2), "token shared": ([1], [3001], 1, 4),
          "32 shared": ([10, 3], [3001, 70], 1, 4), "128 shared": ([30], [3001], 1, 4), "256 shared": ([70], [3001], 1, 4)}
WIDTH = pytest.mark.parametrize("width", WIDTHS)


def _scores(orc, fmt, dim, width, k_of, q_of, scale, tol, what):
    """wq_attn_sinks and wq_attn_tree of one case within `tol`(A, Q) sum (p + 2^-23) |v^| and the output's own rounding, values 1
    and 0 by turns, so that a wrong probability shows."""
    counts, lens, heads, group = WIDTHS[width]
    c = Case(fmt, dim, heads, 64, counts, lens, seed=dim)
    k = [k_of(c, t) for t in lens]
    v = [np.zeros((t, heads, dim), np.float32) for t in lens]
    for x in v:
        x[::2] = 1.0
    v = [f32_to_bf16_bits(x) for x in v]
    c.fill(k, v)
    q = f32_to_bf16_bits(q_of(c, (c.rows, heads * group, dim)))
    qf = bf16_bits_to_f32(q)
    masks = trees(c.rng, counts, "tree")
    ld = -(-max(counts) // 32)
    most = max(np.abs(stored(orc, fmt, bf16_bits_to_f32(x)).astype(np.float64)).sum(-1).max() for x in k)
    Q = abs(scale) * np.abs(qf.astype(np.float64)).max(-1)[..., None] * most
    for window, sinks, tree in ((max(lens), 0, None), (50, 20, None), (0, 0, masks), (100, 7, masks)):
        sees = sees_sinks(c, window, sinks) if tree is None else sees_tree(c, masks, ld, window, sinks)
        ref, ab, A = attend_seen(c, orc, k, v, qf, group, scale, sees)
        bound = tol(A, Q) * ab + 2.0 ** -8 * np.abs(ref) + 1e-30
        for ws in ("asked", None):
            y = run_seen(c, q, group, scale, window, sinks, None if tree is None else dev_words(words(masks, ld, c.rows)), ws=ws)[0]
            err = np.abs(y.astype(np.float64) - ref)
            bad = ~(err <= bound)
            assert not bad.any(), f"{what} {width} {window} {sinks} ws={ws}: {bad.sum()} of {bad.size} outside, {np.nanmax(err / bound):.3g} of the bound"


@WIDTH
@pytest.mark.parametrize("dim", [64, 96, 128, 256])
def test_q4_0_keys_of_bf16_rows_are_exact(orc, dim, width):
    """|y - ref| <= (2^-9 + 2^-14 A) sum (p + 2^-23) |v^| + 2^-8 |ref|, a 32nd of what the scores may be off in general.

    A block's scale is a bf16 number over -8, of 8 bits, and a code less 8 has 3 (8 itself is a power of two): their products have
    11, and are fp16 numbers whether the kernel multiplies codes or values.  Queries of these sizes are exact too, and so is a product of
    the two in fp32.  What is left of a score's error is the fp32 sum of at most 256 of them, 2^-24 of the sum of their magnitudes
    each and as much again for the order that the matrix unit has: 2^-15 A, and a probability twice that."""
    say("exact keys", dim, width)
    _scores(orc, Q4_0, dim, width, lambda c, t: f32_to_bf16_bits(c.rng.standard_normal((t, c.heads, dim), dtype=np.float32) + 0.3),
            lambda c, n: c.rng.standard_normal(n, dtype=np.float32), 24 * dim ** -0.5, lambda A, Q: 2.0 ** -9 + 2.0 ** -14 * A, "exact keys")


def _general(A, Q):
    """The header's bound: half steps of fp16 (2^-11) of probabilities, values, and keys and queries in a score, and what small
    queries beside a large one lose."""
    return 2.0 ** -9 + 2.0 ** -9 * A + 2.0 ** -38 * Q


@WIDTH
@pytest.mark.parametrize("fmt", [Q4_0, Q4_1], ids=["q4_0", "q4_1"])
@pytest.mark.parametrize("outlier", [30.0, -30000.0])
def test_outlier_keys_of_drafts(orc, fmt, outlier, width):
    """Each block of a key has one large channel, where the query is zero: every true score is 0, and all tokens count alike."""
    def keys(c, t):
        k = np.zeros((t, c.heads, 64), np.float32)
        k[::2, :, 5::32], k[1::4, :, 5::32] = outlier, -outlier
        return f32_to_bf16_bits(k)

    def queries(c, n):
        q = c.rng.standard_normal(n, dtype=np.float32) * np.exp2(c.rng.integers(-10, 10, n)).astype(np.float32)
        q[..., 5::32] = 0.0
        return q

    say("outlier", fmt, outlier, width)
    _scores(orc, fmt, 64, width, keys, queries, 0.125, _general, f"outlier {outlier}")


@WIDTH
@pytest.mark.parametrize("fmt", [Q4_0, Q4_1], ids=["q4_0", "q4_1"])
@pytest.mark.parametrize("qs,scale", [(2.0 ** 122, 2.0 ** -124), (2.0 ** -122, 2.0 ** 119), (2.0 ** -129, 2.0 ** 126)], ids=["largest", "small", "subnormal"])
def test_drafts_queries_of_any_magnitude(orc, fmt, qs, scale, width):
    say("magnitude", fmt, qs, width)
    _scores(orc, fmt, 128, width, lambda c, t: f32_to_bf16_bits(c.rng.standard_normal((t, c.heads, 128), dtype=np.float32)),
            lambda c, n: (c.rng.standard_normal(n) * qs).astype(np.float32), scale, _general, f"queries of {qs}")


@pytest.mark.parametrize("batch,rows", [(20, 20000), (300, 90000), (9001, 90000)])
def test_taking_back_puts_the_pages_where_they_were(batch, rows):
    """After a call that takes and one that takes it back the list is the one from before, entry by entry, and so are the lengths
    and the tables' live entries."""
    d = DevPages(64, 30 * batch, batch, 30, rows)
    rng = np.random.default_rng(3)
    at = rng.integers(0, 9 if batch > 1000 else 250, batch)
    d.assign(at)
    d.assign(rng.permutation(at))
    at = d.len.cpu().numpy()
    for grow in (1, 7, 200):
        torch.cuda.synchronize()
        n = int(d.pool[0])
        pool, table = d.pool[4:4 + n].clone(), d.table.clone()
        more = at + np.minimum(rng.integers(0, grow + 1, batch), rows // batch)
        d.assign(more)
        torch.cuda.synchronize()
        assert int(d.pool[0]) == n - int((-(-more // 64) - -(-at // 64)).sum()) and d.pool[1].item() == 0
        d.assign(at)
        torch.cuda.synchronize()
        assert int(d.pool[0]) == n and torch.equal(d.pool[4:4 + n], pool)
        assert d.len.cpu().numpy().tolist() == at.tolist() and d.start[-1].item() == 0
        live = torch.arange(30, device=DEV)[None] < (_i32(at)[:, None] + 63) // 64
        assert torch.equal(d.table[live], table[live])


def _row_bytes(dim, q41):
    """Byte offsets of each of a unit's 32 tokens [32, bytes of a row], by the layout's rule: K's words of 8 channels, V's bytes of
    two, a scale (and an offset) for 32 channels of each."""
    nb, half, plane = dim // 32, dim * (20 if q41 else 18), 2 * dim

    def word(wi, lane):
        c = wi // 4
        return c * 1024 + lane * (16 if 4 * c + 4 <= 2 * nb else 8) + wi % 4 * 4

    out = []
    for t in range(32):
        at = [word(t // 16 * nb + b, g * 16 + t % 16) + i for b in range(nb) for g in range(4) for i in range(4)]
        at += [half + word(2 * b + t // 16, t % 16 // 4 * 16 + c) + t % 4 for b in range(nb) for c in range(16)]
        at += [v + 16 * dim + m + 2 * ((t // 4 * nb + b) * 4 + t % 4) + i for v in (0, half) for m in ((0, plane) if q41 else (0,))
               for b in range(nb) for i in range(2)]
        out.append(at)
    out = np.array(out)
    assert sorted(out.ravel()) == list(range(2 * half))
    return out


@pytest.mark.parametrize("fmt", [Q4_0, Q4_1], ids=["q4_0", "q4_1"])
@pytest.mark.parametrize("i", range(len(KEEP)))
def test_keep_moves_the_kept_rows_and_nothing_else(fmt, i):
    """Every byte of every cache against the same moves on the host: rows that stay, and the places of other tokens, past a
    sequence's end and in other pages too, hold what they held."""
    dim, heads, page, counts, lens, paths = KEEP[i]
    say("keep", fmt, KEEP[i][:5])
    c = Case(fmt, dim, heads, page, counts, lens, seed=70 + i)
    caches = [torch.from_numpy(c.rng.integers(0, 256, c.cache.numel(), dtype=np.uint8)).to(DEV) for _ in range(3)]
    want = [x.cpu().numpy().copy() for x in caches]
    rows, upp = _row_bytes(dim, fmt == Q4_1), page // 32
    unit = rows.size
    for b, p in enumerate(paths):
        def place(t):
            page_no = int(c.table[b, t // page])
            return [((page_no * heads + h) * upp + t % page // 32) * unit + rows[t % 32] for h in range(heads)]
        for j, row in enumerate(p):
            pos0 = lens[b] - counts[b]
            for to, at in zip(place(pos0 + j), place(pos0 + row)):
                for x in want:
                    x[to] = x[at]
    ld = max(1, max(len(p) for p in paths))
    path = np.full((c.batch, ld), -1, np.int32)
    for b, p in enumerate(paths):
        path[b, :len(p)] = p
    wq.wq_cache_keep(c.desc, c.seqs, torch.from_numpy(path).to(DEV), ld, _i32([len(p) for p in paths]), caches)
    torch.cuda.synchronize()
    for x, y in zip(caches, want):
        assert np.array_equal(x.cpu().numpy(), y)


@pytest.mark.parametrize("fmt", [Q4_0, Q4_1], ids=["q4_0", "q4_1"])
@pytest.mark.parametrize("dim,group,counts,lens,paged", [(128, 300, [3, 1], [3001, 70], True), (64, 300, [3] * 40, [40] * 40, True),
                                                         (96, 150, [2, 5], [2500, 5], True), (256, 260, [2, 1], [3001, 33], True),
                                                         (128, 3, [9, 14], [3000, 2999], False), (64, 2, [100, 1], [3001, 17], False)])
def test_heads_of_several_tiles_and_long_pages(orc, fmt, dim, group, counts, lens, paged):
    """More heads for a key/value head than a tile has columns, whole and shared out; sequences that are one page each, without a
    table."""
    say("wide groups", fmt, dim, group, counts, paged)
    c = Case(fmt, dim, 1, 64 if paged else 3104, counts, lens, seed=group, paged=paged)
    k, v = c.random_kv()
    c.fill(k, v)
    q = f32_to_bf16_bits(c.rng.standard_normal((c.rows, group, dim), dtype=np.float32))
    masks = trees(c.rng, counts, "tree")
    ld = -(-max(counts) // 32)
    for window, sinks, tree in ((0, 0, True), (2100, 70, True), (2100, 70, False), (33, 4, False)):
        sees = sees_tree(c, masks, ld, window, sinks) if tree else sees_sinks(c, window, sinks)
        ref, ab, A = attend_seen(c, orc, k, v, bf16_bits_to_f32(q), group, dim ** -0.5, sees)
        for ws in ("asked", None):
            y = run_seen(c, q, group, dim ** -0.5, window, sinks, dev_words(words(masks, ld, c.rows)) if tree else None, ws=ws)[0]
            check_attn(y, ref, ab, A, f"{window} {sinks} {tree} ws={ws}")


@pytest.mark.parametrize("batch,rows", [(3, 90), (60, 9000), (9001, 30000)])
def test_one_of_the_two_maps(batch, rows):
    h, d = Pages(32, 4 * batch, batch, 4), DevPages(32, 4 * batch, batch, 4, rows)
    want = np.random.default_rng(batch).integers(0, 128, batch)
    start, pos, slot = h.assign(want, rows)
    for a, b in ((d.pos, None), (None, d.slot)):
        d.want = _i32(want)
        wq.wq_pages_assign(d.desc, batch, d.len, d.want, d.table, 4, d.pool, rows, d.start, a, b)
        torch.cuda.synchronize()
        assert d.start.cpu().tolist() == start
        assert (a if b is None else b).cpu().tolist()[:start[-1]] == (pos if b is None else slot)
        d.assign(np.zeros(batch, int), maps=False)


@pytest.mark.parametrize("fmt", [Q4_0, Q4_1], ids=["q4_0", "q4_1"])
def test_keep_in_sequences_of_one_page(fmt):
    """Without a table; the rows' lengths past the page are absent, where a path ends."""
    c = Case(fmt, 96, 2, 96, [40, 30, 5], [90, 96, 5], seed=9, paged=False)
    c.d_len.copy_(_i32([90, 120, 5]))                          # the second one's rows are tokens 90 .. 119 of a page of 96
    cache = torch.from_numpy(c.rng.integers(0, 256, c.cache.numel(), dtype=np.uint8)).to(DEV)
    want, rows = cache.cpu().numpy().copy(), _row_bytes(96, fmt == Q4_1)
    paths, kept = [[0, 2, 3, 39], [1, 4, 5, 6, 29], [4]], [4, 3, 1]
    for b, (p, first) in enumerate(zip(paths, (50, 90, 0))):
        for j, row in enumerate(p[:kept[b]]):
            for h in range(2):
                to, at = (((b * 2 + h) * 3 + t // 32) * rows.size + rows[t % 32] for t in (first + j, first + row))
                want[to] = want[at]
    path = np.full((3, 5), -1, np.int32)
    for b, p in enumerate(paths):
        path[b, :len(p)] = p
    got = torch.zeros(3, dtype=torch.int32, device=DEV)
    wq.wq_cache_keep(c.desc, c.seqs, torch.from_numpy(path).to(DEV), 5, _i32([len(p) for p in paths]), [cache], got)
    torch.cuda.synchronize()
    assert got.cpu().tolist() == [54, 93, 1] and np.array_equal(cache.cpu().numpy(), want)
