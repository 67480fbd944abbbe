"""wq_pages_assign and wq_cache_keep: page assignment against the header's rule played out on the host (equal numbers), kept
rows against the bytes of the cache (equal bits), and a serving loop with drafted trees, eager and as a replayed graph."""
import numpy as np
import pytest
import torch

from block_quantized_bit_amd import policy, wq
from block_quantized_bit_amd.inputs import bf16_bits_to_f32, f32_to_bf16_bits

from cache_helpers import Q4_0, Q4_1, Case, check_attn
from gpu_helpers import DEV, dev_bf16, require_gpu, say
from parts_helpers import HostPages, attend_seen, dev_words, sees_tree, trees, words

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def _i32(v):
    return torch.tensor(np.asarray(v, np.int32), device=DEV)


class DevPages:
    def __init__(self, page, pages, batch, per, rows):
        self.desc = wq.cache_desc("q4_0", 64, 1, page, pages)
        self.batch, self.per, self.rows = batch, per, rows
        self.pool = torch.full((4 + pages,), 77, dtype=torch.int32, device=DEV)
        wq.wq_pages_init(pages, self.pool)
        self.len = torch.zeros(batch, dtype=torch.int32, device=DEV)
        self.table = torch.full((batch, per), -1, dtype=torch.int32, device=DEV)
        self.start = torch.full((batch + 1,), -5, dtype=torch.int32, device=DEV)
        self.pos = torch.full((rows,), -9, dtype=torch.int32, device=DEV)
        self.slot = torch.full((rows,), -9, dtype=torch.int64, device=DEV)

    def assign(self, want, maps=True):
        self.want = _i32(want)
        wq.wq_pages_assign(self.desc, self.batch, self.len, self.want, self.table, self.per, self.pool, self.rows, self.start,
                           self.pos if maps else None, self.slot if maps else None)

    def check(self, h, out, what):
        torch.cuda.synchronize()
        start, pos, slot = out
        n = start[-1]
        pool = self.pool.cpu().numpy()
        assert pool[:4].tolist() == [len(h.queue), h.lacking, 0, 0], what
        assert pool[4:4 + len(h.queue)].tolist() == h.queue[::-1], what
        assert self.start.cpu().tolist() == start, what
        assert self.len.cpu().tolist() == h.len, what
        table = self.table.cpu().numpy()
        for b in range(self.batch):
            k = min(-(-h.len[b] // h.page), h.per)
            assert table[b, :k].tolist() == h.table[b][:k], f"{what}: table of {b}"
        if self.rows and pos is not None:
            assert self.pos.cpu().numpy()[:n].tolist() == pos[:n], what
            assert self.slot.cpu().numpy()[:n].tolist() == slot[:n], what


# page, pages, batch, pages per sequence, rows
POOLS = [(32, 1, 1, 1, 40), (32, 40, 1, 20, 700), (64, 100, 5, 12, 4000), (96, 500, 64, 9, 60000), (32, 3000, 65, 50, 120000),
         (32, 900, 300, 9, 90000), (448, 700, 1025, 2, 500000), (32, 5000, 4100, 4, 600000), (2048, 70, 3, 30, 200000),
         (32, 20000, 8192, 6, 1100000), (32, 9000, 9001, 3, 900000)]


@pytest.mark.parametrize("i", range(len(POOLS)))
def test_assign(i):
    """Sequences that grow, shrink, end, start and stay, for several calls; more is wanted than there is now and then."""
    page, pages, batch, per, rows = POOLS[i]
    say("pages", POOLS[i])
    rng = np.random.default_rng(i)
    h, d = HostPages(page, pages, batch, per), DevPages(page, pages, batch, per, rows)
    for step in range(8):
        top = min(per * page, max(1, int(2.2 * pages * page / batch)))
        want = rng.integers(0, top + 1, batch)
        kind = rng.integers(0, 5, batch)
        now = np.array(h.len)
        want = np.where(kind == 0, now, np.where(kind == 1, 0, np.where(kind == 2, np.minimum(now + 1, per * page), want)))
        if step == 5:
            want[:] = 0
        if step == 6:
            want[0] = per * page + 5                      # past the table: tokens without a place
        out = h.assign(want, rows)
        d.assign(want)
        d.check(h, out, f"call {step}")


def test_a_call_that_takes_back_restores(orc):
    h, d = HostPages(64, 300, 20, 30), DevPages(64, 300, 20, 30, 20000)
    rng = np.random.default_rng(3)
    a = rng.integers(0, 500, 20)
    for want in (a, a + 300, a, np.zeros(20, int)):
        before = d.pool.clone()
        out = h.assign(want, 20000)
        d.assign(want)
        d.check(h, out, "")
        if want is a:
            kept = before
    assert d.pool.cpu().numpy()[4:].tolist() == list(range(300))[::-1] and kept is not None


def test_negative_lengths_bad_entries_and_short_maps():
    """Lengths below 0 are 0; entries that are no page are not given back; rows past the maps are cut and the maps' ends
    left; a call without maps."""
    d = DevPages(32, 50, 4, 6, 100)
    d.assign([100, 70, 0, 31])
    torch.cuda.synchronize()
    d.table[0, 1], d.table[1, 2] = -3, 50
    d.assign([-4, -2**31, 5, 31])
    torch.cuda.synchronize()
    assert d.len.cpu().tolist() == [0, 0, 5, 31] and d.start.cpu().tolist() == [0, 0, 0, 5, 5]
    pool = d.pool.cpu().tolist()
    # 0..7 were taken (4, 3, 0, 1 pages); 0 2 3 and 4 5 come back, without the two entries that are none; then 0 is taken
    assert pool[:4] == [46, 0, 0, 0]
    assert pool[4:50][::-1] == [2, 3, 4, 5] + list(range(8, 50))
    assert d.table[2, 0].item() == 0
    d.pos.fill_(-9)
    d.slot.fill_(-9)
    d.assign([60, 60, 65, 31])
    torch.cuda.synchronize()
    assert d.start.cpu().tolist() == [0, 60, 100, 100, 100]
    d2 = DevPages(32, 50, 4, 6, 100)
    d2.assign([10, 0, 3, 0], maps=False)
    torch.cuda.synchronize()
    assert bool((d2.pos == -9).all()) and d2.start.cpu().tolist() == [0, 10, 10, 13, 13]
    d2.assign([10, 7, 3, 0])
    torch.cuda.synchronize()
    assert d2.pos.cpu().tolist() == list(range(7)) + [-9] * 93 and bool((d2.slot[7:] == -9).all())


def test_places_past_32_bits():
    """Slots of a pool of more than 2^31 tokens."""
    page, pages = 1 << 24, 400
    d = DevPages(page, pages, 3, 127, 50)
    d.pool[4:] = _i32(np.arange(pages))                    # the last pages first
    d.assign([20, 0, 30])
    torch.cuda.synchronize()
    assert d.slot.cpu().tolist() == [399 * page + t for t in range(20)] + [398 * page + t for t in range(30)]


def test_pages_graph_replays():
    """A captured call, replayed as lengths change, equals the host's rule."""
    h, d = HostPages(32, 400, 70, 12), DevPages(32, 400, 70, 12, 20000)
    rng = np.random.default_rng(8)
    want = torch.zeros(70, dtype=torch.int32, device=DEV)

    def step():
        wq.wq_pages_assign(d.desc, 70, d.len, want, d.table, 12, d.pool, 20000, d.start, d.pos, d.slot)

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for k in range(6):
        w = rng.integers(0, 260, 70)
        want.copy_(_i32(w))
        out = h.assign(w, 20000)
        g.replay()
        d.check(h, out, f"replay {k}")


def test_two_pools_on_two_streams():
    rng = np.random.default_rng(9)
    h, d = ([f(64, 600, 40, 20) if f is HostPages else f(64, 600, 40, 20, 40000) for _ in range(2)] for f in (HostPages, DevPages))
    streams = [torch.cuda.Stream() for _ in range(2)]
    wants = [_i32(rng.integers(0, 900, 40)) for _ in range(10)]
    torch.cuda.synchronize()
    out = [None, None]
    for k in range(5):
        for i in range(2):
            w = wants[2 * k + i]
            out[i] = h[i].assign(w.cpu().tolist(), 40000)
            x = d[i]
            wq.wq_pages_assign(x.desc, 40, x.len, w, x.table, 20, x.pool, 40000, x.start, x.pos, x.slot, stream=streams[i])
    for i in range(2):
        d[i].check(h[i], out[i], f"pool {i}")


def test_keep_in_many_caches():
    """As many caches as a call takes; each has its own bytes moved."""
    c = Case(Q4_1, 64, 1, 32, [9, 4], [40, 33], seed=2)
    caches = [torch.from_numpy(c.rng.integers(0, 256, c.cache.numel(), dtype=np.uint8)).to(DEV) for _ in range(64)]
    before = [x.clone() for x in caches]
    path, count = _i32([[1, 4, 8], [0, 3, 9]]), _i32([3, 3])
    wq.wq_cache_keep(c.desc, c.seqs, path, 3, count, caches)
    for x, y in zip(caches, before):
        wq.wq_cache_keep(c.desc, c.seqs, path, 3, count, [y])
        assert torch.equal(x, y)
    a, z = _rows_of(c, caches[63], 0, np.array([31, 32, 33])), _rows_of(c, before[63], 0, np.array([31, 32, 33]))
    assert all(np.array_equal(x, y) for x, y in zip(a, z))


def _rows_of(c, cache, b, tokens, fmt=None):
    """Read back tokens of sequence b (values as fp32 bits)."""
    t = c.lens[b]
    s = wq.seqs(1, t, _i32([t]), c.d_table[b:b + 1], _i32([0, t]))
    out = [torch.empty((t, c.heads * c.dim), dtype=torch.float32, device=DEV) for _ in range(2)]
    wq.wq_cache_read(c.desc, s, cache, out[0], c.heads * c.dim, out[1], c.heads * c.dim, wq.WQ_F32)
    torch.cuda.synchronize()
    return [o.cpu().numpy().view(np.uint32)[tokens] for o in out]


# dim, heads, page, rows, tokens, paths
KEEP = [
    (64, 20, 448, [13], [224], [[0, 3, 7, 12]]),
    (64, 2, 32, [5, 1, 0, 9], [5, 33, 40, 100], [[0, 1, 2, 3, 4], [0], [], [8]]),
    (96, 3, 96, [40, 33], [113, 700], [[1, 2, 5, 6, 30, 39], []]),
    (128, 8, 64, [64, 17], [1000, 64], [list(range(0, 64, 5)), [0, 1, 2, 4, 16]]),
    (256, 2, 32, [33, 8], [600, 70], [list(range(20)) + [25, 32], [2, 3]]),
    (128, 1, 32, [200], [250], [list(range(1, 200, 2)) + []]),                    # more entries than are looked up together
    (64, 1, 64, [150], [150], [[2 * j + (j > 60) for j in range(70)]]),
]


@pytest.mark.parametrize("fmt", [Q4_0, Q4_1], ids=["q4_0", "q4_1"])
@pytest.mark.parametrize("i", range(len(KEEP)))
def test_keep(fmt, i):
    """Kept rows have their bits at their new places, every other byte of every cache is as it was."""
    dim, heads, page, counts, lens, paths = KEEP[i]
    say("keep", fmt, KEEP[i][:5])
    c = Case(fmt, dim, heads, page, counts, lens, seed=i)
    c.fill(*c.random_kv())
    caches = [c.cache, torch.from_numpy(c.rng.integers(0, 256, c.cache.numel(), dtype=np.uint8)).to(DEV)]
    before = [x.clone() for x in caches]
    ld = max(1, max(len(p) for p in paths)) + i % 2
    path = np.full((c.batch, ld), 2**31 - 1, np.int32)
    for b, p in enumerate(paths):
        path[b, :len(p)] = p
    want = torch.full((c.batch,), -1, dtype=torch.int32, device=DEV)
    wq.wq_cache_keep(c.desc, c.seqs, torch.from_numpy(path).to(DEV), ld, _i32([len(p) for p in paths]), caches, want)
    torch.cuda.synchronize()
    assert want.cpu().tolist() == [t - n + len(p) for t, n, p in zip(lens, counts, paths)]
    for now, old in zip(caches, before):
        # the same bytes, moved by writing the same tokens' bytes on the host
        place = [np.arange(t) for t in lens]
        for b, p in enumerate(paths):
            pos0 = lens[b] - counts[b]
            place[b][pos0:pos0 + len(p)] = pos0 + np.array(p, int)
            a, z = _rows_of(c, now, b, slice(None)), _rows_of(c, old, b, place[b])
            assert all(np.array_equal(x, y) for x, y in zip(a, z)), f"sequence {b}"
        # and no byte but the moved tokens': written back to where they were, all is as before
        assert int((now != old).sum()) <= sum(2 * len(p) for p in paths) * heads * (dim // 2 + dim // 16 * (2 if fmt == Q4_1 else 1))
    pages = set(int(x) for b in range(c.batch) for x in c.table[b][:-(-lens[b] // page)])
    size = c.cache.numel() // c.desc.pages
    for now, old in zip(caches, before):
        for p in range(c.desc.pages):
            if p not in pages:
                assert torch.equal(now[p * size:(p + 1) * size], old[p * size:(p + 1) * size])


def test_keep_ends_paths():
    """A path ends before an entry that is no row, does not ascend, or has no page; counts past the path, below 0; rows
    without a token; without want."""
    c = Case(Q4_0, 64, 2, 32, [20, 20, 20, 20, 20, 20], [90, 90, 90, 90, 12, 90], seed=3, bad=[(3, 2)])
    c.fill(*c.random_kv())
    path = np.array([[0, 5, 4, 9], [1, 3, 20, 4], [-1, 0, 1, 2], [0, 1, 7, 2], [0, 1, 2, 3], [0, 2, 4, 6]], np.int32)
    want = torch.zeros(6, dtype=torch.int32, device=DEV)
    old = c.cache.clone()
    counts = _i32([4, 4, 4, 4, 4, 9])
    wq.wq_cache_keep(c.desc, c.seqs, torch.from_numpy(path).to(DEV), 4, counts, [c.cache], want)
    torch.cuda.synchronize()
    # rows of sequence 3 from the third page (token 64) on, which is absent: its pos0 is 70, so all of them
    assert want.cpu().tolist() == [72, 72, 70, 70, 0, 74]
    c.cache.copy_(old)
    wq.wq_cache_keep(c.desc, c.seqs, torch.from_numpy(path).to(DEV), 4, _i32([-1, 0, -5, 0, 0, -2**31]), [c.cache], None)
    torch.cuda.synchronize()
    assert torch.equal(c.cache, old)
    one = wq.seqs(6, 6, c.d_len, c.d_table)
    wq.wq_cache_keep(c.desc, one, torch.from_numpy(path[:, :1].copy()).to(DEV), 1, _i32([1] * 6), [c.cache], want)
    torch.cuda.synchronize()
    assert want.cpu().tolist() == [90, 89, 89, 89, 12, 90] and torch.equal(c.cache, old)


def test_keep_past_32_bits():
    """A pool of over 4 GiB; the pages in use are its last ones."""
    d = wq.cache_desc("q4_0", 256, 8, 256, 8700)
    cache = torch.empty(wq.wq_cache_size(d), dtype=torch.uint8, device=DEV)
    c = Case(Q4_0, 256, 8, 256, [60], [300], seed=4, spare=0)
    c.desc, c.cache = d, cache
    c.d_table = torch.tensor([[8699, 8697, -1]], dtype=torch.int32, device=DEV)
    c.seqs = wq.seqs(1, 60, c.d_len, c.d_table, c.d_start)
    c.fill(*c.random_kv())
    old = _rows_of(c, cache, 0, np.array([240 + j for j in (3, 9, 17, 40, 59)]))
    wq.wq_cache_keep(d, c.seqs, _i32([[3, 9, 17, 40, 59]]), 5, _i32([5]), [cache])
    torch.cuda.synchronize()
    new = _rows_of(c, cache, 0, np.arange(240, 245))
    assert all(np.array_equal(a, b) for a, b in zip(old, new))


@pytest.mark.parametrize("captured", [False, True], ids=["eager", "graph"])
def test_serving_with_drafts(orc, captured):
    """The calls as they are used: prompts admitted, then steps of drafting a tree, attention, keeping a path; requests end and
    others start.  The attention of every step is checked against float64 over the tokens that were kept so far."""
    fmt, dim, heads, group, page, batch, most = Q4_1, 64, 2, 2, 32, 5, 12
    width, hq = heads * dim, heads * group
    rng = np.random.default_rng(5)
    pages, per = 60, 12
    desc = wq.cache_desc(fmt, dim, heads, page, pages)
    caches = [torch.from_numpy(rng.integers(0, 256, wq.wq_cache_size(desc), dtype=np.uint8)).to(DEV) for _ in range(2)]
    pool = torch.empty(4 + pages, dtype=torch.int32, device=DEV)
    wq.wq_pages_init(pages, pool)
    zeros = lambda *s: torch.zeros(s, dtype=torch.int32, device=DEV)  # noqa: E731
    length, want, table, start = zeros(batch), zeros(batch), zeros(batch, per), zeros(batch + 1)
    kept, path, count = zeros(batch), zeros(batch, 4), zeros(batch)
    rows = batch * most
    pos, slot = zeros(rows), torch.zeros(rows, dtype=torch.int64, device=DEV)
    seqs = wq.seqs(batch, rows, length, table, start)
    K, V, Q = (torch.zeros((rows, w), dtype=torch.int16, device=DEV) for w in (width, width, hq * dim))
    Y = torch.zeros_like(Q)
    tree = zeros(rows, 1)
    n = wq.wq_attn_tree_workspace_size(desc, seqs, hq, 0, 0)
    ws = torch.empty(max(n, 16), dtype=torch.uint8, device=DEV)
    host_k, host_v = [np.zeros((0, heads, dim), np.uint16) for _ in range(batch)], [np.zeros((0, heads, dim), np.uint16) for _ in range(batch)]

    def step():
        wq.wq_pages_assign(desc, batch, length, want, table, per, pool, rows, start, pos, slot)
        for cache in caches:
            wq.wq_cache_write(desc, seqs, K, width, V, width, wq.WQ_BF16, cache)
        wq.wq_attn_tree(desc, seqs, hq, Q, hq * dim, caches[1], 0.125, 0, 0, tree, 1, Y, hq * dim, ws, n)
        wq.wq_cache_keep(desc, seqs, path, 4, count, caches, kept)

    graph = None
    for t in range(7):
        counts = rng.integers(1, most + 1, batch) if t else np.full(batch, most)
        counts[rng.integers(0, batch)] = 0 if t % 3 == 2 else counts[0]
        if t == 4:                                            # a request ends, and another takes its place
            host_k[1], host_v[1] = host_k[1][:0], host_v[1][:0]
            kept[1] = 0
            cut = kept.clone()
            wq.wq_pages_assign(desc, batch, length, cut, table, per, pool, rows, start)
        lens = [len(x) + int(a) for x, a in zip(host_k, counts)]
        # back to what was kept, and on from there, in one call: a call's rows are the tokens that its lengths grow by
        back = _i32([len(x) for x in host_k])
        wq.wq_pages_assign(desc, batch, length, back, table, per, pool, rows, start)
        want.copy_(_i32(lens))
        masks = trees(rng, counts, "chain" if t == 0 else "tree")
        if int(counts.sum()):
            tree[:int(counts.sum())] = dev_words(words(masks, 1, int(counts.sum())))
        at = np.concatenate([[0], np.cumsum(counts)])
        kb, vb, qb = (f32_to_bf16_bits(rng.standard_normal((rows, w), dtype=np.float32)) for w in (width, width, hq * dim))
        for x, y in ((K, kb), (V, vb), (Q, qb)):
            x.copy_(dev_bf16(y))
        paths = []
        for a, m in zip(counts, masks):                       # the way to a node
            node = int(rng.integers(0, a)) if a else 0
            paths.append(np.flatnonzero(m[node])[:4] if a else np.zeros(0, int))
        p = np.zeros((batch, 4), np.int32)
        for b, x in enumerate(paths):
            p[b, :len(x)] = x
        path.copy_(torch.from_numpy(p).to(DEV))
        count.copy_(_i32([len(x) for x in paths]))
        Y.fill_(0x7BAD)
        if captured and graph is None:
            side = torch.cuda.Stream()
            torch.cuda.synchronize()
            saved = [x.clone() for x in (length, table, pool, start, kept, *caches)]
            with torch.cuda.stream(side):
                step()
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                step()
            for x, y in zip((length, table, pool, start, kept, *caches), saved):
                x.copy_(y)
        graph.replay() if captured else step()
        torch.cuda.synchronize()
        assert start.cpu().tolist() == at.tolist() and pool[1].item() == 0
        assert pos.cpu().tolist()[:at[-1]] == [len(host_k[b]) + j for b in range(batch) for j in range(counts[b])]
        tab = table.cpu().numpy()
        where = [(len(host_k[b]) + j) for b in range(batch) for j in range(counts[b])]
        owner = [b for b in range(batch) for _ in range(counts[b])]
        assert slot.cpu().tolist()[:at[-1]] == [int(tab[b, x // page]) * page + x % page for b, x in zip(owner, where)]

        class Now:
            pass

        now = Now()
        now.fmt, now.dim, now.heads, now.batch, now.rows = fmt, dim, heads, batch, rows
        now.lens, now.counts, now.start = lens, [int(x) for x in counts], at
        now.present = lambda b: np.ones(lens[b], bool)  # noqa: B023
        full = [[np.concatenate([x[b], y.reshape(rows, heads, dim)[at[b]:at[b + 1]]]) for b in range(batch)]
                for x, y in ((host_k, kb), (host_v, vb))]
        ref, ab, A = attend_seen(now, orc, full[0], full[1], bf16_bits_to_f32(qb).reshape(rows, hq, dim), group, 0.125,
                                 sees_tree(now, masks, 1, 0, 0))
        y = Y.cpu().numpy().view(np.uint16)
        m = int(at[-1])
        check_attn(bf16_bits_to_f32(y).reshape(rows, hq, dim)[:m], ref[:m], ab[:m], A[:m], f"step {t}")
        assert np.all(y[m:] == 0x7BAD)
        assert kept.cpu().tolist() == [len(host_k[b]) + len(paths[b]) for b in range(batch)]
        for b in range(batch):
            pick = at[b] + paths[b]
            host_k[b] = np.concatenate([host_k[b], kb.reshape(rows, heads, dim)[pick]])
            host_v[b] = np.concatenate([host_v[b], vb.reshape(rows, heads, dim)[pick]])
    # nothing is lost: when all requests have ended every page is free once
    wq.wq_pages_assign(desc, batch, length, zeros(batch), table, per, pool, rows, start)
    torch.cuda.synchronize()
    assert pool[0].item() == pages and sorted(pool[4:].cpu().tolist()) == list(range(pages))


def test_the_models_decoder(orc):
    """A tree over the decoder's own self-attention caches, one page per utterance (no table)."""
    spec = [x for x in policy.decoder_caches("q4_0", 3) if x.kind == "self"]
    desc = spec[0].desc
    heads, dim = policy.HEADS, policy.HEAD_DIM
    rng = np.random.default_rng(2)
    c = Case(Q4_0, dim, heads, desc.page, [6, 1, 9], [100, 1, 448], seed=8, paged=False)
    k, v = c.random_kv()
    c.fill(k, v)
    masks = trees(rng, c.counts, "tree")
    q = f32_to_bf16_bits(rng.standard_normal((16, heads, dim), dtype=np.float32))
    Q, Y = dev_bf16(q.reshape(16, -1)), torch.zeros((16, heads * dim), dtype=torch.int16, device=DEV)
    tree = dev_words(words(masks, 1, 16))
    wq.wq_attn_tree(c.desc, c.seqs, heads, Q, heads * dim, c.cache, dim ** -0.5, 0, 0, tree, 1, Y, heads * dim)
    torch.cuda.synchronize()
    ref, ab, A = attend_seen(c, orc, k, v, bf16_bits_to_f32(q), 1, dim ** -0.5, sees_tree(c, masks, 1, 0, 0))
    check_attn(bf16_bits_to_f32(Y.cpu().numpy().view(np.uint16)).reshape(ref.shape), ref, ab, A)
    caches = [c.cache.clone() for _ in spec]
    want = torch.zeros(3, dtype=torch.int32, device=DEV)
    wq.wq_cache_keep(c.desc, c.seqs, _i32([[0, 5], [0, 0], [1, 8]]), 2, _i32([2, 1, 2]), caches, want)
    torch.cuda.synchronize()
    assert want.cpu().tolist() == [96, 1, 441] and all(torch.equal(x, caches[0]) for x in caches[1:])
