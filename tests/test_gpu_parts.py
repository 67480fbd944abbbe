"""wq_attn_sinks and wq_attn_tree against float64 attention over the values the cache stands for: windows of one token and of
more than there are, sinks that reach into or past the window, gaps of many pages, trees of any shape over any context, rows
that see nothing, bad pages, strides, split calls, streams and replayed graphs."""
import numpy as np
import pytest
import torch

from block_quantized_bit_amd import wq
from block_quantized_bit_amd.inputs import bf16_bits_to_f32, f32_to_bf16_bits

from cache_helpers import Q4_0, Q4_1, Case, check_attn, run_attn
from gpu_helpers import DEV, dev_bf16, require_gpu, say
from parts_helpers import attend_seen, dev_words, run_seen, sees_sinks, sees_tree, trees, words

pytestmark = pytest.mark.gpu

FMT = [Q4_0, Q4_1]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def _q(c, group, std=1.0):
    return f32_to_bf16_bits(c.rng.standard_normal((c.rows, c.heads * group, c.dim), dtype=np.float32) * std)


def _check(orc, c, group, window, sinks, masks=None, ld=None, *, pad=0, ws=("asked", None), what="", scale=None):
    k, v = c.random_kv()
    c.fill(k, v)
    q = _q(c, group)
    scale = c.dim ** -0.5 if scale is None else scale
    tree = None
    if masks is None:
        sees = sees_sinks(c, window, sinks)
    else:
        ld = ld or max(1, -(-max(c.counts) // 32))
        sees = sees_tree(c, masks, ld, window, sinks)
        tree = dev_words(words(masks, ld, c.rows, c.rng))
    ref, ab, A = attend_seen(c, orc, k, v, bf16_bits_to_f32(q), group, scale, sees)
    n, ys = int(c.start[-1]), []
    for w in ws:
        y, bits = run_seen(c, q, group, scale, window, sinks, tree, ws=w, pad=pad)
        check_attn(y[:n], ref[:n], ab[:n], A[:n], f"{what} ws={w}")
        assert np.all(bits[n:] == 0x7BAD), "rows behind the last sequence were written"
        ys.append(bits)
    return q, ys


# dim, heads, group, page, rows, tokens, window, sinks
SINKS = [
    (64, 20, 1, 448, [1], [448], 224, 4),
    (64, 4, 1, 64, [1] * 6, [0, 1, 4, 5, 33, 700], 1, 4),
    (64, 2, 16, 32, [1] * 5, [0, 1, 32, 33, 5000], 100, 33),           # a gap of more pages than a wave holds entries
    (96, 3, 5, 96, [1] * 4, [95, 96, 97, 700], 300, 0),
    (128, 8, 4, 64, [1] * 6, [1, 15, 16, 17, 64, 1000], 2000, 64),     # a window of more than there are
    (128, 1, 40, 64, [1] * 2, [333, 65], 64, 65),
    (128, 2, 8, 32, [1] * 3, [2000, 100, 31], 128, 1900),              # sinks that reach into the window
    (256, 2, 8, 64, [1] * 3, [513, 64, 2], 31, 1),
    (256, 1, 3, 128, [1] * 2, [700, 129], 33, 2**31 - 1),
    (128, 1, 4, 32, [1] * 2, [9001, 6000], 2**31 - 1, 7),
    (64, 4, 1, 448, [5, 1, 0, 17], [100, 1, 50, 17], 9, 4),
    (64, 2, 3, 64, [3, 9, 4], [2, 5, 4], 2, 1),                        # rows whose token would be negative see nothing
    (96, 2, 2, 96, [40, 150], [40, 400], 50, 3),
    (128, 2, 4, 64, [5] * 4, [300, 5, 64, 3129], 50, 33),
    (256, 2, 2, 32, [7, 2], [1123, 80], 40, 70),
    # more than 128 columns per sequence
    (64, 4, 4, 448, [41, 90, 0, 33], [100, 90, 50, 470], 20, 4),
    (64, 2, 3, 64, [130, 9, 44], [77, 5, 300], 33, 1),
    (96, 3, 2, 32, [140, 77], [3333, 77], 64, 40),
    (128, 2, 4, 64, [64, 33, 64], [300, 64, 5129], 50, 5),
    (128, 1, 2, 32, [257], [2570], 1, 0),
    (128, 1, 5, 64, [70, 70], [70, 200], 1000, 4),
    (256, 1, 4, 64, [65, 30], [2600, 33], 100, 1),
    (256, 2, 2, 32, [90, 80], [123, 80], 40, 200),
    (64, 30, 1, 64, [1500, 100], [1500, 3164], 300, 17),               # enough tiles for 256 columns each
    (128, 20, 2, 96, [800, 333], [850, 333], 129, 65),
]

# dim, heads, group, page, rows, tokens, window, sinks
TREES = [
    (64, 20, 1, 448, [13], [224], 0, 0),
    (64, 4, 1, 64, [1, 2, 31, 32, 33], [1, 2, 31, 33, 95], 0, 0),      # no context, or next to none
    (64, 2, 5, 32, [3, 0, 9], [2, 40, 5], 0, 0),                       # rows whose token would be negative
    (96, 3, 3, 96, [17, 5, 8], [113, 700, 96], 0, 0),
    (128, 8, 4, 64, [25, 7, 31], [1000, 64, 95], 0, 0),
    (128, 2, 8, 32, [25, 16], [2000, 31], 100, 33),
    (128, 2, 2, 64, [60, 1], [5000, 1], 20, 4),                        # deeper than the window at the chain's end
    (256, 2, 8, 64, [9, 2], [513, 64], 64, 1),
    (256, 1, 3, 128, [33, 40], [700, 169], 0, 0),
    (128, 1, 70, 64, [3, 2], [333, 65], 0, 0),                         # one row's heads are several tiles
    # more than 128 columns per sequence
    (64, 4, 4, 448, [41, 90, 0, 33], [100, 90, 50, 470], 0, 0),
    (64, 2, 3, 64, [130, 9, 44], [77, 5, 300], 0, 0),
    (96, 3, 2, 32, [140, 77], [3333, 77], 64, 40),
    (128, 2, 4, 64, [64, 33, 64], [300, 64, 5129], 0, 0),
    (128, 1, 2, 32, [257], [2570], 500, 0),
    (256, 1, 4, 64, [65, 30], [600, 33], 0, 0),
    (256, 2, 2, 32, [90, 80], [123, 2080], 40, 200),
    (64, 30, 1, 64, [700, 1100], [1500, 1100], 300, 17),
    (128, 20, 2, 96, [800, 333], [850, 333], 0, 0),
]


@pytest.mark.parametrize("fmt", FMT, ids=["q4_0", "q4_1"])
@pytest.mark.parametrize("i", range(len(SINKS)))
def test_sinks(orc, fmt, i):
    dim, heads, group, page, counts, lens, window, sinks = SINKS[i]
    say("sinks", fmt, SINKS[i])
    c = Case(fmt, dim, heads, page, counts, lens, seed=i, one_row=max(counts) == 1 and min(counts) == 1, pad_rows=i % 3)
    _check(orc, c, group, window, sinks, pad=8 * (i % 2), what=str(SINKS[i]))


@pytest.mark.parametrize("fmt", FMT, ids=["q4_0", "q4_1"])
@pytest.mark.parametrize("kind", ["tree", "chain", "any", "none"])
@pytest.mark.parametrize("i", range(len(TREES)))
def test_trees(orc, fmt, kind, i):
    dim, heads, group, page, counts, lens, window, sinks = TREES[i]
    if kind in ("chain", "none") and max(counts) > 100:
        kind = "tree" if kind == "chain" else "any"
    say("tree", fmt, kind, TREES[i])
    c = Case(fmt, dim, heads, page, counts, lens, seed=60 + i, pad_rows=i % 3)
    masks = trees(c.rng, counts, kind)
    ld = max(1, -(-max(counts) // 32))
    _check(orc, c, group, window, sinks, masks, ld + i % 2 - (1 if ld > 1 and i % 5 == 0 else 0), pad=8 * (i % 2), what=f"{kind} {TREES[i]}")


@pytest.mark.parametrize("fmt,dim", [(Q4_0, 128), (Q4_1, 64), (Q4_0, 96), (Q4_1, 256)])
def test_long_sequences_shared_out(orc, fmt, dim):
    """Few rows over long sequences: split over workgroups (with a workspace), window and sinks far apart."""
    c = Case(fmt, dim, 2, 256, [1, 1, 1, 1], [20011, 1, 0, 5003], seed=7, one_row=True)
    _check(orc, c, 4, 9000, 100, what="window shared out")
    c = Case(fmt, dim, 1, 64, [2, 3], [9001, 130], seed=8)
    _check(orc, c, 8, 5000, 2000, what="several rows")
    for counts, lens, group in (([9, 3], [9001, 130], 4), ([40], [6001], 2), ([100, 1, 90], [4001, 40, 90], 3)):
        c = Case(fmt, dim, 1, 64, counts, lens, seed=9)
        masks = trees(c.rng, counts, "tree")
        for window, sinks in ((0, 0), (3000, 50)):
            _check(orc, c, group, window, sinks, masks, what=f"tree {counts} {window}")


@pytest.mark.parametrize("fmt", FMT, ids=["q4_0", "q4_1"])
@pytest.mark.parametrize("dim", [64, 96, 128, 256])
def test_one_long_sequence_among_many(orc, fmt, dim):
    counts = [3, 5, 1, 8] * 10
    lens = [6000] + [int(x) for x in np.random.default_rng(dim).integers(8, 300, 39)]
    c = Case(fmt, dim, 2, 64, counts, lens, seed=21)
    _check(orc, c, 2, 0, 0, trees(c.rng, counts, "tree"), what="tree")
    _check(orc, c, 2, 4000, 40, what="sinks")


def test_a_chain_is_causal(orc):
    """A tree that is a chain sees what wq_attn's rows see, and so does a window that leaves nothing out."""
    for counts, group in (([5, 2], 2), ([40, 33], 2), ([90, 70], 3)):
        c = Case(Q4_0, 128, 2, 64, counts, [900, 333], seed=3)
        k, v = c.random_kv()
        c.fill(k, v)
        q, scale = _q(c, group), 128 ** -0.5
        ref, ab, A = attend_seen(c, orc, k, v, bf16_bits_to_f32(q), group, scale, sees_sinks(c, 900, 0))
        tree = dev_words(words(trees(c.rng, counts, "chain"), -(-max(counts) // 32), c.rows))
        check_attn(run_seen(c, q, group, scale, 0, 0, tree)[0], ref, ab, A, "chain")
        check_attn(run_attn(c, q, group, scale, 1, 0)[0], ref, ab, A, "causal")
        for window, sinks in ((900, 0), (1, 900), (500, 400)):
            check_attn(run_seen(c, q, group, scale, window, sinks)[0], ref, ab, A, f"{window} and {sinks}")


@pytest.mark.parametrize("counts", [[1, 1, 1], [33, 1, 8], [200, 32, 60]], ids=["token", "rows", "many"])
def test_bad_pages_are_absent(orc, counts):
    for bad in ([(0, 0), (0, 3), (1, 0), (2, 2)], [(0, 6), (1, 0), (2, 1)], [(0, 1), (2, 0)]):
        c = Case(Q4_1, 64, 2, 32, counts, [200, 32, 70], bad=bad, seed=4, one_row=max(counts) == 1)
        _check(orc, c, 2, 50, 40)
        _check(orc, c, 2, 0, 0, trees(c.rng, counts, "tree"))


@pytest.mark.parametrize("rows", [1, 40, 140])
def test_results_do_not_change(orc, rows):
    c = Case(Q4_0, 128, 2, 64, [rows] * 2, [5000, 3333], seed=11)
    c.fill(*c.random_kv())
    q = _q(c, 4)
    tree = dev_words(words(trees(c.rng, c.counts, "tree"), -(-rows // 32), c.rows))
    for w in ("asked", None):
        for t, window, sinks in ((None, 3500, 100), (tree, 0, 0), (tree, 1000, 33)):
            runs = [run_seen(c, q, 4, 0.1, window, sinks, t, ws=w)[1] for _ in range(3)]
            assert all(np.array_equal(runs[0], r) for r in runs[1:])


@pytest.mark.parametrize("rows", [1, 33, 140])
def test_nan_stays_in_its_row(orc, rows):
    c = Case(Q4_0, 64, 2, 64, [rows, rows], [300, 290], seed=6)
    c.fill(*c.random_kv())
    q = _q(c, 2)
    tree = dev_words(words(trees(c.rng, c.counts, "tree"), -(-rows // 32), c.rows))
    bad = q.copy()
    bad[0, 1, 5], bad[rows, 0, 0] = 0x7FC0, 0x7F80
    keep = np.ones((c.rows, 4), bool)
    keep[0, 1] = keep[rows, 0] = False
    for t, window, sinks in ((None, 50, 4), (tree, 0, 0)):
        clean, got = (run_seen(c, x, 2, 0.125, window, sinks, t)[0] for x in (q, bad))
        assert np.isnan(got[0, 1]).all() and np.array_equal(got[keep], clean[keep])


def test_scores_far_apart(orc):
    """Scores of several hundred in both directions; a scale below zero, and none."""
    for counts in ([1, 1], [40, 9], [140, 30]):
        for scale in (3.0, -2.0, 0.0):
            c = Case(Q4_1, 64, 2, 64, counts, [700, 333], seed=5)
            _check(orc, c, 2, 200, 40, scale=scale)
            _check(orc, c, 2, 0, 0, trees(c.rng, counts, "tree"), scale=scale)


def test_offsets_past_32_bits(orc):
    """A pool of over 4 GiB whose last pages are in use."""
    d = wq.cache_desc("q4_0", 128, 8, 512, 8800)
    assert wq.wq_cache_size(d) > 1 << 32
    cache = torch.empty(wq.wq_cache_size(d), dtype=torch.uint8, device=DEV)
    for n in (1, 7, 64):
        c = Case(Q4_0, 128, 8, 512, [n], [900], seed=17, spare=0)
        c.desc, c.cache = d, cache
        c.d_table = torch.tensor([[8799, 8790, -1]], dtype=torch.int32, device=DEV)
        c.seqs = wq.seqs(1, n, c.d_len, c.d_table, c.d_start)
        _check(orc, c, 4, 100, 40)
        _check(orc, c, 4, 0, 0, trees(c.rng, [n], "tree"))


def test_rows_claimed_twice_stay_in_the_workspace(orc):
    """Starts that do not ascend: the outputs are not specified, but parts stay inside the workspace and masks are read
    inside their array."""
    c = Case(Q4_0, 64, 1, 64, [160, 0, 160], [6000, 0, 5900], seed=33, pad_rows=5)
    c.fill(*c.random_kv())
    c.d_start.copy_(torch.tensor([0, 160, 0, 160], dtype=torch.int32))
    s = wq.seqs(3, 165, c.d_len, c.d_table, row_start=c.d_start)
    tree = torch.full((165, 5), -1, dtype=torch.int32, device=DEV)
    q = torch.ones((165, 256), dtype=torch.bfloat16, device=DEV)
    for window, sinks in ((0, 0), (4500, 40)):
        need = wq.wq_attn_tree_workspace_size(c.desc, s, 4, window, sinks)
        assert need > 0
        ws = torch.full((need + 65536,), 0x5A, dtype=torch.uint8, device=DEV)
        y = torch.full((165, 256), 0x7BAD, dtype=torch.int16, device=DEV)
        wq.wq_attn_tree(c.desc, s, 4, q, 256, c.cache, 0.125, window, sinks, tree, 5, y, 256, ws, need)
        torch.cuda.synchronize()
        assert bool((ws[need:] == 0x5A).all()) and bool((y[160:] == 0x7BAD).all())


@pytest.mark.parametrize("counts,lens", [([1, 1], [9000, 900]), ([40, 3], [2600, 3]), ([150, 2], [2600, 900])],
                         ids=["token", "rows", "many rows"])
def test_graph_replays(orc, counts, lens):
    """Captured once, replayed with other lengths and other trees: every replay equals the eager call."""
    c = Case(Q4_0, 128, 1, 64, counts, lens, seed=30, one_row=max(counts) == 1)
    c.fill(*c.random_kv())
    hq = 2
    Q = dev_bf16(_q(c, hq).reshape(c.rows, -1))
    Y, Z = torch.empty_like(Q), torch.empty_like(Q)
    ld = -(-max(counts) // 32)
    tree = dev_words(words(trees(c.rng, counts, "tree"), ld, c.rows))
    n1 = wq.wq_attn_sinks_workspace_size(c.desc, c.seqs, hq, 4500, 70)
    n2 = wq.wq_attn_tree_workspace_size(c.desc, c.seqs, hq, 0, 0)
    ws = torch.full((max(n1, n2, 16),), 0xFF, dtype=torch.uint8, device=DEV)

    def step():
        wq.wq_attn_sinks(c.desc, c.seqs, hq, Q, hq * 128, c.cache, 0.1, 4500, 70, Y, hq * 128, ws, n1)
        wq.wq_attn_tree(c.desc, c.seqs, hq, Q, hq * 128, c.cache, 0.1, 0, 0, tree, ld, Z, hq * 128, ws, n2)

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for i, cut in enumerate((0, 1, 700, 32, 0)):
        c.d_len.copy_(torch.tensor([max(t - cut, 0) for t in lens], dtype=torch.int32))
        tree.copy_(dev_words(words(trees(c.rng, counts, "any" if i % 2 else "tree"), ld, c.rows)))
        Y.fill_(0x7FC0)
        Z.fill_(0x7FC0)
        g.replay()
        torch.cuda.synchronize()
        got = Y.clone(), Z.clone()
        ws.fill_(0xFF)
        Y.fill_(0x7FC0)
        Z.fill_(0x7FC0)
        step()
        torch.cuda.synchronize()
        assert torch.equal(got[0], Y) and torch.equal(got[1], Z), f"lengths cut by {cut}"


def test_calls_on_two_streams(orc):
    c = Case(Q4_1, 64, 4, 64, [5, 9, 2], [5000, 77, 2500], seed=31)
    c.fill(*c.random_kv())
    qs = [_q(c, 2) for _ in range(2)]
    masks = [dev_words(words(trees(c.rng, c.counts, "tree"), 1, c.rows)) for _ in range(2)]
    want = [run_seen(c, q, 2, 0.125, 0, 0, m)[1] for q, m in zip(qs, masks)]
    n = wq.wq_attn_tree_workspace_size(c.desc, c.seqs, 8, 0, 0)
    Q = [dev_bf16(q.reshape(c.rows, -1)) for q in qs]
    Y = [torch.zeros_like(x) for x in Q]
    W = [torch.empty(max(n, 16), dtype=torch.uint8, device=DEV) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for i in range(2):
            wq.wq_attn_tree(c.desc, c.seqs, 8, Q[i], 512, c.cache, 0.125, 0, 0, masks[i], 1, Y[i], 512, W[i], n, stream=streams[i])
    torch.cuda.synchronize()
    for i in range(2):
        assert np.array_equal(Y[i].cpu().numpy().view(np.uint16).reshape(want[i].shape), want[i])


def test_one_row_each_without_starts(orc):
    """A draft of one token per sequence, without row starts and in pages without a table; lengths below zero and past the
    last page."""
    for fmt, dim, group in ((Q4_0, 64, 2), (Q4_1, 128, 20)):
        c = Case(fmt, dim, 2, 64, [1] * 5, [0, 1, 64, 40, 17], seed=12, one_row=True, paged=False)
        _check(orc, c, group, 0, 0, trees(c.rng, c.counts, "tree"))
        _check(orc, c, group, 10, 3, trees(c.rng, c.counts, "any"))
        _check(orc, c, group, 7, 5)
    c = Case(Q4_0, 64, 2, 64, [1, 7, 1], [100, 90, 30], seed=13)
    c.fill(*c.random_kv())
    q = _q(c, 2)
    tree = dev_words(words(trees(c.rng, c.counts, "chain"), 1, c.rows))
    want = run_seen(c, q, 2, 0.1, 0, 0, tree)[1]
    c.d_len.copy_(torch.tensor([100, -3, 30], dtype=torch.int32))
    for t, window, sinks in ((tree, 0, 0), (tree, 9, 3), (None, 9, 3)):
        got = run_seen(c, q, 2, 0.1, window, sinks, t)[1]
        assert not got[1:8].any()
        if not window:
            assert np.array_equal(got[0], want[0]) and np.array_equal(got[8], want[8])
    c.d_len.copy_(torch.tensor([100000, 90, 2**31 - 1], dtype=torch.int32))
    for t, window, sinks in ((tree, 0, 0), (None, 9, 3)):
        got = run_seen(c, q, 2, 0.1, window, sinks, t)[0]
        assert np.isfinite(got[1:8]).all()                            # (others' pages hold anything past their lengths)


def test_every_width_of_tile(orc):
    """Calls of the sizes at which tiles of 16, 32, 128 and 256 columns are taken, whole and shared out, with and without a
    workspace."""
    for dim, heads, batch, rows, length in ((128, 8, 40, 12, 70), (128, 20, 10, 32, 90), (64, 20, 12, 128, 140), (96, 16, 30, 9, 100),
                                            (256, 4, 6, 45, 120), (128, 1, 2, 20, 5000), (64, 1, 1, 60, 4300), (96, 1, 1, 130, 4400)):
        say("width", dim, heads, batch, rows, length)
        c = Case(Q4_0 if rows % 2 else Q4_1, dim, heads, 64, [max(1, rows - i % 3) for i in range(batch)], [length - i for i in range(batch)], seed=rows)
        masks = trees(c.rng, c.counts, "tree")
        _check(orc, c, 4 if dim * rows < 8000 else 2, 0, 0, masks)
        _check(orc, c, 3, 60, 5, masks)
