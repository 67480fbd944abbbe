"""wq_attn over the 4-bit cache against float64 attention over the values the cache stands for (the oracle's quantizers):
head sizes, groups, lengths from none to long, windows, rows that see nothing, pages that end anywhere or are bad, junk
behind the last token, strides, streams, graphs, and a decoder layer's run of calls."""
import numpy as np
import pytest
import torch

from block_quantized_bit_amd import policy, wq
from block_quantized_bit_amd.inputs import bf16_bits_to_f32, f32_to_bf16_bits

from cache_helpers import Q4_0, Q4_1, Case, attend, check_attn, run_attn
from gpu_helpers import DEV, dev_bf16, gpu_quantize, require_gpu, say

pytestmark = pytest.mark.gpu

FMT = [Q4_0, Q4_1]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def _q(c, group, std=1.0):
    return f32_to_bf16_bits(c.rng.standard_normal((c.rows, c.heads * group, c.dim), dtype=np.float32) * std)


def _check(orc, c, group, causal, window, *, scale=None, kv=None, q=None, pad=0, ws=("asked", None), what=""):
    k, v = kv or c.random_kv()
    c.fill(k, v)
    q = _q(c, group) if q is None else q
    scale = c.dim ** -0.5 if scale is None else scale
    ref, ab, A = attend(c, orc, k, v, bf16_bits_to_f32(q), group, scale, causal, window)
    ys = []
    for w in ws:
        y, bits = run_attn(c, q, group, scale, causal, window, ws=w, pad=pad)
        n = int(c.start[-1])
        check_attn(y[:n], ref[:n], ab[:n], A[:n], f"{what} ws={w}")
        assert np.all(bits[n:] == 0x7BAD), "rows behind the last sequence were written"
        ys.append(bits)
    return ys


# dim, heads, group, page, rows, tokens, causal, window
TOKEN = [
    (64, 20, 1, 448, [1], [224], 1, 0),
    (64, 20, 1, 448, [1], [1], 1, 0),
    (64, 4, 1, 1504, [1] * 3, [1500, 1499, 31], 0, 0),
    (64, 2, 16, 32, [1] * 5, [0, 1, 32, 33, 200], 1, 0),
    (96, 3, 5, 96, [1] * 4, [95, 96, 97, 700], 1, 0),
    (128, 8, 4, 64, [1] * 6, [1, 15, 16, 17, 64, 1000], 1, 0),
    (128, 1, 40, 64, [1] * 2, [333, 65], 1, 0),            # more query heads than one tile of columns has
    (128, 2, 8, 32, [1] * 3, [2000, 100, 31], 1, 128),
    (256, 2, 8, 64, [1] * 3, [513, 64, 2], 1, 0),
    (256, 1, 3, 128, [1] * 2, [700, 129], 1, 33),
]
ROWS = [
    (64, 4, 1, 448, [5, 1, 0, 17], [100, 1, 50, 17], 1, 0),
    (64, 2, 3, 64, [3, 9, 4], [2, 5, 4], 1, 0),            # rows whose token would be negative see nothing
    (96, 2, 2, 96, [40, 150], [40, 400], 1, 0),
    (128, 2, 4, 64, [5] * 4, [300, 5, 64, 129], 1, 0),
    (128, 2, 4, 64, [5] * 4, [300, 5, 64, 129], 1, 50),
    (128, 1, 1, 32, [257], [257], 1, 0),
    (128, 2, 1, 64, [300, 2], [500, 64], 1, 100),
    (128, 1, 5, 64, [70, 70], [70, 200], 0, 0),            # not causal: all rows see all tokens
    (64, 3, 2, 64, [33], [31], 0, 0),                      # more rows than tokens
    (256, 1, 4, 64, [65, 3], [600, 3], 1, 0),
    (256, 2, 2, 32, [90], [123], 1, 40),
    (128, 1, 150, 64, [3], [90], 1, 0),                    # one head's group is wider than any tile
    (128, 1, 300, 64, [2], [70], 1, 0),
    # more than 128 columns per sequence
    (64, 4, 4, 448, [41, 90, 0, 33], [100, 90, 50, 470], 1, 0),
    (64, 2, 3, 64, [130, 9, 44], [77, 5, 300], 1, 0),      # rows whose token would be negative see nothing
    (96, 2, 3, 96, [40, 150], [40, 400], 1, 0),
    (96, 3, 2, 32, [140, 77], [333, 77], 1, 64),
    (128, 2, 4, 64, [64, 33, 64], [300, 64, 129], 1, 50),
    (128, 1, 2, 32, [257], [257], 1, 0),
    (128, 1, 5, 64, [70, 70], [70, 200], 0, 0),
    (64, 1, 140, 64, [2, 1], [31, 900], 0, 0),
    (256, 1, 4, 64, [65, 30], [600, 33], 1, 0),
    (256, 2, 2, 32, [90, 80], [123, 80], 1, 40),
    (64, 30, 1, 64, [1500, 100], [1500, 164], 1, 300),     # enough tiles for 256 columns each
    (128, 20, 2, 96, [800, 333], [850, 333], 1, 0),
    (96, 24, 2, 128, [700], [701], 0, 0),
]


@pytest.mark.parametrize("fmt", FMT, ids=["q4_0", "q4_1"])
@pytest.mark.parametrize("i", range(len(TOKEN)))
def test_single_tokens(orc, fmt, i):
    dim, heads, group, page, counts, lens, causal, window = TOKEN[i]
    say("attn token", fmt, TOKEN[i])
    c = Case(fmt, dim, heads, page, counts, lens, seed=i, one_row=True, pad_rows=i % 3)
    _check(orc, c, group, causal, window, pad=8 * (i % 2), what=str(TOKEN[i]))


@pytest.mark.parametrize("fmt", FMT, ids=["q4_0", "q4_1"])
@pytest.mark.parametrize("i", range(len(ROWS)))
def test_rows(orc, fmt, i):
    dim, heads, group, page, counts, lens, causal, window = ROWS[i]
    say("attn rows", fmt, ROWS[i])
    c = Case(fmt, dim, heads, page, counts, lens, seed=50 + i, pad_rows=i % 3)
    _check(orc, c, group, causal, window, pad=8 * (i % 2), what=str(ROWS[i]))


@pytest.mark.parametrize("fmt,dim", [(Q4_0, 128), (Q4_1, 64)])
def test_long_sequences_shared_out(orc, fmt, dim):
    """Few rows over long sequences of very unequal length: the call is split over workgroups (with a workspace)."""
    c = Case(fmt, dim, 2, 256, [1, 1, 1, 1], [20011, 1, 0, 5003], seed=7, one_row=True)
    a, b = _check(orc, c, 4, 1, 0, what="long")
    c2 = Case(fmt, dim, 1, 64, [2, 3], [9001, 130], seed=8)
    _check(orc, c2, 8, 1, 0, what="long, several rows")
    _check(orc, Case(fmt, dim, 1, 64, [40], [6001], seed=9), 2, 1, 0, what="long, many rows")
    _check(orc, Case(fmt, dim, 1, 64, [40], [6001], seed=10), 2, 1, 1000, what="long, many rows, window")
    _check(orc, Case(fmt, dim, 1, 64, [100], [3001], seed=19), 2, 1, 0, what="long, more rows")
    _check(orc, Case(fmt, dim, 1, 64, [100, 1, 90], [2001, 40, 90], seed=20), 3, 1, 500, what="long, more rows, window")


@pytest.mark.parametrize("fmt", FMT, ids=["q4_0", "q4_1"])
@pytest.mark.parametrize("dim", [64, 96, 128, 256])
def test_one_long_sequence_among_many(orc, fmt, dim):
    """Tiles of one, a few and many parts in one call."""
    lens = [20011, 5003, 1, 0, 2999, 1300] + [7 * i % 331 for i in range(64)]
    say("one long", fmt, dim)
    c = Case(fmt, dim, 1, 256, [1] * len(lens), lens, seed=21, one_row=True, pad_rows=1)
    _check(orc, c, 5, 1, 0, what="one long")
    c = Case(fmt, dim, 1, 256, [2, 1, 1, 0, 3, 1] + [1] * 64, lens, seed=22)
    _check(orc, c, 3, 1, 2500, what="one long, window")


@pytest.mark.parametrize("fmt", FMT, ids=["q4_0", "q4_1"])
@pytest.mark.parametrize("dim", [64, 96, 128, 256])
def test_more_tiles_than_compute_units(orc, fmt, dim):
    lens = [37 * i % 401 for i in range(150)]
    say("many tiles", fmt, dim)
    c = Case(fmt, dim, 2, 96, [1] * len(lens), lens, seed=23, one_row=True, pad_rows=2)
    _check(orc, c, 3, 1, 0, ws=("asked",), what="many tiles")


@pytest.mark.parametrize("fmt", FMT, ids=["q4_0", "q4_1"])
@pytest.mark.parametrize("dim", [64, 96, 128, 256])
def test_many_rows_split(orc, fmt, dim):
    """Tiles of 128 columns whose tokens are shared out: the last part ends anywhere in a unit."""
    for tokens in (3001, 2990):
        say("rows split", fmt, dim, tokens)
        c = Case(fmt, dim, 1, 64, [70, 3], [tokens, 50], seed=24)
        assert wq.wq_attn_workspace_size(c.desc, c.seqs, 4) > 0
        _check(orc, c, 4, 1, 0, ws=("asked",), what="rows split")


def test_results_do_not_change(orc):
    """The same call gives the same bits, with any workspace content, and neighbours in the batch do not matter to
    rows of a call without a workspace."""
    c = Case(Q4_0, 128, 2, 64, [1] * 5, [3000, 40, 1, 777, 64], seed=11, one_row=True)
    k, v = c.random_kv()
    c.fill(k, v)
    q = _q(c, 4)
    for w in ("asked", None):
        runs = [run_attn(c, q, 4, 0.1, 1, 0, ws=w)[1] for _ in range(3)]
        assert all(np.array_equal(runs[0], r) for r in runs[1:])
    Q = dev_bf16(q.reshape(5, -1))
    for b in range(5):
        y = torch.empty((1, 8 * 128), dtype=torch.int16, device=DEV)
        s = wq.seqs(1, 1, c.d_len[b:b + 1], c.d_table[b:b + 1])
        wq.wq_attn(c.desc, s, 8, Q[b:b + 1], 1024, c.cache, 0.1, 1, 0, y, 1024)
        torch.cuda.synchronize()
        assert np.array_equal(y.cpu().numpy().view(np.uint16).reshape(8, 128), runs[0][b])


@pytest.mark.parametrize("counts", [[1, 1, 1], [33, 1, 8], [200, 32, 60]], ids=["token", "rows", "many"])
def test_bad_pages_are_absent(orc, counts):
    c = Case(Q4_1, 64, 2, 32, counts, [200, 32, 70], bad=[(0, 0), (0, 3), (1, 0), (2, 2)], seed=4, one_row=max(counts) == 1)
    _check(orc, c, 2, 1, 0)
    c = Case(Q4_0, 128, 1, 32, counts, [200, 32, 70], bad=[(0, 6), (1, 0), (2, 1)], seed=5, one_row=max(counts) == 1)
    _check(orc, c, 2, 0, 0)


@pytest.mark.parametrize("rows", [1, 40, 140])
def test_scores_far_apart(orc, rows):
    """Scores of several hundred in both directions, a first token that outweighs all others, a scale below zero, none."""
    for seed, scale in ((1, 0.5), (2, -0.3), (3, 0.0), (4, 0.09)):
        c = Case(Q4_0, 64, 1, 64, [rows], [700], seed=seed)
        k, v = c.random_kv(std=4.0)
        k[0][0] = f32_to_bf16_bits(np.full((1, 64), 8.0, np.float32))
        q = _q(c, 1, std=2.0)
        q[: rows // 2 + 1] = f32_to_bf16_bits(np.full((1, 1, 64), 2.5, np.float32))
        _check(orc, c, 1, 1, 0, scale=scale, kv=(k, v), q=q)


@pytest.mark.parametrize("rows", [1, 40, 140])
def test_small_and_large_values(orc, rows):
    """Values near the smallest a scale can hold, at the limit, and both in one head; queries of any magnitude."""
    for seed, (ks, vs, qs, scale) in enumerate([(1e-4, 1e-4, 1e4, 1.0), (1.0, 1e4, 1.0, 0.1), (2e4, 2e4, 1e-6, 1.0), (1.0, 1e-6, 1e20, 1e-20)]):
        c = Case(Q4_1 if seed % 2 else Q4_0, 64, 1, 64, [rows], [300], seed=20 + seed)
        k, v = c.random_kv()
        k = [f32_to_bf16_bits(bf16_bits_to_f32(x) * np.float32(ks)) for x in k]
        v = [f32_to_bf16_bits(bf16_bits_to_f32(x) * np.float32(vs) * np.where(np.arange(64) < 32, 1e-3, 1).astype(np.float32)) for x in v]
        _check(orc, c, 1, 1, 0, scale=scale, kv=(k, v), q=_q(c, 1, std=qs))


@pytest.mark.parametrize("rows", [1, 40, 80])
def test_nan_stays_in_its_row(orc, rows):
    """A query with a NaN or an infinity makes its own row and head NaN at most."""
    c = Case(Q4_0, 64, 2, 64, [rows, rows], [300, 90], seed=6)
    k, v = c.random_kv()
    c.fill(k, v)
    q = _q(c, 2)
    clean, _ = run_attn(c, q, 2, 0.125, 1, 0)
    bad = q.copy()
    bad[0, 1, 5], bad[rows, 0, 0] = 0x7FC0, 0x7F80
    got, _ = run_attn(c, bad, 2, 0.125, 1, 0)
    assert np.isnan(got[0, 1]).all()
    keep = np.ones(got.shape[:2], bool)
    keep[0, 1] = keep[rows, 0] = False
    assert np.array_equal(got[keep], clean[keep])


def test_rows_claimed_twice_stay_in_the_workspace(orc):
    """Starts that do not ascend, so that two sequences claim the same rows: the outputs are not specified, but the parts
    of a split call stay inside the workspace and the rows that no sequence has are left as they were."""
    c = Case(Q4_0, 64, 1, 64, [160, 0, 160], [2000, 0, 1900], seed=33, pad_rows=5)
    c.fill(*c.random_kv())
    c.d_start.copy_(torch.tensor([0, 160, 0, 160], dtype=torch.int32))
    s = wq.seqs(3, 165, c.d_len, c.d_table, row_start=c.d_start)
    need = wq.wq_attn_workspace_size(c.desc, s, 4)
    assert need > 0
    ws = torch.full((need + 65536,), 0x5A, dtype=torch.uint8, device=DEV)
    q = torch.ones((165, 256), dtype=torch.bfloat16, device=DEV)
    y = torch.full((165, 256), 0x7BAD, dtype=torch.int16, device=DEV)
    wq.wq_attn(c.desc, s, 4, q, 256, c.cache, 0.125, 1, 0, y, 256, ws, need)
    torch.cuda.synchronize()
    assert bool((ws[need:] == 0x5A).all()) and bool((y[160:] == 0x7BAD).all())


def test_shared_pages(orc):
    """Two sequences that share their first pages read the same keys and values."""
    c = Case(Q4_0, 128, 2, 32, [1, 1], [96, 96], seed=12, one_row=True)
    k, v = c.random_kv()
    c.fill(k, v)
    t = c.table.copy()
    t[1] = t[0]
    s = wq.seqs(2, 2, c.d_len, torch.from_numpy(t).to(DEV))
    q = _q(c, 2)
    q[1] = q[0]
    Q = dev_bf16(q.reshape(2, -1))
    y = torch.empty((2, 512), dtype=torch.int16, device=DEV)
    wq.wq_attn(c.desc, s, 4, Q, 512, c.cache, 0.1, 1, 0, y, 512)
    torch.cuda.synchronize()
    assert torch.equal(y[0], y[1])


def test_without_a_table(orc):
    for counts in ([1, 1, 1], [60, 1, 30]):
        c = Case(Q4_1, 64, 3, 224, counts, [200, 7, 224], paged=False, seed=13)
        _check(orc, c, 2, 1, 0)


def test_many_sequences(orc):
    """Hundreds of sequences, many short, some empty, some without rows."""
    rng = np.random.default_rng(3)
    counts = [int(n) for n in rng.choice([0, 1, 1, 1, 2, 7], 300)]
    lens = [int(n) for n in rng.integers(0, 70, 300)]
    _check(orc, Case(Q4_0, 64, 1, 32, counts, lens, seed=14), 2, 1, 0, what="mixed")
    _check(orc, Case(Q4_0, 64, 1, 32, [1] * 300, lens, seed=15, one_row=True), 2, 1, 0, what="one row")


def test_lengths_past_the_last_page(orc):
    """A length larger than the table holds: the tokens that are there are attended to; negative lengths: zeros."""
    c = Case(Q4_0, 64, 1, 32, [1, 1, 1], [64, 64, 64], seed=16, one_row=True)
    k, v = c.random_kv()
    c.fill(k, v)
    q = _q(c, 1)
    want, _ = run_attn(c, q, 1, 0.125, 0, 0)
    c.table[:, 2:] = -1
    t = torch.from_numpy(np.ascontiguousarray(c.table[:, :2])).to(DEV)
    c.seqs = wq.seqs(3, 3, torch.tensor([64, 2**31 - 1, -4], dtype=torch.int32, device=DEV), t)
    got, _ = run_attn(c, q, 1, 0.125, 0, 0)
    assert np.array_equal(got[:2], want[:2]) and not got[2].any()
    got, _ = run_attn(c, q, 1, 0.125, 1, 0)
    assert np.array_equal(got[:2], want[:2]) and not got[2].any()


def test_offsets_past_32_bits(orc):
    """A pool of over 4 GiB whose last pages are in use, in both kernels' reach."""
    d = wq.cache_desc("q4_0", 128, 8, 512, 8800)
    assert wq.wq_cache_size(d) > 1 << 32
    cache = torch.empty(wq.wq_cache_size(d), dtype=torch.uint8, device=DEV)
    c = Case(Q4_0, 128, 8, 512, [1], [900], seed=17, spare=0)
    k, v = c.random_kv()
    c.desc, c.cache = d, cache
    c.d_table = torch.tensor([[8799, 8790, -1]], dtype=torch.int32, device=DEV)
    c.seqs = wq.seqs(1, 1, c.d_len, c.d_table, c.d_start)
    _check(orc, c, 4, 1, 0, kv=(k, v))
    c.counts, c.rows, c.start = [64], 64, np.array([0, 64], np.int32)
    c.d_start = torch.from_numpy(c.start).to(DEV)
    c.seqs = wq.seqs(1, 64, c.d_len, c.d_table, c.d_start)
    _check(orc, c, 4, 1, 0, kv=(k, v))


def test_another_stream_and_graph_replays(orc):
    """One token a step: the new row is written and attended to, captured once and replayed with other lengths, rows and
    eager work in between; every replay equals the eager call on its own state."""
    dim, heads, group, page, start = 128, 2, 4, 32, [300, 31, 64]
    c = Case(Q4_1, dim, heads, page, [1] * 3, [n + 8 for n in start], seed=18, one_row=True)
    k, v = c.random_kv()
    full = list(c.lens)
    c.lens = start
    lens = torch.tensor(start, dtype=torch.int32, device=DEV)
    s = wq.seqs(3, 3, lens, c.d_table)
    # the tokens before the first step
    first = Case.fill
    c.d_len = lens
    first(c, [x[:n] for x, n in zip(k, start)], [x[:n] for x, n in zip(v, start)])
    w = heads * dim
    K, V = (torch.zeros((3, w), dtype=torch.int16, device=DEV) for _ in range(2))
    Q = torch.zeros((3, w * group), dtype=torch.int16, device=DEV)
    Y = torch.zeros_like(Q)
    n = wq.wq_attn_workspace_size(c.desc, s, heads * group)
    ws = torch.empty(n, dtype=torch.uint8, device=DEV) if n else None

    def step():
        wq.wq_cache_write(c.desc, s, K, w, V, w, wq.WQ_BF16, c.cache)
        wq.wq_attn(c.desc, s, heads * group, Q, w * group, c.cache, dim ** -0.5, 1, 0, Y, w * group, ws, n)

    def load(i):
        lens.copy_(torch.tensor([m + i + 1 for m in start], dtype=torch.int32))
        for dst, src in ((K, k), (V, v)):
            dst.copy_(dev_bf16(np.stack([x[m + i].reshape(-1) for x, m in zip(src, start)])))
        q = f32_to_bf16_bits(np.random.default_rng(i).standard_normal((3, heads * group, dim), dtype=np.float32))
        Q.copy_(dev_bf16(q.reshape(3, -1)))
        return q

    load(0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for i in range(8):
        q = load(i)
        Y.fill_(0x7FC0)
        g.replay()
        torch.cuda.synchronize()
        got = Y.cpu().numpy().view(np.uint16).copy()
        Y.fill_(0x7FC0)
        step()
        torch.cuda.synchronize()
        assert np.array_equal(got, Y.cpu().numpy().view(np.uint16)), f"replay {i} differs from the eager call"
        c.lens = [m + i + 1 for m in start]
        ref, ab, A = attend(c, orc, [x[:m] for x, m in zip(k, c.lens)], [x[:m] for x, m in zip(v, c.lens)], bf16_bits_to_f32(q),
                            group, dim ** -0.5, 1, 0)
        check_attn(bf16_bits_to_f32(got).reshape(ref.shape), ref, ab, A, f"step {i}")
    assert c.lens == full


@pytest.mark.parametrize("counts,lens", [([1, 1], [3000, 900]), ([40, 3], [2600, 3]), ([150, 2], [2600, 900])],
                         ids=["shared out", "rows", "many rows"])
def test_graph_replays_of_split_calls(orc, counts, lens):
    """Calls that take a workspace and a second launch, captured and replayed with other lengths and a workspace that holds
    the last replay's parts: every replay equals the eager call."""
    c = Case(Q4_0, 128, 1, 64, counts, lens, seed=30, one_row=max(counts) == 1)
    k, v = c.random_kv()
    c.fill(k, v)
    hq = 2
    q = _q(c, hq)
    Q = dev_bf16(q.reshape(c.rows, -1))
    Y = torch.empty_like(Q)
    n = wq.wq_attn_workspace_size(c.desc, c.seqs, hq)
    assert n > 0
    ws = torch.full((n,), 0xFF, dtype=torch.uint8, device=DEV)          # NaN in every float

    def step():
        wq.wq_attn(c.desc, c.seqs, hq, Q, hq * 128, c.cache, 0.1, 1, 0, Y, hq * 128, ws, n)

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for cut in (0, 1, 700, 32, 0):
        c.d_len.copy_(torch.tensor([max(t - cut, 0) for t in lens], dtype=torch.int32))
        Y.fill_(0x7FC0)
        g.replay()
        torch.cuda.synchronize()
        got = Y.clone()
        ws.fill_(0xFF)
        Y.fill_(0x7FC0)
        step()
        torch.cuda.synchronize()
        assert torch.equal(got, Y), f"lengths cut by {cut}"
    c.lens = lens
    ref, ab, A = attend(c, orc, k, v, bf16_bits_to_f32(q), hq, 0.1, 1, 0)
    check_attn(bf16_bits_to_f32(Y.cpu().numpy().view(np.uint16)).reshape(ref.shape), ref, ab, A, "last replay")


def test_calls_on_two_streams(orc):
    """Two calls at the same time on two streams, each with its workspace, on one cache."""
    c = Case(Q4_1, 64, 4, 64, [1, 1, 1], [5000, 77, 2500], seed=31, one_row=True)
    k, v = c.random_kv()
    c.fill(k, v)
    qs = [_q(c, 2) for _ in range(2)]
    want = [run_attn(c, q, 2, 0.125, 1, 0)[1] for q in qs]
    n = wq.wq_attn_workspace_size(c.desc, c.seqs, 8)
    assert n > 0
    Q = [dev_bf16(q.reshape(3, -1)) for q in qs]
    Y = [torch.zeros_like(x) for x in Q]
    W = [torch.empty(n, dtype=torch.uint8, device=DEV) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for i in range(2):
            wq.wq_attn(c.desc, c.seqs, 8, Q[i], 512, c.cache, 0.125, 1, 0, Y[i], 512, W[i], n, stream=streams[i])
    torch.cuda.synchronize()
    for i in range(2):
        assert np.array_equal(Y[i].cpu().numpy().view(np.uint16).reshape(want[i].shape), want[i])


@pytest.mark.parametrize("fmt", ["q4_0", "q4_1"])
def test_a_decoder_layer(orc, fmt):
    """The fused projection's K and V rows into the cache, attention over it, the output projection: a prompt of 5 tokens,
    then tokens one by one, the whole run against the same run in float64 over the same quantized rows."""
    heads, dim, dm = 20, 64, 1280
    rng = np.random.default_rng(0)
    wqkv = (rng.standard_normal((3 * dm, dm), dtype=np.float32) * 0.03).astype(np.float32)
    wo = (rng.standard_normal((dm, dm), dtype=np.float32) * 0.03).astype(np.float32)
    dq, cq, sq = gpu_quantize(wq.WQ_Q4_0, wqkv)
    do, co, so = gpu_quantize(wq.WQ_Q4_0, wo)
    wo_hat = orc.quantize(wq.WQ_Q4_0, wo)["w_hat"]
    c = Case(Q4_0 if fmt == "q4_0" else Q4_1, dim, heads, 448, [1], [12], paged=False, seed=1)
    planned = policy.decoder_caches(fmt, 1)[0].desc
    assert bytes(planned) == bytes(c.desc)                       # the model's own self-attention cache
    lens = torch.zeros(1, dtype=torch.int32, device=DEV)
    keys, values = [], []
    for first, n in [(0, 5)] + [(i, 1) for i in range(5, 12)]:
        x = f32_to_bf16_bits(rng.standard_normal((n, dm), dtype=np.float32))
        out = torch.empty((3, n, dm), dtype=torch.int16, device=DEV)
        ws = wq.wq_workspace_size(dq, n)
        W = torch.empty(ws, dtype=torch.uint8, device=DEV) if ws else None
        wq.wq_matmul_qkv(dq, n, dev_bf16(x), dm, cq, sq, None, [dm] * 3, [out[0], out[1], out[2]], [dm] * 3, wq.WQ_BF16, W, ws)
        lens.fill_(first + n)
        s = wq.seqs(1, n, lens, row_start=torch.tensor([0, n], dtype=torch.int32, device=DEV))
        wq.wq_cache_write(c.desc, s, out[1], dm, out[2], dm, wq.WQ_BF16, c.cache)
        y = torch.empty((n, dm), dtype=torch.int16, device=DEV)
        wq.wq_attn(c.desc, s, heads, out[0], dm, c.cache, dim ** -0.5, 1, 0, y, dm)
        z = torch.empty((n, dm), dtype=torch.float32, device=DEV)
        wq.wq_matmul(do, n, y, dm, co, so, None, z, wq.WQ_F32, dm)
        torch.cuda.synchronize()
        qkv = out.cpu().numpy().view(np.uint16)
        keys.append(qkv[1].reshape(n, heads, dim))
        values.append(qkv[2].reshape(n, heads, dim))
        c.counts, c.lens, c.start, c.rows = [n], [first + n], np.array([0, n], np.int32), n
        ref, ab, A = attend(c, orc, [np.concatenate(keys)], [np.concatenate(values)], bf16_bits_to_f32(qkv[0]).reshape(n, heads, dim),
                            1, dim ** -0.5, 1, 0)
        yb = y.cpu().numpy().view(np.uint16)
        yf = bf16_bits_to_f32(yb)
        check_attn(yf.reshape(ref.shape), ref, ab, A, f"token {first}")
        want = yf.astype(np.float64) @ wo_hat.astype(np.float64).T
        bound = 4e-3 * (np.abs(yf.astype(np.float64)) @ np.abs(wo_hat.astype(np.float64)).T) + 1e-6
        assert np.all(np.abs(z.cpu().numpy() - want) <= bound)


@pytest.mark.parametrize("rows", [1, 5, 140])
def test_queries_and_outputs_side_by_side(orc, rows):
    """Q and Y as the columns of one buffer share no byte: the call is taken, and gives what separate buffers give."""
    c = Case(Q4_0, 64, 2, 64, [rows], [200], seed=40)
    c.fill(*c.random_kv())
    q = _q(c, 2)
    want = run_attn(c, q, 2, 0.125, 1, 0, ws=None)[1]
    both = torch.zeros((rows, 2 * 256 + 8), dtype=torch.int16, device=DEV)
    both[:, :256] = dev_bf16(q.reshape(rows, -1))
    wq.wq_attn(c.desc, c.seqs, 4, both, both.shape[1], c.cache, 0.125, 1, 0, both[:, 256:], both.shape[1])
    torch.cuda.synchronize()
    assert np.array_equal(both[:, 256:512].cpu().numpy().view(np.uint16).reshape(want.shape), want)
    assert not both[:, 512:].any()
