"""Sinks, trees, pages and kept rows without a GPU: every refusal returns before anything is enqueued, and a call with nothing to
do is no launch."""
import numpy as np
import pytest

from block_quantized_bit_amd import wq

from test_cache_host import BAD_DESCS, BAD_SEQS, FAKE, _desc, _seqs, _status, _Tensor

I31 = 2**31 - 1


def _sinks(**kw):
    f = dict(d=_desc(), s=_seqs(), hq=32, q=FAKE, ldq=4096, cache=FAKE, scale=0.1, window=100, sinks=4, y=2 * FAKE, ldy=4096, ws=None, wsb=0)
    f.update(kw)
    return _status(wq.wq_attn_sinks, *f.values(), 0)


def _tree(**kw):
    f = dict(d=_desc(), s=_seqs(), hq=32, q=FAKE, ldq=4096, cache=FAKE, scale=0.1, window=0, sinks=0, tree=FAKE, ld=1, y=2 * FAKE,
             ldy=4096, ws=None, wsb=0)
    f.update(kw)
    return _status(wq.wq_attn_tree, *f.values(), 0)


def _pages(**kw):
    f = dict(d=_desc(), batch=4, len=FAKE, want=2 * FAKE, table=FAKE, ld=10, pool=FAKE, rows=9, start=FAKE, pos=FAKE, slot=FAKE)
    f.update(kw)
    return _status(wq.wq_pages_assign, *f.values(), 0)


def _keep(**kw):
    f = dict(d=_desc(), s=_seqs(), path=FAKE, ld=4, count=FAKE, caches=[FAKE, 2 * FAKE], want=2 * FAKE)
    f.update(kw)
    return _status(wq.wq_cache_keep, *f.values(), 0)


@pytest.mark.parametrize("change,want", BAD_DESCS, ids=str)
def test_descriptor_refusals(change, want):
    d = _desc(**change)
    assert _sinks(d=d) == want and _tree(d=d) == want and _pages(d=d) == want and _keep(d=d) == want
    assert _status(wq.wq_attn_sinks_workspace_size, d, _seqs(), 32, 10, 0) == want
    assert _status(wq.wq_attn_tree_workspace_size, d, _seqs(), 32, 0, 0) == want


@pytest.mark.parametrize("change,want", BAD_SEQS, ids=str)
def test_sequence_refusals(change, want):
    s = _seqs(**change)
    assert _sinks(s=s) == want and _tree(s=s) == want and _keep(s=s) == want


@pytest.mark.parametrize("at", [_sinks, _tree], ids=["sinks", "tree"])
def test_attention_refusals(at):
    assert at(hq=0) == 3 and at(hq=12) == 3 and at(hq=65536) == 3
    assert at(q=None) == 1 and at(y=None) == 1 and at(cache=None) == 1
    assert at(q=FAKE + 2) == 4 and at(y=FAKE + 8) == 4 and at(cache=FAKE + 8) == 4
    assert at(ldq=4088) == 1 and at(ldy=4100) == 1 and at(ldq=1 << 31) == 1
    assert at(scale=float("nan")) == 1 and at(scale=float("inf")) == 1 and at(scale=-3e38) == 1
    assert at(window=-1) == 1 and at(sinks=-1, window=5) == 1
    assert at(ws=FAKE + 8, wsb=1 << 40) == 4
    assert at(y=FAKE) == 1 and at(y=FAKE + 16) == 1                   # shares bytes with q
    assert at(s=_seqs(rows=I31, row_start=FAKE)) == 3


def test_what_a_row_sees():
    assert _sinks(window=0) == 1
    assert _tree(tree=None) == 1 and _tree(tree=FAKE + 2) == 4
    assert _tree(ld=0) == 1 and _tree(ld=-1) == 1 and _tree(ld=65537) == 1
    assert _tree(sinks=4) == 1                                        # first tokens are seen anyway without a window
    d, s = _desc(), _seqs()
    size = lambda f, w, k: _status(f, d, s, 32, w, k)  # noqa: E731
    for f, bad, good in ((wq.wq_attn_sinks_workspace_size, ((0, 4), (-1, 0), (5, -1)), ((1, 0), (I31, I31))),
                         (wq.wq_attn_tree_workspace_size, ((0, 4), (-1, 0), (5, -1)), ((0, 0), (1, 0), (I31, I31)))):
        assert all(size(f, *x) == 1 for x in bad) and all(size(f, *x) == 0 for x in good)


def test_page_refusals():
    assert _pages(batch=-1) == 3 and _pages(batch=(1 << 20) + 1) == 3 and _pages(rows=-1) == 3
    for name in ("len", "want", "table", "pool", "start"):
        assert _pages(**{name: None}) == 1, name
        assert _pages(**{name: 3 * FAKE + 2}) == 4, name
    assert _pages(pos=FAKE + 2) == 4 and _pages(slot=FAKE + 4) == 4
    assert _pages(ld=0) == 1 and _pages(ld=-1) == 1 and _pages(ld=1 << 25) == 3
    assert _pages(want=FAKE) == 1                                     # in and out in one array
    assert _pages(batch=0) == 0
    init = lambda n, p: _status(wq.wq_pages_init, n, p, 0)  # noqa: E731
    assert init(0, FAKE) == 3 and init(-1, FAKE) == 3 and init(1 << 31, FAKE) == 3
    assert init(10, None) == 1 and init(10, FAKE + 1) == 4


def test_keep_refusals():
    for name in ("path", "count"):
        assert _keep(**{name: None}) == 1 and _keep(**{name: FAKE + 2}) == 4, name
    assert _keep(want=FAKE + 1) == 4 and _keep(want=FAKE) == 1        # the lengths are still read
    assert _keep(want=5 * FAKE, count=5 * FAKE) == 1 and _keep(want=5 * FAKE, path=5 * FAKE) == 1
    assert _keep(ld=0) == 1 and _keep(ld=-1) == 1
    assert _keep(caches=[]) == 1 and _keep(caches=[FAKE, None]) == 1 and _keep(caches=[FAKE, 2 * FAKE + 8]) == 4
    assert _keep(caches=[FAKE, 2 * FAKE, FAKE]) == 1                  # one cache twice
    assert _keep(caches=[FAKE * (i + 1) for i in range(65)]) == 2
    assert _keep(s=_seqs(batch=0)) == 0


def test_pages_arrays_are_different_ones():
    apart = dict(len=FAKE, want=2 * FAKE, table=3 * FAKE, pool=4 * FAKE, start=5 * FAKE, pos=6 * FAKE, slot=7 * FAKE)
    for a in apart:
        for b in apart:
            if a != b:
                assert _pages(**{**apart, a: apart[b]}) == 1, (a, b)
    assert _pages(**{**apart, "pos": None, "slot": None, "pool": FAKE}) == 1


def test_keep_more_workgroups_than_a_launch_has():
    many = [FAKE * (i + 1) for i in range(64)]
    s = _seqs(batch=1 << 18, rows=1 << 18)
    assert _keep(d=_desc(kv_heads=1), s=s, caches=many) == 3
    assert _keep(d=_desc(kv_heads=64), s=s, caches=many[:1]) == 3
    assert _keep(d=_desc(kv_heads=8), s=_seqs(batch=1 << 20, rows=1 << 20), caches=many[:2]) == 3


def test_nothing_to_do_is_no_launch():
    for s in (_seqs(rows=0, row_start=FAKE), _seqs(batch=0)):
        assert _sinks(s=s) == 0 and _tree(s=s) == 0
        assert wq.wq_attn_sinks_workspace_size(_desc(), s, 32, 5, 5) == 0
        assert wq.wq_attn_tree_workspace_size(_desc(), s, 32, 0, 0) == 0


def test_workspace_refusals():
    d, s = _desc(pages=5000), _seqs(batch=1, rows=1, table_ld=4096)   # one row, up to 262144 tokens: split
    need = wq.wq_attn_tree_workspace_size(d, s, 32, 0, 0)
    assert need > 0
    assert _tree(d=d, s=s, ws=FAKE, wsb=need - 1) == 6 and _tree(d=d, s=s, ws=FAKE + 8, wsb=need) == 4
    need = wq.wq_attn_sinks_workspace_size(d, s, 32, 100000, 100)
    assert need > 0 and _sinks(d=d, s=s, window=100000, sinks=100, ws=FAKE, wsb=need - 1) == 6
    assert wq.wq_attn_sinks_workspace_size(d, s, 32, 100, 4) == 0     # a short window is not split


def test_more_tiles_than_a_launch_has():
    d = _desc(head_dim=64, kv_heads=128)
    for batch, want in (((1 << 16) - 1, 0), (1 << 16, 3)):
        s = _seqs(batch=batch, rows=batch)
        assert _status(wq.wq_attn_tree_workspace_size, d, s, 128, 0, 0) == want
        assert _status(wq.wq_attn_sinks_workspace_size, d, s, 128, 9, 0) == want


def test_more_tiles_without_a_workspace():
    """Whole tiles of a call without a workspace can be narrower, and more, than those that are shared out."""
    d = _desc(head_dim=64, kv_heads=64)
    s = _seqs(batch=40000, rows=4000000, row_start=FAKE, table_ld=1000)   # 100 columns: 4.5 million tiles of 128, 10.5 of 32
    assert _status(wq.wq_attn_tree_workspace_size, d, s, 64, 0, 0) == 3
    s = _seqs(batch=20000, rows=2000000, row_start=FAKE, table_ld=1000)
    assert _status(wq.wq_attn_tree_workspace_size, d, s, 64, 0, 0) == 0


@pytest.mark.parametrize("past", [1 << 32, -(1 << 32), 1 << 31])
def test_binding_refuses_numbers_past_32_bits(past):
    for call in (lambda: _sinks(window=past + 5), lambda: _sinks(sinks=past), lambda: _sinks(hq=past + 32), lambda: _tree(window=past),
                 lambda: _tree(sinks=past), lambda: _tree(ld=past + 1), lambda: _tree(hq=past + 32), lambda: _pages(batch=past + 1),
                 lambda: _pages(ld=past + 1), lambda: _pages(rows=past + 1), lambda: _keep(ld=past + 1),
                 lambda: wq.wq_attn_sinks_workspace_size(_desc(), _seqs(), 32, past + 1, 0),
                 lambda: wq.wq_attn_tree_workspace_size(_desc(), _seqs(), 32, 1, past)):
        with pytest.raises(ValueError, match="32 bits"):
            call()


def test_binding_refuses_other_tensors():
    import torch
    with pytest.raises(ValueError, match="device buffers"):
        _tree(tree=torch.zeros((4, 1), dtype=torch.int32))
    with pytest.raises(ValueError, match="int32"):
        _tree(tree=torch.zeros((4, 1), dtype=torch.int64))
    with pytest.raises(ValueError, match="needed"):
        _tree(tree=torch.zeros((4, 1), dtype=torch.int32), ld=2)
    for name, n in (("len", 4), ("want", 4), ("table", 40), ("pool", 104), ("start", 5), ("pos", 9)):
        with pytest.raises(ValueError, match="needed"):
            _pages(**{name: torch.zeros(n - 1, dtype=torch.int32)})
        with pytest.raises(ValueError, match="int32"):
            _pages(**{name: torch.zeros(n, dtype=torch.float32)})
        with pytest.raises(ValueError, match="device buffers"):
            _pages(**{name: torch.zeros(n, dtype=torch.int32)})
    with pytest.raises(ValueError, match="int64"):
        _pages(slot=torch.zeros(9, dtype=torch.int32))
    with pytest.raises(ValueError, match="needed"):
        _keep(path=torch.zeros((4, 3), dtype=torch.int32))
    with pytest.raises(ValueError, match="needed"):
        _keep(count=torch.zeros(3, dtype=torch.int32))
    with pytest.raises(ValueError, match="needed"):
        wq.wq_pages_init(10, torch.zeros(13, dtype=torch.int32))


def test_binding_refuses_tensors_of_two_devices():
    s = wq.seqs(4, 4, _Tensor(1), _Tensor(1))
    with pytest.raises(ValueError, match="device"):
        _sinks(s=s, q=_Tensor(0))
    with pytest.raises(ValueError, match="device"):
        _tree(s=s, q=_Tensor(1), tree=_Tensor(0))
    with pytest.raises(ValueError, match="device"):
        _pages(len=_Tensor(0), want=_Tensor(1))
    with pytest.raises(ValueError, match="device"):
        _keep(s=s, path=_Tensor(0))
    with pytest.raises(ValueError, match="device"):
        _keep(s=s, caches=[_Tensor(1), _Tensor(0)])


def test_pages_rule_on_the_host():
    """The rule that the GPU is held to: what a call takes, a call that takes it back puts where it was."""
    from parts_helpers import HostPages
    rng = np.random.default_rng(1)
    h = HostPages(32, 50, 6, 8)
    for _ in range(20):
        a = [int(x) for x in h.len]
        queue = list(h.queue)
        grow = [x + int(y) for x, y in zip(a, rng.integers(0, 60, 6))]
        start, pos, slot = h.assign(grow, 1000)
        assert start[-1] == len(pos) == len(slot) and sorted(s for s in slot if s >= 0) == sorted(set(s for s in slot if s >= 0))
        if h.lacking == 0:
            h.assign(a, 1000)
            assert h.queue == queue
        h.assign(rng.integers(0, 8 * 32, 6) // 2, 1000)
        held = [p for b in range(6) for p in h.table[b][:-(-h.len[b] // 32)] if p >= 0]
        assert sorted(held + h.queue) == list(range(50))
