"""The 4-bit cache and attention calls without a GPU: every refusal returns before anything is enqueued, and the layout
header is compiled on the host and checked whole (places distinct, inside the unit, bad pages and lengths)."""
import ctypes
import subprocess

import numpy as np
import pytest

from block_quantized_bit_amd import build, policy, wq

FAKE = 1 << 20
Q4_0, Q4_1 = wq.WQ_Q4_0, wq.WQ_Q4_1


def _status(fn, *a):
    try:
        fn(*a)
    except wq.WqError as e:
        return e.status
    return 0


def _desc(**kw):
    f = dict(format=Q4_0, head_dim=128, kv_heads=8, page=64, pages=100, reserved=0)
    f.update(kw)
    return wq.wq_cache_desc(*(f[n] for n, _ in wq.wq_cache_desc._fields_))


def _seqs(**kw):
    f = dict(batch=4, rows=4, row_start=None, len=FAKE, table=FAKE, table_ld=10, reserved=0)
    f.update(kw)
    return wq.wq_seqs(*(f[n] for n, _ in wq.wq_seqs._fields_))


BAD_DESCS = [(dict(format=0), 1), (dict(format=9), 1), (dict(format=wq.WQ_NF4), 2), (dict(format=wq.WQ_Q8_0), 2),
             (dict(head_dim=32), 2), (dict(head_dim=80), 2), (dict(head_dim=512), 2), (dict(kv_heads=0), 3),
             (dict(kv_heads=65536), 3), (dict(page=0), 3), (dict(page=16), 3), (dict(page=33), 3), (dict(page=-32), 3),
             (dict(page=(1 << 24) + 32), 3), (dict(pages=0), 3), (dict(pages=1 << 31), 3),
             (dict(pages=(1 << 31) - 1, page=4096), 3), (dict(kv_heads=8192, page=1 << 24, pages=1), 3), (dict(reserved=1), 1)]
BAD_SEQS = [(dict(batch=-1), 3), (dict(batch=(1 << 20) + 1, row_start=FAKE), 3), (dict(rows=-1), 3), (dict(rows=3), 3),
            (dict(len=None), 1), (dict(len=FAKE + 2), 4), (dict(table=FAKE + 1), 4), (dict(row_start=FAKE + 3), 4),
            (dict(table_ld=0), 1), (dict(table_ld=-1), 1), (dict(table=None), 1), (dict(table_ld=1 << 25), 3),
            (dict(reserved=2), 1)]


def _calls(d, s):
    return {"write": _status(wq.wq_cache_write, d, s, FAKE, 1024, FAKE, 1024, wq.WQ_BF16, FAKE, 0),
            "read": _status(wq.wq_cache_read, d, s, FAKE, FAKE, 1024, FAKE, 1024, wq.WQ_F32, 0),
            "attn": _status(wq.wq_attn, d, s, 32, FAKE, 4096, FAKE, 0.1, 1, 0, FAKE, 4096, None, 0, 0),
            "ws": _status(wq.wq_attn_workspace_size, d, s, 32)}


@pytest.mark.parametrize("change,want", BAD_DESCS, ids=str)
def test_descriptor_refusals(change, want):
    assert _status(wq.wq_cache_size, _desc(**change)) == want
    assert set(_calls(_desc(**change), _seqs()).values()) == {want}


@pytest.mark.parametrize("change,want", BAD_SEQS, ids=str)
def test_sequence_refusals(change, want):
    assert set(_calls(_desc(), _seqs(**change)).values()) == {want}


def test_cache_size():
    for dim in (64, 96, 128, 256):
        for heads, page, pages in ((1, 32, 1), (20, 448, 3), (8, 64, 1000)):
            n = heads * page * pages * dim
            assert wq.wq_cache_size(wq.cache_desc("q4_0", dim, heads, page, pages)) == n * 9 // 8
            assert wq.wq_cache_size(wq.cache_desc("q4_1", dim, heads, page, pages)) == n * 10 // 8


def test_row_refusals():
    d, s = _desc(), _seqs()
    for fn in (lambda **kw: _status(wq.wq_cache_write, d, s, kw.get("k", FAKE), kw.get("ldk", 1024), kw.get("v", FAKE),
                                    kw.get("ldv", 1024), kw.get("dt", 1), kw.get("cache", FAKE), 0),
               lambda **kw: _status(wq.wq_cache_read, d, s, kw.get("cache", FAKE), kw.get("k", FAKE), kw.get("ldk", 1024),
                                    kw.get("v", FAKE), kw.get("ldv", 1024), kw.get("dt", 1), 0)):
        assert fn(k=None) == 1 and fn(v=None) == 1 and fn(cache=None) == 1
        assert fn(k=FAKE + 8) == 4 and fn(v=FAKE + 2) == 4 and fn(cache=FAKE + 4) == 4
        assert fn(ldk=1016) == 1 and fn(ldv=1028) == 1 and fn(ldk=1 << 31) == 1
        assert fn(dt=0) == 1 and fn(dt=3) == 1


def test_attention_refusals():
    d, s = _desc(), _seqs()
    at = lambda **kw: _status(wq.wq_attn, d, kw.get("s", s), kw.get("hq", 32), kw.get("q", FAKE), kw.get("ldq", 4096),  # noqa: E731
                              kw.get("cache", FAKE), kw.get("scale", 0.1), kw.get("causal", 1), kw.get("window", 0),
                              kw.get("y", FAKE), kw.get("ldy", 4096), kw.get("ws", None), kw.get("wsb", 0), 0)
    assert at(hq=0) == 3 and at(hq=12) == 3 and at(hq=65536) == 3
    assert at(q=None) == 1 and at(y=None) == 1 and at(cache=None) == 1
    assert at(q=FAKE + 2) == 4 and at(y=FAKE + 8) == 4 and at(cache=FAKE + 8) == 4
    assert at(ldq=4088) == 1 and at(ldy=4100) == 1 and at(ldq=1 << 31) == 1
    assert at(scale=float("nan")) == 1 and at(scale=float("inf")) == 1 and at(scale=-3e38) == 1
    assert at(causal=2) == 1 and at(causal=-1) == 1
    assert at(window=-1) == 1 and at(causal=0, window=5) == 1
    assert at(ws=FAKE + 8, wsb=1 << 40) == 4
    assert at(s=_seqs(rows=(1 << 31) - 1, row_start=FAKE)) == 3


def test_nothing_to_do_is_no_launch():
    """No rows or no sequences: validated, nothing enqueued (there is no GPU here to enqueue on)."""
    for s in (_seqs(rows=0, row_start=FAKE), _seqs(batch=0)):
        assert set(_calls(_desc(), s).values()) == {0}
        assert wq.wq_attn_workspace_size(_desc(), s, 32) == 0


def test_workspace_refusal():
    d, s = _desc(pages=5000), _seqs(batch=1, rows=1, table_ld=4096)   # one row, up to 262144 tokens: split
    need = wq.wq_attn_workspace_size(d, s, 32)
    if need:
        assert _status(wq.wq_attn, d, s, 32, FAKE, 4096, FAKE, 0.1, 1, 0, FAKE, 4096, FAKE, need - 1, 0) == 6


def test_more_tiles_than_a_launch_has():
    size = lambda d, s, hq: _status(wq.wq_attn_workspace_size, d, s, hq)  # noqa: E731
    d = _desc(head_dim=64, kv_heads=128)                  # one tile per sequence and head
    for batch, want in (((1 << 16) - 1, 0), (1 << 16, 3)):
        s = _seqs(batch=batch, rows=batch)
        assert size(d, s, 128) == want and size(d, s, 128 * 16) == want
        if want:
            assert _status(wq.wq_attn, d, s, 128, FAKE, 8192, FAKE, 0.1, 1, 0, FAKE, 8192, None, 0, 0) == 3
    s = _seqs(batch=1 << 15, rows=1 << 15)
    assert size(d, s, 128 * 16) == 0 and size(d, s, 128 * 17) == 3   # two tiles


def test_binding_refuses_other_tensors():
    import torch
    n = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError, match="device buffers"):
        wq.seqs(4, 4, n)
    with pytest.raises(ValueError, match="int32"):
        wq.seqs(4, 4, torch.zeros(4, dtype=torch.int64))
    with pytest.raises(ValueError, match="needed"):
        wq.seqs(4, 4, torch.zeros(3, dtype=torch.int32))
    with pytest.raises(ValueError, match="needed"):
        wq.seqs(4, 9, FAKE, row_start=torch.zeros(4, dtype=torch.int32))
    with pytest.raises(ValueError, match="pages per sequence"):
        wq.seqs(4, 4, FAKE, table=torch.zeros((3, 5), dtype=torch.int32))
    with pytest.raises(ValueError, match="contiguous"):
        wq.seqs(4, 4, FAKE, table=torch.zeros((5, 4), dtype=torch.int32).t())


class _Tensor:
    """A stand-in for a device tensor: an address on a device."""
    is_cuda, dtype = True, "torch.int32"

    def __init__(self, device):
        self.device_index = device

    def get_device(self):
        return self.device_index

    def data_ptr(self):
        return FAKE

    def is_contiguous(self):
        return True

    def numel(self):
        return 100

    def dim(self):
        return 2

    shape = (4, 10)


def test_binding_refuses_tensors_of_two_devices():
    with pytest.raises(ValueError, match="devices 0 and 1"):
        wq.seqs(4, 4, _Tensor(0), _Tensor(1))
    s = wq.seqs(4, 0, _Tensor(1), _Tensor(1), _Tensor(1))
    assert s.device == 1
    for a, b in ((0, 0), (1, 0)):
        with pytest.raises(ValueError, match="device"):
            wq.wq_cache_write(_desc(), s, _Tensor(a), 1024, _Tensor(b), 1024, wq.WQ_BF16, _Tensor(a), stream=0)
        with pytest.raises(ValueError, match="device"):
            wq.wq_attn(_desc(), s, 32, _Tensor(a), 4096, _Tensor(b), 0.1, 1, 0, _Tensor(b), 4096, stream=0)


@pytest.fixture(scope="module")
def layout(tmp_path_factory):
    """cache_layout.h as a host library."""
    d = tmp_path_factory.mktemp("layout")
    (d / "l.cpp").write_text('''
#include "cache_layout.h"
using namespace wq;
extern "C" {
int k_word(int nb, int t, int b, int g) { return cache_k_word(nb, t, b, g); }
int v_byte(int nb, int t, int b, int c) { return cache_v_byte(nb, t, b, c); }
int scale(int nb, int t, int b) { return cache_scale(nb, t, b); }
int half_bytes(int q41, int dim) { return cache_half_bytes(q41 != 0, dim); }
static Seqs mk(const int* rs, const int* len, const int* tab, int batch, int rows, int ld, int page, int heads, long pages, long ub) {
    Seqs s; s.row_start = rs; s.len = len; s.table = tab; s.batch = batch; s.rows = rows; s.table_ld = ld; s.page = page;
    s.upp = page / 32; s.heads = heads; s.pages = pages; s.unit_bytes = ub; return s;
}
int of_row(const int* rs, int batch, int rows, int row) { return seq_of_row(mk(rs, 0, 0, batch, rows, 1, 32, 1, 1, 1), row); }
void rows_of(const int* rs, int batch, int rows, int b, int* out) { seq_rows(mk(rs, 0, 0, batch, rows, 1, 32, 1, 1, 1), b, out, out + 1); }
int tokens(const int* len, int ld, int page, int b) { return seq_tokens(mk(0, len, 0, 1, 1, ld, page, 1, 1, 1), b); }
long unit(const int* tab, int ld, int page, int heads, long pages, long ub, int b, int h, int t) {
    return seq_unit(mk(0, 0, tab, 1, 1, ld, page, heads, pages, ub), b, h, t);
}
}
''')
    so = d / "l.so"
    subprocess.run(["g++", "-O1", "-std=c++17", "-shared", "-fPIC", "-fsanitize=undefined", "-fno-sanitize-recover=all", "-static-libubsan",
                    "-I", build.CSRC, "-o", str(so), str(d / "l.cpp")], check=True)
    L = ctypes.CDLL(str(so))
    L.unit.restype = ctypes.c_long
    L.unit.argtypes = [ctypes.c_void_p, ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_long, ctypes.c_long] + [ctypes.c_int] * 3
    return L


def _i32(*v):
    return np.array(v, np.int32)


def _p(a):
    return a.ctypes.data_as(ctypes.c_void_p)


@pytest.mark.parametrize("q41", [0, 1])
@pytest.mark.parametrize("dim", [64, 96, 128, 256])
def test_unit_is_filled_exactly_once(layout, dim, q41):
    """Every byte of a unit's K part and V part belongs to one (token, 32-channel block) and to one place in it."""
    nb, half = dim // 32, layout.half_bytes(q41, dim)
    assert half == 32 * dim * (10 if q41 else 9) // 16
    k, v = np.zeros(half, int), np.zeros(half, int)
    for t in range(32):
        for b in range(nb):
            for g in range(4):
                w = layout.k_word(nb, t, b, g)
                assert w % 4 == 0
                k[w:w + 4] += 1
            for c in range(16):
                v[layout.v_byte(nb, t, b, c)] += 1
            i = 16 * dim + 2 * layout.scale(nb, t, b)
            for plane in range(1 + q41):
                k[i + 2 * dim * plane:][:2] += 1
                v[i + 2 * dim * plane:][:2] += 1
    assert np.all(k == 1) and np.all(v == 1)


@pytest.mark.parametrize("dim", [64, 128])
def test_layout_positions(layout, dim):
    """Written out from the description: a lane's 16-byte slots and the bytes inside them."""
    nb = dim // 32
    for t, b, g in ((0, 0, 0), (5, 1, 2), (31, 1, 3), (16, 0, 1)):
        word = (t // 16) * nb + b
        assert layout.k_word(nb, t, b, g) == (word // 4) * 1024 + (16 * g + t % 16) * 16 + (word % 4) * 4
    for t, b, c in ((0, 0, 0), (7, 1, 9), (30, 1, 15), (16, 0, 3)):
        word = 2 * b + t // 16
        assert layout.v_byte(nb, t, b, c) == (word // 4) * 1024 + (16 * ((t % 16) // 4) + c) * 16 + (word % 4) * 4 + t % 4


def test_rows_and_sequences(layout):
    rs = _i32(2, 2, 5, 5, 5, 9)                        # rows 0, 1 and 9.. are nobody's; sequences 0, 2, 3 have none
    got = [layout.of_row(_p(rs), 5, 12, r) for r in range(12)]
    assert got == [-1, -1, 1, 1, 1, 4, 4, 4, 4, -1, -1, -1]
    assert [layout.of_row(None, 3, 5, r) for r in range(5)] == [0, 1, 2, -1, -1]
    out = _i32(0, 0)
    for b, want in enumerate([(2, 2), (2, 5), (5, 5), (5, 5), (5, 9)]):
        layout.rows_of(_p(rs), 5, 12, b, _p(out))
        assert tuple(out) == want
    wild = _i32(-5, 100, 3, 2**31 - 1)                 # whatever it holds, rows stay inside [0, rows]
    for b in range(3):
        layout.rows_of(_p(wild), 3, 12, b, _p(out))
        assert 0 <= out[0] <= out[1] <= 12


def test_bad_pages_and_lengths(layout):
    lens = _i32(-3, 0, 1, 640, 641, 2**31 - 1, -2**31)
    assert [layout.tokens(_p(lens), 10, 64, b) for b in range(7)] == [0, 0, 1, 640, 640, 640, 0]
    tab = _i32(3, -1, 4, 2**31 - 1, -2**31, 2, 0, 1)   # a pool of 4 pages, 2 sequences of 4 entries
    at = lambda b, h, t: layout.unit(_p(tab), 4, 64, 5, 4, 1000, b, h, t)  # noqa: E731
    assert at(0, 0, 0) == (3 * 5 * 2) * 1000 and at(0, 4, 63) == ((3 * 5 + 4) * 2 + 1) * 1000
    assert at(0, 0, 64) == at(0, 0, 128) == at(0, 0, 192) == -1 and at(1, 0, 0) == -1
    assert at(1, 2, 70) == ((2 * 5 + 2) * 2) * 1000 and at(1, 0, 255) == ((1 * 5) * 2 + 1) * 1000
    assert at(0, 0, 256) == -1                          # past the last entry
    assert layout.unit(None, 1, 64, 5, 4, 1000, 3, 0, 5) == 3 * 5 * 2 * 1000
    assert layout.unit(None, 1, 64, 5, 4, 1000, 4, 0, 5) == -1
    big = layout.unit(_p(_i32(2**31 - 2)), 1, 64, 5, 2**31 - 1, 9216, 0, 4, 63)   # far past 32 bits
    assert big == (((2**31 - 2) * 5 + 4) * 2 + 1) * 9216


def test_decoder_caches():
    """One self- and one cross-attention cache per decoder layer, pages of whole units that hold the positions and frames."""
    for fmt, bits in (("q4_0", 9), ("Q4_1", 10)):
        caches = policy.decoder_caches(fmt, 3)
        assert [(c.layer, c.kind) for c in caches] == [(l, k) for l in range(4) for k in ("self", "cross")]
        for c in caches:
            tokens = 448 if c.kind == "self" else 1504
            assert (c.desc.page, c.desc.pages, c.causal) == (tokens, 3, c.kind == "self")
            assert c.desc.kv_heads * c.desc.head_dim == policy.D_MODEL
            assert wq.wq_cache_size(c.desc) == 3 * tokens * 1280 * bits // 8
    for bad in ("nf4", "q8_0", "bf16"):
        with pytest.raises(ValueError, match="q4_0 or q4_1"):
            policy.decoder_caches(bad, 1)
    with pytest.raises(ValueError):
        policy.decoder_caches("q4_0", 0)


def test_overlapping_windows_are_refused():
    """Rows that are read or written twice: Y over Q, and the two outputs of a read over each other, at equal and at
    different leading dimensions.  (A window that is accepted would be launched, so only refusals are made here.)"""
    d, s = _desc(), _seqs(rows=6)
    at = lambda q, ldq, y, ldy: _status(wq.wq_attn, d, s, 32, q, ldq, FAKE, 0.1, 1, 0, y, ldy, None, 0, 0)  # noqa: E731
    far = FAKE + 2 * 5 * 4104 + 2 * 4096 - 16             # the last 8 columns of Q's last row
    for ldq in (4096, 4104):
        assert at(FAKE, ldq, FAKE, ldq) == 1
    for y, ldy in ((FAKE + 16, 4104), (FAKE, 8192), (far, 4104), (far, 1 << 20), (FAKE + 2 * 4104 - 16, 4104)):
        assert at(FAKE, 4104, y, ldy) == 1 and at(y, ldy, FAKE, 4104) == 1
    for dt, es in ((wq.WQ_BF16, 2), (wq.WQ_F32, 4)):
        rd = lambda k, ldk, v, ldv: _status(wq.wq_cache_read, d, s, FAKE, k, ldk, v, ldv, dt, 0)  # noqa: E731
        assert rd(FAKE, 1024, FAKE, 1024) == 1
        assert rd(FAKE, 2048, FAKE + es * 1016, 2048) == 1 and rd(FAKE + es * 1016, 2048, FAKE, 2048) == 1
        assert rd(FAKE, 1024, FAKE + es * (6 * 1024 - 8), 1032) == 1


@pytest.mark.parametrize("dim,heads,most", [(64, 1, (1 << 31) - 125), (128, 8, (1 << 27) - 5), (256, 16, (1 << 26) - 1), (96, 5, (1 << 28) - 13)])
def test_more_rows_than_a_launch_has(dim, heads, most):
    """Groups of four tokens, each of heads * dim / 8 threads, K and V side by side: the last number of rows whose launch has
    fewer than 2^32 threads along x.  (No sequences: a call that is taken does nothing.)"""
    d, width = _desc(head_dim=dim, kv_heads=heads), dim * heads
    for rows, want in ((most, 0), (most + 1, 3), ((1 << 31) - 1, 3)):
        s = _seqs(batch=0, rows=rows, row_start=FAKE)
        assert _status(wq.wq_cache_write, d, s, FAKE, width, FAKE, width, wq.WQ_BF16, FAKE, 0) == want
        assert _status(wq.wq_cache_read, d, s, FAKE, FAKE, width, FAKE, width, wq.WQ_F32, 0) == want
    # sequences count too: each may touch two groups more
    s = _seqs(batch=1 << 20, rows=most, row_start=FAKE)
    assert _status(wq.wq_cache_write, d, s, FAKE, width, FAKE, width, wq.WQ_BF16, FAKE, 0) == 3


def test_written_assembly_names_what_it_writes():
    """A statement that writes m0 says so, so that the compiler keeps nothing there across it."""
    import os
    import re
    found = 0
    for name in sorted(os.listdir(build.CSRC)):
        with open(os.path.join(build.CSRC, name)) as f:
            text = f.read()
        for stmt in re.findall(r"\basm\b[^;]*;", text):
            code, *rest = stmt.split(":")
            if "m0" in code:
                found += 1
                assert '"m0"' in "".join(rest), f"{name}: {stmt}"
    assert found > 0


@pytest.mark.parametrize("past", [1 << 32, -(1 << 32), 1 << 31])
def test_binding_refuses_numbers_past_32_bits(past):
    """Such a number would be passed as its low 32 bits: another page size, batch or window.  (Window and heads are tried on
    a descriptor that is refused anyway.)"""
    d, s = _desc(), _seqs()
    for call in (lambda: wq.cache_desc("q4_0", 128, 8, past + 64, 10), lambda: wq.cache_desc("q4_0", 128, past + 8, 64, 10),
                 lambda: wq.cache_desc("q4_0", past + 128, 8, 64, 10), lambda: wq.seqs(past + 4, 4, FAKE, FAKE, FAKE, 10),
                 lambda: wq.seqs(4, past + 4, FAKE, FAKE, FAKE, 10), lambda: wq.seqs(4, 4, FAKE, FAKE, FAKE, past + 10),
                 lambda: wq.wq_attn_workspace_size(d, s, past + 32),
                 lambda: wq.wq_attn(_desc(page=1), s, past + 32, FAKE, 4096, FAKE, 0.1, 1, 0, 2 * FAKE, 4096, stream=0),
                 lambda: wq.wq_attn(_desc(page=1), s, 32, FAKE, 4096, FAKE, 0.1, 1, past + 5, 2 * FAKE, 4096, stream=0),
                 lambda: wq.wq_attn(_desc(page=1), s, 32, FAKE, 4096, FAKE, 0.1, past + 1, 0, 2 * FAKE, 4096, stream=0)):
        with pytest.raises(ValueError, match="32 bits"):
            call()
    assert wq.cache_desc("q4_0", 128, 8, 64, 1 << 33).pages == 1 << 33     # (64 bits in the descriptor)


def test_workspace_refusal_of_a_split_call():
    """The call does ask for a workspace; one byte less is refused, as is a misaligned one."""
    d, s = _desc(pages=5000), _seqs(batch=1, rows=1, table_ld=4096)
    need = wq.wq_attn_workspace_size(d, s, 32)
    assert need > 0
    at = lambda ws, n: _status(wq.wq_attn, d, s, 32, FAKE, 4096, FAKE, 0.1, 1, 0, 2 * FAKE, 4096, ws, n, 0)  # noqa: E731
    assert at(FAKE, need - 1) == 6 and at(FAKE, 0) == 6 and at(FAKE + 8, need) == 4
