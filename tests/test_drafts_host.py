"""Of the calls of a step with drafts, what needs no GPU: refusals of arrays that share bytes, the step's rule, what fp16 holds of
the cache's values."""
import numpy as np
import pytest

from block_quantized_bit_amd import build
from block_quantized_bit_amd.inputs import bf16_bits_to_f32, f32_to_bf16_bits

from cache_helpers import Q4_0, stored
from parts_helpers import HostPages
from test_cache_host import FAKE, _seqs
from test_parts_host import _keep, _pages


@pytest.mark.parametrize("name", ["len", "row_start", "table", "path", "count"])
def test_keep_writes_over_none_of_its_inputs(name):
    """Every workgroup reads a sequence's lengths, starts, pages and path, when another may have written `want` already."""
    at = dict(len=10 * FAKE, row_start=20 * FAKE, table=30 * FAKE, path=40 * FAKE, count=50 * FAKE)
    ints = dict(len=4, row_start=5, table=4 * 10, path=4 * 4, count=4)

    def call(want, **kw):
        s = _seqs(rows=9, **{k: at[k] for k in ("len", "row_start", "table")}, **kw)
        return _keep(s=s, path=at["path"], count=at["count"], want=want)

    for first in (0, ints[name] - 1, -3):                   # want has 4 words: the array's first, its last, the one behind want's
        assert call(at[name] + 4 * first) == 1, first

    s = _seqs(rows=9, row_start=None, len=at["len"], table=None, table_ld=0)
    assert _keep(s=s, path=at["path"], count=at["count"], want=at["len"] + 12) == 1


def test_page_arrays_share_no_byte():
    """Each of a call's arrays, moved to the last bytes of each other one, or so that its own last bytes are the other's first."""
    words = dict(len=4, want=4, table=40, pool=104, start=5, pos=9, slot=18)     # batch 4, 10 entries each, 100 pages, 9 rows
    apart = {k: FAKE * (i + 1) for i, k in enumerate(words)}
    for a in words:
        for b in words:
            if a != b:
                step = 2 if a == "slot" else 1                                   # (aligned to its entries)
                for at in (4 * ((words[b] - 1) // step * step), -4 * ((words[a] - 1) // step * step)):
                    assert _pages(**{**apart, a: apart[b] + at}) == 1, (a, b, at)


def test_a_step_ends_with_the_accepted_length():
    """The header's step: a draft's rows are what the lengths grow by, so the call back to the accepted length cannot be left
    to the next step's first call."""
    def draft(closed):
        h = HostPages(32, 20, 1, 10)
        h.assign([100], 200)
        h.assign([113], 200)                                # 13 drafted tokens, of which 5 are kept
        if closed:
            h.assign([105], 0)
        return h.assign([118], 200)[1]                      # 13 more

    assert draft(True) == list(range(105, 118)) and draft(False) == list(range(113, 118))
    header = open(build.ROOT + "/include/wq.h").read()
    at = header.index("A step of serving with drafted tokens")
    step = header[at:header.index("*/", at)]
    calls = [x.split()[1] for x in step.splitlines() if x.startswith(" *   wq_")]
    assert calls == ["wq_pages_assign", "wq_cache_write", "wq_attn_tree", "wq_cache_keep", "wq_pages_assign"]
    assert "does it too" not in step and "belongs to every step" in step


def test_q4_0_of_bf16_rows_is_exact_in_fp16(orc):
    """A scale of 8 bits times a code less 8: what the kernels hold as fp16 is then the value itself."""
    rng = np.random.default_rng(1)
    for std in (2.0 ** -6, 1.0, 300.0):
        x = bf16_bits_to_f32(f32_to_bf16_bits((rng.standard_normal((200, 256)) * std).astype(np.float32)))
        y = stored(orc, Q4_0, x)
        assert np.array_equal(y.astype(np.float16).astype(np.float32), y)
