"""Pages and kept rows where a call's arrays hold what no ordinary step leaves there: the pool's own words, entries that are no
page among thousands that are given back, rows cut by the maps, lengths without pages; and the whole step, captured."""
import numpy as np
import pytest
import torch

from block_quantized_bit_amd import wq

from gpu_helpers import DEV, require_gpu, say
from parts_helpers import HostPages
from test_gpu_pages import DevPages, _i32

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
