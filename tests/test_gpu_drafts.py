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
