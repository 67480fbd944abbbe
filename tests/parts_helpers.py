"""Helpers for the tests of attention with sinks and of drafted trees, of pages and of kept rows: which tokens a row sees,
float64 attention over them, and page assignment step by step on the host."""
from __future__ import annotations

import numpy as np
import torch

from block_quantized_bit_amd import wq
from block_quantized_bit_amd.inputs import bf16_bits_to_f32

from cache_helpers import stored
from gpu_helpers import DEV, dev_bf16


def sees_sinks(case, window, sinks):
    """[rows of b, tokens of b] truth values per sequence."""
    out = []
    for b in range(case.batch):
        t, n = case.lens[b], case.counts[b]
        p, at = np.arange(t - n, t)[:, None], np.arange(t)[None]
        out.append((at <= p) & ((at > p - window) | (at < sinks)) & case.present(b)[None])
    return out


def words(masks, ld, rows, rng=None):
    """[rows][ld] 32-bit words of per-sequence masks [n, n]; bits that no row of the sequence has, and padding rows, are
    random."""
    w = np.zeros((rows, ld * 32), bool) if rng is None else rng.random((rows, ld * 32)) < 0.5
    at = 0
    for m in masks:
        n = m.shape[0]
        k = min(n, ld * 32)
        w[at:at + n, :k] = m[:, :k]
        at += n
    return np.packbits(w, axis=1, bitorder="little").view(np.uint32).reshape(rows, ld)


def trees(rng, counts, kind):
    """Masks [n, n] of each sequence: a chain, a tree (parents among the 9 before, or the context), any bits, none."""
    out = []
    for n in counts:
        if kind == "chain":
            m = np.tril(np.ones((n, n), bool))
        elif kind == "any":
            m = rng.random((n, n)) < 0.4
        elif kind == "none":
            m = np.zeros((n, n), bool)
        else:
            m = np.zeros((n, n), bool)
            for i in range(n):
                parent = i - 1 - int(rng.integers(0, 9))
                if parent >= 0:
                    m[i] = m[parent]
                m[i, i] = True
        out.append(m)
    return out


def sees_tree(case, masks, ld, window, sinks):
    out = []
    for b in range(case.batch):
        t, n = case.lens[b], case.counts[b]
        at, before = np.arange(t), t - n
        m = masks[b].copy()
        m[:, ld * 32:] = False
        see = np.tile((at < before)[None], (n, 1))
        if window:
            see &= (at[None] >= before - window + m.sum(1)[:, None]) | (at[None] < sinks)
        for j in range(n):
            if before + j >= 0:
                see[:, before + j] = m[:, j]
        out.append(see & case.present(b)[None])
    return out


def attend_seen(case, O, k, v, q, group, scale, sees):
    """float64 attention over the tokens that `sees` says: (y, sum (p + 2^-23) |v^|, A) as cache_helpers.attend."""
    hq = case.heads * group
    y = np.zeros((case.rows, hq, case.dim))
    ab, A = np.zeros_like(y), np.zeros((case.rows, hq, 1))
    for b in range(case.batch):
        t, n, r = case.lens[b], case.counts[b], int(case.start[b])
        if t == 0 or n == 0:
            continue
        kh = stored(O, case.fmt, bf16_bits_to_f32(k[b])).astype(np.float64)
        vh = stored(O, case.fmt, bf16_bits_to_f32(v[b])).astype(np.float64)
        see = sees[b]
        some = see.any(1)[:, None]
        for h in range(hq):
            Q, K, V = q[r:r + n, h].astype(np.float64), kh[:, h // group], vh[:, h // group]
            s = np.where(see, (Q @ K.T) * scale, -np.inf)
            e = np.exp(s - np.where(some, s.max(1, keepdims=True), 0.0))
            e = e / np.where(some, e.sum(1, keepdims=True), 1.0)
            y[r:r + n, h] = e @ V
            ab[r:r + n, h] = np.where(see, e + 2.0 ** -23, 0.0) @ np.abs(V)
            A[r:r + n, h, 0] = np.where(see, abs(scale) * (np.abs(Q) @ np.abs(K).T), 0.0).max(1)
    return y, ab, A


def run_seen(case, q_bits, group, scale, window, sinks, tree=None, *, ws="asked", pad=0, stream=None, fill=0x7BAD):
    """wq_attn_sinks, or wq_attn_tree with a device tensor of mask words: Y as float32 [rows, heads, dim] and its bits."""
    hq = case.heads * group
    width = hq * case.dim
    qb = np.full((case.rows, width + pad), 0x7FC0, np.uint16)
    qb[:, :width] = q_bits.reshape(case.rows, width)
    Q = dev_bf16(qb)
    Y = torch.full((case.rows, width + pad), fill, dtype=torch.int16, device=DEV)
    size = wq.wq_attn_sinks_workspace_size if tree is None else wq.wq_attn_tree_workspace_size
    w, wb = None, 0
    if ws == "asked":
        wb = size(case.desc, case.seqs, hq, window, sinks)
        if wb:
            w = torch.from_numpy(np.random.default_rng(5).integers(0, 256, wb, dtype=np.uint8)).to(DEV)
    if tree is None:
        wq.wq_attn_sinks(case.desc, case.seqs, hq, Q, width + pad, case.cache, scale, window, sinks, Y, width + pad, w, wb, stream=stream)
    else:
        wq.wq_attn_tree(case.desc, case.seqs, hq, Q, width + pad, case.cache, scale, window, sinks, tree, tree.shape[1], Y,
                        width + pad, w, wb, stream=stream)
    torch.cuda.synchronize()
    y = Y.cpu().numpy().view(np.uint16)
    if pad:
        assert np.all(y[:, width:] == np.uint16(fill)), "columns beyond the heads were written"
    y = np.ascontiguousarray(y[:, :width]).reshape(case.rows, hq, case.dim)
    return bf16_bits_to_f32(y), y


def dev_words(w):
    return torch.from_numpy(np.ascontiguousarray(w).view(np.int32)).to(DEV)


class HostPages:
    """Page assignment as the header says it, one page at a time."""

    def __init__(self, page, pages, batch, per, free=None):
        self.page, self.pages, self.per = page, pages, per
        self.queue = list(range(pages)) if free is None else list(free)
        self.len = [0] * batch
        self.table = [[-1] * per for _ in range(batch)]
        self.lacking = 0

    def assign(self, want, rows):
        want = [max(int(w), 0) for w in want]
        n_of = lambda t: min(-(-t // self.page), self.per)  # noqa: E731
        back = []
        for b, w in enumerate(want):
            for j in range(n_of(w), n_of(self.len[b])):
                if 0 <= self.table[b][j] < self.pages:
                    back.append(self.table[b][j])
        self.queue = back + self.queue
        self.lacking = 0
        start, pos, slot = [0], [], []
        for b, w in enumerate(want):
            for j in range(n_of(self.len[b]), n_of(w)):
                if self.queue:
                    self.table[b][j] = self.queue.pop(0)
                else:
                    self.table[b][j] = -1
                    self.lacking += 1
            for t in range(self.len[b], w):
                pos.append(t)
                j = t // self.page
                p = self.table[b][j] if j < self.per else -1
                slot.append(p * self.page + t % self.page if 0 <= p < self.pages else -1)
            start.append(min(rows, start[-1] + max(w - self.len[b], 0)))
            self.len[b] = w
        return start, pos[:rows], slot[:rows]
