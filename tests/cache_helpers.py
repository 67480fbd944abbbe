"""Helpers for the cache and attention tests: the values the cache stands for (from the oracle's q4_0 / q4_1 quantizers,
after the clamp), attention over them in float64, and calls of the library on seeded sequences."""
from __future__ import annotations

import ctypes

import numpy as np
import torch

from block_quantized_bit_amd import wq
from block_quantized_bit_amd.inputs import bf16_bits_to_f32, f32_to_bf16_bits

from gpu_helpers import DEV, dev_bf16

Q4_0, Q4_1 = wq.WQ_Q4_0, wq.WQ_Q4_1


def stored(O, fmt, x):
    """fp32 [..., dim] -> the fp32 values a cache of this format holds for them."""
    x = np.ascontiguousarray(np.clip(np.where(np.isnan(x), np.float32(-32768), x), -32768, 32768), np.float32)
    n, k = int(np.prod(x.shape[:-1])), x.shape[-1]
    if n == 0:
        return x
    p = lambda a: a.ctypes.data_as(ctypes.c_void_p)  # noqa: E731
    codes, out = np.empty((n, k), np.uint8), np.empty((n, k), np.float32)
    scales = np.empty((n, k // 32, 2 if fmt == Q4_1 else 1), np.uint16)
    L = O.lib()
    quant, dequant = ((L.or_q4_0_quantize, L.or_q4_0_dequantize) if fmt == Q4_0 else (L.or_q4_1_quantize, L.or_q4_1_dequantize))
    quant(n, k, p(x), p(codes), p(scales))
    dequant(n, k, p(codes), p(scales), p(out))
    return out.reshape(x.shape)


class Case:
    """Sequences with rows `counts` and lengths `lens` (rows included) in a paged cache whose pages are in a random order.
    `bad`: (sequence, logical page) entries that point outside the pool."""

    def __init__(self, fmt, dim, heads, page, counts, lens, *, seed=0, one_row=False, paged=True, bad=(), pad_rows=0, spare=2,
                 junk=True):
        self.fmt, self.dim, self.heads, self.page = fmt, dim, heads, page
        self.counts, self.lens, self.batch = list(counts), list(lens), len(counts)
        self.rng = np.random.default_rng(seed)
        per = max([1] + [-(-t // page) for t in lens]) + (1 if paged else 0)
        need = [-(-t // page) for t in lens]
        pages = sum(need) + spare if paged else self.batch
        if not paged:
            assert per == 1
        order = self.rng.permutation(pages).astype(np.int32)
        self.table = None
        if paged:
            self.table = np.full((self.batch, per), -7, np.int32)
            at = 0
            for b, n in enumerate(need):
                self.table[b, :n] = order[at:at + n]
                at += n
            for i, (b, j) in enumerate(bad):
                self.table[b, j] = (pages, -1, 2**31 - 1, -2**31)[i % 4]
        self.bad = set(bad)
        self.rows = sum(counts) + pad_rows
        self.start = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
        self.desc = wq.cache_desc(fmt, dim, heads, page, pages)
        n = wq.wq_cache_size(self.desc)
        fill = self.rng.integers(0, 256, n, dtype=np.uint8) if junk else np.zeros(n, np.uint8)
        self.cache = torch.from_numpy(fill).to(DEV)                  # scales among the junk are infinite and NaN
        self.d_table = None if self.table is None else torch.from_numpy(self.table).to(DEV)
        self.d_len = torch.tensor(self.lens, dtype=torch.int32, device=DEV)
        self.d_start = None if one_row else torch.from_numpy(self.start).to(DEV)
        self.seqs = wq.seqs(self.batch, self.rows, self.d_len, self.d_table, self.d_start)

    def present(self, b):
        """Which of the sequence's tokens have a place in the cache."""
        t = np.arange(self.lens[b])
        return np.array([(b, int(x) // self.page) not in self.bad for x in t], bool)

    def fill(self, k, v, xdt=wq.WQ_BF16):
        """Write all tokens: k, v lists of [len, heads, dim] (bf16 bits, or fp32)."""
        n = sum(self.lens)
        if n == 0:
            return
        cat = [np.ascontiguousarray(np.concatenate(x).reshape(n, -1)) for x in (k, v)]
        dev = [torch.from_numpy(x).to(DEV) if xdt == wq.WQ_F32 else dev_bf16(x) for x in cat]
        start = torch.tensor(np.concatenate([[0], np.cumsum(self.lens)]).astype(np.int32), device=DEV)
        s = wq.seqs(self.batch, n, self.d_len, self.d_table, start)
        wq.wq_cache_write(self.desc, s, dev[0], cat[0].shape[1], dev[1], cat[1].shape[1], xdt, self.cache)
        torch.cuda.synchronize()

    def random_kv(self, std=1.0):
        def draw():
            return [f32_to_bf16_bits(self.rng.standard_normal((t, self.heads, self.dim), dtype=np.float32) * std + 0.3)
                    for t in self.lens]
        return draw(), draw()


def attend(case, O, k, v, q, group, scale, causal, window):
    """float64 attention: (y, sum (p + 2^-23) |v^|, A) with A the largest |scale| sum |q k^| of a row's visible tokens."""
    hq = case.heads * group
    y = np.zeros((case.rows, hq, case.dim))
    ab, A = np.zeros_like(y), np.zeros((case.rows, hq, 1))
    for b in range(case.batch):
        t, n = case.lens[b], case.counts[b]
        if t == 0:
            continue
        kh = stored(O, case.fmt, bf16_bits_to_f32(k[b])).astype(np.float64)
        vh = stored(O, case.fmt, bf16_bits_to_f32(v[b])).astype(np.float64)
        pos = np.arange(t)
        for i in range(n):
            row = case.start[b] + i
            see = case.present(b).copy()
            if causal:
                p = t - n + i
                see &= pos <= p
                if window:
                    see &= pos > p - window
            if not see.any():
                continue
            for h in range(hq):
                qv = q[row, h].astype(np.float64)
                K, V = kh[see, h // group], vh[see, h // group]
                s = (K @ qv) * scale
                e = np.exp(s - s.max())
                e /= e.sum()
                y[row, h] = e @ V
                ab[row, h] = (e + 2.0 ** -23) @ np.abs(V)
                A[row, h] = abs(scale) * (np.abs(K) @ np.abs(qv)).max()
    return y, ab, A


def run_attn(case, q_bits, group, scale, causal, window, *, ws="asked", pad=0, stream=None, fill=0x7BAD):
    """Y as float32 [rows, heads, dim] (and its raw bits); `pad` adds columns to the rows of q and y."""
    hq = case.heads * group
    width = hq * case.dim
    qb = np.full((case.rows, width + pad), 0x7FC0, np.uint16)
    qb[:, :width] = q_bits.reshape(case.rows, width)
    Q = dev_bf16(qb)
    Y = torch.full((case.rows, width + pad), fill, dtype=torch.int16, device=DEV)
    w, wb = None, 0
    if ws == "asked":
        wb = wq.wq_attn_workspace_size(case.desc, case.seqs, hq)
        if wb:
            w = torch.from_numpy(np.random.default_rng(5).integers(0, 256, wb, dtype=np.uint8)).to(DEV)
    wq.wq_attn(case.desc, case.seqs, hq, Q, width + pad, case.cache, scale, causal, window, Y, width + pad, w, wb, stream=stream)
    torch.cuda.synchronize()
    y = Y.cpu().numpy().view(np.uint16)
    if pad:
        assert np.all(y[:, width:] == np.uint16(fill)), "columns beyond the heads were written"
    y = np.ascontiguousarray(y[:, :width]).reshape(case.rows, hq, case.dim)
    return bf16_bits_to_f32(y), y


def check_attn(y, ref, ab, A, what=""):
    """|y - ref| <= (2^-9 + 2^-9 A) sum (p + 2^-23) |v^| + the bf16 rounding of y.

    Where it comes from, in steps of u = 2^-11 (half a step of fp16): a probability is off by u from its rounding to
    fp16, a value by u, and each score by at most u A where keys are rounded (their products with q by u each), which
    moves p by a factor e^(+-2 u A) (its own score and the sum's).  Together (2 u + 2 u A) (1 + o(1)) of sum p |v^|, and
    the fp32 sums of up to 2^17 terms in tiles and exp2 add under u (1 + A).  2^-9 = 4 u leaves a third to spare.
    Below 2^-14 fp16's steps are 2^-24, whatever the number: a small probability is off by up to 2^-25.  The kernels hold
    2^(x - ref) with the largest at least 2^7 (ref is set 7 below the largest score so far, and larger scores only add), so
    the sum that divides is at least 2^7 and a probability is off by at most 2^-32 = 2^-9 2^-23 that way.
    The output is off by half a step, 2^-8 |y| at most."""
    tol = (2.0 ** -9 + 2.0 ** -9 * A) * ab + 2.0 ** -8 * np.abs(ref) + 1e-30
    err = np.abs(y.astype(np.float64) - ref)
    bad = ~(err <= tol)
    if bad.any():
        i = tuple(np.argwhere(bad)[0])
        raise AssertionError(f"{what}: {bad.sum()} of {bad.size} outside; first {i}: y={y[i]} ref={ref[i]} tol={tol[i]}")
