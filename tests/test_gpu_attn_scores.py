"""Scores of wq_attn where their error shows: blocks whose largest key meets a query near zero (the other products then
have to stay small by themselves, not by cancelling), heavy-tailed queries, and queries of any magnitude under a scale that
brings the scores back to ordinary ones.  Few rows, many rows, and long sequences that are shared out."""
import numpy as np
import pytest

from block_quantized_bit_amd.inputs import bf16_bits_to_f32, f32_to_bf16_bits

from cache_helpers import Q4_0, Q4_1, Case, attend, run_attn, stored
from gpu_helpers import require_gpu, say

pytestmark = pytest.mark.gpu

FMT = pytest.mark.parametrize("fmt", [Q4_0, Q4_1], ids=["q4_0", "q4_1"])
# rows and tokens: one row, several, more than 128 columns, one row over a sequence that is shared out
SHAPE = pytest.mark.parametrize("rows,tokens", [(1, 70), (40, 70), (140, 70), (1, 3001)], ids=["token", "rows", "many", "shared"])


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def _check(orc, c, k, v, q, scale, what):
    """|y - ref| <= (2^-9 + 2^-9 A + 2^-38 Q) sum (p + 2^-23) |v^| + 2^-8 |ref|, Q = |scale| max |q| max_t sum |k^_t|.

    The first two terms are those of check_attn.  The third: queries are brought to fp16 by a power of two that puts a row's
    largest into [2^14, 2^15); the others keep all their bits down to 2^-14, and below that are off by half of 2^-24, which is
    2^-39 of the largest at most.  A score is then off by 2^-39 Q, and a probability by twice that."""
    c.fill([k], [v])
    qf = bf16_bits_to_f32(q)
    ref, ab, A = attend(c, orc, [k], [v], qf, 1, scale, 0, 0)
    kh = np.abs(stored(orc, c.fmt, bf16_bits_to_f32(k)).astype(np.float64)).sum(-1).max(0)          # [heads]
    Q = abs(scale) * np.abs(qf.astype(np.float64)).max(-1) * kh
    tol = (2.0 ** -9 + 2.0 ** -9 * A + 2.0 ** -38 * Q[..., None]) * ab + 2.0 ** -8 * np.abs(ref) + 1e-30
    for ws in ("asked", None):
        y, _ = run_attn(c, q, 1, scale, 0, 0, ws=ws)
        err = np.abs(y.astype(np.float64) - ref)
        bad = ~(err <= tol)
        assert not bad.any(), f"{what} ws={ws}: {bad.sum()} of {bad.size} outside, worst {np.nanmax(err / tol):.3g} of the bound"


def _values(c, tokens):
    """Values that differ from token to token, so that a wrong probability shows: 1 in every other token, 0 between."""
    v = np.zeros((tokens, c.heads, c.dim), np.float32)
    v[::2] = 1.0
    return f32_to_bf16_bits(v)


@FMT
@SHAPE
def test_largest_key_beside_a_small_query(orc, fmt, rows, tokens):
    """One block (32768, 0 ..., 32768) against (0, 1.5 ..., 1.25 2^-13): a score of 0.625 that is made by one product."""
    c = Case(fmt, 64, 1, 64, [rows], [tokens], seed=1, one_row=rows == 1)
    say("largest key", fmt, rows, tokens)
    k = np.zeros((tokens, 1, 64), np.float32)
    k[::2, :, 0] = k[::2, :, 31] = 32768.0
    q = np.zeros((rows, 1, 64), np.float32)
    q[..., 1:31] = 1.5
    q[..., 31] = 1.25 * 2.0 ** -13
    _check(orc, c, f32_to_bf16_bits(k), _values(c, tokens), f32_to_bf16_bits(q), 0.125, "largest key")


@FMT
@SHAPE
@pytest.mark.parametrize("dim", [64, 96, 128, 256])
def test_outlier_keys(orc, fmt, rows, tokens, dim):
    """Each block of a key has one large channel, where the query is zero, and zeros elsewhere, under a query of many
    binades: every true score is 0, and every token counts alike."""
    for seed, outlier in enumerate([30.0, -300.0, 30000.0, -30000.0]):
        c = Case(fmt, dim, 2, 64, [rows], [tokens], seed=seed, one_row=rows == 1)
        say("outlier", fmt, rows, tokens, dim, outlier)
        k = np.zeros((tokens, 2, dim), np.float32)
        k[::2, :, 5::32] = outlier
        k[1::4, :, 5::32] = -outlier
        q = c.rng.standard_normal((rows, 2, dim), dtype=np.float32) * np.exp2(c.rng.integers(-10, 10, (rows, 2, dim))).astype(np.float32)
        q[..., 5::32] = 0.0
        _check(orc, c, f32_to_bf16_bits(k), _values(c, tokens), f32_to_bf16_bits(q), dim ** -0.5, f"outlier {outlier}")


RANGE = pytest.mark.parametrize("qs,scale", [(2.0 ** 122, 2.0 ** -124), (2.0 ** 110, 2.0 ** -113), (2.0 ** -110, 2.0 ** 107), (2.0 ** -122, 2.0 ** 119),
                                             (2.0 ** -129, 2.0 ** 126)], ids=["largest", "large", "small", "smaller", "subnormal"])


def _magnitude(orc, fmt, rows, tokens, qs, scale):
    c = Case(fmt, 128, 1, 64, [rows], [tokens], seed=3, one_row=rows == 1)
    say("magnitude", fmt, rows, tokens, qs, scale)
    k, v = (x[0] for x in c.random_kv())
    q = (c.rng.standard_normal((rows, 1, 128)) * qs).astype(np.float32)
    _check(orc, c, k, v, f32_to_bf16_bits(q), scale, f"queries of {qs}")


@FMT
@pytest.mark.parametrize("rows,tokens", [(1, 70), (40, 70), (1, 3001)], ids=["token", "rows", "shared"])
@RANGE
def test_queries_of_any_magnitude(orc, fmt, rows, tokens, qs, scale):
    _magnitude(orc, fmt, rows, tokens, qs, scale)


@FMT
@RANGE
def test_many_rows_of_queries_of_any_magnitude(orc, fmt, qs, scale):
    _magnitude(orc, fmt, 140, 70, qs, scale)
