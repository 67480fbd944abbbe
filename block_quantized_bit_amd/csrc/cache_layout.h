// cache_layout.h -- where a token's keys and values are in a 4-bit cache.  Plain C++ (no HIP types), so that the map
// is also compiled and checked on the host.
//
// The pool is one buffer of pages; a page holds `page` tokens of every head, head by head, in units of 32 tokens of
// one head.  A unit is what one wave of the decode attention takes per step, kept in the order its matrix
// instructions take operands, so that a lane's 16-byte loads are operands without any exchange between lanes:
//
//   [K codes 16 dim][K scales][V codes 16 dim][V scales]          scales: 2 dim bytes (q4_0) or 4 dim (q4_1)
//
//   K codes: word (tile, b, lane 16 g + r): token 16 tile + r, channels 32 b + 8 g + 0..7 (nibble n = channel + n):
//            the 8 values that lane supplies to a 16 x 16 x 32 product as the row `token`, for the 32-channel block b.
//   V codes: word (b, tile, lane 16 g + c): byte i = token 16 tile + 4 g + i, low nibble channel 32 b + c, high nibble
//            channel 32 b + 16 + c.  The product's result for K leaves a lane the scores of exactly the tokens
//            4 g + i of each tile, so the probabilities are the other operand as they stand.
//   word wi of a lane (K: tile nb + b; V: 2 b + tile; 2 nb words) is in 1 KiB chunks of 4 words per lane, the last
//   chunk of 2 words per lane where 2 nb is not a multiple of 4.
//   scales:  fp16 [tile][g][b][i] of token 16 tile + 4 g + i: d, then for q4_1 a second such plane with m.
//
// One token's row of one head touches whole bytes that no other token shares, so rows are written independently.
#pragma once

#include <stdint.h>

#ifdef __HIPCC__
#define WQ_HD __host__ __device__
#else
#define WQ_HD
#endif

namespace wq {

constexpr int kUnit = 32;        // tokens per unit
constexpr int kCacheBlock = 32;  // channels per scale
// Magnitudes above this are stored as this: every value the cache stands for (at most 15 d + m with d and m rounded
// to fp16, below 32800) is then a finite fp16 number for the kernels that compute on fp16 values.
constexpr float kCacheLimit = 32768.0f;

// Byte offset of word wi of a lane inside a unit's K or V codes (nb = dim / 32).
WQ_HD constexpr int cache_word(int nb, int wi, int lane) {
    const int c = wi >> 2;
    const bool full = 4 * c + 4 <= 2 * nb;
    return c * 1024 + lane * (full ? 16 : 8) + (wi & 3) * 4;
}
// K: token t (0..31), 8-channel group b * 4 + g.
WQ_HD constexpr int cache_k_word(int nb, int t, int b, int g) {
    return cache_word(nb, (t >> 4) * nb + b, g * 16 + (t & 15));
}
// V: the byte of token t with the channels 32 b + c (low nibble) and 32 b + 16 + c (high), c = 0..15.
WQ_HD constexpr int cache_v_byte(int nb, int t, int b, int c) {
    return cache_word(nb, 2 * b + (t >> 4), ((t & 15) >> 2) * 16 + c) + (t & 3);
}
// fp16 index inside a scale plane.
WQ_HD constexpr int cache_scale(int nb, int t, int b) { return ((t >> 2) * nb + b) * 4 + (t & 3); }

WQ_HD constexpr int cache_plane_bytes(int dim) { return 2 * dim; }                    // one scale plane of K or of V
WQ_HD constexpr int cache_half_bytes(bool q41, int dim) { return dim * (q41 ? 20 : 18); }  // K part, or V part
WQ_HD constexpr int cache_unit_bytes(bool q41, int dim) { return 2 * cache_half_bytes(q41, dim); }

// The sequences of a call: which rows are whose, and where their tokens are.
struct Seqs {
    const int32_t* row_start;  // [batch + 1], or null: row b is sequence b's only row
    const int32_t* len;        // [batch]
    const int32_t* table;      // [batch][table_ld], or null: sequence b is page b
    int32_t batch, rows;
    int32_t table_ld;          // pages a sequence can have (1 without a table)
    int32_t page;              // tokens per page
    int32_t upp;               // units per page
    int32_t heads;
    int64_t pages;
    int64_t unit_bytes;
};

// Rows [r0, r1) of sequence b: inside [0, rows) whatever row_start holds.
WQ_HD inline void seq_rows(const Seqs& s, int b, int* r0, int* r1) {
    if (!s.row_start) {
        *r0 = b;
        *r1 = b + 1;
        return;
    }
    int a = s.row_start[b], e = s.row_start[b + 1];
    a = a < 0 ? 0 : a > s.rows ? s.rows : a;
    e = e < a ? a : e > s.rows ? s.rows : e;
    *r0 = a;
    *r1 = e;
}

// Sequence of a row, or -1 (a row that is no sequence's).
WQ_HD inline int seq_of_row(const Seqs& s, int row) {
    if (!s.row_start) return row < s.batch ? row : -1;
    if (row < s.row_start[0] || row >= s.row_start[s.batch]) return -1;
    int lo = 0, hi = s.batch;  // the last b with row_start[b] <= row
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (s.row_start[mid] <= row) lo = mid;
        else hi = mid;
    }
    return row < s.row_start[lo + 1] ? lo : -1;
}

// Tokens of sequence b that are in the cache: len, within what its pages can hold.
WQ_HD inline int seq_tokens(const Seqs& s, int b) {
    const int n = s.len[b], cap = s.table_ld * s.page;
    return n < 0 ? 0 : n < cap ? n : cap;
}

// Pool page of logical page j of sequence b, or -1: an entry outside the pool is no page, and its tokens are absent.
WQ_HD inline int64_t seq_page(const Seqs& s, int b, int j) {
    if (j < 0 || j >= s.table_ld) return -1;
    const int64_t p = s.table ? (int64_t)s.table[(int64_t)b * s.table_ld + j] : (int64_t)b;
    return p >= 0 && p < s.pages ? p : -1;
}

// Byte offset in the pool of head h's unit with token t of sequence b, or -1.
WQ_HD inline int64_t seq_unit(const Seqs& s, int b, int h, int t) {
    const int j = t / s.page;
    const int64_t p = seq_page(s, b, j);
    if (p < 0) return -1;
    return ((p * s.heads + h) * s.upp + (t - j * s.page) / kUnit) * s.unit_bytes;
}

}  // namespace wq
