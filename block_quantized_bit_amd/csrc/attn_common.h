// attn_common.h -- shared by the attention kernels: which rows and tokens a tile has, where a sequence's units are, and
// the cross-lane and conversion helpers.
//
// Both kernels compute the transposed products S^T = K Q^T and Y^T = V^T P^T.  A tile's columns are query rows times the
// query heads that share a key/value head, so the keys and values of one head serve a whole tile; and a lane's scores
// after the first product are, in the cache's order of tokens, the lane's operand of the second.
#pragma once

#include <cfloat>

#include "cache_device.h"
#include "wq_device.h"
#include "wq_launch.h"

namespace wq {

typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// Columns per tile: `rows` rows of the sequence times the group's heads, or one row's `ht` runs of heads.
struct TileShape {
    int rows, ht;
};
__host__ __device__ inline TileShape tile_shape(int cols, int group) {
    return group <= cols ? TileShape{cols / group, 1} : TileShape{1, (group + cols - 1) / cols};
}
// Tiles of a call with `rows` rows and `batch` sequences: at most this many.
__host__ __device__ inline int64_t tile_bound(const TileShape& ts, int rows, int batch, bool one_row) {
    if (one_row) return (int64_t)batch * ts.ht;
    return ((int64_t)rows / ts.rows + (ts.rows > 1 ? (rows < batch ? rows : batch) : 0)) * ts.ht;
}

// Rows, tokens and units of a sequence.
struct SeqInfo {
    int r0, n;        // its rows
    int tokens;       // in the cache
    int64_t pos0;     // token of its first row (causal)
};

__device__ inline SeqInfo seq_info(const AttnArgs& a, int b) {   // b per lane
    SeqInfo q;
    int r0, r1;
    seq_rows(a.s, b, &r0, &r1);
    q.r0 = r0;
    q.n = r1 - r0;
    q.tokens = seq_tokens(a.s, b);
    q.pos0 = (int64_t)a.s.len[b] - q.n;
    return q;
}

// The same for a uniform b, through scalar loads.
__device__ inline SeqInfo seq_info_uniform(const AttnArgs& a, int b) {
    const SeqRows r = seq_rows_uniform(a.s, b);
    const int len = r.len, cap = a.s.table_ld * a.s.page;
    SeqInfo q;
    q.r0 = r.r0;
    q.n = r.r1 - r.r0;
    q.tokens = len < 0 ? 0 : len < cap ? len : cap;
    q.pos0 = (int64_t)len - q.n;
    return q;
}

// Tokens [lo, hi) that row i of the sequence sees.
__device__ inline void row_tokens(const AttnArgs& a, const SeqInfo& q, int i, int* lo, int* hi) {
    *lo = 0;
    *hi = q.tokens;
    if (a.causal) {
        const int64_t p = q.pos0 + i + 1;
        *hi = p < 0 ? 0 : p < *hi ? (int)p : *hi;
        if (a.window > 0 && p > a.window) *lo = p - a.window < *hi ? (int)(p - a.window) : *hi;
    }
}

// Units [u0, u1) that hold the tokens of rows [i0, i1) of the sequence.
__device__ inline void row_units(const AttnArgs& a, const SeqInfo& q, int i0, int i1, int* u0, int* u1) {
    int lo, hi, x;
    row_tokens(a, q, i0, &lo, &x);
    row_tokens(a, q, i1 - 1, &x, &hi);
    *u0 = lo / kUnit;
    *u1 = hi > lo ? (hi + kUnit - 1) / kUnit : *u0;
}

// The same with sinks, or of a tree of drafted tokens: the rows' units in ascending order, without those that no row sees.
struct UnitList {
    int far, near, count;    // units 0 .. far - 1, then near, near + 1 ...: `count` in all
    __device__ int operator[](int i) const { return i < far ? i : i - far + near; }
    // Whether units are left out between the i-th and the one `step` after it.
    __device__ bool gap(int i, int step) const { return i < far && i + step >= far && near > far; }
};

// Tokens [lo, hi) that row i of the sequence sees besides sinks and drafted tokens: with a tree, those before the first row,
// as far back as the window goes when the drafted tokens that the row sees (itself among them) are the nearest part of it.
__device__ inline int drafts_seen(const AttnArgs& a, const SeqInfo& q, int i) {
    const uint32_t* const w = a.tree + (int64_t)(q.r0 + i) * a.tree_ld;
    int seen = 0;
    for (int k = 0; k < a.tree_ld && k * 32 < q.n; k++) seen += __popc(q.n - k * 32 < 32 ? w[k] & ((1u << (q.n - k * 32)) - 1) : w[k]);
    return seen;
}
__device__ inline int clamped(int64_t v, int most) { return v < 0 ? 0 : v < most ? (int)v : most; }
__device__ inline void row_context(const AttnArgs& a, const SeqInfo& q, int i, int* lo, int* hi) {
    if (!a.tree) return row_tokens(a, q, i, lo, hi);
    *lo = 0;
    *hi = clamped(q.pos0, q.tokens);
    if (a.window > 0) *lo = clamped(q.pos0 + drafts_seen(a, q, i) - a.window, *hi);
}
// What rows [i0, i1] see all of: the tokens [lo_most, hi_least), at least.
__device__ inline void parts_between(const AttnArgs& a, const SeqInfo& q, int i0, int i1, int* lo_most, int* hi_least) {
    if (!a.tree) {
        int x;
        row_tokens(a, q, i0, &x, hi_least);
        row_tokens(a, q, i1, lo_most, &x);
        return;
    }
    *hi_least = clamped(q.pos0, q.tokens);
    *lo_most = a.window > 0 ? clamped(q.pos0 + q.n - a.window, *hi_least) : 0;
}
// Units of rows [i0, i1).
__device__ inline UnitList row_parts(const AttnArgs& a, const SeqInfo& q, int i0, int i1) {
    int lo, hi, x, sinks;
    if (a.tree) {
        const int context = clamped(q.pos0, q.tokens);
        lo = a.window > 0 ? clamped(q.pos0 - a.window, context) : 0;
        hi = q.tokens;
        sinks = min(a.sinks, context);
    } else {
        row_tokens(a, q, i0, &lo, &x);
        row_tokens(a, q, i1 - 1, &x, &hi);
        sinks = min(a.sinks, hi);
    }
    UnitList r;
    r.near = lo / kUnit;
    r.far = min((sinks + kUnit - 1) / kUnit, r.near);
    r.count = r.far + (hi > lo ? (hi + kUnit - 1) / kUnit - r.near : 0);
    return r;
}
// Which of the 32 tokens from t0 on are drafted ones that row i sees, a bit each.
__device__ inline uint32_t seen_nodes(const AttnArgs& a, const SeqInfo& q, int i, int t0) {
    if (!a.tree || t0 >= q.tokens || t0 + kUnit <= q.pos0) return 0;
    const int64_t at = t0 - q.pos0;   // bit of token t0, -31 or more
    const uint32_t* const w = a.tree + (int64_t)(q.r0 + i) * a.tree_ld;
    const int64_t k = at >> 5;        // floor
    const uint32_t low = k >= 0 && k < a.tree_ld ? w[k] : 0, high = k + 1 < a.tree_ld ? w[k + 1] : 0;   // (k >= -1)
    const uint32_t bits = __builtin_amdgcn_alignbit(high, low, (uint32_t)at & 31);
    return q.tokens - t0 < kUnit ? bits & ((1u << (q.tokens - t0)) - 1) : bits;
}

// Which of the 32 tokens from t0 on are seen, a bit each, where [lo, hi), the first `sinks` below hi and `nodes` are.
__device__ inline uint32_t bits_below(int n) { return n >= 32 ? ~0u : n > 0 ? (1u << n) - 1 : 0u; }
__device__ inline uint32_t seen_tokens(int lo, int hi, int sinks, uint32_t nodes, int t0) {
    return (bits_below(hi - t0) & (~bits_below(lo - t0) | bits_below(sinks - t0))) | nodes;
}

__device__ inline int tiles_of(const TileShape& ts, int n) { return (n + ts.rows - 1) / ts.rows * ts.ht; }

// With as many tiles, the n rows spread evenly over them.
__device__ inline TileShape even_shape(const TileShape& ts, int n) {
    if (ts.ht != 1 || n <= ts.rows) return ts.ht == 1 && n > 0 ? TileShape{n, 1} : ts;
    const int tiles = (n + ts.rows - 1) / ts.rows;
    return TileShape{(n + tiles - 1) / tiles, 1};
}
struct TileCount {
    const AttnArgs& a;
    TileShape ts;
    __device__ uint32_t operator()(int b) const {
        int r0, r1;
        seq_rows(a.s, b, &r0, &r1);
        return (uint32_t)tiles_of(ts, r1 - r0);
    }
};

// Where the units of one head of one sequence are, unit by unit.  The wave holds 64 table entries, one a lane: an entry
// read when it is needed would be a scalar load, whose wait is also one for every LDS read that is on its way.
struct UnitWalk {
    const int32_t* table;   // this sequence's row, or null
    int upp, table_ld, seq, pages;
    int j, k;               // page and unit within it
    int j0, entries;        // entries (per lane): of page j0 + lane
    int per_page, head_units, unit_bytes;
    int64_t cur;            // byte offset of the unit (the pool's first one's where it is absent)
    int there;              // whether it has a page

    __device__ void start(const Seqs& q, int sequence, int head, int unit) {
        upp = q.upp;
        table_ld = q.table_ld;
        table = q.table ? q.table + (int64_t)sequence * q.table_ld : nullptr;
        seq = sequence;
        pages = (int)q.pages;
        unit_bytes = (int)q.unit_bytes;
        per_page = q.heads * q.upp;     // (below 2^31: a cache is at most 2^41 bytes)
        head_units = head * q.upp;
        j = uniform(unit / upp);   // (a quotient is made by the vector unit, and would keep what follows from it there)
        k = unit - j * upp;
        hold();
        place();
    }
    __device__ void hold() {
        j0 = j;
        const int at = j + (threadIdx.x & 63);
        entries = -1;
        if (at < table_ld) entries = table ? table[at] : seq;
        asm volatile("" : "+v"(entries));   // waited for here, and not wherever an entry is used
    }
    __device__ void place() {
        const int entry = __builtin_amdgcn_readlane(entries, j - j0);
        there = (unsigned)entry < (unsigned)pages;
        cur = there ? ((int64_t)entry * per_page + (head_units + k)) * unit_bytes : 0;
    }
    __device__ void seek(int unit) {   // on to a later unit
        j = uniform(unit / upp);
        k = unit - j * upp;
        if (j - j0 >= 64) hold();
        place();
    }
    __device__ void step(int n) {
        k += n;
        if (k < upp) {
            cur += there ? n * unit_bytes : 0;
            return;
        }
        do {
            k -= upp;
            j++;
        } while (k >= upp);
        if (j - j0 >= 64) hold();
        place();
    }
    // The unit's address.
    __device__ const uint8_t* at(const uint8_t* cache) const { return cache + cur; }
};
// An address in scalar registers whose origin the compiler does not see: it would else add the lanes' offsets to the
// part that does not change, and hold 64-bit sums of them in vector registers.
typedef const uint8_t __attribute__((address_space(1))) * global_bytes;
__device__ inline global_bytes scalar_address(const uint8_t* p) {
    uint64_t v = (uint64_t)(uintptr_t)p;
    asm("" : "+s"(v));
    return (global_bytes)v;
}
template <class T>
__device__ inline T load_at(global_bytes p, uint32_t offset) {
    return *(const T __attribute__((address_space(1)))*)(p + offset);
}

__device__ inline float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

__device__ inline f16x2 as_f16x2(uint32_t v) { return __builtin_bit_cast(f16x2, v); }

// (w & mask) | bits, in one instruction where neither is a literal to the compiler (an instruction takes one).  Not as
// written assembly: the compiler counts no waiting states between a matrix instruction and that.
__device__ inline uint32_t and_or(uint32_t w, uint32_t mask, uint32_t bits) {
    asm("" : "+s"(mask));
    return (w & mask) | bits;
}
// A constant in a register.
__device__ inline uint32_t held(uint32_t c) {
    uint32_t r = c;
    asm("" : "+v"(r));
    return r;
}
// The codes of a word, two to a register, nibbles i and i + 4, under the bits of a number whose last place is 1
// (fp16 1024: 0x64006400).
__device__ inline uint32_t nibble_pair(uint32_t w, int i, uint32_t bits) { return and_or(w >> (4 * i), 0x000F000Fu, bits); }
// V words (masked to one nibble per byte): bytes 0, 1 or 2, 3.
__device__ inline f16x2 byte_pair(uint32_t w, int hi) {
    return __builtin_bit_cast(f16x2, __builtin_amdgcn_perm(0x64646464u, w, hi ? 0x04030402u : 0x04010400u));
}
// 1024 + 16 q -> q - OFF, exactly: a code where it lies, four bits up, costs no shift.  s16: 1/16.
template <int OFF>
__device__ inline f16x2 sixteenth(f16x2 u, f16x2 s16) {
    const _Float16 c = -(_Float16)(64 + OFF);
    return __builtin_elementwise_fma(u, s16, (f16x2){c, c});
}
// Nibbles i and i + 4 of a word, less OFF.
template <int OFF>
__device__ inline f16x2 code_pair(uint32_t w, int i, uint32_t f1024, f16x2 s16) {
    if (i >= 2) w >>= 8;
    if (i & 1) return sixteenth<OFF>(as_f16x2(and_or(w, 0x00F000F0u, f1024)), s16);
    return as_f16x2(and_or(w, 0x000F000Fu, f1024)) - (_Float16)(1024 + OFF);
}
// 1024 + q -> the value: (q - 8) d, or q d + m with one rounding.  Both subtractions are exact.
template <bool Q41>
__device__ inline f16x2 code_value(f16x2 u, f16x2 d, f16x2 m) {
    if constexpr (Q41) {
        const f16x2 c = u - (_Float16)1024.0f;
        return __builtin_elementwise_fma(c, d, m);
    } else {
        const f16x2 c = u - (_Float16)1032.0f;
        return c * d;
    }
}
__device__ inline uint32_t pack_f16(float a, float b) { return __builtin_bit_cast(uint32_t, f16x2{(_Float16)a, (_Float16)b}); }
__device__ inline uint32_t pack_bf16(float a, float b) {
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, bf16x2{(__bf16)a, (__bf16)b});
}

// Queries as fp16: a row's values times 2^query_shift, which puts the largest into [2^14, 2^15) (subnormal bf16 numbers get as
// far as 2^141 takes them, and all of them are exact then).  The others keep all their bits down to 2^-14, and are off by
// 2^-39 of the largest at most below that.  The factor is taken back in the scale of the scores.
__device__ inline uint32_t largest_bf16(u32x4 v) {   // bits, without the sign
    uint32_t big = 0;
#pragma unroll
    for (int i = 0; i < 4; i++) big = max(big, max(v[i] & 0x7FFFu, (v[i] >> 16) & 0x7FFFu));
    return big;
}
__device__ inline int query_shift(uint32_t big) { return 141 - (int)(big >> 7); }   // exponent bits of bf16: value < 2^(e - 126)
// In the order of a K word's nibble pairs: 0, 4, 1, 5, 2, 6, 3, 7.
__device__ inline f16x8 query_f16(u32x4 v, int up) {
    float f[8];
#pragma unroll
    for (int i = 0; i < 4; i++) {
        f[2 * i] = ldexpf(__uint_as_float(v[i] << 16), up);
        f[2 * i + 1] = ldexpf(__uint_as_float(v[i] & 0xFFFF0000u), up);
    }
    return __builtin_bit_cast(f16x8, (u32x4){pack_f16(f[0], f[4]), pack_f16(f[1], f[5]), pack_f16(f[2], f[6]), pack_f16(f[3], f[7])});
}

// Probabilities are held as 2^(x - ref): at most 2^15, the top of fp16, and 2^7 when ref is set, so that ref moves
// seldom and a probability keeps all of fp16's bits down to 2^-21 of the largest.
constexpr float kRefBelow = 7.0f, kRefMost = 15.0f;

// Partial results of a sequence that is shared out: [slot][cols][dim] sums, then [slot][cols] (reference, sum of p).
struct Partials {
    float* o;
    float* ml;
    int dim, cols;
    __device__ explicit Partials(const AttnArgs& a)
        : o(reinterpret_cast<float*>(a.ws)), ml(o + (int64_t)a.slots * a.tile_cols * a.dim), dim(a.dim), cols(a.tile_cols) {}
    __device__ float* sums(int slot, int col) const { return o + ((int64_t)slot * cols + col) * dim; }
    __device__ float* stat(int slot, int col) const { return ml + ((int64_t)slot * cols + col) * 2; }
    // (at most 2^17 columns of 256 channels: offsets fit 32 bits)
    __device__ f32x4 read(int slot, int col, int ch) const {
        return load_at<f32x4>((global_bytes)(uintptr_t)o, (uint32_t)(((slot * cols + col) * dim + ch) * 4));
    }
    __device__ f32x2 read_stat(int slot, int col) const {
        return load_at<f32x2>((global_bytes)(uintptr_t)ml, (uint32_t)((slot * cols + col) * 8));
    }
};
__host__ __device__ inline int64_t partial_bytes(int slots, int cols, int dim) { return (int64_t)slots * cols * (dim + 2) * 4; }

// The query column of a tile: row within the sequence and query head, or no column.
__device__ inline bool tile_col(const AttnArgs& a, const TileShape& ts, int tile, int col, int n, int* row, int* head) {
    if (ts.ht == 1) {
        const int r = col / a.group;
        *row = tile * ts.rows + r;
        *head = col - r * a.group;
        return r < ts.rows && *row < n;
    }
    *row = tile / ts.ht;
    *head = (tile - *row * ts.ht) * a.tile_cols + col;
    return *head < a.group;
}

}  // namespace wq
