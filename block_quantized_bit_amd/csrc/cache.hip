// cache.hip -- keys and values quantized as they are written into a 4-bit cache, and read back.
//
// Each block of 32 channels of one token of one head is quantized by the format's rule for a weight block (q4_0: d =
// fp16(x_big / -8), q = clamp(rint(x / d), -8, 7) + 8, x^ = (q - 8) d; q4_1: d = fp16((max - min) / 15), m = fp16(min),
// q = clamp(rint((x - m) / d), 0, 15), x^ = q d + m), after clamping x to +-32768.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "cache_device.h"
#include "wq_device.h"
#include "wq_launch.h"

namespace wq {

namespace {

typedef uint16_t u16x8 __attribute__((ext_vector_type(8)));
typedef uint16_t u16x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

template <bool F32>
__device__ inline void load8(const void* p, int64_t i, float v[8]) {
    if constexpr (F32) {
        const f32x4* q = reinterpret_cast<const f32x4*>(static_cast<const float*>(p) + i);
        const f32x4 a = q[0], b = q[1];
#pragma unroll
        for (int j = 0; j < 4; j++) {
            v[j] = a[j];
            v[4 + j] = b[j];
        }
    } else {
        const u16x8 a = *reinterpret_cast<const u16x8*>(static_cast<const uint16_t*>(p) + i);
#pragma unroll
        for (int j = 0; j < 8; j++) v[j] = bf16_value(a[j]);
    }
}

template <bool F32>
__device__ inline void store8(void* p, int64_t i, const float v[8]) {
    if constexpr (F32) {
        f32x4* q = reinterpret_cast<f32x4*>(static_cast<float*>(p) + i);
        q[0] = f32x4{v[0], v[1], v[2], v[3]};
        q[1] = f32x4{v[4], v[5], v[6], v[7]};
    } else {
        u16x8 a;
#pragma unroll
        for (int j = 0; j < 8; j++) a[j] = __builtin_bit_cast(uint16_t, (__bf16)v[j]);
        *reinterpret_cast<u16x8*>(static_cast<uint16_t*>(p) + i) = a;
    }
}

// Lane ^ 1, lane ^ 2.
template <int X>
__device__ inline uint32_t quad_xor(uint32_t v) {
    return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, X == 1 ? 0xB1 : 0x4E, 0xF, 0xF, true);
}
template <int X>
__device__ inline float quad_xor(float v) { return __uint_as_float(quad_xor<X>(__float_as_uint(v))); }

// Quantizes a block of 32 held by 4 neighbouring lanes (8 values each, in lane order).  Returns the 8 codes, nibble n =
// value n; d, m: fp16 bits (m only for q4_1).
//
// The codes are rint of the correctly rounded quotients RN(x / d), in 3 instructions a value in place of a division's 10
// (and d itself likewise from (max - min) / 15): with r = 1/d to 1 ulp, q = RN(x r) is (x / d)(1 + a), |a| < 2^-21, and
// q + r RN(x - d q) is x / d to 2^-44 before its rounding.  A tie of the rounding to 24 bits is mid d = x with mid of 25
// bits and d of at most 11: unless it is met exactly, x / d is at least 2^-36 away from it, so the corrected quotient
// rounds to the same side.  (Where the remainder underflows, the quotient is far below 1/2.)  d = 0: r = 0 gives the code
// of 0.
__device__ inline float corrected_quotient(float x, float d, float r) {
    const float q = x * r;
    return fmaf(fmaf(-q, d, x), r, q);
}
template <bool Q41>
__device__ inline uint32_t quantize_block(float v[8], uint16_t* d, uint16_t* m) {
#pragma unroll
    for (int j = 0; j < 8; j++) v[j] = __builtin_amdgcn_fmed3f(v[j], -kCacheLimit, kCacheLimit);   // a NaN becomes the lesser, -32768
    float low;
    if constexpr (Q41) {
        float lo = v[0], hi = v[0];
#pragma unroll
        for (int j = 1; j < 8; j++) {
            lo = fminf(lo, v[j]);
            hi = fmaxf(hi, v[j]);
        }
        lo = fminf(lo, quad_xor<1>(lo));
        hi = fmaxf(hi, quad_xor<1>(hi));
        lo = fminf(lo, quad_xor<2>(lo));
        hi = fmaxf(hi, quad_xor<2>(hi));
        *d = f16_sat_bits(corrected_quotient(hi - lo, 15.0f, 1.0f / 15.0f));
        *m = f16_sat_bits(lo);
        const float mu = f16_value(*m);
#pragma unroll
        for (int j = 0; j < 8; j++) v[j] -= mu;
        low = 0.0f;
    } else {
        float big = v[0];                                    // the first of the largest magnitude
#pragma unroll
        for (int j = 1; j < 8; j++) big = fabsf(v[j]) > fabsf(big) ? v[j] : big;
        const float o1 = quad_xor<1>(big);                   // the other lane's values come first where the bit is set
        big = fabsf(o1) > fabsf(big) || ((threadIdx.x & 1) && fabsf(o1) == fabsf(big)) ? o1 : big;
        const float o2 = quad_xor<2>(big);
        big = fabsf(o2) > fabsf(big) || ((threadIdx.x & 2) && fabsf(o2) == fabsf(big)) ? o2 : big;
        *d = f16_sat_bits(big * -0.125f);
        *m = 0;
        low = -8.0f;
    }
    const float delta = f16_value(*d), r = delta != 0.0f ? __builtin_amdgcn_rcpf(delta) : 0.0f;
    float c[8];
#pragma unroll
    for (int j = 0; j < 8; j++) {
        const float q = corrected_quotient(v[j], delta, r);
        c[j] = rintf(__builtin_amdgcn_fmed3f(q, low, low + 15.0f));   // (the limits are whole: before or after rint is the same)
    }
    // four codes as one whole number
    uint32_t w[2];
#pragma unroll
    for (int k = 0; k < 2; k++)
        w[k] = (uint32_t)fmaf(4096.0f, c[4 * k + 3], fmaf(256.0f, c[4 * k + 2], fmaf(16.0f, c[4 * k + 1], c[4 * k] - low * 4369.0f)));
    return w[0] | (w[1] << 16);
}

// Four nibbles to the low halves of four bytes, and back.
__device__ inline uint32_t spread4(uint32_t x) {
    x = (x | (x << 8)) & 0x00FF00FFu;
    return (x | (x << 4)) & 0x0F0F0F0Fu;
}
__device__ inline uint32_t gather4(uint32_t x) {   // (bytes are below 16)
    x = (x | (x >> 4)) & 0x00FF00FFu;
    return (x | (x >> 8)) & 0x0000FFFFu;
}
// Rows and columns of a 4 x 4 byte square exchanged.
__device__ inline void transpose4(uint32_t (&w)[4]) {
    const uint32_t a = __builtin_amdgcn_perm(w[1], w[0], 0x05010400u), b = __builtin_amdgcn_perm(w[1], w[0], 0x07030602u);
    const uint32_t c = __builtin_amdgcn_perm(w[3], w[2], 0x05010400u), d = __builtin_amdgcn_perm(w[3], w[2], 0x07030602u);
    w[0] = __builtin_amdgcn_perm(c, a, 0x05040100u);
    w[1] = __builtin_amdgcn_perm(c, a, 0x07060302u);
    w[2] = __builtin_amdgcn_perm(d, b, 0x05040100u);
    w[3] = __builtin_amdgcn_perm(d, b, 0x07060302u);
}

// A thread takes 8 channels of four neighbouring tokens of one head, whose place in a unit is whole words (K), words of
// one byte per token (V) and 8 bytes of scales: tokens 4 k .. 4 k + 3 of a sequence, as many of them as are the call's.
struct GroupCount {
    const Seqs& s;
    int log2;             // tokens per group: 4, or 32 for whole units
    __device__ uint32_t operator()(int b) const {
        int r0, r1;
        seq_rows(s, b, &r0, &r1);
        if (r0 == r1) return 0;
        const int64_t p0 = (int64_t)s.len[b] - (r1 - r0);
        return (uint32_t)(((p0 + (r1 - r0) - 1) >> log2) - (p0 >> log2) + 1);
    }
};
struct Group {
    int seq, h, b, g;     // sequence, head, 32-channel block, 8 channels of it
    int64_t row;          // of token 0 of the group (the call's rows are row + i, i in [first, end))
    int first, end;
    int64_t token;        // of i = 0; may be below 0
};
// per_row: threads per group; false: no work for this thread.
__device__ inline bool thread_group(const Seqs& s, int nb, int per_row, int groups_per_block, Group* q) {
    const int in_block = groups_per_block > 1 ? threadIdx.x / (unsigned)per_row : 0;
    const int in = threadIdx.x - in_block * per_row + blockIdx.y * blockDim.x;
    const uint32_t first = blockIdx.x * groups_per_block;
    uint32_t before;
    int seq, r0, r1;
    if (s.row_start) {
        const GroupCount count{s, 2};
        seq = SeqTotals(s.batch, count).find(first, &before);
        if (seq < 0) return false;
        if (in >= per_row || in_block >= groups_per_block) return false;
        uint32_t n = count(seq);
        while (first + in_block - before >= n) {
            before += n;
            if (++seq >= s.batch) return false;
            n = count(seq);
        }
    } else {
        if (in >= per_row || in_block >= groups_per_block) return false;
        seq = before = first + in_block;
        if (seq >= s.batch) return false;
    }
    seq_rows(s, seq, &r0, &r1);
    const int64_t p0 = (int64_t)s.len[seq] - (r1 - r0), t = ((p0 >> 2) + (first + in_block - before)) * 4;
    q->seq = seq;
    q->token = t;
    q->row = r0 + (t - p0);
    q->first = t < p0 ? (int)(p0 - t) : 0;
    q->end = t + 4 - p0 > r1 - r0 ? (int)(p0 + (r1 - r0) - t) : 4;
    const int c8 = nb * 4, h = in / (unsigned)c8, cg = in - h * c8;
    q->h = h;
    q->b = cg >> 2;
    q->g = cg & 3;
    return true;
}

}  // namespace

// 8 channels of the group's tokens [first, end): codes and scales.  A row that is not the call's is read as its neighbour
// that is.
struct GroupCodes {
    uint32_t w[4];
    uint16_t d[4], m[4];
};
template <bool Q41, bool F32>
__device__ inline GroupCodes quantize_group(const void* src, int64_t ld, int64_t row, int col, int first, int end) {
    float x[4][8];
#pragma unroll
    for (int i = 0; i < 4; i++) load8<F32>(src, (row + max(first, min(i, end - 1))) * ld + col, x[i]);
    GroupCodes c;
#pragma unroll
    for (int i = 0; i < 4; i++) c.w[i] = quantize_block<Q41>(x[i], &c.d[i], &c.m[i]);
    return c;
}
// V's bytes: channels 8 g + n of a lane's codes are the low nibbles of the bytes for g < 2, and the high ones of the lane
// g ^ 2's channels: a lane makes the bytes of channels 8 (g & 1) + 4 (g >> 1) + 0..3, one token each.
__device__ inline int v_first(int g) { return 8 * (g & 1) + 4 * (g >> 1); }
__device__ inline void codes_to_bytes(int g, uint32_t (&w)[4]) {
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const uint32_t other = quad_xor<2>(w[i]);
        const uint32_t lo = g < 2 ? w[i] & 0xFFFFu : other >> 16, hi = g < 2 ? other & 0xFFFFu : w[i] >> 16;
        w[i] = spread4(lo) | (spread4(hi) << 4);
    }
}
// All four tokens, from place u0 (a multiple of 4) of the unit's K or V part at `to` (memory or LDS).
template <bool Q41, int NB>
__device__ inline void store_whole(GroupCodes& c, bool is_v, int u0, int b, int g, uint8_t* to) {
    constexpr int dim = 32 * NB;
    if (g == 0) {
        uint16_t* const sc = reinterpret_cast<uint16_t*>(to + 16 * dim) + cache_scale(NB, u0, b);
        *reinterpret_cast<u16x4*>(sc) = (u16x4){c.d[0], c.d[1], c.d[2], c.d[3]};
        if constexpr (Q41) *reinterpret_cast<u16x4*>(sc + dim) = (u16x4){c.m[0], c.m[1], c.m[2], c.m[3]};
    }
    if (is_v) {
        codes_to_bytes(g, c.w);
        transpose4(c.w);
    }
#pragma unroll
    for (int i = 0; i < 4; i++)
        *reinterpret_cast<uint32_t*>(to + (is_v ? cache_v_byte(NB, u0, b, v_first(g) + i) : cache_k_word(NB, u0 + i, b, g))) = c.w[i];
}
// The tokens [first, end) of the four, and no byte of the others.
template <bool Q41, int NB>
__device__ inline void store_some(GroupCodes& c, bool is_v, int u0, int b, int g, int first, int end, uint8_t* to) {
    constexpr int dim = 32 * NB;
    uint16_t* const sc = reinterpret_cast<uint16_t*>(to + 16 * dim) + cache_scale(NB, u0, b);
    if (is_v) codes_to_bytes(g, c.w);
#pragma unroll
    for (int i = 0; i < 4; i++) {
        if (i < first || i >= end) continue;
        if (g == 0) {
            sc[i] = c.d[i];
            if constexpr (Q41) sc[dim + i] = c.m[i];
        }
        if (is_v) {
#pragma unroll
            for (int n = 0; n < 4; n++) to[cache_v_byte(NB, u0 + i, b, v_first(g) + n)] = (uint8_t)(c.w[i] >> (8 * n));
        } else {
            *reinterpret_cast<uint32_t*>(to + cache_k_word(NB, u0 + i, b, g)) = c.w[i];
        }
    }
}

// Few rows per sequence: a thread takes 8 channels of four tokens, K or V (blockIdx.z), so that a whole group's words and
// scales are whole stores.  Bound by the way to memory and back (lengths, pages, rows): one row of 20 heads of 64 3.3-3.7 us,
// 96 sequences of one row, 8 heads of 128, 4.2-4.9 us.
template <bool Q41, bool F32, int NB>
__global__ __launch_bounds__(256) void k_cache_write(Seqs s, int per_row, int groups_per_block, const void* __restrict__ k, int64_t ldk,
                                                     const void* __restrict__ v, int64_t ldv, uint8_t* __restrict__ cache) {
    constexpr int dim = 32 * NB;
    Group q;
    if (!thread_group(s, NB, per_row, groups_per_block, &q)) return;
    const int first = max(q.first, q.token < 0 ? (int)min((int64_t)4, -q.token) : 0);
    if (first >= q.end || q.token >= (int64_t)s.table_ld * s.page) return;   // (the capacity is a multiple of 4)
    const int token = q.token < 0 ? 0 : (int)q.token;
    const int64_t at = seq_unit(s, q.seq, q.h, token);
    if (at < 0) return;
    const bool is_v = blockIdx.z;
    GroupCodes c = quantize_group<Q41, F32>(is_v ? v : k, is_v ? ldv : ldk, q.row, q.h * dim + q.b * 32 + q.g * 8, first, q.end);
    uint8_t* const to = cache + at + (is_v ? cache_half_bytes(Q41, dim) : 0);
    const int u0 = token % s.page % kUnit;   // (below 0: only tokens of a group that ends before the first one)
    if (first == 0 && q.end == 4) store_whole<Q41, NB>(c, is_v, u0, q.b, q.g, to);
    else store_some<Q41, NB>(c, is_v, u0, q.b, q.g, first, q.end, to);
}

// Many rows per sequence: a workgroup makes one unit of one head.  In the unit's order a lane's results are
// 4-byte pieces 16 bytes apart, so a whole unit is put together in LDS and written in 16-byte pieces side by side.
// Bound by memory, with the quantization's arithmetic close behind: 36176 rows of 8 heads of 128, bf16 to q4_1 (195 MB)
// 44 us, 4.4 TB/s; 4 x 1500 rows of 20 heads of 64, fp32 to q4_0 (70 MB) 14 us, 4.9 TB/s.  Written from registers,
// as k_cache_write does, the first took 62 us.
template <bool Q41, bool F32, int NB>
__global__ __launch_bounds__(NB == 3 ? 128 : 32 * NB) void k_cache_write_units(Seqs s, const void* __restrict__ k, int64_t ldk,
                                                                               const void* __restrict__ v, int64_t ldv,
                                                                               uint8_t* __restrict__ cache) {
    constexpr int dim = 32 * NB, half = cache_half_bytes(Q41, dim), threads = NB == 3 ? 128 : 32 * NB;
    __shared__ __attribute__((aligned(16))) uint8_t lds[2 * half];
    uint32_t before;
    const int seq = SeqTotals(s.batch, GroupCount{s, 5}).find(blockIdx.x, &before);
    if (seq < 0) return;
    const SeqRows r = seq_rows_uniform(s, seq);
    const int r0 = r.r0, r1 = r.r1;
    const int64_t p0 = (int64_t)r.len - (r1 - r0), t0 = ((p0 >> 5) + (blockIdx.x - before)) * kUnit;   // the unit's token 0
    if (t0 < 0 || t0 >= (int64_t)s.table_ld * s.page) return;   // (units before the first token, past the last page)
    const int h = blockIdx.y;
    const int gi = threadIdx.x / (4 * NB), cg = threadIdx.x - gi * (4 * NB), b = cg >> 2, g = cg & 3;
    const int64_t t = t0 + 4 * gi, lo = p0 > 0 ? p0 : 0, hi = p0 + (r1 - r0);
    const int first = t < lo ? (int)min((int64_t)4, lo - t) : 0, end = t + 4 > hi ? (int)max((int64_t)0, hi - t) : 4;
    const bool whole = t0 >= lo && t0 + kUnit <= hi;
    const int64_t at = seq_unit_uniform(s, seq, h, (int)t0);
    if (at < 0) return;
    uint8_t* const to = cache + at;
    if (gi < 8 && first < end) {
        const int64_t row = r0 + (t - p0);
        const int col = h * dim + b * 32 + g * 8;
        GroupCodes ck = quantize_group<Q41, F32>(k, ldk, row, col, first, end);
        GroupCodes cv = quantize_group<Q41, F32>(v, ldv, row, col, first, end);
        if (whole) {
            store_whole<Q41, NB>(ck, false, 4 * gi, b, g, lds);
            store_whole<Q41, NB>(cv, true, 4 * gi, b, g, lds + half);
        } else {
            store_some<Q41, NB>(ck, false, 4 * gi, b, g, first, end, to);
            store_some<Q41, NB>(cv, true, 4 * gi, b, g, first, end, to + half);
        }
    }
    if (!whole) return;
    __syncthreads();
    typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
    for (int i = threadIdx.x; i < 2 * half / 16; i += threads) reinterpret_cast<u32x4*>(to)[i] = reinterpret_cast<const u32x4*>(lds)[i];
}

// A thread takes 8 channels of four tokens, K or V.  36176 rows of 8 heads of 128, q4_1 to bf16 (195 MB), 40 us, 4.8 TB/s:
// near the copy's 5.1, with the vector unit issuing in 87 % of the cycles.  Fewer rows are bound by each thread's chain of row
// starts, lengths, table and unit: 4 x 1500 rows of 20 heads of 64, q4_0 to bf16 (39 MB), 13-15 us, where the bytes take 7.8.
template <bool Q41, bool F32, int NB>
__global__ __launch_bounds__(256) void k_cache_read(Seqs s, int per_row, int groups_per_block, const uint8_t* __restrict__ cache,
                                                    void* __restrict__ k, int64_t ldk, void* __restrict__ v, int64_t ldv) {
    constexpr int dim = 32 * NB, half = cache_half_bytes(Q41, dim);
    Group q;
    if (!thread_group(s, NB, per_row, groups_per_block, &q)) return;
    const int64_t cap = (int64_t)s.table_ld * s.page;
    const int64_t at = q.token <= -4 || q.token >= cap ? -1 : seq_unit(s, q.seq, q.h, (int)(q.token < 0 ? 0 : q.token));
    const bool is_v = blockIdx.z;
    const int c0 = 8 * (q.g & 1) + 4 * (q.g >> 1);
    uint32_t w[4] = {};
    u16x4 d = {}, m = {};
    if (at >= 0) {
        const int u0 = q.token < 0 ? 0 : (int)(q.token % s.page) % kUnit;
        const uint8_t* const from = cache + at + (is_v ? half : 0);
#pragma unroll
        for (int i = 0; i < 4; i++)
            w[i] = *reinterpret_cast<const uint32_t*>(from + (is_v ? cache_v_byte(NB, u0, q.b, c0 + i) : cache_k_word(NB, u0 + i, q.b, q.g)));
        const uint16_t* const sc = reinterpret_cast<const uint16_t*>(from + 16 * dim) + cache_scale(NB, u0, q.b);
        d = *reinterpret_cast<const u16x4*>(sc);
        if constexpr (Q41) m = *reinterpret_cast<const u16x4*>(sc + dim);
    }
    if (is_v) {
        transpose4(w);   // now row i's bytes of channels c0 .. c0 + 3
        // to this lane's 8 channels: four nibbles of its own bytes and four of lane g ^ 2's
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const uint32_t lo = gather4(w[i] & 0x0F0F0F0Fu), hi = gather4((w[i] >> 4) & 0x0F0F0F0Fu);
            const uint32_t own = q.g < 2 ? lo : hi, got = quad_xor<2>(q.g < 2 ? hi : lo);
            w[i] = q.g < 2 ? own | (got << 16) : got | (own << 16);
        }
    }
    void* const dst = is_v ? v : k;
    const int64_t ld = is_v ? ldv : ldk;
#pragma unroll
    for (int i = 0; i < 4; i++) {
        if (i < q.first || i >= q.end) continue;
        // no token: codes and scales that give +0
        const bool none = at < 0 || q.token + i < 0;
        const uint32_t codes = none ? 0x88888888u : w[i], lo = codes & 0x0F0F0F0Fu, hi = (codes >> 4) & 0x0F0F0F0Fu;
        const float delta = none ? 0.0f : f16_value(d[i]), mu = none ? 0.0f : f16_value(m[i]);
        float x[8];
#pragma unroll
        for (int n = 0; n < 8; n++) {
            const float c = (float)(((n & 1 ? hi : lo) >> (8 * (n >> 1))) & 0xFFu);
            if constexpr (Q41) x[n] = fmaf(c, delta, mu);   // (c d is exact: one rounding either way)
            else x[n] = (c - 8.0f) * delta;
        }
        store8<F32>(dst, (q.row + i) * ld + q.h * dim + q.b * 32 + q.g * 8, x);
    }
}

namespace {

// What a token's row of one head has in a unit, in pieces: V's bytes of 2 channels, K's words of 8, and the scales.  A
// piece of the token at place u is at base[u / 16] + (u / 4 % 4) row[u / 16] + (u % 4) step[u / 16].
template <bool Q41, int NB>
struct Pieces {
    static constexpr int dim = 32 * NB, half = cache_half_bytes(Q41, dim), scales = NB * (Q41 ? 2 : 1);
    static constexpr int bytes = 16 * NB, words = 4 * NB, all = bytes + words + 2 * scales, threads = (all + 63) / 64 * 64;
    int size, base[2], row[2], step[2];

    __device__ explicit Pieces(int i) {
        const auto at = [&](int u) {
            if (size == 1) return half + cache_v_byte(NB, u, i >> 4, i & 15);
            if (size == 4) return cache_k_word(NB, u, i >> 2, i & 3);
            const int v = i >= scales ? 1 : 0, s = i - v * scales, m = s >= NB ? 1 : 0;
            return v * half + 16 * dim + m * cache_plane_bytes(dim) + 2 * cache_scale(NB, u, s - m * NB);
        };
        size = i < bytes ? 1 : i < bytes + words ? 4 : 2;
        i -= size == 1 ? 0 : size == 4 ? bytes : bytes + words;
#pragma unroll
        for (int tile = 0; tile < 2; tile++) {
            base[tile] = at(16 * tile);
            row[tile] = at(16 * tile + 4) - base[tile];
            step[tile] = at(16 * tile + 1) - base[tile];
        }
    }
    __device__ int at(int u) const {   // (u is uniform)
        return u < 16 ? base[0] + (u >> 2) * row[0] + (u & 3) * step[0] : base[1] + ((u >> 2) - 4) * row[1] + (u & 3) * step[1];
    }
};

}  // namespace

// The accepted rows of a draft, moved to the places behind its context, a workgroup per sequence, head and pool.  A thread
// has one piece of a row, and moves it for one entry of the path after the other: an entry's source lies behind all places
// that earlier entries were moved to (a path ascends), so whole groups are read before they are written.  Every wave looks the
// entries up for itself, one a lane, and takes them from there.  Bound by its instructions and the way to memory and back
// (path, pages, rows): 256 sequences' 1.7 thousand rows of 8 heads of 128, q4_1, 13 us; one draft in four pools 4.9.
template <bool Q41, int NB>
__global__ __launch_bounds__((Pieces<Q41, NB>::threads)) void k_cache_keep(KeepArgs a) {
    constexpr int at_once = 64, group = 16;   // entries that are looked up together, and moved together
    const Seqs& s = a.s;
    const int b = blockIdx.x, h = blockIdx.y, lane = threadIdx.x & 63;
    uint8_t* const cache = a.cache[blockIdx.z];
    const int32_t* const path = a.path + (int64_t)b * a.path_ld;
    const auto row_at = [&](int j) { return j >= 0 && j < a.path_ld ? path[j] : -1; };
    int i = row_at(lane), last = row_at(lane - 1);   // (requested with the lengths)
    const int count = min(a.count[b], a.path_ld);
    int r0, r1;
    seq_rows(s, b, &r0, &r1);
    const int n = r1 - r0;
    const int64_t pos0 = (int64_t)s.len[b] - n, capacity = (int64_t)s.table_ld * s.page;
    const Pieces<Q41, NB> piece(threadIdx.x);
    const bool has_piece = threadIdx.x < Pieces<Q41, NB>::all;
    int kept = 0;
    for (int j0 = 0; j0 < count; j0 += at_once) {
        // the path ends before an entry that is no row, is not above the one before it, or has no place to be or to go
        const int j = j0 + lane;
        if (j0 > 0) {
            i = row_at(j);
            last = row_at(j - 1);
        }
        int64_t source = -1, target = -1;
        int places = 0;                       // in their units; -1: it is where it belongs
        const int64_t st = pos0 + i, tt = pos0 + j;
        if (j < count && i > last && i >= 0 && i < n && tt >= 0 && st < capacity) {
            source = seq_unit(s, b, h, (int)st);
            target = seq_unit(s, b, h, (int)tt);
            places = st == tt ? -1 : (int)(st % kUnit) | (int)(tt % kUnit) << 8;   // (a page is whole units)
        }
        const uint64_t good = __ballot(source >= 0 && target >= 0);
        const int m = good == ~0ull ? at_once : __builtin_ctzll(~good);
        const auto entry = [&](int64_t v, int k) {
            return (int64_t)((uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(v >> 32), k) << 32 | (uint32_t)__builtin_amdgcn_readlane((int)v, k));
        };
        for (int k0 = 0; k0 < m; k0 += group) {
            uint32_t v[group];
#pragma unroll
            for (int k = 0; k < group; k++) {
                if (k0 + k >= m) break;
                const int where = __builtin_amdgcn_readlane(places, k0 + k);
                if (where < 0 || !has_piece) continue;
                const uint8_t* const p = cache + entry(source, k0 + k) + piece.at(where & 0xFF);
                v[k] = piece.size == 4 ? *reinterpret_cast<const uint32_t*>(p) : piece.size == 2 ? *reinterpret_cast<const uint16_t*>(p) : *p;
            }
#pragma unroll
            for (int k = 0; k < group; k++) {
                if (k0 + k >= m) break;
                const int where = __builtin_amdgcn_readlane(places, k0 + k);
                if (where < 0 || !has_piece) continue;
                uint8_t* const p = cache + entry(target, k0 + k) + piece.at(where >> 8);
                if (piece.size == 4) *reinterpret_cast<uint32_t*>(p) = v[k];
                else if (piece.size == 2) *reinterpret_cast<uint16_t*>(p) = (uint16_t)v[k];
                else *p = (uint8_t)v[k];
            }
        }
        kept += m;
        if (m < at_once) break;
    }
    if (threadIdx.x == 0 && h == 0 && blockIdx.z == 0 && a.want) a.want[b] = (int)max(pos0 + kept, (int64_t)0);
}

namespace {

// Rows per sequence, on average, from which whole units are written.
constexpr int64_t kManyRows = 16;

// Threads per group, groups per workgroup, the launch.
struct Launch {
    int per_row, groups;
    dim3 grid, block;
};
// Units of 32 tokens: n rows touch at most n / 32 + 2.  Threads per workgroup: whole waves.
int64_t unit_bound(const Seqs& s) { return (int64_t)s.rows / kUnit + 2 * (int64_t)std::min(s.rows, s.batch); }
constexpr int unit_threads(int nb) { return nb == 3 ? 128 : 32 * nb; }

Launch group_launch(const Seqs& s, int nb) {
    Launch l;
    l.per_row = s.heads * nb * 4;
    l.groups = std::max(1, 256 / l.per_row);
    const int threads = std::min(256, (l.per_row * l.groups + 63) / 64 * 64);
    // groups of four tokens: n rows touch at most n / 4 + 2
    const int64_t n = s.row_start ? (int64_t)s.rows / 4 + 2 * (int64_t)std::min(s.rows, s.batch) : s.batch;
    l.grid = dim3((unsigned)((n + l.groups - 1) / l.groups), (unsigned)((l.per_row + threads - 1) / threads), 2);   // z: K, V
    l.block = dim3((unsigned)threads);
    return l;
}

template <int NB>
void write_nb(const Seqs& q, bool q41, bool f32, const void* k, int64_t ldk, const void* v, int64_t ldv, uint8_t* cache, hipStream_t s) {
    if (q.row_start && (int64_t)q.rows >= kManyRows * (int64_t)q.batch) {
        const dim3 grid((unsigned)unit_bound(q), (unsigned)q.heads);
        auto f = q41 ? (f32 ? k_cache_write_units<true, true, NB> : k_cache_write_units<true, false, NB>)
                     : (f32 ? k_cache_write_units<false, true, NB> : k_cache_write_units<false, false, NB>);
        hipLaunchKernelGGL(f, grid, dim3(unit_threads(NB)), 0, s, q, k, ldk, v, ldv, cache);
        return;
    }
    const Launch l = group_launch(q, NB);
    auto f = q41 ? (f32 ? k_cache_write<true, true, NB> : k_cache_write<true, false, NB>)
                 : (f32 ? k_cache_write<false, true, NB> : k_cache_write<false, false, NB>);
    hipLaunchKernelGGL(f, l.grid, l.block, 0, s, q, l.per_row, l.groups, k, ldk, v, ldv, cache);
}
template <int NB>
void read_nb(const Seqs& q, bool q41, bool f32, const uint8_t* cache, void* k, int64_t ldk, void* v, int64_t ldv, hipStream_t s) {
    const Launch l = group_launch(q, NB);
    auto f = q41 ? (f32 ? k_cache_read<true, true, NB> : k_cache_read<true, false, NB>)
                 : (f32 ? k_cache_read<false, true, NB> : k_cache_read<false, false, NB>);
    hipLaunchKernelGGL(f, l.grid, l.block, 0, s, q, l.per_row, l.groups, cache, k, ldk, v, ldv);
}

}  // namespace

// A launch has fewer than 2^32 threads along x, whichever kernel the call takes.  (The workgroups fit 32 bits before that.)
bool cache_fits(const Seqs& q, int dim) {
    const Launch l = group_launch(q, dim / 32);
    const int64_t most = (int64_t(1) << 32) - 1;
    return (int64_t)l.grid.x * l.block.x <= most && unit_bound(q) * unit_threads(dim / 32) <= most;
}

hipError_t launch_cache_write(const Seqs& q, bool q41, int dim, bool f32, const void* k, int64_t ldk, const void* v, int64_t ldv,
                              uint8_t* cache, hipStream_t s) {
    switch (dim) {
    case 64: write_nb<2>(q, q41, f32, k, ldk, v, ldv, cache, s); break;
    case 96: write_nb<3>(q, q41, f32, k, ldk, v, ldv, cache, s); break;
    case 128: write_nb<4>(q, q41, f32, k, ldk, v, ldv, cache, s); break;
    default: write_nb<8>(q, q41, f32, k, ldk, v, ldv, cache, s); break;
    }
    return hipGetLastError();
}

template <int NB>
void keep_nb(const KeepArgs& a, bool q41, hipStream_t s) {
    const dim3 grid((unsigned)a.s.batch, (unsigned)a.s.heads, (unsigned)a.caches);
    if (q41) hipLaunchKernelGGL((k_cache_keep<true, NB>), grid, dim3(Pieces<true, NB>::threads), 0, s, a);
    else hipLaunchKernelGGL((k_cache_keep<false, NB>), grid, dim3(Pieces<false, NB>::threads), 0, s, a);
}

hipError_t launch_cache_keep(const KeepArgs& a, bool q41, int dim, hipStream_t s) {
    switch (dim) {
    case 64: keep_nb<2>(a, q41, s); break;
    case 96: keep_nb<3>(a, q41, s); break;
    case 128: keep_nb<4>(a, q41, s); break;
    default: keep_nb<8>(a, q41, s); break;
    }
    return hipGetLastError();
}

hipError_t launch_cache_read(const Seqs& q, bool q41, int dim, bool f32, const uint8_t* cache, void* k, int64_t ldk, void* v,
                             int64_t ldv, hipStream_t s) {
    switch (dim) {
    case 64: read_nb<2>(q, q41, f32, cache, k, ldk, v, ldv, s); break;
    case 96: read_nb<3>(q, q41, f32, cache, k, ldk, v, ldv, s); break;
    case 128: read_nb<4>(q, q41, f32, cache, k, ldk, v, ldv, s); break;
    default: read_nb<8>(q, q41, f32, cache, k, ldk, v, ldv, s); break;
    }
    return hipGetLastError();
}

}  // namespace wq
