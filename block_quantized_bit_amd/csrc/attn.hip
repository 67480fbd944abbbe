// attn.hip -- attention over the 4-bit cache: y = sum_t softmax_t(scale q . k^_t) v^_t over the tokens a row sees.
//
// One pass over the tokens: with x_t the scores times log2(e), a column holds a reference ref, l = sum 2^(x_t - ref) and
// o = sum 2^(x_t - ref) v^_t in fp32; where a score passes ref by too much, o and l are scaled to a new one.  Parts of a
// column (waves, workgroups) are joined by y = sum_i 2^(ref_i - ref) o_i / sum_i 2^(ref_i - ref) l_i.  Nothing of the size
// rows x tokens is written, and keys and values are read packed.
//
// Rounded to fp16, because the matrix instructions take 16-bit operands and fp16 has three bits more than bf16: probabilities
// (2^(x - ref), at most 2^15; the sum that divides is of the unrounded ones), values, queries (times a power of two per row and
// head, mostly exact), and keys, but for q4_0 in calls with few rows, whose codes are exact there.  Each is off by half a step,
// 2^-11 of itself.  In calls with ordinary scores the outputs' error is that of their own rounding to bf16 (0.0017 of their
// magnitude against 64 bits, as for the same computed in fp32).
#include <hip/hip_runtime.h>

#include <algorithm>

#include "attn_common.h"

namespace wq {

// ---------------------------------------------------------------------------------------------------------------
// Few columns per sequence (single tokens, drafted tokens): tiles of 16 columns, every wave its own units.
// ---------------------------------------------------------------------------------------------------------------

// What bounds it: with one row per sequence a group's heads share every unit that is read, at 2 x 16 columns of products
// per 4.5 or 5 bits, so a call with enough tokens is bound by memory, and a short one by the way to memory and back
// (lengths, pages, units, one after the other).  Measured (a copy runs at 5.1 TB/s on the card): 32 sequences
// of 30011 to 32768 tokens, 8 x 5 heads of 128, q4_0 (1.16 GB) 227-233 us with the join, 5.0-5.1 TB/s; one of 131077 tokens,
// 8 x 8 heads (151 MB) 43 us; 16 of 1500 tokens, 20 heads of 64 (35 MB) 16 us, with neither memory (2.1 TB/s) nor the vector
// unit (32 % of the cycles) busy; one of 224 tokens 6 us; 16 x 5 rows that see 4096 tokens, 2 x 8 heads of 256, q4_1 (43 MB)
// 43 us, where three tiles take each unit and their conversions bound it.
// 16 columns, since a group's heads of one token are seldom more; with 32 columns a wave spills, and was slower in all of
// these.
//
// Each wave keeps a ring of units in LDS, filled by loads that go there directly (no registers), so that several units
// per wave are on their way while one is computed on.  The unit is contiguous in the cache and keeps its layout.
template <int NB, bool Q41>
struct UnitRing {
    static constexpr int dim = 32 * NB, half = cache_half_bytes(Q41, dim), bytes = 2 * half, plane = cache_plane_bytes(dim);
    static constexpr int full = bytes / 1024, rest = bytes % 1024 / 16;   // whole 1 KiB loads, lanes of a last one
    static constexpr int loads = full + (rest ? 1 : 0);
};

// The request for one unit: 16 bytes a lane, to LDS at m0 + offset + 16 lane.  The compiler does not see the write to LDS; the
// memory clobbers keep LDS reads in order with it, and the counted waits below are the only ones there are for it.  Five
// waiting states (s_nop 4) are what a load's address needs that the vector unit wrote: the compiler counts none before written
// assembly.
template <int BYTES>
__device__ inline void request_unit(const uint8_t* src, uint32_t lds) {
    const int lane = threadIdx.x & 63;
    const uint32_t off = lane * 16;
    constexpr int full = BYTES / 1024, rest = BYTES % 1024 / 16;
#pragma unroll
    for (int c = 0; c < full + (rest ? 1 : 0); c++) {
        if (c < full || lane < rest) {
            asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tglobal_load_lds_dwordx4 %1, %2"
                         :: "s"(lds + c * 1024), "v"(off), "s"(src + c * 1024) : "m0", "memory");
        }
    }
}
template <int N>
__device__ inline void wait_loads() {
    asm volatile("s_waitcnt vmcnt(%0)" :: "n"(N) : "memory");
}
__device__ inline void wait_lds() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }

template <int NB>
__device__ inline void read_words(const uint8_t* p, int lane, uint32_t* w) {
#pragma unroll
    for (int c = 0; c < NB / 2; c++) {
        const u32x4 v = *reinterpret_cast<const u32x4*>(p + c * 1024 + lane * 16);
#pragma unroll
        for (int i = 0; i < 4; i++) w[4 * c + i] = v[i];
    }
    if constexpr (NB % 2) {
        const u32x2 v = *reinterpret_cast<const u32x2*>(p + NB / 2 * 1024 + lane * 8);
        w[2 * NB - 2] = v[0];
        w[2 * NB - 1] = v[1];
    }
}

// Scales of blocks b0 .. b0 + BG - 1 of one tile: [block][token pair].
template <int NB, int BG>
__device__ inline void read_scales(const uint8_t* p, int g, int tile, int b0, uint32_t (&d)[BG][2]) {
    const uint8_t* q = p + ((tile * 4 + g) * NB + b0) * 8;
    if constexpr (NB % 2 == 0) {
#pragma unroll
        for (int b = 0; b < BG; b += 2) {
            const u32x4 v = *reinterpret_cast<const u32x4*>(q + b * 8);
            d[b][0] = v[0];
            d[b][1] = v[1];
            d[b + 1][0] = v[2];
            d[b + 1][1] = v[3];
        }
    } else {
#pragma unroll
        for (int b = 0; b < BG; b++) {
            const u32x2 v = *reinterpret_cast<const u32x2*>(q + b * 8);
            d[b][0] = v[0];
            d[b][1] = v[1];
        }
    }
}

// A column's running softmax and its part of the sums.
template <int NB>
struct ColState {
    f32x4 o[2 * NB];     // channels 16 i + 4 g + 0..3 of column lane % 16
    float ref, l;        // l: this lane's tokens only
};

// What K is multiplied as: q4_0's codes less 8, which fp16 holds exactly, with a block's scale applied to its product in fp32;
// q4_1's values d q + m, rounded to fp16 once.  Either way a product's terms are the keys' own, so its fp32 error follows
// sum |q k^|.  (Terms that only cancel, codes from 128 on against a start of -136 sum q, or m sum q beside q4_1's codes, leave
// errors of the size of the block's scale times sum |q|: a key of 32768 beside a query of nearly zero moved scores of 0.6 by
// 0.1.  They took 223-227 us where this takes 227-233, for 32 sequences of 30011 to 32768 tokens, 8 x 5 heads of 128, q4_0.)
template <int NB, bool Q41, bool MASKED>
__device__ inline void unit_step(const uint8_t* unit, const f16x8 (&qf)[NB], float sl2, int t0, int lo, int hi, int tokens,
                                 uint32_t f1024, f16x2 s16, ColState<NB>* st) {
    using R = UnitRing<NB, Q41>;
    const int lane = threadIdx.x & 63, g = lane >> 4;
    float x[8];
    uint32_t kw[2 * NB];
    read_words<NB>(unit, lane, kw);
#pragma unroll
    for (int tile = 0; tile < 2; tile++) {
        f32x4 s = {0.0f, 0.0f, 0.0f, 0.0f};
        if (NB > 4 && tile) asm volatile("" ::: "memory");
        if constexpr (Q41) {
            // (the lane's words are one token's: 4 (r / 4) + r % 4 of the tile)
            const uint8_t* const sc = unit + 16 * R::dim + ((tile * 4 + ((lane & 15) >> 2)) * NB) * 8 + (lane & 3) * 2;
#pragma unroll
            for (int b = 0; b < NB; b++) {
                const _Float16 d1 = *reinterpret_cast<const _Float16*>(sc + b * 8), m1 = *reinterpret_cast<const _Float16*>(sc + b * 8 + R::plane);
                const f16x2 d = {d1, d1}, m = {m1, m1};
                u32x4 u;
#pragma unroll
                for (int i = 0; i < 4; i++)
                    u[i] = __builtin_bit_cast(uint32_t, __builtin_elementwise_fma(code_pair<0>(kw[tile * NB + b], i, f1024, s16), d, m));
                s = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, u), qf[b], s, 0, 0, 0);
            }
        } else {
            uint32_t kd[NB][2];
            read_scales<NB, NB>(unit + 16 * R::dim, g, tile, 0, kd);
#pragma unroll
            for (int b = 0; b < NB; b++) {
                u32x4 u;
#pragma unroll
                for (int i = 0; i < 4; i++) u[i] = __builtin_bit_cast(uint32_t, code_pair<8>(kw[tile * NB + b], i, f1024, s16));
                const f32x4 p = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, u), qf[b], (f32x4){0, 0, 0, 0}, 0, 0, 0);
                const f16x2 d01 = as_f16x2(kd[b][0]), d23 = as_f16x2(kd[b][1]);
                s[0] = fmaf((float)d01[0], p[0], s[0]);
                s[1] = fmaf((float)d01[1], p[1], s[1]);
                s[2] = fmaf((float)d23[0], p[2], s[2]);
                s[3] = fmaf((float)d23[1], p[3], s[3]);
            }
        }
#pragma unroll
        for (int i = 0; i < 4; i++) x[4 * tile + i] = s[i];
    }
    uint32_t keep[4] = {~0u, ~0u, ~0u, ~0u};    // token pairs that are in the cache: what lies behind them is anything
    float e[8];
#pragma unroll
    for (int j = 0; j < 8; j++) {
        e[j] = fmaf(x[j], sl2, -st->ref);
        if constexpr (MASKED) {
            const int t = t0 + (j >> 2) * 16 + 4 * g + (j & 3);
            e[j] = t >= lo && t < hi ? e[j] : -INFINITY;
            if (t >= tokens) keep[j >> 1] &= (j & 1) ? 0x0000FFFFu : 0xFFFF0000u;
        }
    }
    const float most = fmaxf(fmaxf(fmaxf(e[0], e[1]), fmaxf(e[2], e[3])), fmaxf(fmaxf(e[4], e[5]), fmaxf(e[6], e[7])));
    if (__any(most > kRefMost)) {
        float mx = -INFINITY;
#pragma unroll
        for (int j = 0; j < 8; j++) mx = fmaxf(mx, e[j] == -INFINITY ? -INFINITY : x[j] * sl2);
        mx = fmaxf(mx, __shfl_xor(mx, 16, 64));
        mx = fmaxf(mx, __shfl_xor(mx, 32, 64));
        const float ref = fmaxf(st->ref, mx - kRefBelow);
        const float alpha = ref == st->ref ? 1.0f : exp2_fast(st->ref - ref);
#pragma unroll
        for (int i = 0; i < 2 * NB; i++) st->o[i] *= alpha;
        st->l *= alpha;
        st->ref = ref;
#pragma unroll
        for (int j = 0; j < 8; j++) e[j] = e[j] == -INFINITY ? -INFINITY : fmaf(x[j], sl2, -ref);
    }
    u32x4 p;
#pragma unroll
    for (int j = 0; j < 8; j++) x[j] = exp2_fast(e[j]);
    st->l += ((x[0] + x[1]) + (x[2] + x[3])) + ((x[4] + x[5]) + (x[6] + x[7]));
#pragma unroll
    for (int j = 0; j < 4; j++) p[j] = pack_f16(x[2 * j], x[2 * j + 1]);
    const f16x8 pf = __builtin_bit_cast(f16x8, p);
    // (at most four blocks' scales in registers at a time)
    constexpr int BG = NB > 4 ? 4 : NB;
#pragma unroll
    for (int b0 = 0; b0 < NB; b0 += BG) {
        if (b0 > 0) asm volatile("" ::: "memory");
        uint32_t vw[2 * BG], vd[2][BG][2], vm[2][BG][2];
        read_words<BG>(unit + R::half + b0 * 512, lane, vw);
#pragma unroll
        for (int tile = 0; tile < 2; tile++) {
            read_scales<NB, BG>(unit + R::half + 16 * R::dim, g, tile, b0, vd[tile]);
            if constexpr (Q41) read_scales<NB, BG>(unit + R::half + 16 * R::dim + R::plane, g, tile, b0, vm[tile]);
        }
#pragma unroll
        for (int b = 0; b < BG; b++) {
            u32x4 vlo, vhi;
#pragma unroll
            for (int tile = 0; tile < 2; tile++) {
                const uint32_t w = vw[2 * b + tile], wl = w & 0x0F0F0F0Fu, wh = w & 0xF0F0F0F0u;
#pragma unroll
                for (int i = 0; i < 2; i++) {
                    const uint32_t in = MASKED ? keep[2 * tile + i] : ~0u;
                    const f16x2 d = as_f16x2(vd[tile][b][i] & in);
                    const f16x2 cl = byte_pair(wl, i) - (_Float16)(Q41 ? 1024.0f : 1032.0f), ch = sixteenth<Q41 ? 0 : 8>(byte_pair(wh, i), s16);
                    f16x2 lo2 = cl * d, hi2 = ch * d;
                    if constexpr (Q41) {
                        const f16x2 m = as_f16x2(vm[tile][b][i] & in);
                        lo2 = __builtin_elementwise_fma(cl, d, m);
                        hi2 = __builtin_elementwise_fma(ch, d, m);
                    }
                    vlo[2 * tile + i] = __builtin_bit_cast(uint32_t, lo2);
                    vhi[2 * tile + i] = __builtin_bit_cast(uint32_t, hi2);
                }
            }
            f32x4* const o = st->o + 2 * (b0 + b);
            o[0] = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, vlo), pf, o[0], 0, 0, 0);
            o[1] = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, vhi), pf, o[1], 0, 0, 0);
        }
    }
}

constexpr int kTokenCols = 16;

// Units [*u0, *u0 + return) of a sequence's rows: every tile of it takes all of them.
__device__ inline int span_units(const AttnArgs& a, const SeqInfo& q, int* u0) {
    int u1;
    *u0 = 0;
    if (q.n == 0) return 0;
    row_units(a, q, 0, q.n, u0, &u1);
    return u1 - *u0;
}

// What beginning a tile costs a workgroup (queries, the first requests' way to memory, joining the waves), in units: the
// work that is shared out counts it, so that workgroups with many short sequences end with the others.
constexpr int kTileCost = 8;

// The stretch of the call's work, in units over all (sequence, tile, head), that a workgroup takes: `share` each.
__device__ inline uint32_t work_share(uint32_t total, int workgroups, int least) {
    const uint32_t s = (total + workgroups - 1) / workgroups;
    return s > (uint32_t)least ? s : (uint32_t)least;
}

// The tile that a workgroup began and did not end, for k_attn_join_token: parts 0 if there is none.
struct OpenTile {
    int parts, tile, head, r0, n;
};
__device__ inline OpenTile* open_tile(const AttnArgs& a, int workgroup) {
    return reinterpret_cast<OpenTile*>(a.ws + partial_bytes(a.slots, a.tile_cols, a.dim)) + workgroup;
}

struct SpanWeight {
    const AttnArgs& a;
    TileShape ts;
    __device__ uint32_t operator()(int b) const {
        const SeqInfo q = seq_info(a, b);
        int u0;
        return (uint32_t)(tiles_of(ts, q.n) * a.s.heads * (kTileCost + span_units(a, q, &u0)));
    }
};
struct TokenShare {
    SeqTotals<SpanWeight> t;
    uint32_t total, share;
    __device__ TokenShare(const AttnArgs& a, const TileShape& ts) : t(a.s.batch, SpanWeight{a, ts}) {
        total = t.total();
        share = work_share(total, a.workgroups, a.least_units);
    }
};

// A tile's columns x units [ua, ub) of one head, by the workgroup.  part: where the sums go (null: the tile is whole,
// and y is written).
template <int NB, bool Q41, int NW, int D>
__device__ void token_segment(const AttnArgs& a, const TileShape& ts, const SeqInfo& q, int seq, int tile, int h, int ua, int ub,
                              float* part_o, float* part_ml, uint8_t* lds) {
    constexpr int dim = 32 * NB, ld = dim + 4;
    float* const lds_o = reinterpret_cast<float*>(lds);
    float* const lds_f = lds_o + NW * 16 * ld;
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6), g = lane >> 4, col = lane & 15;
    int row, head;
    const bool valid = tile_col(a, ts, tile, col, q.n, &row, &head);
    const int first = ts.ht == 1 ? tile * ts.rows : tile / ts.ht, last = min(first + ts.rows, q.n) - 1;
    int lo, hi, lo_most, hi_least, x;
    row_tokens(a, q, valid ? row : first, &lo, &hi);
    row_tokens(a, q, first, &x, &hi_least);
    row_tokens(a, q, last, &lo_most, &x);

    constexpr int bytes = UnitRing<NB, Q41>::bytes, loads = UnitRing<NB, Q41>::loads;
    const uint8_t* const ring = lds + wave * D * bytes;
    const uint32_t ring_at = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const uint8_t*)ring;
    const int n = ub > ua + wave ? (ub - ua - wave + NW - 1) / NW : 0;   // this wave's units: ua + wave + NW i
    UnitWalk walk;
    walk.start(a.s, seq, h, ua + wave);
    uint32_t absent = 0;    // bit i % 32: unit i's page is none; its request is then any unit, for the count
    int put = 0, get = 0;   // byte offsets of the slots to fill and to read next
    const auto next = [](int at) { return at + bytes == D * bytes ? 0 : at + bytes; };
    const auto request = [&](int i) {
        request_unit<bytes>(walk.at(a.cache), uniform(ring_at + put));
        put = next(put);
        absent = walk.there ? absent & ~(1u << (i & 31)) : absent | 1u << (i & 31);
        walk.step(NW);
    };
#pragma unroll
    for (int i = 0; i < D - 1; i++)
        if (i < n) request(i);
    u32x4 qv[NB];
    const uint16_t* qp = a.q + (int64_t)(q.r0 + row) * a.ldq + (int64_t)(h * a.group + head) * dim + 8 * g;
#pragma unroll
    for (int b = 0; b < NB; b++) {
        qv[b] = (u32x4){0, 0, 0, 0};
        if (valid) qv[b] = *reinterpret_cast<const u32x4*>(qp + 32 * b);
    }
    uint32_t big = 0;
#pragma unroll
    for (int b = 0; b < NB; b++) big = max(big, largest_bf16(qv[b]));
    big = max(big, (uint32_t)__shfl_xor((int)big, 16, 64));
    big = max(big, (uint32_t)__shfl_xor((int)big, 32, 64));
    const int up = query_shift(big);
    const float sl2 = ldexpf(a.scale_log2, -up);
    f16x8 qf[NB];
#pragma unroll
    for (int b = 0; b < NB; b++) qf[b] = query_f16(qv[b], up);

    const uint32_t f1024 = held(0x64006400u);
    const f16x2 s16 = as_f16x2(held(0x2C002C00u));   // 1/16
    ColState<NB> st;
#pragma unroll
    for (int i = 0; i < 2 * NB; i++) st.o[i] = (f32x4){0, 0, 0, 0};
    st.ref = -FLT_MAX;
    st.l = 0.0f;

    for (int i = 0; i < n; i++) {
        if (i + D - 1 < n) {
            wait_lds();     // unit i - 1's reads, whose slot the request fills
            request(i + D - 1);
            wait_loads<(D - 1) * loads>();
        } else {
            wait_loads<0>();
        }
        const int t0 = (ua + wave + NW * i) * kUnit;
        const bool masked = t0 < lo_most || t0 + kUnit > hi_least;
        if (!(absent >> (i & 31) & 1)) {
            if (masked) unit_step<NB, Q41, true>(ring + get, qf, sl2, t0, lo, hi, q.tokens, f1024, s16, &st);
            else unit_step<NB, Q41, false>(ring + get, qf, sl2, t0, lo, hi, q.tokens, f1024, s16, &st);
        }
        get = next(get);
    }
    __syncthreads();   // the rings' space is the join's now

    // the waves' sums, joined in LDS
    st.l += __shfl_xor(st.l, 16, 64);
    st.l += __shfl_xor(st.l, 32, 64);
    if (lane < 16) {
        lds_f[wave * 16 + lane] = st.ref;
        lds_f[(NW + wave) * 16 + lane] = st.l;
    }
#pragma unroll
    for (int i = 0; i < 2 * NB; i++)
        *reinterpret_cast<f32x4*>(lds_o + (wave * 16 + col) * ld + 16 * i + 4 * g) = st.o[i];
    __syncthreads();
    for (int i = threadIdx.x; i < kTokenCols * (dim / 4); i += NW * 64) {
        const int c = i / (dim / 4), ch = (i - c * (dim / 4)) * 4;
        int r2, h2;
        if (!tile_col(a, ts, tile, c, q.n, &r2, &h2)) continue;
        float ref = lds_f[c];
#pragma unroll
        for (int w = 1; w < NW; w++) ref = fmaxf(ref, lds_f[w * 16 + c]);
        f32x4 o = {0, 0, 0, 0};
        float l = 0.0f;
#pragma unroll
        for (int w = 0; w < NW; w++) {
            const float f = exp2_fast(lds_f[w * 16 + c] - ref);
            l += f * lds_f[(NW + w) * 16 + c];
            o += f * *reinterpret_cast<const f32x4*>(lds_o + (w * 16 + c) * ld + ch);
        }
        if (part_o) {
            *reinterpret_cast<f32x4*>(part_o + c * dim + ch) = o;
            if (ch == 0) {
                part_ml[2 * c] = ref;
                part_ml[2 * c + 1] = l;
            }
        } else {
            const float inv = l != 0.0f ? 1.0f / l : 0.0f;
            const u32x2 y = {pack_bf16(o[0] * inv, o[1] * inv), pack_bf16(o[2] * inv, o[3] * inv)};
            *reinterpret_cast<u32x2*>(a.y + (int64_t)(q.r0 + r2) * a.ldy + (int64_t)(h * a.group + h2) * dim + ch) = y;
        }
    }
    __syncthreads();
}

// Sequences shared out evenly: workgroup i takes units [i share, (i + 1) share) of the call's work, whatever the lengths
// are; a tile that more than one workgroup has a part of is joined by k_attn_join_token.  With `workgroups` 0 every
// workgroup has one whole tile.  (61 sequences of 1 to 8191 tokens, 8 x 4 heads of 128, q4_1: 80 us with 5 for the join,
// 4.0 TB/s; counting what beginning a tile costs took it from 102 us to 81.)
template <int NB, bool Q41, int NW, int D>
__global__ __launch_bounds__(NW * 64) __attribute__((amdgpu_waves_per_eu(2))) void k_attn_token(AttnArgs a) {
    constexpr int ring_bytes = NW * D * UnitRing<NB, Q41>::bytes, join_bytes = NW * 16 * (32 * NB + 4 + 2) * 4;
    __shared__ __attribute__((aligned(16))) uint8_t lds[ring_bytes > join_bytes ? ring_bytes : join_bytes];
    const TileShape ts = tile_shape(kTokenCols, a.group);
    const int heads = a.s.heads;
    if (a.workgroups == 0) {
        const int item = blockIdx.x;
        int seq;
        uint32_t before;
        if (!a.s.row_start) {
            seq = item / (ts.ht * heads);
            before = seq * (ts.ht * heads);
        } else {
            seq = SeqTotals(a.s.batch, TileCount{a, ts}).find(item / heads, &before);
            before *= heads;
        }
        if (seq < 0 || seq >= a.s.batch) return;
        const SeqInfo q = seq_info_uniform(a, seq);
        const int in = item - (int)before, tile = in / heads, h = in - tile * heads;
        const int first = ts.ht == 1 ? tile * ts.rows : tile / ts.ht, end = min(first + ts.rows, q.n);
        if (first >= end) return;
        int u0, u1;
        row_units(a, q, first, end, &u0, &u1);
        token_segment<NB, Q41, NW, D>(a, ts, q, seq, tile, h, u0, u1, nullptr, nullptr, lds);
        return;
    }
    const TokenShare sh(a, ts);
    uint32_t w = blockIdx.x * sh.share, before;
    const uint32_t end = min(w + sh.share, sh.total);
    OpenTile open = {};
    int seq = w < end ? sh.t.find(w, &before) : 0;
    while (w < end) {
        const SeqInfo q = seq_info_uniform(a, seq);
        int u0;
        const int units = span_units(a, q, &u0), span = kTileCost + units;
        const uint32_t items = tiles_of(ts, q.n) * heads;
        while (w < end && w - before < items * span) {
            const int item = (w - before) / span, s0 = (w - before) - item * span, s1 = min((uint32_t)span, s0 + (end - w));
            const int tile = item / heads, h = item - tile * heads;
            float *po = nullptr, *pm = nullptr;
            if (s1 - s0 < span) {
                const Partials p(a);
                const int slot = 2 * blockIdx.x + (s0 > 0 ? 0 : 1);
                po = p.sums(slot, 0);
                pm = p.stat(slot, 0);
                // (the rows' starts are the caller's: whatever they hold, the parts are workgroups)
                if (s0 == 0) open = {(int)(min((w + span - 1) / sh.share, gridDim.x - 1) - blockIdx.x) + 1, tile, h, q.r0, q.n};
            }
            token_segment<NB, Q41, NW, D>(a, ts, q, seq, tile, h, u0 + max(0, s0 - kTileCost), u0 + max(0, s1 - kTileCost), po, pm, lds);
            w += s1 - s0;
        }
        before += items * span;
        seq++;
    }
    if (threadIdx.x == 0) *open_tile(a, blockIdx.x) = open;
}

// Joins the parts of a tile's column: y = sum_i 2^(ref_i - ref) o_i / sum_i 2^(ref_i - ref) l_i.  Every thread sums four
// channels of some of the parts; their sums meet in LDS, in order.  Bound by the way to memory: 5.5 us for 64 columns of 64
// parts of 128 channels.
constexpr int kJoinParts = 512;
struct JoinLds {
    float f[kJoinParts], red[4], sum[1024];
};
template <class F>
__device__ inline void join_column(const AttnArgs& a, const Partials& p, int n, int col, uint16_t* y, F slot, JoinLds& lds) {
    const int tid = threadIdx.x, quads = a.dim / 4, groups = 256 / quads, gr = tid / quads, c = tid - gr * quads;
    float ref = -FLT_MAX, m0[2], l0[2];
    constexpr int ahead = 8;                  // parts requested before their factors are known
    f32x4 early[ahead];
#pragma unroll
    for (int k = 0; k < ahead; k++) {
        const int i = gr + k * groups;
        early[k] = (f32x4){0, 0, 0, 0};
        if (gr < groups && i < n) early[k] = p.read(slot(i), col, 4 * c);
    }
#pragma unroll
    for (int k = 0; k < 2; k++) {
        const int i = tid + 256 * k;
        m0[k] = -FLT_MAX;
        l0[k] = 0.0f;
        if (i < n) {
            const f32x2 st = p.read_stat(slot(i), col);
            m0[k] = st[0];
            l0[k] = st[1];
        }
        ref = fmaxf(ref, m0[k]);
    }
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) ref = fmaxf(ref, __shfl_xor(ref, d, 64));
    __syncthreads();                          // (the last column's reads of lds are done)
    if ((tid & 63) == 0) lds.red[tid >> 6] = ref;
    __syncthreads();
    ref = fmaxf(fmaxf(lds.red[0], lds.red[1]), fmaxf(lds.red[2], lds.red[3]));
    float l = 0.0f;
#pragma unroll
    for (int k = 0; k < 2; k++) {
        const int i = tid + 256 * k;
        const float f = exp2_fast(m0[k] - ref);
        if (i < n) lds.f[i] = f;
        l += i < n ? f * l0[k] : 0.0f;
    }
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) l += __shfl_xor(l, d, 64);
    __syncthreads();
    if ((tid & 63) == 0) lds.red[tid >> 6] = l;
    f32x4 o = {0, 0, 0, 0};
    if (gr < groups) {
#pragma unroll
        for (int k = 0; k < ahead; k++)
            if (gr + k * groups < n) o += lds.f[gr + k * groups] * early[k];
#pragma unroll 4
        for (int i = gr + ahead * groups; i < n; i += groups) o += lds.f[i] * p.read(slot(i), col, 4 * c);
        *reinterpret_cast<f32x4*>(lds.sum + tid * 4) = o;
    }
    __syncthreads();
    if (tid < quads) {
        for (int k = 1; k < groups; k++) o += *reinterpret_cast<const f32x4*>(lds.sum + (k * quads + c) * 4);
        l = (lds.red[0] + lds.red[1]) + (lds.red[2] + lds.red[3]);
        const float inv = l != 0.0f ? 1.0f / l : 0.0f;
        *reinterpret_cast<u32x2*>(y + 4 * c) = (u32x2){pack_bf16(o[0] * inv, o[1] * inv), pack_bf16(o[2] * inv, o[3] * inv)};
    }
}

// The same by a wave, for few parts: no barriers, and a workgroup has four columns at a time (488 tiles of 4 columns, at most
// three parts each: 5.1 us, by workgroups 8.4).
constexpr int kWaveParts = 16;
__device__ inline void join_column_wave(const AttnArgs& a, const Partials& p, int n, int col, uint16_t* y, int slot0) {
    const int lane = threadIdx.x & 63, quads = a.dim / 4, groups = 64 / quads, gr = lane / quads, c = lane - gr * quads;
    const auto slot = [&](int i) { return slot0 + 2 * i + (i == 0); };
    const auto part = [&](int i) {
        return gr < groups && i < n ? p.read(slot(i), col, 4 * c) : (f32x4){0, 0, 0, 0};
    };
    constexpr int ahead = 8;                  // parts requested before their factors are known
    f32x4 early[ahead];
#pragma unroll
    for (int k = 0; k < ahead; k++) early[k] = part(gr + k * groups);
    float m0 = -FLT_MAX, l = 0.0f;
    if (lane < n) {
        const f32x2 st = p.read_stat(slot(lane), col);
        m0 = st[0];
        l = st[1];
    }
    float ref = m0;
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) ref = fmaxf(ref, __shfl_xor(ref, d, 64));
    const float f = exp2_fast(m0 - ref);
    l *= f;
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) l += __shfl_xor(l, d, 64);
    f32x4 o = {0, 0, 0, 0};
#pragma unroll
    for (int k = 0; k < ahead; k++) {
        const float fk = __shfl(f, (gr + k * groups) & 63, 64);
        if (gr + k * groups < n) o += fk * early[k];
    }
    for (int i0 = ahead * groups; i0 < n; i0 += groups) {
        const float fk = __shfl(f, (gr + i0) & 63, 64);
        if (gr + i0 < n) o += fk * part(gr + i0);
    }
    f32x4 sum = o;
    for (int k = 1; k < groups; k++)
#pragma unroll
        for (int i = 0; i < 4; i++) sum[i] += __shfl(o[i], (lane + k * quads) & 63, 64);
    if (lane < quads) {
        const float inv = l != 0.0f ? 1.0f / l : 0.0f;
        *reinterpret_cast<u32x2*>(y + 4 * c) = (u32x2){pack_bf16(sum[0] * inv, sum[1] * inv), pack_bf16(sum[2] * inv, sum[3] * inv)};
    }
}

// Workgroup i: the tile, if there is one, that workgroup i of k_attn_token began and did not end.  WAVES: tiles of few parts
// by waves.  (A kernel of its own: with both ways in it, eight tiles of 64 parts took 6.5 us in place of 5.7.)
template <bool WAVES>
__global__ __launch_bounds__(256) void k_attn_join_token(AttnArgs a) {
    __shared__ __attribute__((aligned(16))) JoinLds lds;
    const TileShape ts = tile_shape(kTokenCols, a.group);
    const int32_t* const d = &open_tile(a, blockIdx.x)->parts;
    const OpenTile t = {read_const(d, 0), read_const(d, 1), read_const(d, 2), read_const(d, 3), read_const(d, 4)};
    if (t.parts == 0) return;
    const Partials p(a);
    // the first part is the one that starts the tile, the others start their workgroups
    const auto slot = [](int i) { return 2 * ((int)blockIdx.x + i) + (i == 0); };
    const bool few = WAVES && t.parts <= kWaveParts;
    for (int col = few ? blockIdx.y * 4 + uniform(threadIdx.x >> 6) : blockIdx.y; col < kTokenCols; col += (few ? 4 : 1) * gridDim.y) {
        int row, head;
        if (!tile_col(a, ts, t.tile, col, t.n, &row, &head)) break;   // columns without a query are the last ones
        uint16_t* const y = a.y + (int64_t)(t.r0 + row) * a.ldy + (int64_t)(t.head * a.group + head) * a.dim;
        if (few) join_column_wave(a, p, t.parts, col, y, 2 * (int)blockIdx.x);
        else join_column(a, p, t.parts, col, y, slot, lds);
    }
}

// ---------------------------------------------------------------------------------------------------------------
// Many rows per sequence (prompts): tiles of 128 or 256 columns, keys and values made fp16 once per workgroup.
// ---------------------------------------------------------------------------------------------------------------

// What a thread makes fp16 in a step: two neighbouring words of a unit's K codes and the same two of its V codes.  K's
// words have one scale each (a token's), V's four (the tokens').
template <bool Q41>
struct Pair {
    uint32_t kw[2], kd[2], km[Q41 ? 2 : 1];
    uint32_t vw[2], vd[2][2], vm[Q41 ? 2 : 1][2];
};

// Where the words' scales are and their fp16 values go.  The values are in the order in which the 32 x 32 x 16 products
// take them, 1 KiB fragments of 16 bytes a lane: K: fragment (16 channels) lane 32 (g % 2) + token; V: fragment (block,
// 16-token tile) lane 32 (g % 2) + channel, half g / 2 of its 16 bytes.  V's two words are the block's two tiles.
struct PairPlace {
    uint32_t kc, vc, ks[2], vs;              // byte offsets in the unit: words, scales
    int ko[2], vo, token;                    // token: V's byte 0 within a tile
};
template <int NB, bool Q41>
__device__ inline PairPlace pair_place(int p) {   // p: which 8 bytes of the unit's codes
    constexpr int dim = 32 * NB, half = cache_half_bytes(Q41, dim);
    const bool tail = NB % 2 && p >= NB / 2 * 128;
    const int lane = tail ? p - NB / 2 * 128 : (p & 127) >> 1, w0 = tail ? 2 * NB - 2 : (p >> 7) * 4 + (p & 1) * 2;
    const int g = lane >> 4, x = lane & 15;
    PairPlace r;
    r.kc = p * 8;
    r.vc = half + p * 8;
#pragma unroll
    for (int j = 0; j < 2; j++) {
        const int tile = (w0 + j) / NB, b = (w0 + j) - tile * NB;
        r.ks[j] = 16 * dim + ((tile * 4 + (x >> 2)) * NB + b) * 8 + (x & 3) * 2;
        r.ko[j] = (2 * b + (g >> 1)) * 1024 + ((g & 1) * 32 + 16 * tile + x) * 16;
    }
    r.vs = half + 16 * dim + (g * NB + (w0 >> 1)) * 8;
    r.vo = w0 * 1024 + ((g & 1) * 32 + x) * 16 + (g >> 1) * 8;
    r.token = 4 * g;
    return r;
}

template <int NB, bool Q41>
__device__ inline void load_pair(global_bytes unit, const PairPlace& at, Pair<Q41>* r) {
    constexpr int plane = cache_plane_bytes(32 * NB);
    // (a uniform address and a 32-bit offset per lane each)
    const u32x2 k = load_at<u32x2>(unit, at.kc);
    const u32x2 v = load_at<u32x2>(unit, at.vc);
#pragma unroll
    for (int j = 0; j < 2; j++) {
        r->kw[j] = k[j];
        r->vw[j] = v[j];
        r->kd[j] = load_at<uint16_t>(unit, at.ks[j]);
        const u32x2 d = load_at<u32x2>(unit + j * 32 * NB, at.vs);
        r->vd[j][0] = d[0];
        r->vd[j][1] = d[1];
        if constexpr (Q41) {
            r->km[j] = load_at<uint16_t>(unit + plane, at.ks[j]);
            const u32x2 m = load_at<u32x2>(unit + (plane + j * 32 * NB), at.vs);
            r->vm[j][0] = m[0];
            r->vm[j][1] = m[1];
        }
    }
}

// Only `left` (< 32) of the unit's tokens are in the cache: the others become zeros.
template <bool Q41>
__device__ inline void clear_pair(const PairPlace& at, int left, Pair<Q41>* r) {
#pragma unroll
    for (int j = 0; j < 2; j++) {
        const int t = 16 * j + at.token;
        const uint32_t k0 = (t < left ? 0x0000FFFFu : 0u) | (t + 1 < left ? 0xFFFF0000u : 0u);
        const uint32_t k1 = (t + 2 < left ? 0x0000FFFFu : 0u) | (t + 3 < left ? 0xFFFF0000u : 0u);
        r->vd[j][0] &= k0;
        r->vd[j][1] &= k1;
        if (left <= 0) r->kd[j] = 0;
        if constexpr (Q41) {
            r->vm[j][0] &= k0;
            r->vm[j][1] &= k1;
            if (left <= 0) r->km[j] = 0;
        }
    }
}

template <bool Q41>
__device__ inline void store_pair(const Pair<Q41>& r, const PairPlace& at, uint32_t f1024, uint8_t* k, uint8_t* v) {
#pragma unroll
    for (int j = 0; j < 2; j++) {
        const f16x2 d = as_f16x2(r.kd[j] * 0x10001u);
        f16x2 m = {};
        if constexpr (Q41) m = as_f16x2(r.km[j] * 0x10001u);
        u32x4 x;
#pragma unroll
        for (int i = 0; i < 4; i++) x[i] = __builtin_bit_cast(uint32_t, code_value<Q41>(as_f16x2(nibble_pair(r.kw[j], i, f1024)), d, m));
        *reinterpret_cast<u32x4*>(k + at.ko[j]) = x;
    }
#pragma unroll
    for (int j = 0; j < 2; j++) {
        const uint32_t wl = r.vw[j] & 0x0F0F0F0Fu, wh = (r.vw[j] >> 4) & 0x0F0F0F0Fu;
        u32x2 lo, hi;
#pragma unroll
        for (int i = 0; i < 2; i++) {
            const f16x2 d = as_f16x2(r.vd[j][i]);
            f16x2 m = {};
            if constexpr (Q41) m = as_f16x2(r.vm[j][i]);
            lo[i] = __builtin_bit_cast(uint32_t, code_value<Q41>(byte_pair(wl, i), d, m));
            hi[i] = __builtin_bit_cast(uint32_t, code_value<Q41>(byte_pair(wh, i), d, m));
        }
        *reinterpret_cast<u32x2*>(v + at.vo + j * 1024) = lo;
        *reinterpret_cast<u32x2*>(v + at.vo + j * 1024 + 256) = hi;
    }
}

// Per step of KS units: every wave makes its share of a later step's keys and values fp16 and puts them in LDS, in the
// order the products take them; and it multiplies this step's with its 32 columns.  A ring of LDS buffers, one barrier per
// step; the codes of the step after are on their way meanwhile.  A wave's products and its vector arithmetic are
// independent of each other, so that the matrix unit works beside the vector unit: the scores of unit i + 1 beside the
// exponentials of unit i, the sums over unit i's values beside the maximum of unit i + 1 and the conversions to fp16.
//
// Bound by the vector unit beside the matrix unit (issuing in 51 % and busy in 46 % of the cycles): 2048 rows of 8 x 4 heads of
// 128 over 18432 tokens (584 GFLOP), q4_0, 604-617 us, 947-967 TFLOP/s, where a large fp16 matrix product reaches 1405; the
// conversions and their loads come on top of the products, which is why 256 columns share each of them.  64 columns per wave
// would halve them again, but the accumulators then leave no registers (spills, and moves to and from the accumulation
// registers every step: slower); a ring of 4 buffers, or two units per step with 128 columns of heads of 128, gained nothing.
// The same rows and tokens, q4_0 and q4_1: heads of 64 402 and 425 us (292 GFLOP), of 96 526 and 528 (438 GFLOP), of 128 609 and
// 643, 4 x 4 heads of 256 875 and 1552 (584 GFLOP).  Heads of 256 have one wave per SIMD and reload 18 (q4_0) and 25 (q4_1)
// spilled registers inside the step loop, q4_1 with heads of 128 one (256 columns) or 6 (128 columns); the others none.
template <int NB, bool Q41, int NW, int KS>
__global__ __launch_bounds__(NW * 64) __attribute__((amdgpu_waves_per_eu(NB > 4 ? 1 : 2))) void k_attn_rows(AttnArgs a) {
    constexpr int dim = 32 * NB, unit_lds = 64 * dim, buffer = 2 * KS * unit_lds;   // fp16 bytes of a unit's K, or V; a step
    constexpr int threads = NW * 64, pairs = KS * 2 * dim, rounds = (pairs + threads - 1) / threads;
    constexpr int ahead = KS > 1 ? 2 : 3;   // steps: keys are read a unit before their product, two before their use
    __shared__ __attribute__((aligned(16))) uint8_t lds[(ahead + 1) * buffer];
    const TileShape ts = tile_shape(NW * 32, a.group);
    const int heads = a.s.heads, tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6), hl = lane >> 5;
    // heads vary fastest, so that a head's tiles (which read the same keys and values) tend to the same die; later tiles,
    // which see more, come first
    int at = blockIdx.x;
    const int h = uniform(at % heads);
    at = uniform(at / heads);
    const int split = uniform(at % a.splits);
    at = uniform(at / a.splits);
    const int item = at * heads + h;        // of the parts' places: below the grid's bound whatever row_start holds
    uint32_t before;
    const int seq = SeqTotals(a.s.batch, TileCount{a, ts}).find(at, &before);
    if (seq < 0) return;
    const SeqInfo q = seq_info_uniform(a, seq);
    const int tile = uniform(tiles_of(ts, q.n) - 1 - (at - (int)before));
    const int first = uniform(ts.ht == 1 ? tile * ts.rows : tile / ts.ht), end = min(first + ts.rows, q.n);
    int u0, u1;
    row_units(a, q, first, end, &u0, &u1);
    u0 = uniform(u0);
    u1 = uniform(u1);
    if (a.splits > 1) {
        const int per = uniform(((u1 - u0 + a.splits - 1) / a.splits + KS - 1) / KS * KS);
        u0 += split * per;
        u1 = min(u1, u0 + per);
    }

    // this wave's 32 columns
    int row, head, lo, hi, lo_most, hi_least, x;
    const bool valid = tile_col(a, ts, tile, wave * 32 + (lane & 31), q.n, &row, &head);
    row_tokens(a, q, valid ? row : first, &lo, &hi);
    row_tokens(a, q, first, &x, &hi_least);
    row_tokens(a, q, end - 1, &lo_most, &x);

    // this thread's pairs of words: unit (id / 2 dim) of the step, 8 bytes (id % 2 dim) of its codes
    const uint32_t f1024 = held(0x64006400u);
    Pair<Q41> r[rounds];                    // the fetched step's
    PairPlace place[rounds];
#pragma unroll
    for (int i = 0; i < rounds; i++) place[i] = pair_place<NB, Q41>((i * threads + tid) % (2 * dim));
    UnitWalk walk;
    walk.start(a.s, seq, h, u0);
    const auto pair_unit = [&](int i) { return uniform((i * threads + wave * 64) / (2 * dim)); };   // (2 dim % 64 == 0)
    int fetched = u0;                       // unit
    // requests a step's words; returns which of its units have tokens (a bit each)
    const auto fetch = [&](Pair<Q41>* r) {
        uint32_t has = 0;
        global_bytes unit[KS];
#pragma unroll
        for (int k = 0; k < KS; k++) {
            const bool there = fetched + k < u1 && walk.there;
            has |= (there ? 1u : 0u) << k;
            unit[k] = scalar_address(there ? walk.at(a.cache) : a.cache);   // (an absent unit's loads are of the pool's first one: cleared below)
            walk.step(1);
        }
        fetched += KS;
#pragma unroll
        for (int i = 0; i < rounds; i++) {
            if (rounds * threads > pairs && i * threads + wave * 64 >= pairs) break;
            load_pair<NB, Q41>(KS > 1 && pair_unit(i) ? unit[KS - 1] : unit[0], place[i], &r[i]);
        }
        return has;
    };
    // the tokens of step u that are not in the cache are made zeros
    const auto clear = [&](Pair<Q41>* r, uint32_t has, int u) {
        if (has == (1u << KS) - 1 && (u + KS) * kUnit <= q.tokens) return;
#pragma unroll
        for (int i = 0; i < rounds; i++) {
            const int k = pair_unit(i), left = has >> k & 1 ? q.tokens - (u + k) * kUnit : 0;
            if (left < kUnit) clear_pair<Q41>(place[i], left, &r[i]);
        }
    };
    const auto put = [&](const Pair<Q41>* r, uint8_t* to) {
#pragma unroll
        for (int i = 0; i < rounds; i++) {
            if (rounds * threads > pairs && i * threads + wave * 64 >= pairs) break;
            const int k = pair_unit(i);
            store_pair<Q41>(r[i], place[i], f1024, to + k * unit_lds, to + (KS + k) * unit_lds);
        }
    };

    // The first `ahead` steps, all requested before the first is used.
    uint32_t has = 0, got;                  // units with tokens: of this step and the `ahead` - 1 after it; of the fetched one
    const uint16_t* const qp = a.q + (int64_t)(q.r0 + row) * a.ldq + (int64_t)(h * a.group + head) * dim + 8 * hl;
    u32x4 qv[2 * NB];
    {
        Pair<Q41> r0[ahead][rounds];
        uint32_t h0[ahead];
#pragma unroll
        for (int i = 0; i < ahead; i++) h0[i] = fetch(r0[i]);
#pragma unroll
        for (int s = 0; s < 2 * NB; s++) {
            qv[s] = (u32x4){0, 0, 0, 0};
            if (valid) qv[s] = *reinterpret_cast<const u32x4*>(qp + 16 * s);
        }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = 0; i < ahead; i++) {
            has |= h0[i] << (i * KS);
            clear(r0[i], h0[i], u0 + i * KS);
            put(r0[i], lds + i * buffer);
        }
    }
    got = fetch(r);

    uint32_t big = 0;
#pragma unroll
    for (int s = 0; s < 2 * NB; s++) big = max(big, largest_bf16(qv[s]));
    big = max(big, (uint32_t)__shfl_xor((int)big, 32, 64));
    const int up = query_shift(big);
    const float sl2 = ldexpf(a.scale_log2, -up);
    f16x8 qf[2 * NB];
#pragma unroll
    for (int s = 0; s < 2 * NB; s++) qf[s] = query_f16(qv[s], up);

    f32x16 o[NB];
#pragma unroll
    for (int b = 0; b < NB; b++)
#pragma unroll
        for (int i = 0; i < 16; i++) o[b][i] = 0.0f;
    float ref = -FLT_MAX, l = 0.0f;
    constexpr int F = 2 * NB;               // operands of a unit's keys, and of its values
    f16x8 kf[F], vf[F];
    f32x16 s;                               // the scores of the unit after the one whose exponentials are taken
    float e[16], most;
    const auto read_k = [&](const uint8_t* at) {
#pragma unroll
        for (int f = 0; f < F; f++) kf[f] = *reinterpret_cast<const f16x8*>(at + f * 1024 + lane * 16);
    };
    const auto read_v = [&](const uint8_t* at, int c) {   // of the unit's first, second 16 tokens
#pragma unroll
        for (int b = 0; b < NB; b++) vf[2 * b + c] = *reinterpret_cast<const f16x8*>(at + (2 * b + c) * 1024 + lane * 16);
    };
    const auto scores = [&]() {
#pragma unroll
        for (int i = 0; i < 16; i++) s[i] = 0.0f;
#pragma unroll
        for (int f = 0; f < F; f++) s = __builtin_amdgcn_mfma_f32_32x32x16_f16(kf[f], qf[f], s, 0, 0, 0);
    };
    const auto exponents = [&]() {
#pragma unroll
        for (int i = 0; i < 16; i++) e[i] = fmaf(s[i], sl2, -ref);
        most = e[0];
#pragma unroll
        for (int i = 1; i < 16; i++) most = fmaxf(most, e[i]);
    };
    // masks, and a new reference, where the unit needs them
    const auto settle = [&](int u, bool there) {
        const int t0 = u * kUnit;
        if (t0 < lo_most || t0 + kUnit > hi_least || !there) {
            const int lo2 = there ? lo - t0 : kUnit, hi2 = hi - t0;
            most = -INFINITY;
#pragma unroll
            for (int i = 0; i < 16; i++) {
                const int t = 8 * (i >> 2) + 4 * hl + (i & 3);
                e[i] = t >= lo2 && t < hi2 ? e[i] : -INFINITY;
                most = fmaxf(most, e[i]);
            }
        }
        if (__any(most > kRefMost)) {
            float mx = -INFINITY;
#pragma unroll
            for (int i = 0; i < 16; i++) mx = fmaxf(mx, e[i] == -INFINITY ? -INFINITY : s[i] * sl2);
            mx = fmaxf(mx, __shfl_xor(mx, 32, 64));
            const float r2 = fmaxf(ref, mx - kRefBelow), alpha = r2 == ref ? 1.0f : exp2_fast(ref - r2);
#pragma unroll
            for (int b = 0; b < NB; b++) o[b] *= alpha;
            l *= alpha;
            ref = r2;
#pragma unroll
            for (int i = 0; i < 16; i++) e[i] = e[i] == -INFINITY ? -INFINITY : fmaf(s[i], sl2, -ref);
        }
    };
    if (u0 < u1) {
        __syncthreads();
        read_k(lds);
        scores();
        exponents();
        settle(u0, has & 1);
        read_k(lds + (KS > 1 ? unit_lds : buffer));
        uint8_t *lk = lds, *ln = lds + buffer, *lp = lds + ahead * buffer;   // this step's, the next one's, the one to fill
        const auto next = [&](uint8_t* at) { return at == lds + ahead * buffer ? lds : at + buffer; };
        for (int u = u0; u < u1; u += KS) {
            has |= got << (ahead * KS);
            clear(r, got, u + ahead * KS);
#pragma unroll
            for (int k = 0; k < KS; k++) {
                // (behind the last unit the scores are of zeros, and not used)
                read_v(lk + (KS + k) * unit_lds, 0);
                __builtin_amdgcn_sched_barrier(0);
                scores();
                float sum = 0.0f;
#pragma unroll
                for (int i = 0; i < 16; i++) {
                    e[i] = exp2_fast(e[i]);
                    sum += e[i];
                }
                l += sum;
                f16x8 pf[2];
#pragma unroll
                for (int c = 0; c < 2; c++)
                    pf[c] = __builtin_bit_cast(f16x8, (u32x4){pack_f16(e[8 * c], e[8 * c + 1]), pack_f16(e[8 * c + 2], e[8 * c + 3]),
                                                              pack_f16(e[8 * c + 4], e[8 * c + 5]), pack_f16(e[8 * c + 6], e[8 * c + 7])});
                asm volatile("" : "+v"(l));
#pragma unroll
                for (int f = 0; f < F; f++) {
                    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
                    __builtin_amdgcn_sched_group_barrier(0x402, (40 + F - 1) / F, 0);
                }
                __builtin_amdgcn_sched_barrier(0);
                // (the second half of V now: its registers were the probabilities'); keys of the unit after the next
                read_v(lk + (KS + k) * unit_lds, 1);
                read_k(KS == 1 ? next(ln) : k == 0 ? ln : ln + unit_lds);
#pragma unroll
                for (int f = 0; f < F; f++) {
                    const int b = f % NB, c = f / NB;
                    o[b] = __builtin_amdgcn_mfma_f32_32x32x16_f16(vf[2 * b + c], pf[c], o[b], 0, 0, 0);
                }
                if (k == 0) put(r, lp);
                exponents();
                asm volatile("" : "+v"(most));
#pragma unroll
                for (int f = 0; f < F; f++) {
                    __builtin_amdgcn_sched_group_barrier(0x008, 1, 1);
                    if (k == 0) __builtin_amdgcn_sched_group_barrier(0x402, (24 + 64 * rounds + F - 1) / F, 1);
                    else __builtin_amdgcn_sched_group_barrier(0x402, (24 + F - 1) / F, 1);
                }
                __builtin_amdgcn_sched_barrier(0);
                if (k == 0) got = fetch(r);
                settle(u + k + 1, has >> (k + 1) & 1);
            }
            has >>= KS;
            lk = ln;
            ln = next(ln);
            lp = next(lp);
            __syncthreads();
        }
    }
    l += __shfl_xor(l, 32, 64);
    if (!valid) return;
    if (a.splits > 1) {
        const Partials p(a);
        const int slot = item * a.splits + split, col = wave * 32 + (lane & 31);
        float* const po = p.sums(slot, col);
#pragma unroll
        for (int b = 0; b < NB; b++)
#pragma unroll
            for (int k = 0; k < 4; k++)
                *reinterpret_cast<f32x4*>(po + 32 * b + 8 * k + 4 * hl) = (f32x4){o[b][4 * k], o[b][4 * k + 1], o[b][4 * k + 2], o[b][4 * k + 3]};
        if (hl == 0) {
            float* const st = p.stat(slot, col);
            st[0] = ref;
            st[1] = l;
        }
        return;
    }
    const float inv = l != 0.0f ? 1.0f / l : 0.0f;
    uint16_t* const y = a.y + (int64_t)(q.r0 + row) * a.ldy + (int64_t)(h * a.group + head) * dim;
#pragma unroll
    for (int b = 0; b < NB; b++)
#pragma unroll
        for (int k = 0; k < 4; k++)
            *reinterpret_cast<u32x2*>(y + 32 * b + 8 * k + 4 * hl) = (u32x2){pack_bf16(o[b][4 * k] * inv, o[b][4 * k + 1] * inv),
                                                                            pack_bf16(o[b][4 * k + 2] * inv, o[b][4 * k + 3] * inv)};
}

// Workgroup (tile, head): the tile's columns, each shared out over a.splits workgroups of k_attn_rows.
__global__ __launch_bounds__(256) void k_attn_join_rows(AttnArgs a) {
    __shared__ __attribute__((aligned(16))) JoinLds lds;
    const TileShape ts = tile_shape(a.tile_cols, a.group);
    const int heads = a.s.heads, h = blockIdx.x % heads, at = blockIdx.x / heads;
    uint32_t before;
    const int seq = SeqTotals(a.s.batch, TileCount{a, ts}).find(at, &before);
    if (seq < 0) return;
    const SeqInfo q = seq_info_uniform(a, seq);
    const int tile = tiles_of(ts, q.n) - 1 - (at - (int)before);
    const Partials p(a);
    const auto slot = [&](int i) { return (int)blockIdx.x * a.splits + i; };
    for (int col = blockIdx.y; col < a.tile_cols; col += gridDim.y) {
        int row, head;
        if (!tile_col(a, ts, tile, col, q.n, &row, &head)) break;
        join_column(a, p, a.splits, col, a.y + (int64_t)(q.r0 + row) * a.ldy + (int64_t)(h * a.group + head) * a.dim, slot, lds);
    }
}

namespace {

// Workgroups that a shared-out call has, and the units that each takes at least.
constexpr int kShareWorkgroups = kJoinParts, kShareLeast = 24;
// Columns per sequence, on average, from which a call takes tiles of 128 or 256 columns: measured in us, tiles of 16 and
// of 128, 16 sequences of 4096 tokens, 8 x 4 heads of 128: 64 columns 60 and 121, 128 columns 110 and 122; one of 65536
// tokens, 64 columns 69 and 71, 256 columns 214 and 199.
constexpr int kManyCols = 129;
// Tiles of 128 columns: with fewer (tiles x heads) than this their tokens are shared out; units that a part has at least.
constexpr int kRowItems = 128, kRowLeast = 16;

// How a call runs.
struct Schedule {
    int cols;            // columns per tile: 16, 128 or 256
    int64_t items;       // tiles x heads (at most)
    int workgroups;      // 16 columns: sequences shared out over so many (0: not)
    int splits;          // 128, 256 columns: parts per tile
    int slots() const { return cols == kTokenCols ? 2 * workgroups : splits > 1 ? (int)items * splits : 0; }
};

Schedule schedule(const AttnArgs& a, bool share) {
    Schedule s{};
    const auto items = [&](int cols) {
        s.cols = cols;
        s.items = tile_bound(tile_shape(cols, a.group), a.s.rows, a.s.batch, !a.s.row_start) * a.s.heads;
    };
    const int64_t units = ((int64_t)a.s.table_ld * a.s.page) / kUnit;   // of the longest sequence there can be
    s.splits = 1;
    if (a.s.row_start && (int64_t)a.s.rows * a.group >= (int64_t)kManyCols * a.s.batch) {
        // Twice as many columns share a conversion to fp16, with one workgroup per compute unit instead of two: in us, 256
        // and 128 columns, 2048 rows of 8 x 4 heads of 128 over 18432 tokens 610 and 712, two prompts of 2048 rows 95 and
        // 108, but 8 prompts of 700 rows, 12 heads of 96, 49 and 41, 4 of 1500, 20 heads of 64, 76 and 70.
        items(256);
        if (s.items < 256 || units < 64 || a.dim == 256) items(128);
        if (share && s.items <= kRowItems)
            s.splits = (int)std::max<int64_t>(1, std::min<int64_t>({2 * kRowItems / s.items, units / kRowLeast, 64}));
    } else {
        items(kTokenCols);
        // Shared out, and joined by a second launch, where a sequence can be long.  Measured in us, whole and shared out,
        // 8 heads of 128: 8 tiles of 1024 tokens 11.4 and 17.7, of 2048 tokens 17.9 and 17.4; 256 tiles of 2048 22 and 29,
        // of 4096 34 and 42, of 8192 65 and 72, but 288 tiles of 4096, of which 64 share a compute unit, 57 and 46 (equal
        // lengths: unequal ones only gain).  Work is counted in 32 bits.
        if (share && units > (s.items < 256 ? 64 : 128) && s.items * (units + kTileCost) <= 0x7FFFFFFF)
            s.workgroups = kShareWorkgroups;
    }
    return s;
}

template <int NB, int NW, int D>
void launch_token(const AttnArgs& a, dim3 grid, hipStream_t s) {
    if (a.q41) hipLaunchKernelGGL((k_attn_token<NB, true, NW, D>), grid, dim3(NW * 64), 0, s, a);
    else hipLaunchKernelGGL((k_attn_token<NB, false, NW, D>), grid, dim3(NW * 64), 0, s, a);
}
template <int NB, int NW, int KS>
void launch_rows(const AttnArgs& a, dim3 grid, hipStream_t s) {
    if (a.q41) hipLaunchKernelGGL((k_attn_rows<NB, true, NW, KS>), grid, dim3(NW * 64), 0, s, a);
    else hipLaunchKernelGGL((k_attn_rows<NB, false, NW, KS>), grid, dim3(NW * 64), 0, s, a);
}

}  // namespace

// A launch has fewer than 2^32 threads.
bool attn_fits(const AttnArgs& a) {
    const Schedule s = schedule(a, true);
    return s.items * s.splits < (int64_t(1) << 23);
}

size_t attn_workspace_bytes(const AttnArgs& a) {
    const Schedule s = schedule(a, true);
    return (size_t)partial_bytes(s.slots(), s.cols, a.dim) + s.workgroups * sizeof(OpenTile);
}

hipError_t launch_attn(const AttnArgs& args, hipStream_t s) {
    AttnArgs a = args;
    const Schedule c = schedule(a, a.ws != nullptr);
    a.tile_cols = c.cols;
    a.workgroups = c.workgroups;
    a.least_units = kShareLeast;
    a.splits = c.splits;
    a.slots = c.slots();
    const TileShape ts = tile_shape(a.tile_cols, a.group);
    const int cols = std::min(a.tile_cols, (a.s.row_start ? ts.rows : 1) * a.group);   // that a tile can have
    if (c.cols != kTokenCols) {
        const dim3 grid((unsigned)(c.items * c.splits));
        const bool wide = c.cols == 256;
        switch (a.dim) {
        case 64: wide ? launch_rows<2, 8, 2>(a, grid, s) : launch_rows<2, 4, 2>(a, grid, s); break;
        case 96: wide ? launch_rows<3, 8, 2>(a, grid, s) : launch_rows<3, 4, 1>(a, grid, s); break;
        case 128: wide ? launch_rows<4, 8, 2>(a, grid, s) : launch_rows<4, 4, 1>(a, grid, s); break;
        default: launch_rows<8, 4, 1>(a, grid, s); break;
        }
        if (c.splits > 1) hipLaunchKernelGGL(k_attn_join_rows, dim3((unsigned)c.items, std::min(cols, 64)), dim3(256), 0, s, a);
        return hipGetLastError();
    }
    const dim3 grid((unsigned)(c.workgroups ? c.workgroups : c.items));
    // With at most a tile per compute unit eight waves share a tile's tokens (1024 tokens, 8 tiles of 4 x 128: 13.6 ->
    // 11.4 us; 80 tiles of 1500 x 64: 12.3 -> 10.3); with more, four (320 tiles of 1500 x 64: 20.2 -> 16.5 us).
    const bool few = !c.workgroups && c.items <= 256;
    switch (a.dim) {
    case 64: few ? launch_token<2, 8, 3>(a, grid, s) : launch_token<2, 4, 4>(a, grid, s); break;
    case 96: few ? launch_token<3, 8, 3>(a, grid, s) : launch_token<3, 4, 3>(a, grid, s); break;
    case 128: few ? launch_token<4, 8, 3>(a, grid, s) : launch_token<4, 4, 3>(a, grid, s); break;
    default: launch_token<8, 4, 2>(a, grid, s); break;
    }
    // (with few tiles each has many parts, and a workgroup takes one column at a time, not four)
    if (c.workgroups) {
        if (c.items * 8 >= c.workgroups) hipLaunchKernelGGL(k_attn_join_token<true>, dim3(c.workgroups - 1, (cols + 3) / 4), dim3(256), 0, s, a);
        else hipLaunchKernelGGL(k_attn_join_token<false>, dim3(c.workgroups - 1, std::min(cols, 8)), dim3(256), 0, s, a);
    }
    return hipGetLastError();
}

}  // namespace wq
