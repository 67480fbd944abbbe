// attn.hip -- attention over the 4-bit cache: y = sum_t softmax_t(scale q . k^_t) v^_t over the tokens a row sees.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "attn_common.h"

namespace wq {

// ---------------------------------------------------------------------------------------------------------------
// Few columns per sequence (single tokens, drafted tokens): tiles of 16 columns, every wave its own units.
// ---------------------------------------------------------------------------------------------------------------

// One unit's operands in a lane's registers.
template <int NB, bool Q41>
struct UnitRegs {
    uint32_t kw[2 * NB], vw[2 * NB];
    uint32_t kd[2][NB][2], vd[2][NB][2];                            // [tile][block][token pair]
    uint32_t km[Q41 ? 2 : 1][Q41 ? NB : 1][2], vm[Q41 ? 2 : 1][Q41 ? NB : 1][2];
};

template <int NB>
__device__ inline void load_words(const uint8_t* p, int lane, uint32_t* w) {
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

template <int NB>
__device__ inline void load_scales(const uint8_t* p, int g, uint32_t (*d)[NB][2]) {
#pragma unroll
    for (int tile = 0; tile < 2; tile++) {
        const uint8_t* q = p + (tile * 4 + g) * NB * 8;
        if constexpr (NB % 2 == 0) {
#pragma unroll
            for (int b = 0; b < NB; b += 2) {
                const u32x4 v = *reinterpret_cast<const u32x4*>(q + b * 8);
                d[tile][b][0] = v[0];
                d[tile][b][1] = v[1];
                d[tile][b + 1][0] = v[2];
                d[tile][b + 1][1] = v[3];
            }
        } else {
#pragma unroll
            for (int b = 0; b < NB; b++) {
                const u32x2 v = *reinterpret_cast<const u32x2*>(q + b * 8);
                d[tile][b][0] = v[0];
                d[tile][b][1] = v[1];
            }
        }
    }
}

template <int NB, bool Q41>
__device__ inline void load_unit(const uint8_t* p, int lane, UnitRegs<NB, Q41>* r) {
    constexpr int dim = 32 * NB, half = cache_half_bytes(Q41, dim), plane = cache_plane_bytes(dim);
    const int g = lane >> 4;
    load_words<NB>(p, lane, r->kw);
    load_scales<NB>(p + 16 * dim, g, r->kd);
    if constexpr (Q41) load_scales<NB>(p + 16 * dim + plane, g, r->km);
    load_words<NB>(p + half, lane, r->vw);
    load_scales<NB>(p + half + 16 * dim, g, r->vd);
    if constexpr (Q41) load_scales<NB>(p + half + 16 * dim + plane, g, r->vm);
}

// A column's running softmax and its part of the sums.
template <int NB>
struct ColState {
    f32x4 o[2 * NB];     // channels 16 i + 4 g + 0..3 of column lane % 16
    float ref, l;        // l: this lane's tokens only
};

// K codes are multiplied as the bf16 integers 128 + q, exact, with the sum's start at -(128 + 8) sum q (q4_0; -128 sum q
// for q4_1), so that a block's product is the exact-code sum in fp32, and its fp16 scale is applied after it.
template <int NB, bool Q41>
__device__ inline void unit_step(const UnitRegs<NB, Q41>& r, const bf16x8 (&qf)[NB], const float (&c0)[NB], float sl2, int t0,
                                 int lo, int hi, int tokens, bool masked, ColState<NB>* st) {
    const int g = (threadIdx.x & 63) >> 4;
    float x[8];
#pragma unroll
    for (int tile = 0; tile < 2; tile++) {
        f32x4 s = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int b = 0; b < NB; b++) {
            const uint32_t w = r.kw[tile * NB + b];
            u32x4 u;
#pragma unroll
            for (int i = 0; i < 4; i++) u[i] = ((w >> (4 * i)) & 0x000F000Fu) | 0x43004300u;
            const f32x4 c = {c0[b], c0[b], c0[b], c0[b]};
            const f32x4 p = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, u), qf[b], c, 0, 0, 0);
            const f16x2 d01 = as_f16x2(r.kd[tile][b][0]), d23 = as_f16x2(r.kd[tile][b][1]);
            s[0] = fmaf((float)d01[0], p[0], s[0]);
            s[1] = fmaf((float)d01[1], p[1], s[1]);
            s[2] = fmaf((float)d23[0], p[2], s[2]);
            s[3] = fmaf((float)d23[1], p[3], s[3]);
            if constexpr (Q41) {
                const f16x2 m01 = as_f16x2(r.km[tile][b][0]), m23 = as_f16x2(r.km[tile][b][1]);
                const float sx = c0[b] * -0.0078125f;   // sum q over the block
                s[0] = fmaf((float)m01[0], sx, s[0]);
                s[1] = fmaf((float)m01[1], sx, s[1]);
                s[2] = fmaf((float)m23[0], sx, s[2]);
                s[3] = fmaf((float)m23[1], sx, s[3]);
            }
        }
#pragma unroll
        for (int i = 0; i < 4; i++) x[4 * tile + i] = s[i] * sl2;
    }
    uint32_t keep[4] = {~0u, ~0u, ~0u, ~0u};    // token pairs that are in the cache: what lies behind them is anything
    if (masked) {
#pragma unroll
        for (int j = 0; j < 8; j++) {
            const int t = t0 + (j >> 2) * 16 + 4 * g + (j & 3);
            x[j] = t >= lo && t < hi ? x[j] : -INFINITY;
            if (t >= tokens) keep[j >> 1] &= (j & 1) ? 0x0000FFFFu : 0xFFFF0000u;
        }
    }
    float mx = fmaxf(fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])), fmaxf(fmaxf(x[4], x[5]), fmaxf(x[6], x[7])));
    if (__any(mx - st->ref > kRefMost)) {
        mx = fmaxf(mx, __shfl_xor(mx, 16, 64));
        mx = fmaxf(mx, __shfl_xor(mx, 32, 64));
        const float ref = fmaxf(st->ref, mx - kRefBelow);
        const float alpha = ref == st->ref ? 1.0f : exp2_fast(st->ref - ref);
#pragma unroll
        for (int i = 0; i < 2 * NB; i++) st->o[i] *= alpha;
        st->l *= alpha;
        st->ref = ref;
    }
    u32x4 p;
#pragma unroll
    for (int j = 0; j < 8; j++) x[j] = exp2_fast(x[j] - st->ref);
    st->l += ((x[0] + x[1]) + (x[2] + x[3])) + ((x[4] + x[5]) + (x[6] + x[7]));
#pragma unroll
    for (int j = 0; j < 4; j++) p[j] = pack_f16(x[2 * j], x[2 * j + 1]);
    const f16x8 pf = __builtin_bit_cast(f16x8, p);
#pragma unroll
    for (int b = 0; b < NB; b++) {
        u32x4 vlo, vhi;
#pragma unroll
        for (int tile = 0; tile < 2; tile++) {
            const uint32_t w = r.vw[2 * b + tile], wl = w & 0x0F0F0F0Fu, wh = (w >> 4) & 0x0F0F0F0Fu;
#pragma unroll
            for (int i = 0; i < 2; i++) {
                const f16x2 d = as_f16x2(r.vd[tile][b][i] & keep[2 * tile + i]);
                f16x2 m = {};
                if constexpr (Q41) m = as_f16x2(r.vm[tile][b][i] & keep[2 * tile + i]);
                vlo[2 * tile + i] = __builtin_bit_cast(uint32_t, code_value<Q41>(byte_pair(wl, i), d, m));
                vhi[2 * tile + i] = __builtin_bit_cast(uint32_t, code_value<Q41>(byte_pair(wh, i), d, m));
            }
        }
        st->o[2 * b] = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, vlo), pf, st->o[2 * b], 0, 0, 0);
        st->o[2 * b + 1] = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, vhi), pf, st->o[2 * b + 1], 0, 0, 0);
    }
}

constexpr int kTokenCols = 16;

// Units of a sequence's items, for sharing out: every tile of it takes all of them; at least one, so that tiles whose
// rows see nothing are visited (and written).
__device__ inline int span_units(const AttnArgs& a, const SeqInfo& q, int* u0) {
    int u1;
    if (q.n == 0) {
        *u0 = 0;
        return 0;
    }
    row_units(a, q, 0, q.n, u0, &u1);
    return u1 > *u0 ? u1 - *u0 : 1;
}

// The stretch of the call's work, in units over all (sequence, tile, head), that a workgroup takes: `share` each.
__device__ inline uint32_t work_share(uint32_t total, int workgroups, int least) {
    const uint32_t s = (total + workgroups - 1) / workgroups;
    return s > (uint32_t)least ? s : (uint32_t)least;
}

// A tile's columns x units [ua, ub) of one head, by the workgroup.  part: where the sums go (null: the tile is whole,
// and y is written).
template <int NB, bool Q41, int NW>
__device__ void token_segment(const AttnArgs& a, const TileShape& ts, const SeqInfo& q, int seq, int tile, int h, int ua, int ub,
                              float* part_o, float* part_ml, float* lds_o, float* lds_f) {
    constexpr int dim = 32 * NB, ld = dim + 4;
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6), g = lane >> 4, col = lane & 15;
    int row, head;
    const bool valid = tile_col(a, ts, tile, col, q.n, &row, &head);
    const int first = ts.ht == 1 ? tile * ts.rows : tile / ts.ht, last = min(first + ts.rows, q.n) - 1;
    int lo, hi, lo_most, hi_least, x;
    row_tokens(a, q, valid ? row : first, &lo, &hi);
    row_tokens(a, q, first, &x, &hi_least);
    row_tokens(a, q, last, &lo_most, &x);

    bf16x8 qf[NB];
    const uint16_t* qp = a.q + (int64_t)(q.r0 + row) * a.ldq + (int64_t)(h * a.group + head) * dim + 8 * g;
#pragma unroll
    for (int b = 0; b < NB; b++) {
        u32x4 v = {};
        if (valid) v = *reinterpret_cast<const u32x4*>(qp + 32 * b);
        // to the order of a K word's nibble pairs: 0, 4, 1, 5, 2, 6, 3, 7
        u32x4 w;
        w[0] = __builtin_amdgcn_perm(v[2], v[0], 0x05040100u);
        w[1] = __builtin_amdgcn_perm(v[2], v[0], 0x07060302u);
        w[2] = __builtin_amdgcn_perm(v[3], v[1], 0x05040100u);
        w[3] = __builtin_amdgcn_perm(v[3], v[1], 0x07060302u);
        qf[b] = __builtin_bit_cast(bf16x8, w);
    }
    float c0[NB];
    {
        const uint32_t minus = Q41 ? 0xC300C300u : 0xC308C308u;   // bf16 -128, -136
        const bf16x8 k = __builtin_bit_cast(bf16x8, (u32x4){minus, minus, minus, minus});
#pragma unroll
        for (int b = 0; b < NB; b++) c0[b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(k, qf[b], (f32x4){0, 0, 0, 0}, 0, 0, 0)[0];
    }

    ColState<NB> st;
#pragma unroll
    for (int i = 0; i < 2 * NB; i++) st.o[i] = (f32x4){0, 0, 0, 0};
    st.ref = -FLT_MAX;
    st.l = 0.0f;

    int u = ua + wave;
    if (u < ub) {
        UnitWalk walk;
        walk.start(a.s, seq, h, u);
        UnitRegs<NB, Q41> A, B;
        int64_t at = walk.at();
        if (at >= 0) load_unit<NB, Q41>(a.cache + at, lane, &A);
        const auto step = [&](const UnitRegs<NB, Q41>& r, int unit) {
            const int t0 = unit * kUnit;
            const bool masked = t0 < lo_most || t0 + kUnit > hi_least;
            unit_step<NB, Q41>(r, qf, c0, a.scale_log2, t0, lo, hi, q.tokens, masked, &st);
        };
        while (true) {
            int64_t at2 = -1;
            if (u + NW < ub) {
                walk.step(NW);
                at2 = walk.at();
                if (at2 >= 0) load_unit<NB, Q41>(a.cache + at2, lane, &B);
            }
            if (at >= 0) step(A, u);
            u += NW;
            if (u >= ub) break;
            at = -1;
            if (u + NW < ub) {
                walk.step(NW);
                at = walk.at();
                if (at >= 0) load_unit<NB, Q41>(a.cache + at, lane, &A);
            }
            if (at2 >= 0) step(B, u);
            u += NW;
            if (u >= ub) break;
        }
    }

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
// are; a tile that more than one workgroup has a part of is joined by k_attn_join.  With `splits` 0 every workgroup has
// one whole tile.
template <int NB, bool Q41, int NW>
__global__ __launch_bounds__(NW * 64) void k_attn_token(AttnArgs a) {
    __shared__ float lds_o[NW * 16 * (32 * NB + 4)];
    __shared__ float lds_f[2 * NW * 16];
    const TileShape ts = tile_shape(kTokenCols, a.group);
    const int heads = a.s.heads;
    if (a.workgroups == 0) {
        const int item = blockIdx.x;
        int seq = -1;
        uint32_t before = 0;
        if (!a.s.row_start) {
            seq = item / (ts.ht * heads);
            before = seq * (ts.ht * heads);
        } else {
            find_seq(a.s.batch, item, [&](int b) { int r0, r1; seq_rows(a.s, b, &r0, &r1); return (uint32_t)(tiles_of(ts, r1 - r0) * heads); },
                     &seq, &before);
            seq = uniform(seq);
            before = uniform(before);
        }
        if (seq < 0 || seq >= a.s.batch) return;
        const SeqInfo q = seq_info_uniform(a, seq);
        const int in = item - (int)before, tile = in / heads, h = in - tile * heads;
        const int first = ts.ht == 1 ? tile * ts.rows : tile / ts.ht, end = min(first + ts.rows, q.n);
        if (first >= end) return;
        int u0, u1;
        row_units(a, q, first, end, &u0, &u1);
        token_segment<NB, Q41, NW>(a, ts, q, seq, tile, h, u0, u1, nullptr, nullptr, lds_o, lds_f);
        return;
    }
    const auto weight = [&](int b) {
        const SeqInfo q = seq_info(a, b);
        int u0;
        return (uint32_t)(tiles_of(ts, q.n) * heads * span_units(a, q, &u0));
    };
    int seq;
    uint32_t before;
    const uint32_t total = find_seq(a.s.batch, 0u, weight, &seq, &before);
    const uint32_t share = work_share(total, a.workgroups, a.least_units);
    uint32_t w = blockIdx.x * share;
    const uint32_t end = min(w + share, total);
    if (w >= end) return;
    find_seq(a.s.batch, w, weight, &seq, &before);
    seq = uniform(seq);
    before = uniform(before);
    while (w < end) {
        const SeqInfo q = seq_info_uniform(a, seq);
        int u0;
        const int span = span_units(a, q, &u0);
        const uint32_t items = tiles_of(ts, q.n) * heads;
        while (w < end && w - before < items * span) {
            const int item = (w - before) / span, s0 = (w - before) - item * span, s1 = min((uint32_t)span, s0 + (end - w));
            const int tile = item / heads, h = item - tile * heads;
            float *po = nullptr, *pm = nullptr;
            if (s1 - s0 < span) {
                const int slot = 2 * blockIdx.x + (s0 > 0 ? 0 : 1);
                const Partials p = {reinterpret_cast<float*>(a.ws), reinterpret_cast<float*>(a.ws) + (int64_t)2 * a.workgroups * kTokenCols * a.dim,
                                    a.dim, kTokenCols};
                po = p.sums(slot, 0);
                pm = p.stat(slot, 0);
            }
            // (a span of one unit stands for none where the rows see nothing)
            int r0, r1;
            row_units(a, q, 0, q.n, &r0, &r1);
            token_segment<NB, Q41, NW>(a, ts, q, seq, tile, h, u0 + s0, min(u0 + s1, r1), po, pm, lds_o, lds_f);
            w += s1 - s0;
        }
        before += items * span;
        seq++;
    }
}

// Joins the parts of a shared-out tile: y = sum_i 2^(ref_i - ref) o_i / sum_i 2^(ref_i - ref) l_i, in order.  One wave
// per column.
__device__ inline void join_column(const AttnArgs& a, const Partials& p, int n, int col, uint16_t* y, int first_slot, int step) {
    const int lane = threadIdx.x & 63;
    const auto slot = [&](int i) { return i == 0 ? first_slot : first_slot - (step == 2 ? 1 : 0) + step * i; };
    float ref = -FLT_MAX;
    for (int i = lane; i < n; i += 64) ref = fmaxf(ref, p.stat(slot(i), col)[0]);
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) ref = fmaxf(ref, __shfl_xor(ref, d, 64));
    float l = 0.0f, o[4] = {};
    for (int i = 0; i < n; i++) {
        const float* st = p.stat(slot(i), col);
        const float f = exp2_fast(st[0] - ref);
        l += f * st[1];
        const float* s = p.sums(slot(i), col);
#pragma unroll
        for (int j = 0; j < 4; j++)
            if (lane + 64 * j < a.dim) o[j] += f * s[lane + 64 * j];
    }
    const float inv = l != 0.0f ? 1.0f / l : 0.0f;
#pragma unroll
    for (int j = 0; j < 4; j++)
        if (lane + 64 * j < a.dim) y[lane + 64 * j] = __builtin_bit_cast(uint16_t, (__bf16)(o[j] * inv));
}

__global__ __launch_bounds__(256) void k_attn_join_token(AttnArgs a) {
    const TileShape ts = tile_shape(kTokenCols, a.group);
    const int heads = a.s.heads, wave = uniform(threadIdx.x >> 6);
    const uint32_t item = blockIdx.x;
    const auto weight = [&](int b) {
        const SeqInfo q = seq_info(a, b);
        int u0;
        return (uint32_t)(tiles_of(ts, q.n) * heads * span_units(a, q, &u0));
    };
    const auto count = [&](int b) { int r0, r1; seq_rows(a.s, b, &r0, &r1); return (uint32_t)(tiles_of(ts, r1 - r0) * heads); };
    int seq, other;
    uint32_t before, items_before, x;
    find_seq(a.s.batch, item, count, &seq, &items_before);
    seq = uniform(seq);
    if (seq < 0) return;
    // the total, and what comes before this sequence
    const uint32_t total = find_seq(a.s.batch, 0u, weight, &other, &x);
    before = find_seq(seq, 0u, weight, &other, &x);
    const uint32_t share = work_share(total, a.workgroups, a.least_units);
    const SeqInfo q = seq_info_uniform(a, seq);
    int u0;
    const uint32_t span = span_units(a, q, &u0), in = item - uniform(items_before);
    const uint32_t w0 = before + in * span, w1 = w0 + span;
    const int i0 = w0 / share, i1 = (w1 - 1) / share;
    if (i0 == i1) return;
    const int tile = in / heads, h = in - tile * heads;
    const Partials p = {reinterpret_cast<float*>(a.ws), reinterpret_cast<float*>(a.ws) + (int64_t)2 * a.workgroups * kTokenCols * a.dim, a.dim,
                        kTokenCols};
    const int first = 2 * i0 + 1;   // the part that starts the tile; the others start their workgroups
    for (int col = wave; col < kTokenCols; col += 4) {
        int row, head;
        if (!tile_col(a, ts, tile, col, q.n, &row, &head)) continue;
        join_column(a, p, i1 - i0 + 1, col, a.y + (int64_t)(q.r0 + row) * a.ldy + (int64_t)(h * a.group + head) * a.dim, first, 2);
    }
}

namespace {

// Workgroups that a shared-out call has, and the units that each takes at least.
constexpr int kShareWorkgroups = 512, kShareLeast = 16;

// Sequences are shared out where their tiles alone would leave compute units without work, and a sequence can be long
// enough to be worth the second launch that joins the parts.
int share_workgroups(const AttnArgs& a) {
    const TileShape ts = tile_shape(kTokenCols, a.group);
    const int64_t items = tile_bound(ts, a.s.rows, a.s.batch, !a.s.row_start) * a.s.heads;
    const int64_t units = ((int64_t)a.s.table_ld * a.s.page) / kUnit;
    if (units < 32 || items >= 4096) return 0;
    if (items * units > 0x7FFFFFFF) return 0;     // work is counted in 32 bits
    return kShareWorkgroups;
}

template <int NB, int NW>
void launch_token(const AttnArgs& a, dim3 grid, hipStream_t s) {
    if (a.q41) hipLaunchKernelGGL((k_attn_token<NB, true, NW>), grid, dim3(NW * 64), 0, s, a);
    else hipLaunchKernelGGL((k_attn_token<NB, false, NW>), grid, dim3(NW * 64), 0, s, a);
}

}  // namespace

size_t attn_workspace_bytes(const AttnArgs& a) {
    return (size_t)partial_bytes(2 * share_workgroups(a), kTokenCols, a.dim);
}

hipError_t launch_attn(const AttnArgs& args, hipStream_t s) {
    AttnArgs a = args;
    a.tile_cols = kTokenCols;
    a.workgroups = a.ws ? share_workgroups(a) : 0;
    a.least_units = kShareLeast;
    const TileShape ts = tile_shape(kTokenCols, a.group);
    const int64_t items = tile_bound(ts, a.s.rows, a.s.batch, !a.s.row_start) * a.s.heads;
    const dim3 grid((unsigned)(a.workgroups ? a.workgroups : items));
    switch (a.dim) {
    case 64: launch_token<2, 4>(a, grid, s); break;
    case 96: launch_token<3, 4>(a, grid, s); break;
    case 128: launch_token<4, 4>(a, grid, s); break;
    default: launch_token<8, 4>(a, grid, s); break;
    }
    if (a.workgroups) hipLaunchKernelGGL(k_attn_join_token, dim3((unsigned)items), dim3(256), 0, s, a);
    return hipGetLastError();
}

}  // namespace wq
