// attn_wide.hip -- attention of drafts, whose rows and heads are several tiles of 16 columns per key/value head: a wave takes
// CT of them together (two).
//
// As in k_attn_token a wave has units of its own, fetched into a ring in LDS, and a lane's words are the operands of the
// products as they lie; here a unit's words are made fp16 once for 16 CT columns.  Per unit of 128 channels that is some 224
// instructions beside 16 CT products of 16 x 16 x 32 and some 45 instructions and 8 exponentials per tile of columns.  No values
// go through LDS, and no wave waits for another before the end.
//
// Bound by the vector unit and the matrix unit, which take turns more than they overlap: 32 sequences of 300 to 8191 tokens with
// 8 drafted rows each, 8 x 4 heads of 128, q4_0: 71 us, tiles of 16 columns 94.  Four tiles (64 columns) leave one wave per SIMD and
// were slower wherever tiles of 128 columns were not the better choice anyway.
// Keys are made fp16 in both formats.  q4_0's codes as they are, each block's products scaled in fp32 (as k_attn_token has it),
// need a product of their own per block and tile and 16 multiplications more, and registers for both: 71 -> 83 us for those 32
// sequences (67 registers spilled), 62 -> 64 with heads of 96, 49 -> 54 with 64, and 81 -> 112 with the 16 sequences below (159
// spilled), with the same error to four digits.
// Heads of 256 have one wave per SIMD, which nothing hides the reads of LDS for: issued early (below) they take 16 sequences' 25 rows
// over 4096 tokens and 4 first ones, 2 x 8 heads, q4_1, from 97 to 87 us.  A ring of three units there gained nothing.
// (The compiler spills registers for heads of 128 in q4_1 alone, 6.)
#include "attn_kernel.h"

namespace wq {

namespace {

template <int NB, int CT>
struct WideState {
    f32x4 o[CT][2 * NB];   // channels 16 i + 4 g + 0..3 of column 16 c + lane % 16
    float ref[CT], l[CT];  // l: this lane's tokens only
};

// One unit.  EDGE: it is masked, and columns get a new reference where they need one.  Else all columns see all of it; false
// is returned, with nothing done, if a column needs a new reference.  (The sums are touched in no branch that way: they are in
// accumulation registers, and where such a branch meets the other all of them would be copied.)
template <int NB, bool Q41, bool EDGE, int CT>
__device__ inline bool wide_step(const AttnArgs& a, const SeqInfo& q, const uint8_t* unit, const uint8_t* queries, const float (&sl2)[CT],
                                 int t0, const Column* columns, uint32_t f1024, f16x2 s16, WideState<NB, CT>* st) {
    using R = UnitRing<NB, Q41>;
    // Heads of 256 leave one wave per SIMD, so reads of LDS are issued well before their use, which takes registers that there are.
    constexpr bool early = NB > 4;
    const int lane = threadIdx.x & 63, g = lane >> 4;
    f32x4 s[CT][2];
    uint32_t kw[2 * NB], vw[2 * NB], vd[2][NB][2], vm[2][NB][2];
    const auto read_values = [&]() {
        read_words<NB>(unit + R::half, lane, vw);
#pragma unroll
        for (int tile = 0; tile < 2; tile++) {
            read_scales<NB, NB>(unit + R::half + 16 * R::dim, g, tile, 0, vd[tile]);
            if constexpr (Q41) read_scales<NB, NB>(unit + R::half + 16 * R::dim + R::plane, g, tile, 0, vm[tile]);
        }
    };
    read_words<NB>(unit, lane, kw);
#pragma unroll
    for (int c = 0; c < CT; c++) s[c][0] = s[c][1] = (f32x4){0.0f, 0.0f, 0.0f, 0.0f};
    // (the lane's words are one token's: 4 (r / 4) + r % 4 of the tile)
    const uint8_t* const sc = unit + 16 * R::dim + ((lane & 15) >> 2) * NB * 8 + (lane & 3) * 2;
    _Float16 kd[2][NB], km[2][NB];
    const auto read_key_scales = [&](int b) {
#pragma unroll
        for (int tile = 0; tile < 2; tile++) {
            const uint8_t* const at = sc + (tile * 4 * NB + b) * 8;
            kd[tile][b] = *reinterpret_cast<const _Float16*>(at);
            if constexpr (Q41) km[tile][b] = *reinterpret_cast<const _Float16*>(at + R::plane);
        }
    };
    f16x8 qf[2][CT];
    const auto read_queries = [&](int b) {
#pragma unroll
        for (int c = 0; c < CT; c++) qf[b & 1][c] = *reinterpret_cast<const f16x8*>(queries + ((c * NB + b) * 64 + lane) * 16);
    };
    if constexpr (early) {
#pragma unroll
        for (int b = 0; b < NB; b++) read_key_scales(b);
        read_queries(0);
        __builtin_amdgcn_sched_barrier(0);
    }
#pragma unroll
    for (int b = 0; b < NB; b++) {
        if constexpr (early) {
            if (b + 1 < NB) read_queries(b + 1);
            __builtin_amdgcn_sched_barrier(0);
        } else {
            read_key_scales(b);
        }
        f16x8 k[2];
#pragma unroll
        for (int tile = 0; tile < 2; tile++) {
            const f16x2 d = {kd[tile][b], kd[tile][b]};
            f16x2 m = {};
            if constexpr (Q41) m = (f16x2){km[tile][b], km[tile][b]};
            u32x4 u;
#pragma unroll
            for (int i = 0; i < 4; i++) {
                const f16x2 v = code_pair<Q41 ? 0 : 8>(kw[tile * NB + b], i, f1024, s16);
                u[i] = __builtin_bit_cast(uint32_t, Q41 ? __builtin_elementwise_fma(v, d, m) : v * d);
            }
            k[tile] = __builtin_bit_cast(f16x8, u);
        }
        if constexpr (!early) read_queries(b);
#pragma unroll
        for (int c = 0; c < CT; c++) {
            s[c][0] = __builtin_amdgcn_mfma_f32_16x16x32_f16(k[0], qf[b & 1][c], s[c][0], 0, 0, 0);
            s[c][1] = __builtin_amdgcn_mfma_f32_16x16x32_f16(k[1], qf[b & 1][c], s[c][1], 0, 0, 0);
        }
    }
    uint32_t keep[4] = {~0u, ~0u, ~0u, ~0u};    // token pairs that are in the cache: what lies behind them is anything
    if constexpr (EDGE) {
#pragma unroll
        for (int j = 0; j < 8; j++)
            if (t0 + (j >> 2) * 16 + 4 * g + (j & 3) >= q.tokens) keep[j >> 1] &= (j & 1) ? 0x0000FFFFu : 0xFFFF0000u;
    }
    if constexpr (early) {
        read_values();
        __builtin_amdgcn_sched_barrier(0);
    }
    float e[CT][8], most = -INFINITY;
#pragma unroll
    for (int c = 0; c < CT; c++) {
        const Column& col = columns[16 * c + (lane & 15)];
        uint32_t seen = 0;
        if constexpr (EDGE) seen = seen_tokens(col.lo, col.hi, a.sinks, column_nodes(a, q, col, t0), t0) >> (4 * g);
#pragma unroll
        for (int j = 0; j < 8; j++) {
            e[c][j] = fmaf(s[c][j >> 2][j & 3], sl2[c], -st->ref[c]);
            if constexpr (EDGE) e[c][j] = seen >> ((j >> 2) * 16 + (j & 3)) & 1 ? e[c][j] : -INFINITY;
            most = fmaxf(most, e[c][j]);
        }
    }
    if constexpr (!EDGE) {
        if (__any(most > kRefMost)) return false;
    } else if (__any(most > kRefMost)) {
#pragma unroll
        for (int c = 0; c < CT; c++) {
            float mx = -INFINITY;
#pragma unroll
            for (int j = 0; j < 8; j++) mx = fmaxf(mx, e[c][j] == -INFINITY ? -INFINITY : s[c][j >> 2][j & 3] * sl2[c]);
            mx = fmaxf(mx, __shfl_xor(mx, 16, 64));
            mx = fmaxf(mx, __shfl_xor(mx, 32, 64));
            const float ref = fmaxf(st->ref[c], mx - kRefBelow);
            const float alpha = ref == st->ref[c] ? 1.0f : exp2_fast(st->ref[c] - ref);
#pragma unroll
            for (int i = 0; i < 2 * NB; i++) st->o[c][i] *= alpha;
            st->l[c] *= alpha;
            st->ref[c] = ref;
#pragma unroll
            for (int j = 0; j < 8; j++) e[c][j] = e[c][j] == -INFINITY ? -INFINITY : fmaf(s[c][j >> 2][j & 3], sl2[c], -ref);
        }
    }
    f16x8 pf[CT];
#pragma unroll
    for (int c = 0; c < CT; c++) {
        float x[8];
#pragma unroll
        for (int j = 0; j < 8; j++) x[j] = exp2_fast(e[c][j]);
        st->l[c] += ((x[0] + x[1]) + (x[2] + x[3])) + ((x[4] + x[5]) + (x[6] + x[7]));
        u32x4 p;
#pragma unroll
        for (int j = 0; j < 4; j++) p[j] = pack_f16(x[2 * j], x[2 * j + 1]);
        pf[c] = __builtin_bit_cast(f16x8, p);
    }
    if constexpr (!early) read_values();
#pragma unroll
    for (int b = 0; b < NB; b++) {
        u32x4 vlo, vhi;
#pragma unroll
        for (int tile = 0; tile < 2; tile++) {
            const uint32_t w = vw[2 * b + tile], wl = w & 0x0F0F0F0Fu, wh = w & 0xF0F0F0F0u;
#pragma unroll
            for (int i = 0; i < 2; i++) {
                const uint32_t in = EDGE ? keep[2 * tile + i] : ~0u;
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
#pragma unroll
        for (int c = 0; c < CT; c++) {
            f32x4* const o = st->o[c] + 2 * (b);
            o[0] = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, vlo), pf[c], o[0], 0, 0, 0);
            o[1] = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, vhi), pf[c], o[1], 0, 0, 0);
        }
    }
    return true;
}

template <int NB, bool Q41, int NW, int D, int CT>
struct WideLds {
    static constexpr int ld = 32 * NB + 4, ring = NW * D * UnitRing<NB, Q41>::bytes, join = NW * 16 * (ld + 2) * 4;
    union {
        __attribute__((aligned(16))) uint8_t rings[ring];
        struct {
            float o[NW * 16 * ld], ref[NW * 16], l[NW * 16];
        } join16;
    };
    __attribute__((aligned(16))) uint8_t queries[CT * NB * 1024];   // operands of the products, the same for all waves
    Column columns[16 * CT];
};

// A tile's columns x units [ua, ub) of the list un of one head, by the workgroup (as token_segment).
template <int NB, bool Q41, int NW, int D, int CT>
__device__ void wide_segment(const AttnArgs& a, const TileShape& ts, const SeqInfo& q, int seq, int tile, int h, const UnitList& un,
                             int ua, int ub, float* part_o, float* part_ml, WideLds<NB, Q41, NW, D, CT>& lds) {
    constexpr int dim = 32 * NB, ld = dim + 4;
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6), g = lane >> 4, col = lane & 15;
    const int first = ts.ht == 1 ? tile * ts.rows : tile / ts.ht, last = min(first + ts.rows, q.n) - 1;
    int lo_most, hi_least;
    parts_between(a, q, first, last, &lo_most, &hi_least);

    constexpr int bytes = UnitRing<NB, Q41>::bytes, loads = UnitRing<NB, Q41>::loads;
    const uint8_t* const ring = lds.rings + wave * D * bytes;
    const uint32_t ring_at = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const uint8_t*)ring;
    const int n = ub > ua + wave ? (ub - ua - wave + NW - 1) / NW : 0;   // this wave's units: ua + wave + NW i
    UnitWalk walk;
    walk.start(a.s, seq, h, un[ua + wave]);
    uint32_t absent = 0;    // bit i % 32: unit i's page is none; its request is then any unit, for the count
    int put = 0, get = 0;   // byte offsets of the slots to fill and to read next
    const auto next = [](int at) { return at + bytes == D * bytes ? 0 : at + bytes; };
    const auto request = [&](int i) {
        request_unit<bytes>(walk.at(a.cache), uniform(ring_at + put));
        put = next(put);
        absent = walk.there ? absent & ~(1u << (i & 31)) : absent | 1u << (i & 31);
        if (un.gap(ua + wave + NW * i, NW)) walk.seek(un[ua + wave + NW * (i + 1)]);
        else walk.step(NW);
    };
#pragma unroll
    for (int i = 0; i < D - 1; i++)
        if (i < n) request(i);
    // each wave makes some of the columns' queries
    for (int c = wave; c < CT; c += NW) {
        int row, head;
        const bool valid = tile_col(a, ts, tile, 16 * c + col, q.n, &row, &head);
        u32x4 qv[NB];
        const uint16_t* qp = a.q + (int64_t)(q.r0 + row) * a.ldq + (int64_t)(h * a.group + head) * dim + 8 * g;
        uint32_t big = 0;
#pragma unroll
        for (int b = 0; b < NB; b++) {
            qv[b] = (u32x4){0, 0, 0, 0};
            if (valid) qv[b] = *reinterpret_cast<const u32x4*>(qp + 32 * b);
        }
        const int of = valid ? row : first;
        int lo, hi;
        row_context(a, q, of, &lo, &hi);
        const uint32_t nodes = a.tree ? seen_nodes(a, q, of, (first_node_unit(q) + g) * kUnit) : 0;
#pragma unroll
        for (int b = 0; b < NB; b++) big = max(big, largest_bf16(qv[b]));
        big = max(big, (uint32_t)__shfl_xor((int)big, 16, 64));
        big = max(big, (uint32_t)__shfl_xor((int)big, 32, 64));
        const int up = query_shift(big);
        Column* const to = &lds.columns[16 * c + col];
        if (g == 0) {
            to->lo = lo;
            to->hi = hi;
            to->row = of;
            to->sl2 = ldexpf(a.scale_log2, -up);
        }
        static_assert(kNodeWords == 4);
        to->nodes[g] = nodes;
#pragma unroll
        for (int b = 0; b < NB; b++) *reinterpret_cast<f16x8*>(lds.queries + ((c * NB + b) * 64 + lane) * 16) = query_f16(qv[b], up);
    }
    const uint32_t f1024 = held(0x64006400u);
    const f16x2 s16 = as_f16x2(held(0x2C002C00u));   // 1/16
    WideState<NB, CT> st;
#pragma unroll
    for (int c = 0; c < CT; c++) {
#pragma unroll
        for (int i = 0; i < 2 * NB; i++) st.o[c][i] = (f32x4){0, 0, 0, 0};
        st.ref[c] = -FLT_MAX;
        st.l[c] = 0.0f;
    }
    __syncthreads();   // the queries
    float sl2[CT];
#pragma unroll
    for (int c = 0; c < CT; c++) sl2[c] = lds.columns[16 * c + col].sl2;

    int i = 0;
    const auto fetch = [&]() {     // unit i's bytes are there
        if (i + D - 1 < n) {
            wait_lds();     // unit i - 1's reads, whose slot the request fills
            request(i + D - 1);
            wait_loads<(D - 1) * loads>();
        } else {
            wait_loads<0>();
        }
    };
    while (i < n) {
        fetch();
        while (true) {
            const int t0 = un[ua + wave + NW * i] * kUnit;
            if (t0 < lo_most || t0 + kUnit > hi_least || (absent >> (i & 31) & 1)) break;
            if (!wide_step<NB, Q41, false, CT>(a, q, ring + get, lds.queries, sl2, t0, lds.columns, f1024, s16, &st)) break;
            get = next(get);
            if (++i >= n) break;
            fetch();
        }
        if (i >= n) break;
        if (!(absent >> (i & 31) & 1))
            wide_step<NB, Q41, true, CT>(a, q, ring + get, lds.queries, sl2, un[ua + wave + NW * i] * kUnit, lds.columns, f1024, s16, &st);
        get = next(get);
        i++;
    }

    // the waves' sums, joined in LDS (where the rings were), 16 columns at a time
#pragma unroll
    for (int c = 0; c < CT; c++) {
        __syncthreads();
        float l = st.l[c];
        l += __shfl_xor(l, 16, 64);
        l += __shfl_xor(l, 32, 64);
        if (lane < 16) {
            lds.join16.ref[wave * 16 + lane] = st.ref[c];
            lds.join16.l[wave * 16 + lane] = l;
        }
#pragma unroll
        for (int i = 0; i < 2 * NB; i++) *reinterpret_cast<f32x4*>(lds.join16.o + (wave * 16 + col) * ld + 16 * i + 4 * g) = st.o[c][i];
        __syncthreads();
        for (int i = threadIdx.x; i < 16 * (dim / 4); i += NW * 64) {
            const int k = i / (dim / 4), ch = (i - k * (dim / 4)) * 4;
            int row, head;
            if (!tile_col(a, ts, tile, 16 * c + k, q.n, &row, &head)) continue;
            float ref = lds.join16.ref[k];
#pragma unroll
            for (int w = 1; w < NW; w++) ref = fmaxf(ref, lds.join16.ref[w * 16 + k]);
            f32x4 o = {0, 0, 0, 0};
            float sum = 0.0f;
#pragma unroll
            for (int w = 0; w < NW; w++) {
                const float f = exp2_fast(lds.join16.ref[w * 16 + k] - ref);
                sum += f * lds.join16.l[w * 16 + k];
                o += f * *reinterpret_cast<const f32x4*>(lds.join16.o + (w * 16 + k) * ld + ch);
            }
            if (part_o) {
                *reinterpret_cast<f32x4*>(part_o + (16 * c + k) * dim + ch) = o;
                if (ch == 0) {
                    part_ml[2 * (16 * c + k)] = ref;
                    part_ml[2 * (16 * c + k) + 1] = sum;
                }
            } else {
                const float inv = sum != 0.0f ? 1.0f / sum : 0.0f;
                const u32x2 y = {pack_bf16(o[0] * inv, o[1] * inv), pack_bf16(o[2] * inv, o[3] * inv)};
                *reinterpret_cast<u32x2*>(a.y + (int64_t)(q.r0 + row) * a.ldy + (int64_t)(h * a.group + head) * dim + ch) = y;
            }
        }
    }
    __syncthreads();
}

template <int NB, bool Q41, int NW, int D, int CT, int EU>
__global__ __launch_bounds__(NW * 64) __attribute__((amdgpu_waves_per_eu(EU))) void k_attn_wide(AttnArgs a) {
    __shared__ WideLds<NB, Q41, NW, D, CT> lds;
    each_part(a, tile_shape(16 * CT, a.group),
              [&](const TileShape& ts, const SeqInfo& q, int seq, int tile, int h, const UnitList& un, int ua, int ub, float* po,
                  float* pm) { wide_segment<NB, Q41, NW, D, CT>(a, ts, q, seq, tile, h, un, ua, ub, po, pm, lds); });
}

constexpr int kTiles = 2;

// Rings of two units leave LDS for three workgroups per compute unit, and EU 3 the registers for as many waves per SIMD.
template <int NB, int NW, int D, int EU>
void launch_as(const AttnArgs& a, dim3 grid, hipStream_t s) {
    if (a.q41) hipLaunchKernelGGL((k_attn_wide<NB, true, NW, D, kTiles, EU>), grid, dim3(NW * 64), 0, s, a);
    else hipLaunchKernelGGL((k_attn_wide<NB, false, NW, D, kTiles, EU>), grid, dim3(NW * 64), 0, s, a);
}

}  // namespace

void launch_attn_wide(const AttnArgs& a, dim3 grid, hipStream_t s) {
    switch (a.dim) {
    case 64: launch_as<2, 4, 3, 3>(a, grid, s); break;
    case 96: launch_as<3, 4, 2, 3>(a, grid, s); break;
    case 128: launch_as<4, 4, 2, 3>(a, grid, s); break;
    default: launch_as<8, 4, 2, 1>(a, grid, s); break;
    }
}

}  // namespace wq
