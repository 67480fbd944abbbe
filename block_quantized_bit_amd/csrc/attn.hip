// attn.hip -- attention over the 4-bit cache: how a call runs, its kernels over one range of tokens per row (those with sinks
// or trees are attn_parts.hip's), and the joins of shared-out work.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "attn_kernel.h"

namespace wq {

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

// Four columns by a wave, for the few parts of a draft's tiles, which have many columns: 16 lanes each, a lane's channels 64
// apart in runs of four.
__device__ inline void join_four_columns(const AttnArgs& a, const Partials& p, int n, int col, uint16_t* y, int slot0) {
    const int lane = threadIdx.x & 15, group = threadIdx.x & 48, quads = a.dim / 4;
    const auto slot = [&](int i) { return slot0 + 2 * i + (i == 0); };
    constexpr int most = 4, ahead = 2;        // runs of a lane; parts requested before their factors are known
    f32x4 o[most], early[ahead][most];
#pragma unroll
    for (int i = 0; i < ahead; i++)
#pragma unroll
        for (int k = 0; k < most; k++)
            if (y && lane + 16 * k < quads && i < n) early[i][k] = p.read(slot(i), col, 4 * lane + 64 * k);
    float m = -FLT_MAX, l = 0.0f;
    if (y && lane < n) {
        const f32x2 st = p.read_stat(slot(lane), col);
        m = st[0];
        l = st[1];
    }
    float ref = m;
#pragma unroll
    for (int d = 8; d >= 1; d >>= 1) ref = fmaxf(ref, __shfl_xor(ref, d, 64));
    const float f = exp2_fast(m - ref);
    l *= f;
#pragma unroll
    for (int d = 8; d >= 1; d >>= 1) l += __shfl_xor(l, d, 64);
#pragma unroll
    for (int k = 0; k < most; k++) o[k] = (f32x4){0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < ahead; i++) {
        const float fi = __shfl(f, group + i, 64);
#pragma unroll
        for (int k = 0; k < most; k++)
            if (y && lane + 16 * k < quads && i < n) o[k] += fi * early[i][k];
    }
    for (int i = ahead; i < n; i++) {
        const float fi = __shfl(f, group + i, 64);
#pragma unroll
        for (int k = 0; k < most; k++)
            if (y && lane + 16 * k < quads) o[k] += fi * p.read(slot(i), col, 4 * lane + 64 * k);
    }
    const float inv = l != 0.0f ? 1.0f / l : 0.0f;
#pragma unroll
    for (int k = 0; k < most; k++)
        if (y && lane + 16 * k < quads)
            *reinterpret_cast<u32x2*>(y + 4 * lane + 64 * k) = (u32x2){pack_bf16(o[k][0] * inv, o[k][1] * inv), pack_bf16(o[k][2] * inv, o[k][3] * inv)};
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

// The same for a draft's tiles, with COLS columns each, by workgroup (tile, run of columns).  FIND: few tiles, that have many parts
// each: workgroup i takes the i-th tile there is (looking for it costs 2 us; a workgroup for each one that may have begun a
// tile would leave most with nothing: 8 tiles of 128 columns in 64 parts took 70 us, and take 12).
template <bool FIND, int COLS>
__global__ __launch_bounds__(256) void k_attn_join_draft(AttnArgs a) {
    __shared__ __attribute__((aligned(16))) JoinLds lds;
    __shared__ int found;
    int first = blockIdx.x;                   // the workgroup that began the tile
    if (FIND) {
        const int tid = threadIdx.x, i = 2 * tid;   // (at most 512)
        const uint32_t one = i < a.workgroups && open_tile(a, i)->parts > 0, two = i + 1 < a.workgroups && open_tile(a, i + 1)->parts > 0;
        const uint32_t in = wave_scan(one + two);
        uint32_t* const sums = reinterpret_cast<uint32_t*>(lds.red);
        if (tid == 0) found = -1;
        if ((tid & 63) == 63) sums[tid >> 6] = in;
        __syncthreads();
        uint32_t before = in - one - two;
        for (int w = 0; w < tid >> 6; w++) before += sums[w];
        if (one && before == blockIdx.x) found = i;
        if (two && before + one == blockIdx.x) found = i + 1;
        __syncthreads();
        first = uniform(found);
        if (first < 0) return;
    }
    const int32_t* const d = &open_tile(a, first)->parts;
    const OpenTile t = {read_const(d, 0), read_const(d, 1), read_const(d, 2), read_const(d, 3), read_const(d, 4)};
    if (t.parts == 0) return;
    const TileShape ts = even_shape(tile_shape(COLS, a.group), t.n);
    const Partials p(a);
    const auto slot = [&](int i) { return 2 * (first + i) + (i == 0); };
    const auto to = [&](int col) {
        int row, head;
        return tile_col(a, ts, t.tile, col, t.n, &row, &head) ? a.y + (int64_t)(t.r0 + row) * a.ldy + (int64_t)(t.head * a.group + head) * a.dim : nullptr;
    };
    if (t.parts <= kWaveParts) {
        for (int col = blockIdx.y * 16; col < COLS && to(col); col += 16 * gridDim.y)
            join_four_columns(a, p, t.parts, col + (threadIdx.x >> 4), to(col + (threadIdx.x >> 4)), 2 * first);
        return;
    }
    for (int col = blockIdx.y; col < COLS && to(col); col += gridDim.y) join_column(a, p, t.parts, col, to(col), slot, lds);
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
    int cols;            // columns per tile: 16, 128 or 256; drafts: 32 too
    int64_t items;       // tiles x heads (at most)
    int workgroups;      // 16 columns, and drafts: sequences shared out over so many (0: not)
    int splits;          // 128, 256 columns: parts per tile
    bool token() const { return cols < 128; }
    int slots() const { return workgroups > 0 || token() ? 2 * workgroups : splits > 1 ? (int)items * splits : 0; }
};

// Units that a sequence's rows see, of the `most` that it can have: with sinks and a window, those and the rows themselves.
int64_t seen_units(const AttnArgs& a, int64_t most) {
    if (!a.parts || a.window == 0) return most;
    const int64_t rows = a.s.row_start ? (a.s.rows + (int64_t)a.s.batch - 1) / a.s.batch : 1;   // on average
    return std::min(most, ((int64_t)a.sinks + kUnit - 1) / kUnit + (a.window + rows + kUnit - 1) / kUnit + 1);
}

// Drafts: `cols` columns per sequence on average, more than 16.  Measured in us, q4_0, 8 x 4 heads of 128 / of 96 / of 64, contexts of
// one length (whole) or of 300 to so many tokens (shared out, over 256 workgroups for tiles of 256, else 512):
//   tiles of                          16           32          128          256
//   whole     4 x 128,  1500     21/ 18/ 16   31/ 26/ 21   58/ 52/ 40   48/ 44/ 40
//            32 x  80,  1500     68/ 51/ 39   54/ 48/ 37   62/ 58/ 41   52/ 48/ 42
//            32 x 128,   500     55/ 39/ 29   43/ 37/ 31   33/ 28/ 23   30/ 27/ 24
//            32 x 200,  1000    121/ 88/ 64   89/ 77/ 61   68/ 57/ 46   57/ 50/ 42
//            64 x 28 to 320, 300 to 1000
//                               156/111/ 83  118/101/ 80  100/ 88/ 69  113/101/ 87
//            32 x 256,  1500    204/140/105  132/112/ 89   92/ 79/ 63   84/ 72/ 58
//            16 x 512,  3000    345/237/178  206/174/135  152/134/106  135/117/ 98
//   shared   32 x  32,  8191     95/ 78/ 64   73/ 63/ 51   95/ 91/ 67  121/120/104
//   out       8 x  64, 30000    147/123/ 96  109/ 97/ 75  105/100/ 74  120/117/ 99
//            32 x 128,  8191    286/244/189  209/186/145  143/122/ 94  155/138/122
//            32 x 28 to 256, 8191
//                               323/275/216  232/200/156  181/159/123  179/158/136
//            32 x 200,  8191    358/305/236  272/240/187  211/182/147  184/159/137   (120 to 200)
//             8 x 256, 30000    488/417/327  343/308/237  214/183/143  188/154/130
// Wider tiles share conversions, but take more registers and longer to begin: they pay where there are enough of them for the
// chip, or they are shared out.  Sharing out costs some 15 us (finding the work, and the join), as for single tokens.  Between 129
// and 255 columns equal drafts would gain up to a fifth by tiles of 256, and unequal ones, that the average says nothing of, lose up to a
// fifth: those of 128 are taken.
// Heads of 256 leave tiles of 32 columns one wave per SIMD, and those of 128 one workgroup per compute unit.  2 x 8 heads, q4_1
// (=: all of that length), shared out over 512 workgroups for tiles of 16, else 256:
//   tiles of                    16     32    128
//   whole    16 x 200,  4000   103     81    280
//            32 x 200,  1000    67     70     91
//            64 x 512,   500   164    196    126
//   shared   16 x  96, =12000  130    108    128
//   out      16 x 200, =12000  257    200    236
//            16 x 200,  12000  154    177    151
//            16 x 200,  20000  237    243    215
//            16 x 512,   8191  252    273    204
//             8 x 200, =12000  140    118    138
//             8 x 200,  30000  197    227    182
//             4 x 512,  =8000  113     90    118
// Shared out, contexts of one length are faster in tiles of 32, unequal ones in tiles of 128, and the table's width, which is all that the
// host knows, does not say which there are: with 64 tiles or more it goes by unequal ones, with fewer by equal ones.
void draft_schedule(const AttnArgs& a, bool share, int64_t most, int64_t units, int64_t cols, Schedule* s) {
    const auto items = [&](int c) { return tile_bound(tile_shape(c, a.group), a.s.rows, a.s.batch, false) * a.s.heads; };
    const auto take = [&](int c, int workgroups) {
        s->cols = c;
        s->items = items(c);
        s->workgroups = share && s->items * (most + kTileCost) <= 0x7FFFFFFF ? workgroups : 0;
    };
    const bool lengthy = units > (items(kTokenCols) < 256 ? 64 : 128);
    if (a.dim == 256) {
        const bool out = lengthy && share;
        if (cols >= 160 && items(128) >= (out ? 64 : 256) && (!out || units >= 256 || cols >= 512)) take(128, out ? kShareWorkgroups / 2 : 0);
        else if (units >= 64 && cols >= (out ? 80 : 160)) take(32, out && (items(32) < 192 || units >= 256) ? kShareWorkgroups / 2 : 0);
        else take(kTokenCols, out ? kShareWorkgroups : 0);
    } else if (lengthy && share) {
        if (cols > 64) take(cols < 256 ? 128 : 256, cols < 256 ? kShareWorkgroups : kShareWorkgroups / 2);
        else take(32, kShareWorkgroups);
    } else if (cols >= 112 && items(128) >= 256) {
        take(cols >= 256 && items(256) >= 256 ? 256 : 128, 0);
    } else {
        take(items(32) >= 512 ? 32 : kTokenCols, 0);
    }
}

Schedule schedule(const AttnArgs& a, bool share) {
    Schedule s{};
    const auto items = [&](int cols) {
        s.cols = cols;
        s.items = tile_bound(tile_shape(cols, a.group), a.s.rows, a.s.batch, !a.s.row_start) * a.s.heads;
    };
    const int64_t most = ((int64_t)a.s.table_ld * a.s.page) / kUnit, units = seen_units(a, most);   // of the longest sequence there can be
    s.splits = 1;
    const int64_t pairs = (int64_t)a.s.rows * a.group, batch = a.s.batch;
    if (a.parts && a.s.row_start && pairs > kTokenCols * batch && (a.tree_rows || pairs < kManyCols * batch)) {
        draft_schedule(a, share, most, units, pairs / batch, &s);
        return s;
    }
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
        if (share && units > (s.items < 256 ? 64 : 128) && s.items * (most + kTileCost) <= 0x7FFFFFFF)
            s.workgroups = kShareWorkgroups;
    }
    return s;
}

template <int COLS>
void launch_join(const AttnArgs& a, int64_t items, int cols, hipStream_t s) {
    if (items >= 64) hipLaunchKernelGGL((k_attn_join_draft<false, COLS>), dim3(a.workgroups - 1, (cols + 15) / 16), dim3(256), 0, s, a);
    else hipLaunchKernelGGL((k_attn_join_draft<true, COLS>), dim3((unsigned)items, cols), dim3(256), 0, s, a);
}

}  // namespace

// A launch has fewer than 2^32 threads.
bool attn_fits(const AttnArgs& a) {
    const Schedule s = schedule(a, true), w = schedule(a, false);   // with and without a workspace
    return std::max(s.items * s.splits, w.items) < (int64_t(1) << 23);
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
    if (!c.token()) {
        const dim3 grid((unsigned)(c.items * c.splits));
        if (c.workgroups) {
            launch_parts_shared(a, dim3(c.workgroups), c.cols == 256, s);
            c.cols == 256 ? launch_join<256>(a, c.items, cols, s) : launch_join<128>(a, c.items, cols, s);
            return hipGetLastError();
        }
        if (a.parts) launch_parts_rows(a, grid, c.cols == 256, s);
        else launch_rows<false>(a, grid, c.cols == 256, s);
        if (c.splits > 1) hipLaunchKernelGGL(k_attn_join_rows, dim3((unsigned)c.items, std::min(cols, 64)), dim3(256), 0, s, a);
        return hipGetLastError();
    }
    const dim3 grid((unsigned)(c.workgroups ? c.workgroups : c.items));
    // With at most a tile per compute unit eight waves share a tile's tokens (1024 tokens, 8 tiles of 4 x 128: 13.6 ->
    // 11.4 us; 80 tiles of 1500 x 64: 12.3 -> 10.3); with more, four (320 tiles of 1500 x 64: 20.2 -> 16.5 us).
    const bool few = !c.workgroups && c.items <= 256;
    if (c.cols != kTokenCols) launch_attn_wide(a, grid, s);
    else if (a.parts) launch_parts_token(a, grid, few, s);
    else launch_token<false>(a, grid, few, s);
    // (with few tiles each has many parts, and a workgroup takes one column at a time, not four)
    if (c.workgroups) {
        if (c.cols == 32) launch_join<32>(a, c.items, cols, s);
        else if (c.items * 8 >= c.workgroups) hipLaunchKernelGGL(k_attn_join_token<true>, dim3(c.workgroups - 1, (cols + 3) / 4), dim3(256), 0, s, a);
        else hipLaunchKernelGGL(k_attn_join_token<false>, dim3(c.workgroups - 1, std::min(cols, 8)), dim3(256), 0, s, a);
    }
    return hipGetLastError();
}

}  // namespace wq
