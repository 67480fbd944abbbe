// pages.hip -- the pages of a cache's sequences: taken from a list of free ones as sequences grow, given back as they shrink or
// end, with the block table, the row starts and the rows' places that the other calls take.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "cache_device.h"
#include "wq_launch.h"

namespace wq {

namespace {

constexpr int kThreads = 1024;

// Exclusive prefix sums over the workgroup; returns the total.
__device__ inline int64_t block_scan(int64_t v, int64_t* before, int64_t* lds) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    int64_t in = v;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int64_t x = __shfl_up(in, d, 64);
        if (lane >= d) in += x;
    }
    __syncthreads();
    if (lane == 63) lds[wave] = in;
    __syncthreads();
    int64_t run = 0, total = 0;
    for (int w = 0; w < kThreads / 64; w++) {
        if (w < wave) run += lds[w];
        total += lds[w];
    }
    *before = run + in - v;
    return total;
}

// A division by the page's 32s takes five instructions this way, where the compiler's takes some 25.
__device__ inline uint32_t page_of(const PagesArgs& a, uint32_t token) { return (uint32_t)((uint64_t)(token / kUnit) * a.times >> a.shift); }
__device__ inline int pages_of(const PagesArgs& a, int tokens) {
    return (int)min(page_of(a, (uint32_t)tokens + (uint32_t)a.page - 1), (uint32_t)a.table_ld);   // (below 2^31 + 2^24)
}
__device__ inline bool is_page(const PagesArgs& a, int p) { return p >= 0 && p < a.pages; }

}  // namespace

__global__ __launch_bounds__(256) void k_pages_init(int pages, int32_t* pool) {
    const uint32_t i = blockIdx.x * 256 + threadIdx.x;   // (past 2^31 in the last workgroup of the largest list)
    if (i < 4) pool[i] = i == 0 ? pages : 0;
    if (i < (uint32_t)pages) pool[4 + (int64_t)i] = pages - 1 - (int)i;
}

// The call for up to kSeqsAtOnce sequences.  Every workgroup makes the sums over all sequences for itself, in LDS (rows, pages
// wanted, pages given back, each before a sequence), and then does its share of the rows, of the table's new entries and of the
// list's.  Nothing that a workgroup reads is written by another: the page of a wanted entry comes from the entry that is given
// back or from the list itself, not from the table; what is put on the list goes where nothing was; and the lengths and the
// count of free pages, which all of them read, are written by a launch after it (k_pages_settle) if there are several.  (The
// workgroup that is the last to be done could write them, by a counter in the pool; but that goes by what the caller has there,
// and its round trips cost more: two calls, of 4096 drafts 28.3 us and 27.0 now, of 61 prompts 19.3 and 17.7.)
constexpr int kSeqsAtOnce = 8192, kAtOnce = 4;   // kAtOnce: items of a thread that are on their way together
// What bounds it: the sums' instructions, which every workgroup has for itself, and the way to memory and back (lengths, table,
// list, one after the other).  In us as traced, a call that takes and one that gives back: 96 sequences of one row 4.9 and 4.9, 61
// prompts of 282 thousand rows and 4400 pages 7.7, with 1.3 of k_pages_settle, and 8.1, 4096 drafts of 139 thousand rows and 4300 pages
// 11.1, with 4.0, and 14.4.  The workgroups go by the rows, so that pages are given back without rows by one: 200 thousand of 40
// sequences 227 us.  Up to kFewSeqs sequences take little LDS, which leaves a compute unit room for others' workgroups, and some 0.05 us
// a call (two calls of the 96 in a replayed graph 9.8 us, with the LDS of more 9.9).
constexpr int kFewSeqs = 1024;

// a + b, at most `most`: associative for numbers that are at most that.
__device__ inline uint32_t add_to(uint32_t a, uint32_t b, uint32_t most) { return min(a + b, most); }

template <int CTRL, int ROWS>
__device__ inline uint32_t add_dpp_to(uint32_t v, uint32_t most) {
    return add_to(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, ROWS, 0xF, false), most);
}

template <int SEQS>
struct PagesLds {
    uint32_t wave[3][kThreads / 64];
    uint32_t row[SEQS + 1], come[SEQS + 1], gone[SEQS + 1];   // before a sequence
    int had[SEQS];                                            // its pages
};

// The last sequence whose sum before it is at most i (that has the i-th item, for an i below the total).
__device__ inline int holder(const uint32_t* before, int batch, uint32_t i) {
    int lo = 0, hi = batch;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (before[mid] <= i) lo = mid;
        else hi = mid;
    }
    return lo;
}

struct SumArrays {
    uint32_t* of[3];
};
// Numbers per sequence become the sums before each (one entry more: the total), K arrays at once.  A thread has `per`
// neighbouring sequences, an odd number, so that the threads' places are in different banks.
template <int K, int SEQS>
__device__ inline void sums_before(const SumArrays& arrays, int batch, const uint32_t* most, PagesLds<SEQS>& lds, uint32_t* total) {
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int per = ((batch + kThreads - 1) / kThreads) | 1, b0 = min(tid * per, batch), b1 = min(b0 + per, batch);
    uint32_t sum[K];
#pragma unroll
    for (int k = 0; k < K; k++) {
        uint32_t in = 0;
        for (int b = b0; b < b1; b++) in = add_to(in, arrays.of[k][b], most[k]);
        in = add_dpp_to<0x111, 0xF>(in, most[k]);   // over rows of 16 lanes, then the rows' totals (as wave_scan)
        in = add_dpp_to<0x112, 0xF>(in, most[k]);
        in = add_dpp_to<0x114, 0xF>(in, most[k]);
        in = add_dpp_to<0x118, 0xF>(in, most[k]);
        in = add_dpp_to<0x142, 0xA>(in, most[k]);
        in = add_dpp_to<0x143, 0xC>(in, most[k]);
        if (lane == 63) lds.wave[k][wave] = in;
        const uint32_t x = __shfl_up(in, 1, 64);
        sum[k] = lane ? x : 0;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < K; k++) {
        uint32_t run = 0;
        total[k] = 0;
        for (int w = 0; w < kThreads / 64; w++) {
            if (w < wave) run = add_to(run, lds.wave[k][w], most[k]);
            total[k] = add_to(total[k], lds.wave[k][w], most[k]);
        }
        run = add_to(run, sum[k], most[k]);
        for (int b = b0; b < b1; b++) {
            const uint32_t n = arrays.of[k][b];
            arrays.of[k][b] = run;
            run = add_to(run, n, most[k]);
        }
        if (tid == 0) arrays.of[k][batch] = total[k];
    }
    __syncthreads();
}

template <int SEQS>
__global__ __launch_bounds__(kThreads) void k_pages_assign(PagesArgs a) {
    __shared__ PagesLds<SEQS> lds;
    const int tid = threadIdx.x, batch = a.batch;
    const uint32_t most[3] = {0x7FFFFFFFu, 0x7FFFFFFFu, (uint32_t)a.rows};
    const int free0 = a.pool[0];
    const uint32_t free = (uint32_t)(free0 < 0 ? 0 : min(free0, a.pages));
    int32_t* const list = a.pool + 4;
    for (int b0 = 0; b0 < batch; b0 += kAtOnce * kThreads) {   // (what a run of sequences leaves out is left out by all)
        int len[kAtOnce], want[kAtOnce];
#pragma unroll
        for (int k = 0; k < kAtOnce; k++) {
            if (b0 + k * kThreads >= batch) break;
            const int b = min(b0 + k * kThreads + tid, batch - 1);
            len[k] = a.len[b];
            want[k] = a.want[b];
        }
#pragma unroll
        for (int k = 0; k < kAtOnce; k++) {
            if (b0 + k * kThreads >= batch) break;
            const int b = b0 + k * kThreads + tid, l = max(len[k], 0), w = max(want[k], 0), had = pages_of(a, l), gets = pages_of(a, w);
            if (b >= batch) continue;
            lds.row[b] = (uint32_t)min(max(w - l, 0), a.rows);
            lds.come[b] = (uint32_t)max(gets - had, 0);
            lds.gone[b] = (uint32_t)max(had - gets, 0);
            lds.had[b] = had;
        }
    }
    __syncthreads();
    uint32_t total[3];
    sums_before<3>({lds.gone, lds.come, lds.row}, batch, most, lds, total);
    const uint32_t rows = total[2], come = total[1], entries = total[0];

    // Entries that are given back, by their number.
    const auto entry = [&](uint32_t i) {
        const int b = holder(lds.gone, batch, i);
        return a.table[(int64_t)b * a.table_ld + (lds.had[b] - (int)(lds.gone[b + 1] - i))];
    };
    bool holes = false;                       // whether some of them are no page
    uint32_t none = 0;                        // how many: of this thread's, then of all
    int first[kAtOnce];                       // entries tid + k kThreads
    if (entries > 0) {
#pragma unroll
        for (int k = 0; k < kAtOnce; k++)
            if (tid + k * kThreads < entries) first[k] = entry(tid + k * kThreads);
#pragma unroll
        for (int k = 0; k < kAtOnce; k++)
            if (tid + k * kThreads < entries) none += !is_page(a, first[k]);
        for (uint32_t i0 = tid + kAtOnce * kThreads; i0 < entries; i0 += kAtOnce * kThreads) {
            int p[kAtOnce];
#pragma unroll
            for (int k = 0; k < kAtOnce; k++)
                if (i0 + k * kThreads < entries) p[k] = entry(i0 + k * kThreads);
#pragma unroll
            for (int k = 0; k < kAtOnce; k++)
                if (i0 + k * kThreads < entries) none += !is_page(a, p[k]);
        }
        holes = __syncthreads_or(none > 0);
    }
    // Pages are numbered then, not entries, which a workgroup does as it goes over them in order: the first does all there is to
    // do.  (30000 pages of one sequence with such an entry 39 us, without one 22; each page counted from its sequence's start 62 ms.)
    if (holes && blockIdx.x > 0) return;
    if (holes) {
        none = wave_scan(none);
        if ((tid & 63) == 63) lds.wave[0][tid >> 6] = none;
        __syncthreads();
        none = 0;
        for (int w = 0; w < kThreads / 64; w++) none += lds.wave[0][w];
    }
    const uint32_t gone = entries - none, top = free + gone;   // pages given back, pages there are to take
    const uint32_t threads = holes ? kThreads : gridDim.x * kThreads, at = blockIdx.x * kThreads + tid;
    const auto on_list = [&](uint32_t i) { return i < top ? list[free - 1 - (i - gone)] : -1; };   // the i-th wanted page, from the gone-th on
    const auto taken = [&](uint32_t i) { return i < gone ? entry(i) : on_list(i); };               // (without holes)
    const auto take = [&](uint32_t i, int page) {
        const int b = holder(lds.come, batch, i);
        a.table[(int64_t)b * a.table_ld + lds.had[b] + (i - lds.come[b])] = page;
    };
    const auto put = [&](uint32_t i, int page) {
        if (i >= come && i < gone && top - 1 - i < (uint32_t)a.pages) list[top - 1 - i] = page;
    };
    if (holes) {
        uint32_t run = 0;
        for (uint32_t i0 = 0; i0 < entries; i0 += kThreads) {
            const int page = i0 + tid < entries ? entry(i0 + tid) : -1;
            const bool is = is_page(a, page);
            const uint64_t which = __ballot(is);
            __syncthreads();                  // (the last counts are read)
            if ((tid & 63) == 0) lds.wave[0][tid >> 6] = __popcll(which);
            __syncthreads();
            uint32_t i = run + __popcll(which & ((1ull << (tid & 63)) - 1));
            for (int w = 0; w < kThreads / 64; w++) {
                if (w < tid >> 6) i += lds.wave[0][w];
                run += lds.wave[0][w];
            }
            if (is && i < come) take(i, page);
            else if (is) put(i, page);
        }
        for (uint32_t i = gone + tid; i < come; i += kThreads) take(i, on_list(i));
        __syncthreads();                      // the rows' pages are in the table
    }
    // Else the table's new entries, and what goes on the list: by the last threads first, the rows by the first.
    if (!holes) {
        const uint32_t last = threads - 1 - at;
        for (uint32_t i0 = last; i0 < come; i0 += kAtOnce * threads) {
            int p[kAtOnce];
#pragma unroll
            for (int k = 0; k < kAtOnce; k++)
                if (i0 + k * threads < come) p[k] = taken(i0 + k * threads);
#pragma unroll
            for (int k = 0; k < kAtOnce; k++)
                if (i0 + k * threads < come) take(i0 + k * threads, p[k]);
        }
        const bool kept = gridDim.x == 1;
        if (kept) {
#pragma unroll
            for (int k = 0; k < kAtOnce; k++) put(tid + k * kThreads, first[k]);
        }
        const uint32_t behind = kept ? kAtOnce * kThreads : 0;
        for (uint32_t i0 = max(come, behind) + last; i0 < gone; i0 += kAtOnce * threads) {
            int p[kAtOnce];
#pragma unroll
            for (int k = 0; k < kAtOnce; k++)
                if (i0 + k * threads < gone) p[k] = entry(i0 + k * threads);
#pragma unroll
            for (int k = 0; k < kAtOnce; k++) put(i0 + k * threads, p[k]);
        }
    }
    if (a.pos || a.slot) {
        for (uint32_t r0 = at; r0 < rows; r0 += kAtOnce * threads) {
            int b[kAtOnce], t[kAtOnce], j[kAtOnce], p[kAtOnce];
#pragma unroll
            for (int k = 0; k < kAtOnce; k++) {
                const uint32_t r = r0 + k * threads;
                if (r >= rows) break;
                b[k] = holder(lds.row, batch, r);
                t[k] = max(a.want[b[k]], 0) - (int)(lds.row[b[k] + 1] - r);
            }
            if (a.slot) {
#pragma unroll
                for (int k = 0; k < kAtOnce; k++) {
                    if (r0 + k * threads >= rows) break;
                    j[k] = (int)page_of(a, (uint32_t)t[k]);
                    const int had = lds.had[b[k]];
                    p[k] = -1;
                    if (j[k] < (holes ? a.table_ld : had)) p[k] = a.table[(int64_t)b[k] * a.table_ld + j[k]];
                    else if (j[k] < a.table_ld) p[k] = taken(lds.come[b[k]] + (j[k] - had));
                }
            }
#pragma unroll
            for (int k = 0; k < kAtOnce; k++) {
                const uint32_t r = r0 + k * threads;
                if (r >= rows) break;
                if (a.pos) a.pos[r] = t[k];
                if (a.slot) a.slot[r] = is_page(a, p[k]) ? (int64_t)p[k] * a.page + (t[k] - j[k] * a.page) : -1;
            }
        }
    }
    for (int b = at; b <= batch; b += threads) a.row_start[b] = (int)lds.row[b];
    // what others may still read
    const int left = (int)min(top > come ? top - come : 0u, (uint32_t)a.pages), lacking = (int)(come > top ? come - top : 0u);
    if (gridDim.x > 1) {
        if (at == 0) {
            a.pool[1] = lacking;
            a.pool[2] = left;
        }
        return;
    }
    __syncthreads();
    for (int b0 = 0; b0 < batch; b0 += kAtOnce * kThreads) {
        int want[kAtOnce];
#pragma unroll
        for (int k = 0; k < kAtOnce; k++) {
            if (b0 + k * kThreads >= batch) break;
            want[k] = a.want[min(b0 + k * kThreads + tid, batch - 1)];
        }
#pragma unroll
        for (int k = 0; k < kAtOnce; k++) {
            if (b0 + k * kThreads >= batch) break;
            const int b = b0 + k * kThreads + tid;
            if (b < batch) a.len[b] = max(want[k], 0);
        }
    }
    if (tid == 0) {
        a.pool[0] = left;
        a.pool[1] = lacking;
        a.pool[2] = 0;
    }
}

// What the workgroups of k_pages_assign read, and the pool's count, which the first of them left in word 2.
__global__ __launch_bounds__(256) void k_pages_settle(PagesArgs a) {
    const int b = blockIdx.x * 256 + threadIdx.x;
    if (b < a.batch) a.len[b] = max(a.want[b], 0);
    if (b == 0) {
        a.pool[0] = a.pool[2];
        a.pool[2] = 0;
    }
}

// More sequences, or more entries than 32 bits count: one workgroup, and the rows by a launch of their own.  First what is given
// back goes on the list's end (its front), the first sequence's first page last; then what is wanted is taken from there.  Bound by
// the one workgroup's three walks, one after the other (with 11 registers spilled): 16384 sequences of a row each 87 us, 65536 316.
__global__ __launch_bounds__(kThreads) void k_pages_assign_many(PagesArgs a) {
    __shared__ int64_t lds[kThreads / 64];
    int32_t* const list = a.pool + 4;
    const int64_t free = a.pool[0] < 0 ? 0 : a.pool[0] < a.pages ? a.pool[0] : a.pages;
    const auto lengths = [&](int b, int* had, int* gets) {
        const int len = max(a.len[b], 0), want = max(a.want[b], 0);
        *had = pages_of(a, len);
        *gets = pages_of(a, want);
        return max(want - len, 0);
    };
    const auto returned = [&](int b, int had, int gets) {
        int64_t n = 0;
        for (int j = gets; j < had; j++) n += is_page(a, a.table[(int64_t)b * a.table_ld + j]);
        return n;
    };
    int64_t gone = 0, come = 0, rows = 0, before;
    for (int b0 = 0; b0 < a.batch; b0 += kThreads) {
        const int b = b0 + threadIdx.x;
        int had = 0, gets = 0;
        if (b < a.batch) lengths(b, &had, &gets);
        gone += block_scan(b < a.batch ? returned(b, had, gets) : 0, &before, lds);
    }
    const int64_t top = free + gone;   // entries of the list with what is given back
    int64_t run = 0;
    for (int b0 = 0; b0 < a.batch; b0 += kThreads) {
        const int b = b0 + threadIdx.x;
        int had = 0, gets = 0;
        if (b < a.batch) lengths(b, &had, &gets);
        const int64_t n = block_scan(b < a.batch ? returned(b, had, gets) : 0, &before, lds);
        if (b < a.batch) {
            int64_t at = top - 1 - (run + before);
            for (int j = gets; j < had; j++) {
                const int p = a.table[(int64_t)b * a.table_ld + j];
                if (!is_page(a, p)) continue;
                if (at < a.pages) list[at] = p;
                at--;
            }
        }
        run += n;
    }
    __syncthreads();
    for (int b0 = 0; b0 < a.batch; b0 += kThreads) {
        const int b = b0 + threadIdx.x;
        int had = 0, gets = 0, grown = 0;
        if (b < a.batch) grown = lengths(b, &had, &gets);
        int64_t row;
        const int64_t n = block_scan(max(gets - had, 0), &before, lds), r = block_scan(grown, &row, lds);
        if (b < a.batch) {
            int64_t at = top - 1 - (come + before);
            for (int j = had; j < gets; j++, at--) a.table[(int64_t)b * a.table_ld + j] = at >= 0 && at < a.pages ? list[at] : -1;
            a.row_start[b] = (int)min(rows + row, (int64_t)a.rows);
            a.len[b] = max(a.want[b], 0);
        }
        come += n;
        rows += r;
    }
    if (threadIdx.x == 0) {
        a.row_start[a.batch] = (int)min(rows, (int64_t)a.rows);
        a.pool[0] = (int)min(max(top - come, (int64_t)0), (int64_t)a.pages);
        a.pool[1] = (int)min(max(come - top, (int64_t)0), (int64_t)0x7FFFFFFF);
    }
}

// A row's token and its place in the pool.
__global__ __launch_bounds__(256) void k_pages_rows(Seqs s, int32_t* pos, int64_t* slot) {
    const uint32_t i = blockIdx.x * 256 + threadIdx.x;
    if (i >= (uint32_t)s.rows) return;
    const int r = (int)i;
    const int b = seq_of_row(s, r);
    if (b < 0) return;
    int r0, r1;
    seq_rows(s, b, &r0, &r1);
    const int t = s.len[b] - (r1 - r0) + (r - r0), j = t / s.page;   // (a call's rows are new tokens: t >= 0)
    const int64_t p = seq_page(s, b, j);
    if (pos) pos[r] = t;
    if (slot) slot[r] = p < 0 ? -1 : p * s.page + (t - j * s.page);
}

hipError_t launch_pages_init(int pages, int32_t* pool, hipStream_t s) {
    hipLaunchKernelGGL(k_pages_init, dim3((unsigned)(((int64_t)pages + 3) / 256 + 1)), dim3(256), 0, s, pages, pool);
    return hipGetLastError();
}

hipError_t launch_pages_assign(const PagesArgs& a, hipStream_t s) {
    if (a.batch <= kSeqsAtOnce && (int64_t)a.batch * a.table_ld <= 0x7FFFFFFF) {
        const int64_t rows = a.pos || a.slot ? a.rows : 0;
        const bool few = a.batch <= kFewSeqs;
        const int64_t n = std::max<int64_t>(1, std::min<int64_t>(128, (rows + kThreads - 1) / kThreads));
        if (few) hipLaunchKernelGGL((k_pages_assign<kFewSeqs>), dim3((unsigned)n), dim3(kThreads), 0, s, a);
        else hipLaunchKernelGGL((k_pages_assign<kSeqsAtOnce>), dim3((unsigned)n), dim3(kThreads), 0, s, a);
        if (n > 1) hipLaunchKernelGGL(k_pages_settle, dim3((a.batch + 255) / 256), dim3(256), 0, s, a);
        return hipGetLastError();
    }
    hipLaunchKernelGGL(k_pages_assign_many, dim3(1), dim3(kThreads), 0, s, a);
    if (a.rows > 0 && (a.pos || a.slot)) {
        Seqs q{};
        q.row_start = a.row_start;
        q.len = a.len;
        q.table = a.table;
        q.batch = a.batch;
        q.rows = a.rows;
        q.table_ld = a.table_ld;
        q.page = a.page;
        q.pages = a.pages;
        hipLaunchKernelGGL(k_pages_rows, dim3((unsigned)(((int64_t)a.rows + 255) / 256)), dim3(256), 0, s, q, a.pos, a.slot);
    }
    return hipGetLastError();
}

}  // namespace wq
