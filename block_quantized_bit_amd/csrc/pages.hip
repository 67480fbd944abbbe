// pages.hip -- the pages of a cache's sequences: taken from a list of free ones as sequences grow, given back as they shrink or
// end, with the block table, the row starts and the rows' places that the other calls take.
#include <hip/hip_runtime.h>

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

__device__ inline int pages_of(const PagesArgs& a, int tokens) {
    return (int)min((tokens + (int64_t)a.page - 1) / a.page, (int64_t)a.table_ld);
}
__device__ inline bool is_page(const PagesArgs& a, int p) { return p >= 0 && p < a.pages; }

}  // namespace

__global__ __launch_bounds__(256) void k_pages_init(int pages, int32_t* pool) {
    const uint32_t i = blockIdx.x * 256 + threadIdx.x;   // (past 2^31 in the last workgroup of the largest list)
    if (i < 4) pool[i] = i == 0 ? pages : 0;
    if (i < (uint32_t)pages) pool[4 + (int64_t)i] = pages - 1 - (int)i;
}

// One workgroup.  First what is given back goes on the list's end (its front), the first sequence's first page last; then what
// is wanted is taken from there.
__global__ __launch_bounds__(kThreads) void k_pages_assign(PagesArgs a) {
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
    hipLaunchKernelGGL(k_pages_assign, dim3(1), dim3(kThreads), 0, s, a);
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
