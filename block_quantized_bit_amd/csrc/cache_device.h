// cache_device.h -- device helpers of the cache and attention kernels: uniform reads, and finding a sequence's share of a
// call's work.
#pragma once

#include <hip/hip_runtime.h>

#include "cache_layout.h"

namespace wq {

// The call's int32 arrays are only read and indexed uniformly: as constant memory they are scalar loads.
typedef const int32_t __attribute__((address_space(4))) * const_i32;
__device__ inline int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ inline int read_const(const int32_t* p, int64_t i) { return ((const_i32)(uintptr_t)p)[i]; }

// seq_rows, the length and seq_unit for a uniform sequence, through scalar loads.
struct SeqRows {
    int r0, r1, len;
};
__device__ inline SeqRows seq_rows_uniform(const Seqs& s, int b) {
    SeqRows r = {b, b + 1, read_const(s.len, b)};
    if (s.row_start) {
        const int a = read_const(s.row_start, b), e = read_const(s.row_start, b + 1);
        r.r0 = a < 0 ? 0 : a > s.rows ? s.rows : a;
        r.r1 = e < r.r0 ? r.r0 : e > s.rows ? s.rows : e;
    }
    return r;
}
__device__ inline int64_t seq_unit_uniform(const Seqs& s, int b, int h, int t) {
    const int j = t / s.page;
    if (j >= s.table_ld) return -1;
    const int64_t p = s.table ? (int64_t)read_const(s.table, (int64_t)b * s.table_ld + j) : (int64_t)b;
    if (p < 0 || p >= s.pages) return -1;
    return ((p * s.heads + h) * s.upp + (t - j * s.page) / kUnit) * s.unit_bytes;
}

// Inclusive prefix sum over the wave: lanes 1, 2, 4, 8 below within rows of 16, then the rows' totals.
template <int CTRL, int ROWS>
__device__ inline uint32_t add_dpp(uint32_t v) {
    return v + (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, ROWS, 0xF, false);
}
__device__ inline uint32_t wave_scan(uint32_t v) {
    v = add_dpp<0x111, 0xF>(v);   // row_shr
    v = add_dpp<0x112, 0xF>(v);
    v = add_dpp<0x114, 0xF>(v);
    v = add_dpp<0x118, 0xF>(v);
    v = add_dpp<0x142, 0xA>(v);   // row_bcast: lane 15 to the next row, lane 31 to the upper half
    return add_dpp<0x143, 0xC>(v);
}

// Running totals over the sequences of a call: weight(b) is sequence b's share (b per lane).  The first 64 sequences'
// shares stay in registers, so that a call of at most 64 reads their lengths once for all questions.
template <class F>
struct SeqTotals {
    F weight;
    int batch;
    uint32_t w, incl;   // of sequence `lane`

    __device__ SeqTotals(int n, F f) : weight(f), batch(n) {
        const int lane = threadIdx.x & 63;
        w = lane < n ? weight(lane) : 0;
        incl = wave_scan(w);
    }
    static __device__ uint32_t last(uint32_t v) { return (uint32_t)__builtin_amdgcn_readlane((int)v, 63); }
    __device__ uint32_t total() const {
        uint32_t run = last(incl);
        for (int b0 = 64; b0 < batch; b0 += 64) {
            const int b = b0 + (threadIdx.x & 63);
            run += last(wave_scan(b < batch ? weight(b) : 0));
        }
        return run;
    }
    // The sequence whose share contains `target` (below the total), and the total before it; -1 if there is none.
    __device__ int find(uint32_t target, uint32_t* before) const {
        uint32_t run = 0, v = w, in = incl;
        for (int b0 = 0; b0 < batch; b0 += 64) {
            if (b0 > 0) {
                const int b = b0 + (threadIdx.x & 63);
                v = b < batch ? weight(b) : 0;
                in = wave_scan(v);
            }
            const uint32_t sum = last(in);
            if (target - run < sum) {
                const int l = __builtin_ctzll(__ballot(in > target - run));
                *before = run + (uint32_t)__builtin_amdgcn_readlane((int)(in - v), l);
                return b0 + l;
            }
            run += sum;
        }
        *before = run;
        return -1;
    }
};

}  // namespace wq
