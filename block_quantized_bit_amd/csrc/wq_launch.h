// wq_launch.h -- host-side launchers implemented by the kernel translation units
// and called by the C ABI layer after it has validated every argument.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "cache_layout.h"

namespace wq {

// Offsets inside the scales buffer (bytes).
struct ScaleLayout {
    int64_t nb;        // number of blocks
    int64_t ng;        // NF4+DQ: number of 256-block groups
    int64_t d_off;     // NF4+DQ: fp32 d[ng]
    int64_t mu_off;    // NF4+DQ: fp32 mean
    int64_t g_off;     // NVFP4: fp32 global scale
    int64_t hb_off;    // Q5_0: 32-bit fifth-bit words, one per block, tile order
    int64_t kd_off;    // Q4_K: fp16 (d, dmin) per super-block; Q6_K: fp16 d per super-block;
                       //   row-major [n][k/256]
    int64_t bytes;     // total scales bytes
};

ScaleLayout scale_layout(int fmt, bool dq, int64_t n, int64_t k);

hipError_t launch_quantize(int fmt, bool dq, int64_t n, int64_t k, const float* w,
                           uint8_t* codes, uint8_t* scales, hipStream_t s);
hipError_t launch_dequantize(int fmt, bool dq, int64_t n, int64_t k, const uint8_t* codes,
                             const uint8_t* scales, float* out, hipStream_t s);

// Output description shared by the matmul kernels: columns [0, end0) -> y0,
// [end0, end1) -> y1, [end1, n) -> y2.
struct OutSplit {
    void* y[3];
    int64_t ldy[3];
    int64_t end[3];   // exclusive column end of each split (end[nsplit-1] == n)
    int nsplit;
    int f32;          // 1: fp32 output, 0: bf16
};

struct MatmulProblem {
    int fmt;
    bool dq;
    int64_t m, n, k;
    const uint16_t* x;
    int64_t ldx;
    const uint8_t* codes;
    const uint8_t* scales;
    const uint16_t* bias;
    OutSplit out;
    void* ws;
    size_t ws_bytes;
    const float* gscale;   // NVFP4: epilogue factor in device memory; null = the weights' global scale
};

// Workspace bytes the schedule for (fmt, m, n, k) would like (0 = none).
size_t matmul_workspace_bytes(int fmt, int64_t m, int64_t n, int64_t k);

hipError_t launch_gemv(const MatmulProblem& p, hipStream_t s);   // m <= 16
hipError_t launch_gemm(const MatmulProblem& p, hipStream_t s);   // m >= 17

size_t gemv_workspace_bytes(int fmt, int64_t m, int64_t n, int64_t k);
size_t gemm_workspace_bytes(int fmt, int64_t m, int64_t n, int64_t k);

// NVFP4 activations (act.hip): packed row-major codes [m][k/2] and scales [m][k/16]
// followed by the fp32 global scale at align16(m*k/16).
int64_t act_scales_bytes(int64_t m, int64_t k);
hipError_t launch_quantize_act(int64_t m, int64_t k, const uint16_t* x, int64_t ldx, uint8_t* codes,
                               uint8_t* scales, hipStream_t s);
// xe[m][k] = bf16(+-e2m1 * s) (exact) and *gprod = g_w * g_x, with g_w read at gw.
hipError_t launch_expand_act(int64_t m, int64_t k, const uint8_t* codes, const uint8_t* scales,
                             const uint8_t* gw, uint16_t* xe, float* gprod, hipStream_t s);

// 4-bit key/value cache (cache.hip): whether a call's launches are small enough; rows of K and V, bf16 or fp32, into and out of the pool.
bool cache_fits(const Seqs& q, int dim);
hipError_t launch_cache_write(const Seqs& q, bool q41, int dim, bool f32, const void* k, int64_t ldk, const void* v,
                              int64_t ldv, uint8_t* cache, hipStream_t s);
hipError_t launch_cache_read(const Seqs& q, bool q41, int dim, bool f32, const uint8_t* cache, void* k, int64_t ldk,
                             void* v, int64_t ldv, hipStream_t s);

// Attention over the cache (attn.hip).
struct AttnArgs {
    Seqs s;
    const uint16_t* q;
    const uint8_t* cache;
    uint16_t* y;
    int64_t ldq, ldy;
    uint8_t* ws;           // null: no split of a sequence over workgroups
    float scale_log2;      // softmax scale times log2(e)
    int32_t group, dim, window;
    int32_t tile_cols;     // columns (rows x heads) per tile of the kernel that runs
    int32_t workgroups;    // > 0: sequences are shared out over so many
    int32_t least_units;   // units that each then takes at least
    int32_t splits;        // tiles of 128 columns: parts that each tile's tokens are shared out in
    int32_t slots;         // partial results that the workspace holds
    bool q41, causal;
};
bool attn_fits(const AttnArgs& a);
size_t attn_workspace_bytes(const AttnArgs& a);
hipError_t launch_attn(const AttnArgs& a, hipStream_t s);

}  // namespace wq
