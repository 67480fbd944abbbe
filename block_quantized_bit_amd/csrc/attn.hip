// attn.hip -- attention over the 4-bit cache: y = sum_t softmax_t(scale q . k^_t) v^_t over the tokens a row sees.
#include <hip/hip_runtime.h>

#include <cfloat>

#include "cache_layout.h"
#include "wq_device.h"
#include "wq_launch.h"

namespace wq {

// One workgroup per row and query head; 256 tokens a step: a thread takes a token's score, then a channel's sum.
template <bool Q41>
__global__ __launch_bounds__(256) void k_attn(AttnArgs a) {
    __shared__ float qs[256], ps[256], red[4];
    const Seqs& s = a.s;
    const int hq = blockIdx.x % a.q_heads, row = blockIdx.x / a.q_heads, h = hq / a.group, tid = threadIdx.x;
    const int seq = seq_of_row(s, row);
    if (seq < 0) return;
    int r0, r1;
    seq_rows(s, seq, &r0, &r1);
    const int nb = a.dim / 32, half = cache_half_bytes(Q41, a.dim);
    int lo = 0, hi = seq_tokens(s, seq);
    if (a.causal) {
        const int64_t t = (int64_t)s.len[seq] - r1 + row;
        hi = (int)(t + 1 < hi ? t + 1 : hi);
        if (a.window > 0 && t - a.window + 1 > 0) lo = (int)(t - a.window + 1);
    }
    if (tid < a.dim) qs[tid] = bf16_value(a.q[row * a.ldq + (int64_t)hq * a.dim + tid]) * a.scale_log2;
    __syncthreads();
    float m = -FLT_MAX, l = 0.0f, o = 0.0f;
    for (int t0 = lo / 32 * 32; t0 < hi; t0 += 256) {
        const int t = t0 + tid;
        float x = -INFINITY;
        if (t >= lo && t < hi) {
            const int64_t at = seq_unit(s, seq, h, t);
            if (at >= 0) {
                const uint8_t* kb = a.cache + at;
                const uint16_t* ks = reinterpret_cast<const uint16_t*>(kb + 16 * a.dim);
                const int u = t % s.page % kUnit;
                x = 0.0f;
                for (int b = 0; b < nb; b++) {
                    const float d = f16_value(ks[cache_scale(nb, u, b)]);
                    const float off = Q41 ? f16_value(ks[a.dim + cache_scale(nb, u, b)]) : -8.0f * d;
                    for (int g = 0; g < 4; g++) {
                        const uint32_t w = *reinterpret_cast<const uint32_t*>(kb + cache_k_word(nb, u, b, g));
                        for (int n = 0; n < 8; n++) x += qs[32 * b + 8 * g + n] * ((float)((w >> (4 * n)) & 15u) * d + off);
                    }
                }
            }
        }
        float mx = x;
        for (int d = 32; d >= 1; d >>= 1) mx = fmaxf(mx, __shfl_xor(mx, d, 64));
        if ((tid & 63) == 0) red[tid >> 6] = mx;
        __syncthreads();
        mx = fmaxf(fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3])), m);
        const float p = exp2f(x - mx);
        ps[tid] = p;
        float sum = p;
        for (int d = 32; d >= 1; d >>= 1) sum += __shfl_xor(sum, d, 64);
        __syncthreads();
        if ((tid & 63) == 0) red[tid >> 6] = sum;
        __syncthreads();
        const float alpha = exp2f(m - mx);
        l = l * alpha + ((red[0] + red[1]) + (red[2] + red[3]));
        o *= alpha;
        m = mx;
        if (tid < a.dim) {
            const int b = tid >> 5, c = tid & 15, sh = (tid & 16) ? 4 : 0;
            for (int i = 0; i < 256 && t0 + i < hi; i++) {
                if (t0 + i < lo) continue;
                const int64_t at = seq_unit(s, seq, h, t0 + i);
                if (at < 0) continue;
                const uint8_t* vb = a.cache + at + half;
                const uint16_t* vs = reinterpret_cast<const uint16_t*>(vb + 16 * a.dim);
                const int u = (t0 + i) % s.page % kUnit;
                const float d = f16_value(vs[cache_scale(nb, u, b)]);
                const float off = Q41 ? f16_value(vs[a.dim + cache_scale(nb, u, b)]) : -8.0f * d;
                o += ps[i] * ((float)((vb[cache_v_byte(nb, u, b, c)] >> sh) & 15u) * d + off);
            }
        }
        __syncthreads();
    }
    if (tid < a.dim) a.y[row * a.ldy + (int64_t)hq * a.dim + tid] = __builtin_bit_cast(uint16_t, (__bf16)(l != 0.0f ? o / l : 0.0f));   // NaN stays NaN
}

size_t attn_workspace_bytes(const AttnArgs&) { return 0; }

hipError_t launch_attn(const AttnArgs& a, hipStream_t s) {
    const dim3 grid((unsigned)(a.s.rows * a.q_heads));
    if (a.q41) hipLaunchKernelGGL(k_attn<true>, grid, dim3(256), 0, s, a);
    else hipLaunchKernelGGL(k_attn<false>, grid, dim3(256), 0, s, a);
    return hipGetLastError();
}

}  // namespace wq
