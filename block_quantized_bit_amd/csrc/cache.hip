// cache.hip -- keys and values quantized as they are written into a 4-bit cache, and read back.
//
// Each block of 32 channels of one token of one head is quantized by the format's rule for a weight block (q4_0: d =
// fp16(x_big / -8), q = clamp(rint(x / d), -8, 7) + 8, x^ = (q - 8) d; q4_1: d = fp16((max - min) / 15), m = fp16(min),
// q = clamp(rint((x - m) / d), 0, 15), x^ = q d + m), after clamping x to +-32768.
#include <hip/hip_runtime.h>

#include "cache_layout.h"
#include "wq_device.h"
#include "wq_launch.h"

namespace wq {

namespace {

typedef uint16_t u16x8 __attribute__((ext_vector_type(8)));
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

// Quantizes a block of 32 held by 4 neighbouring lanes (8 values each, in lane order).  word: the 8 codes, nibble n =
// value n; d, m: fp16 bits (m only for q4_1).
template <bool Q41>
__device__ inline void quantize_block(float v[8], uint32_t* word, uint16_t* d, uint16_t* m) {
#pragma unroll
    for (int j = 0; j < 8; j++) v[j] = fminf(fmaxf(v[j], -kCacheLimit), kCacheLimit);   // a NaN becomes -32768
    float base, low;
    if constexpr (Q41) {
        float lo = v[0], hi = v[0];
#pragma unroll
        for (int j = 1; j < 8; j++) {
            lo = fminf(lo, v[j]);
            hi = fmaxf(hi, v[j]);
        }
#pragma unroll
        for (int s = 1; s <= 2; s <<= 1) {
            lo = fminf(lo, __shfl_xor(lo, s, 64));
            hi = fmaxf(hi, __shfl_xor(hi, s, 64));
        }
        *d = f16_sat_bits((hi - lo) / 15.0f);
        *m = f16_sat_bits(lo);
        base = f16_value(*m);
        low = 0.0f;
    } else {
        float big = v[0];                                    // the first of the largest magnitude
#pragma unroll
        for (int j = 1; j < 8; j++) big = fabsf(v[j]) > fabsf(big) ? v[j] : big;
#pragma unroll
        for (int s = 1; s <= 2; s <<= 1) {
            const float o = __shfl_xor(big, s, 64);
            const bool other_first = (threadIdx.x & s) != 0;   // the other lane's values come before this one's
            big = fabsf(o) > fabsf(big) || (other_first && fabsf(o) == fabsf(big)) ? o : big;
        }
        *d = f16_sat_bits(big / -8.0f);
        *m = 0;
        base = 0.0f;
        low = -8.0f;
    }
    const float delta = f16_value(*d);
    uint32_t w = 0;
#pragma unroll
    for (int j = 0; j < 8; j++) {
        float q = -low;
        if (delta != 0.0f) q = fminf(fmaxf(rintf((v[j] - base) / delta), low), low + 15.0f) - low;
        w |= (uint32_t)q << (4 * j);
    }
    *word = w;
}

}  // namespace

// One thread per 8 channels of one row of one head (4 threads: a block).
template <bool Q41, bool F32>
__global__ __launch_bounds__(256) void k_cache_write(Seqs s, int nb, const void* __restrict__ k, int64_t ldk,
                                                     const void* __restrict__ v, int64_t ldv, uint8_t* __restrict__ cache) {
    const int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int c8 = nb * 4, per_row = s.heads * c8;
    const int64_t row = c / per_row;
    if (row >= s.rows) return;
    const int in_row = (int)(c - row * per_row), h = in_row / c8, cg = in_row - h * c8, b = cg >> 2, g = cg & 3;
    const int seq = seq_of_row(s, (int)row);
    if (seq < 0) return;
    int r0, r1;
    seq_rows(s, seq, &r0, &r1);
    const int64_t t = (int64_t)s.len[seq] - r1 + row;   // its position
    if (t < 0 || t >= (int64_t)s.table_ld * s.page) return;
    const int64_t at = seq_unit(s, seq, h, (int)t);
    if (at < 0) return;
    const int u = (int)(t % s.page) % kUnit, dim = nb * 32;
    uint8_t* const kb = cache + at;
    uint8_t* const vb = kb + cache_half_bytes(Q41, dim);
    float x[8];
    uint32_t word;
    uint16_t d, m;
    load8<F32>(k, row * ldk + h * dim + cg * 8, x);
    quantize_block<Q41>(x, &word, &d, &m);
    *reinterpret_cast<uint32_t*>(kb + cache_k_word(nb, u, b, g)) = word;
    uint16_t* sc = reinterpret_cast<uint16_t*>(kb + 16 * dim) + cache_scale(nb, u, b);
    if (g == 0) {
        sc[0] = d;
        if constexpr (Q41) sc[dim] = m;
    }
    load8<F32>(v, row * ldv + h * dim + cg * 8, x);
    quantize_block<Q41>(x, &word, &d, &m);
    // channels 8 g + n: the low nibble of channel's byte for g < 2, the high one of channel - 16's for g >= 2
    const uint32_t other = __shfl_xor(word, 2, 64);
    const uint32_t lo = g < 2 ? word : other, hi = g < 2 ? other : word;
    // this lane writes the bytes of channels 8 (g & 1) + 4 (g >> 1) + 0..3
#pragma unroll
    for (int n = 0; n < 4; n++) {
        const int e = 4 * (g >> 1) + n;
        vb[cache_v_byte(nb, u, b, 8 * (g & 1) + e)] = (uint8_t)(((lo >> (4 * e)) & 15u) | (((hi >> (4 * e)) & 15u) << 4));
    }
    sc = reinterpret_cast<uint16_t*>(vb + 16 * dim) + cache_scale(nb, u, b);
    if (g == 0) {
        sc[0] = d;
        if constexpr (Q41) sc[dim] = m;
    }
}

// One thread per 8 channels of one row of one head.
template <bool Q41, bool F32>
__global__ __launch_bounds__(256) void k_cache_read(Seqs s, int nb, const uint8_t* __restrict__ cache, void* __restrict__ k,
                                                    int64_t ldk, void* __restrict__ v, int64_t ldv) {
    const int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int c8 = nb * 4, per_row = s.heads * c8;
    const int64_t row = c / per_row;
    if (row >= s.rows) return;
    const int in_row = (int)(c - row * per_row), h = in_row / c8, cg = in_row - h * c8, b = cg >> 2, g = cg & 3;
    const int seq = seq_of_row(s, (int)row);
    if (seq < 0) return;
    int r0, r1;
    seq_rows(s, seq, &r0, &r1);
    const int64_t t = (int64_t)s.len[seq] - r1 + row;
    const int dim = nb * 32;
    const int64_t at = t < 0 || t >= (int64_t)s.table_ld * s.page ? -1 : seq_unit(s, seq, h, (int)t);
    float x[8], y[8];
    if (at < 0) {
#pragma unroll
        for (int n = 0; n < 8; n++) x[n] = y[n] = 0.0f;
    } else {
        const int u = (int)(t % s.page) % kUnit;
        const uint8_t* const kb = cache + at;
        const uint8_t* const vb = kb + cache_half_bytes(Q41, dim);
        const uint16_t* ks = reinterpret_cast<const uint16_t*>(kb + 16 * dim) + cache_scale(nb, u, b);
        const uint16_t* vs = reinterpret_cast<const uint16_t*>(vb + 16 * dim) + cache_scale(nb, u, b);
        const float kd = f16_value(ks[0]), vd = f16_value(vs[0]);
        const uint32_t word = *reinterpret_cast<const uint32_t*>(kb + cache_k_word(nb, u, b, g));
#pragma unroll
        for (int n = 0; n < 8; n++) {
            const uint32_t kq = (word >> (4 * n)) & 15u;
            const uint32_t vq = (vb[cache_v_byte(nb, u, b, 8 * (g & 1) + n)] >> (g < 2 ? 0 : 4)) & 15u;
            if constexpr (Q41) {
                x[n] = (float)kq * kd + f16_value(ks[dim]);
                y[n] = (float)vq * vd + f16_value(vs[dim]);
            } else {
                x[n] = ((float)kq - 8.0f) * kd;
                y[n] = ((float)vq - 8.0f) * vd;
            }
        }
    }
    store8<F32>(k, row * ldk + h * dim + cg * 8, x);
    store8<F32>(v, row * ldv + h * dim + cg * 8, y);
}

namespace {
unsigned chunk_blocks(const Seqs& s, int nb) { return (unsigned)(((int64_t)s.rows * s.heads * nb * 4 + 255) / 256); }
}  // namespace

hipError_t launch_cache_write(const Seqs& q, bool q41, int dim, bool f32, const void* k, int64_t ldk, const void* v, int64_t ldv,
                              uint8_t* cache, hipStream_t s) {
    const int nb = dim / 32;
    auto f = q41 ? (f32 ? k_cache_write<true, true> : k_cache_write<true, false>)
                 : (f32 ? k_cache_write<false, true> : k_cache_write<false, false>);
    hipLaunchKernelGGL(f, dim3(chunk_blocks(q, nb)), dim3(256), 0, s, q, nb, k, ldk, v, ldv, cache);
    return hipGetLastError();
}

hipError_t launch_cache_read(const Seqs& q, bool q41, int dim, bool f32, const uint8_t* cache, void* k, int64_t ldk, void* v,
                             int64_t ldv, hipStream_t s) {
    const int nb = dim / 32;
    auto f = q41 ? (f32 ? k_cache_read<true, true> : k_cache_read<true, false>)
                 : (f32 ? k_cache_read<false, true> : k_cache_read<false, false>);
    hipLaunchKernelGGL(f, dim3(chunk_blocks(q, nb)), dim3(256), 0, s, q, nb, cache, k, ldk, v, ldv);
    return hipGetLastError();
}

}  // namespace wq
