// moe_q4.cuh -- products of (token, slot) rows with 4-bit expert weights.
//
// W[e] (n x k, out x in) is held as codes [n, k/2] bytes (value 2j of a row in
// the low nibble of byte j, 2j+1 in the high one) and one scale per row and
// group of consecutive values along k:
//   int4  value = (code - 8) s,          s bf16, groups of 32, 64 or 128
//   e2m1  value = E2M1[code] 2^(s-127),  s one byte, groups of 32
// For pair p with expert e = expert[p] and input row x[p / x_div]:
//   a[i] = sum_j W[e][i, j] x[j],  y[p] = gate[p] * act(a).
#pragma once

#include "moe_common.cuh"

namespace moe {
namespace q4 {

enum { INT4 = 0, E2M1 = 1 };
enum { GELU = 0, SWIGLU = 1, NONE = 2 };
constexpr int kThreads = 256;

struct Params {
    const __nv_bfloat16 *x;
    const int *expert;
    const uint8_t *codes;
    const void *scales;
    const float *gate;
    void *y;
    int64_t pairs;
    int x_div, N, n, k, group_shift, groups;   // groups = scales of a row
};

__device__ __forceinline__ float e2m1_value(uint32_t c) {
    const int m = c & 7;   // 0, .5, 1, 1.5, 2, 3, 4, 6
    const float v = m < 2 ? 0.5f * m : __int_as_float((((m >> 1) + 126) << 23) | ((m & 1) << 22));
    return c & 8 ? -v : v;
}
template <int FMT>
__device__ __forceinline__ float code_value(uint32_t c) {
    return FMT == INT4 ? (float)((int)c - 8) : e2m1_value(c);
}
template <int FMT>
__device__ __forceinline__ float scale_of(const void *s, int64_t i) {
    if (FMT == INT4) return __bfloat162float(static_cast<const __nv_bfloat16 *>(s)[i]);
    const uint32_t b = static_cast<const uint8_t *>(s)[i];
    return b == 255u ? __int_as_float(0x7fffffff) : b == 0u ? __int_as_float(0x00400000) : __int_as_float(b << 23);
}

__device__ __forceinline__ float gelu(float v) { return 0.5f * v * (1.0f + erff(v * 0.70710678118654752f)); }
__device__ __forceinline__ float silu(float v) { return v / (1.0f + expf(-v)); }

template <int FMT>
__device__ __forceinline__ float row_dot(const Params &p, int64_t row, const __nv_bfloat16 *x) {
    const int lane = threadIdx.x & 31;
    float sum = 0.f;
    for (int j = lane * 8; j < p.k; j += 256) {   // 8 codes: inside one group
        const uint32_t c = *reinterpret_cast<const uint32_t *>(p.codes + row * (p.k / 2) + j / 2);
        const uint4 xv = *reinterpret_cast<const uint4 *>(x + j);
        const uint32_t xw[4] = {xv.x, xv.y, xv.z, xv.w};
        float part = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            part = fmaf(code_value<FMT>((c >> (8 * i)) & 15u), __uint_as_float(xw[i] << 16), part);
            part = fmaf(code_value<FMT>((c >> (8 * i + 4)) & 15u), __uint_as_float(xw[i] & 0xffff0000u), part);
        }
        sum = fmaf(part, scale_of<FMT>(p.scales, row * p.groups + (j >> p.group_shift)), sum);
    }
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    return sum;
}

// One warp per result of a pair.
template <int FMT, int ACT, typename TO>
__global__ void __launch_bounds__(kThreads) matvec_kernel(const Params p) {
    pdl_enter();
    const int cols = ACT == SWIGLU ? p.n / 2 : p.n;
    const int i = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    if (i >= cols) return;
    for (int64_t pr = blockIdx.y; pr < p.pairs; pr += gridDim.y) {
        const int e = p.expert[pr];
        float v = 0.f;
        if (e >= 0 && e < p.N) {
            const __nv_bfloat16 *x = p.x + pr / p.x_div * p.k;
            v = row_dot<FMT>(p, (int64_t)e * p.n + i, x);
            if (ACT == SWIGLU) v = silu(v) * row_dot<FMT>(p, (int64_t)e * p.n + cols + i, x);
            if (ACT == GELU) v = gelu(v);
            if (p.gate) v *= p.gate[pr];
        } else if (e != -1 && (threadIdx.x & 31) == 0) {
            set_status(kStatusBounds);
        }
        if ((threadIdx.x & 31) == 0) {
            TO *y = static_cast<TO *>(p.y) + pr * cols + i;
            if (sizeof(TO) == 4) *reinterpret_cast<float *>(y) = v;
            else *reinterpret_cast<__nv_bfloat16 *>(y) = __float2bfloat16(v);
        }
    }
}

// Codes and scales of fp32 or bf16 weights: one warp per group of values.
//   int4  s = bf16(max|w| / 7), code = 8 + round(w / s) clamped to 0..15
//   e2m1  s = 2^e, e the smallest integer with max|w| <= 6 2^e; round(w / s) to
//         the nearest of 0, .5, 1, 1.5, 2, 3, 4, 6, ties to the even code
// A group with an infinity or a NaN gets a NaN scale.
template <int FMT, typename T>
__global__ void __launch_bounds__(kThreads) quantize_kernel(const T *__restrict__ W, int64_t rows, int k,
                                                            int group_shift, int groups, uint8_t *__restrict__ codes,
                                                            void *__restrict__ scales) {
    pdl_enter();
    const int lane = threadIdx.x & 31;
    const int64_t total = rows * groups, stride = (int64_t)gridDim.x * (kThreads / 32);
    for (int64_t i = blockIdx.x * (int64_t)(kThreads / 32) + (threadIdx.x >> 5); i < total; i += stride) {
        const int64_t row = i / groups;
        const int j0 = (int)(i - row * groups) << group_shift, j1 = min(j0 + (1 << group_shift), k);
        uint32_t m = 0;
        for (int j = j0 + lane; j < j1; j += 32) m = max(m, __float_as_uint(to_f32(W[row * k + j])) & 0x7fffffffu);
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
        const bool bad = m >= 0x7f800000u;
        float s;
        int e = 0;
        if (FMT == INT4) {
            s = __bfloat162float(__float2bfloat16(__uint_as_float(m) / 7.0f));
            if (bad) s = __int_as_float(0x7fffffff);
            if (lane == 0) static_cast<__nv_bfloat16 *>(scales)[i] = __float2bfloat16(s);
        } else {
            e = max((int)(m >> 23) - 127 - 2 + ((m & 0x7fffffu) > 0x400000u ? 1 : 0), -126);
            s = __int_as_float((e + 127) << 23);
            if (lane == 0) static_cast<uint8_t *>(scales)[i] = bad ? 255 : (uint8_t)(e + 127);
        }
        for (int j = j0 + 2 * lane; j < j1; j += 64) {
            uint32_t byte = 0;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float w = to_f32(W[row * k + j + h]);
                uint32_t c;
                if (FMT == INT4) {
                    c = bad || s == 0.f ? 8u : (uint32_t)min(max(__float2int_rn(w / s) + 8, 0), 15);
                } else {
                    const float a = fabsf(w / s);
                    // halfway points 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5; a tie takes the even code
                    c = (a > 0.25f) + (a >= 0.75f) + (a > 1.25f) + (a >= 1.75f) + (a > 2.5f) + (a >= 3.5f) + (a > 5.0f);
                    c = bad ? 0u : c | (__float_as_uint(w) >> 31 << 3);
                }
                byte |= c << (4 * h);
            }
            codes[(row * k + j) >> 1] = (uint8_t)byte;
        }
    }
}

// The values of codes and scales, rounded once to T.
template <int FMT, typename T>
__global__ void __launch_bounds__(kThreads) dequantize_kernel(const uint8_t *__restrict__ codes,
                                                              const void *__restrict__ scales, int64_t rows, int k,
                                                              int group_shift, int groups, T *__restrict__ W) {
    pdl_enter();
    const int64_t total = rows * (k / 8);
    for (int64_t i = blockIdx.x * (int64_t)kThreads + threadIdx.x; i < total; i += (int64_t)gridDim.x * kThreads) {
        const int64_t row = i / (k / 8);
        const int j = (int)(i - row * (k / 8)) * 8;
        const uint32_t c = *reinterpret_cast<const uint32_t *>(codes + row * (k / 2) + j / 2);
        const float s = scale_of<FMT>(scales, row * groups + (j >> group_shift));
        float v[8];
#pragma unroll
        for (int h = 0; h < 8; ++h) v[h] = code_value<FMT>((c >> (4 * h)) & 15u) * s;
        T *dst = W + row * k + j;
        if (sizeof(T) == 4) {
            reinterpret_cast<float4 *>(dst)[0] = make_float4(v[0], v[1], v[2], v[3]);
            reinterpret_cast<float4 *>(dst)[1] = make_float4(v[4], v[5], v[6], v[7]);
        } else {
            *reinterpret_cast<uint4 *>(dst) = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                                         pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
        }
    }
}

}  // namespace q4
}  // namespace moe
