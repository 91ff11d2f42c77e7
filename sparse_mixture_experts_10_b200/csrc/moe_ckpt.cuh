// moe_ckpt.cuh -- 8-bit activation checkpoints and the activation's backward pass from them.
//
// A checkpoint of a row u holds, for every group of 32, 64 or 128 consecutive
// values, one exponent byte s (the scale 2^(s-127)) and one byte q per value:
//   e = the smallest integer from -126 to E with max|u| <= L 2^e, else E;
//       L = 127, E = 121 (int8) or L = 448, E = 119 (e4m3): L 2^E is the last
//       such value below 2^128, larger magnitudes saturate to it
//   q = round(u 2^-e) (to nearest, ties to even),  s = e + 127,  u^ = q 2^e.
// The scale is a power of two, so u 2^-e and u^ are exact in fp32 and the only
// rounding is q's own: at most 2^(e-1) for int8, 2^-4 |u| (or 2^(e-10) below
// 2^(e-6)) for e4m3.  A group with an infinity or a NaN has s = 255 and reads
// back as NaN everywhere, so a bad step stays visible.
//
// Bound by HBM: a few dozen instructions per value beside 8 to 12 bytes.  One
// warp takes 16 bytes per lane of one row at a time; the group's maximum is a
// shuffle tree over the 4 to 32 lanes that hold it.
#pragma once

#include <cuda_fp8.h>

#include "moe_common.cuh"

namespace moe {
namespace ckpt {

enum { INT8 = 0, E4M3 = 1 };
enum { GELU = 0, SWIGLU = 1, NONE = 2 };

constexpr int kThreads = 256;

// 16 bytes of a row: 8 bf16 or 4 fp32 values.
template <typename T>
struct Vec;
template <>
struct Vec<__nv_bfloat16> {
    static constexpr int N = 8;
    static __device__ __forceinline__ void load(const __nv_bfloat16 *p, float (&v)[8]) {
        const uint4 u = *reinterpret_cast<const uint4 *>(p);
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
    static __device__ __forceinline__ void store(__nv_bfloat16 *p, const float (&v)[8]) {
        *reinterpret_cast<uint4 *>(p) = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                                   pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
    }
    static __device__ __forceinline__ void store_q(uint8_t *p, const uint32_t (&q)[2]) {
        *reinterpret_cast<uint2 *>(p) = make_uint2(q[0], q[1]);
    }
    static __device__ __forceinline__ void load_q(const uint8_t *p, uint32_t (&q)[2]) {
        const uint2 u = *reinterpret_cast<const uint2 *>(p);
        q[0] = u.x;
        q[1] = u.y;
    }
};
template <>
struct Vec<float> {
    static constexpr int N = 4;
    static __device__ __forceinline__ void load(const float *p, float (&v)[4]) {
        const float4 u = *reinterpret_cast<const float4 *>(p);
        v[0] = u.x; v[1] = u.y; v[2] = u.z; v[3] = u.w;
    }
    static __device__ __forceinline__ void store(float *p, const float (&v)[4]) {
        *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
    }
    static __device__ __forceinline__ void store_q(uint8_t *p, const uint32_t (&q)[1]) {
        *reinterpret_cast<uint32_t *>(p) = q[0];
    }
    static __device__ __forceinline__ void load_q(const uint8_t *p, uint32_t (&q)[1]) {
        q[0] = *reinterpret_cast<const uint32_t *>(p);
    }
};

__device__ __forceinline__ float pow2i(int e) { return __int_as_float((e + 127) << 23); }   // -126 <= e <= 127

template <int FMT>
constexpr int kMostExp = FMT == INT8 ? 121 : 119;   // E

// The scale byte of a group from its largest magnitude (NaN where a value is none).
// L = 1.984375 * 2^6 (int8) or 1.75 * 2^8 (e4m3): one more power of two where the
// leading bits of amax are above L's.
template <int FMT>
__device__ __forceinline__ int scale_byte(float amax) {
    const uint32_t b = __float_as_uint(amax);
    if (b >= 0x7f800000u) return 255;
    constexpr int kLead = FMT == INT8 ? 6 : 8;
    constexpr uint32_t kMant = FMT == INT8 ? 0x7e0000u : 0x600000u;
    const int e = (int)(b >> 23) - 127 - kLead + ((b & 0x7fffffu) > kMant ? 1 : 0);
    return min(max(e, -126), kMostExp<FMT>) + 127;
}

// Four values (already multiplied by 2^-e) as four bytes.
template <int FMT>
__device__ __forceinline__ uint32_t quant4(float a, float b, float c, float d) {
    if (FMT == INT8) {
        const uint32_t x = (uint32_t)__float2int_rn(a) & 0xffu, y = (uint32_t)__float2int_rn(b) & 0xffu;
        const uint32_t z = (uint32_t)__float2int_rn(c) & 0xffu, w = (uint32_t)__float2int_rn(d) & 0xffu;
        return x | (y << 8) | (z << 16) | (w << 24);
    }
    const __nv_fp8x2_storage_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
    const __nv_fp8x2_storage_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
    return (uint32_t)lo | ((uint32_t)hi << 16);
}

template <int FMT>
__device__ __forceinline__ void dequant4(uint32_t q, float s, float *v) {
    if (FMT == INT8) {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = (float)((int)(q << (24 - 8 * i)) >> 24) * s;
    } else {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(q >> (16 * i)), __NV_E4M3);
            const float2 f = __half22float2(__half2(h));
            v[2 * i] = f.x * s;
            v[2 * i + 1] = f.y * s;
        }
    }
}

// The scale of a byte; 255 stands for NaN.
__device__ __forceinline__ float scale_value(uint32_t byte) {
    return byte == 255u ? __int_as_float(0x7fffffff) : pow2i(max((int)byte, 1) - 127);
}

// NaN-keeping maximum of magnitudes, as unsigned bit patterns (NaN is above infinity).
template <int N>
__device__ __forceinline__ float amax_bits(const float (&v)[N], int lanes) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) m = max(m, __float_as_uint(v[i]) & 0x7fffffffu);
    for (int o = lanes >> 1; o >= 1; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
    return __uint_as_float(m);
}

// Phi(v), the normal distribution function, and act / act' in the accuracy of the row type: exact-erf
// GELU, sigmoid with expf and a division.
__device__ __forceinline__ float phi(float v) { return 0.5f * (1.0f + erff(v * 0.70710678118654752f)); }
__device__ __forceinline__ float sigmoid(float v) { return 1.0f / (1.0f + expf(-v)); }

struct Params {
    const void *u;
    const uint8_t *q_in, *s_in;
    uint8_t *q, *s;
    void *h;                 // forward: act(u); load: the values
    const void *dh;
    const float *w;
    void *du, *hw;
    float *dw;
    int64_t rows, ldu, ldh;  // row strides (elements) of u / du and of h / dh / hw
    int width, group_shift;  // values per group = 1 << group_shift
    int sgroups;             // scale bytes of one half of a row
    int row_warps;           // warps that share a row (a power of two, at most kThreads / 32)
};

// One vector of a row's half: the checkpoint's bytes written, the values left as they are.
template <typename T, int FMT>
__device__ __forceinline__ void save_vec(const Params &p, int64_t row, int half, int halves, int c, bool in,
                                         const float (&v)[Vec<T>::N]) {
    constexpr int N = Vec<T>::N;
    const int lanes = (1 << p.group_shift) / N;
    const int sb = scale_byte<FMT>(amax_bits(v, lanes));
    if (!in) return;
    const float inv = pow2i(sb == 255 ? 0 : 127 - sb);
    float t[N];
#pragma unroll
    for (int i = 0; i < N; ++i) t[i] = sb == 255 ? 0.f : v[i] * inv;
    if (FMT == INT8 && sb == kMostExp<FMT> + 127) {   // the cvt to e4m3 saturates by itself
#pragma unroll
        for (int i = 0; i < N; ++i) t[i] = fminf(fmaxf(t[i], -127.f), 127.f);
    }
    uint32_t q[N / 4];
#pragma unroll
    for (int i = 0; i < N / 4; ++i) q[i] = quant4<FMT>(t[4 * i], t[4 * i + 1], t[4 * i + 2], t[4 * i + 3]);
    Vec<T>::store_q(p.q + (row * halves + half) * p.width + c, q);
    if ((c & ((1 << p.group_shift) - 1)) == 0)
        p.s[(row * halves + half) * p.sgroups + (c >> p.group_shift)] = (uint8_t)sb;
}

template <typename T, int FMT>
__device__ __forceinline__ void load_vec(const Params &p, int64_t row, int half, int halves, int c, bool in,
                                         float (&v)[Vec<T>::N]) {
    constexpr int N = Vec<T>::N;
    uint32_t q[N / 4];
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < N / 4; ++i) q[i] = 0;
    if (in) {
        Vec<T>::load_q(p.q_in + (row * halves + half) * p.width + c, q);
        s = scale_value(p.s_in[(row * halves + half) * p.sgroups + (c >> p.group_shift)]);
    }
#pragma unroll
    for (int i = 0; i < N / 4; ++i) dequant4<FMT>(q[i], s, v + 4 * i);
}

template <typename T, int ACT, int FMT>
__global__ void __launch_bounds__(kThreads) forward_kernel(const Params p) {
    pdl_enter();
    constexpr int N = Vec<T>::N, kHalves = ACT == SWIGLU ? 2 : 1;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t row = (int64_t)blockIdx.x * ((kThreads / 32) / p.row_warps) + warp / p.row_warps;
    if (row >= p.rows) return;
    const T *u = static_cast<const T *>(p.u) + row * p.ldu;
    for (int c0 = (warp % p.row_warps) * 32 * N; c0 < p.width; c0 += p.row_warps * 32 * N) {
        const int c = c0 + lane * N;
        const bool in = c < p.width;
        float a[N] = {}, b[N] = {}, o[N];
        if (in) {
            Vec<T>::load(u + c, a);
            if (ACT == SWIGLU) Vec<T>::load(u + p.width + c, b);
        }
        save_vec<T, FMT>(p, row, 0, kHalves, c, in, a);
        if (ACT == SWIGLU) save_vec<T, FMT>(p, row, 1, kHalves, c, in, b);
        if (ACT == NONE) continue;
#pragma unroll
        for (int i = 0; i < N; ++i) o[i] = ACT == GELU ? a[i] * phi(a[i]) : a[i] * sigmoid(a[i]) * b[i];
        if (in) Vec<T>::store(static_cast<T *>(p.h) + row * p.ldh + c, o);
    }
}

template <typename T, int FMT>
__global__ void __launch_bounds__(kThreads) load_kernel(const Params p, int halves) {
    pdl_enter();
    constexpr int N = Vec<T>::N;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t row = (int64_t)blockIdx.x * ((kThreads / 32) / p.row_warps) + warp / p.row_warps;
    if (row >= p.rows) return;
    for (int half = 0; half < halves; ++half)
        for (int c0 = (warp % p.row_warps) * 32 * N; c0 < p.width; c0 += p.row_warps * 32 * N) {
            const int c = c0 + lane * N;
            if (c >= p.width) continue;
            float v[N];
            load_vec<T, FMT>(p, row, half, halves, c, true, v);
            Vec<T>::store(static_cast<T *>(p.h) + row * p.ldh + (int64_t)half * p.width + c, v);
        }
}

// hw = w act(u^), du = w dh act'(u^), dw = <dh, act(u^)>; the row's sum is taken lane by lane, then
// over the lanes and warps of the row, in an order set by the width alone.
template <typename T, int ACT, int FMT>
__global__ void __launch_bounds__(kThreads) backward_kernel(const Params p) {
    pdl_enter();
    constexpr int N = Vec<T>::N, kHalves = ACT == SWIGLU ? 2 : 1;
    __shared__ float s_dot[kThreads / 32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t row = (int64_t)blockIdx.x * ((kThreads / 32) / p.row_warps) + warp / p.row_warps;
    float dot = 0.f;
    if (row < p.rows) {
        const float w = p.w ? p.w[row] : 1.0f;
        const T *dh = static_cast<const T *>(p.dh) + row * p.ldh;
        T *du = static_cast<T *>(p.du) + row * p.ldu;
        for (int c0 = (warp % p.row_warps) * 32 * N; c0 < p.width; c0 += p.row_warps * 32 * N) {
            const int c = c0 + lane * N;
            const bool in = c < p.width;
            float a[N], b[N] = {}, d[N] = {}, hv[N], da[N], db[N];
            if (in) Vec<T>::load(dh + c, d);
            load_vec<T, FMT>(p, row, 0, kHalves, c, in, a);
            if (ACT == SWIGLU) load_vec<T, FMT>(p, row, 1, kHalves, c, in, b);
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const float g = w * d[i];
                if (ACT == GELU) {
                    const float ph = phi(a[i]);
                    hv[i] = a[i] * ph;
                    da[i] = g * (ph + a[i] * expf(-0.5f * a[i] * a[i]) * 0.39894228040143268f);
                } else {
                    const float sg = sigmoid(a[i]), si = a[i] * sg;
                    hv[i] = si * b[i];
                    da[i] = g * b[i] * sg * (1.0f + a[i] * (1.0f - sg));
                    db[i] = g * si;
                }
                if (in) dot = fmaf(d[i], hv[i], dot);
                hv[i] *= w;
            }
            if (!in) continue;
            Vec<T>::store(du + c, da);
            if (ACT == SWIGLU) Vec<T>::store(du + p.width + c, db);
            if (p.hw) Vec<T>::store(static_cast<T *>(p.hw) + row * p.ldh + c, hv);
        }
    }
    if (!p.dw) return;
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
    if (lane == 0) s_dot[warp] = dot;
    __syncthreads();
    if (threadIdx.x < (kThreads / 32) / p.row_warps) {
        const int64_t r = (int64_t)blockIdx.x * ((kThreads / 32) / p.row_warps) + threadIdx.x;
        float sum = 0.f;
        for (int i = 0; i < p.row_warps; ++i) sum += s_dot[threadIdx.x * p.row_warps + i];
        if (r < p.rows) p.dw[r] = sum;
    }
}

}  // namespace ckpt
}  // namespace moe
