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
// Bound by HBM: a few dozen instructions per value beside 8 to 12 bytes.  A
// lane takes four 16-byte pieces of each operand of a row at a time (one: 227
// and 270 us, two: 210 and 261 us, four: 208 and 251 us forward and backward
// for 65536 rows of 2 x 2048 bf16, that is 5.2 and 5.4 TB/s); the group's
// maximum is a shuffle tree over the 4 to 32 lanes that hold it.  GELU and e4m3 in
// 12289 rows of 2200: 36 and 45 us, 3.8 and 4.2 TB/s (the activation's
// instructions); in fp32 54 and 72 us, 4.5 and 4.9 TB/s.  SwiGLU and int8 in 32768
// rows of 2 x 2048 fp32: 190 and 240 us, 4.9 and 5.0 TB/s.  Reading back, one piece a
// lane: 65536 rows of 2 x 2048 bf16 in 188 us, 4.3 TB/s (two thirds of it writes);
// 32768 in fp32 in 151 us, 4.4 TB/s.
#pragma once

#include <cuda_fp8.h>

#include "moe_common.cuh"

namespace moe {
namespace ckpt {

enum { INT8 = 0, E4M3 = 1 };
enum { GELU = 0, SWIGLU = 1, NONE = 2 };

constexpr int kThreads = 256;
// 16-byte pieces of each operand that a lane loads before it computes: kUnroll of the kernels.  Four where
// there is work for every warp several times over, one for few rows (37 rows of 2 x 2880, forward and backward in a
// graph: 9.9 us with four, 5.6 us with one; 677 of 2 x 2120: 12.4 and 9.4; 3000 of 2 x 1024: 12.8 and 13.2).
constexpr int kManyUnroll = 4;

__device__ __forceinline__ void load16(const void *p, uint32_t (&w)[4]) {
    const uint4 u = __ldcs(static_cast<const uint4 *>(p));   // read once: ahead of everything else out of L2
    w[0] = u.x; w[1] = u.y; w[2] = u.z; w[3] = u.w;
}

// 16 bytes of a row: 8 bf16 or 4 fp32 values.
template <typename T>
struct Vec;
template <>
struct Vec<__nv_bfloat16> {
    static constexpr int N = 8;
    static __device__ __forceinline__ void widen(const uint32_t (&w)[4], float (&v)[8]) {
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
    static __device__ __forceinline__ void widen(const uint32_t (&w)[4], float (&v)[4]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = __uint_as_float(w[i]);
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

// Four values v 2^-e (inv = 2^-e) as four bytes.  int8: 1.5 2^23 + x holds round(x), ties to even, in its low
// bits (the product with a power of two is exact, so the fused sum rounds once); the conversion instructions
// run at an eighth of its rate.
template <int FMT>
__device__ __forceinline__ uint32_t quant4(const float *v, float inv) {
    if (FMT == INT8) {
        uint32_t b[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) b[i] = __float_as_uint(fmaf(v[i], inv, 12582912.0f));
        return __byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410);
    }
    const __nv_fp8x2_storage_t lo = __nv_cvt_float2_to_fp8x2(make_float2(v[0] * inv, v[1] * inv), __NV_SATFINITE, __NV_E4M3);
    const __nv_fp8x2_storage_t hi = __nv_cvt_float2_to_fp8x2(make_float2(v[2] * inv, v[3] * inv), __NV_SATFINITE, __NV_E4M3);
    return (uint32_t)lo | ((uint32_t)hi << 16);
}

// int8: a byte q + 128 in the low bits of 2^23 is the float 2^23 + 128 + q.
template <int FMT>
__device__ __forceinline__ void dequant4(uint32_t q, float s, float *v) {
    if (FMT == INT8) {
        const uint32_t u = q ^ 0x80808080u;
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = (__uint_as_float(__byte_perm(u, 0x4b000000u, 0x7440 + i)) - 8388736.0f) * s;
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
    return byte == 255u ? __int_as_float(0x7fffffff) : pow2i((int)max(byte, 1u) - 127);
}

// NaN-keeping maximum of magnitudes over the lanes of a group, as bit patterns (NaN is above infinity).  Magnitudes
// of bf16 compare as 16-bit integers, two at a time.
template <typename T>
__device__ __forceinline__ float amax_group(const uint32_t (&raw)[4], int lanes) {
    uint32_t m = 0;
    if (sizeof(T) == 2) {
#pragma unroll
        for (int i = 0; i < 4; ++i) m = __vmaxu2(m, raw[i] & 0x7fff7fffu);
        for (int o = lanes >> 1; o >= 1; o >>= 1) m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, o));
        return __uint_as_float(max(m & 0xffff0000u, m << 16));
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) m = max(m, raw[i] & 0x7fffffffu);
    for (int o = lanes >> 1; o >= 1; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
    return __uint_as_float(m);
}

// Phi(v), the normal distribution function, with its density, and the sigmoid, in the accuracy of the row type, for
// v < 0 relative to Phi itself: fp32 rows take normal_cdf, expf and a division.  bf16 rows (rounded to 2^-8 afterwards)
// take the special-function unit, and for Phi fewer terms of the same form: Phi(-|v|) = t (q1 + t (q2 + ... + t q6)) exp(-v^2 / 2), t = 1 / (1 + c |v|), whose
// exponential is the density's too.  c and q are a fit of Phi(-x) exp(x^2 / 2) for x from 0 to 13.5 (Phi(-13.2) is
// 2^-130) that minimises the larger of error / 7.5e-8 and relative error / 2^-11: it is off by at most 3e-8 and by at
// most 2^-12.3 of Phi; the rounding of t and of the exponential adds up to 4e-7 near 0.
template <typename T>
__device__ __forceinline__ float phi(float v, float *density) {
    if (sizeof(T) == 4) return normal_cdf(v, density);
    const float t = rcp_approx(fmaf(fabsf(v), 0.287f, 1.0f));
    const float e = ex2_approx(v * v * -0.7213475204444817f);         // log2(e) / 2
    float q = fmaf(t, -0.0936281755566597f, 0.3131586015224457f);
    q = fmaf(t, q, -0.12920913100242615f);
    q = fmaf(t, q, 0.19976626827690674f);
    q = fmaf(t, q, 0.09363754838705063f);
    q = fmaf(t, q, 0.11627483367919922f);
    const float below = q * t * e;
    if (density) *density = e * 0.39894228040143268f;                 // 1 / sqrt(2 pi)
    return v < 0.f ? below : 1.0f - below;
}
template <typename T>
__device__ __forceinline__ float sigmoid(float v) {
    if (sizeof(T) == 4) return 1.0f / (1.0f + expf(-v));
    return rcp_approx(1.0f + ex2_approx(v * -1.4426950408889634f));
}

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

// One vector of a row's half: the checkpoint's bytes written.
template <typename T, int FMT>
__device__ __forceinline__ void save_vec(const Params &p, int64_t row, int half, int halves, int c, bool in,
                                         const uint32_t (&raw)[4], float (&v)[Vec<T>::N]) {
    constexpr int N = Vec<T>::N;
    const int lanes = (1 << p.group_shift) / N;
    const int sb = scale_byte<FMT>(amax_group<T>(raw, lanes));
    Vec<T>::widen(raw, v);
    if (!in) return;
    const float inv = pow2i(sb == 255 ? 0 : 127 - sb);
    uint32_t q[N / 4];
    if (FMT == INT8 && sb == kMostExp<FMT> + 127) {   // may saturate (the conversion to e4m3 does so by itself)
        float w[N];
#pragma unroll
        for (int i = 0; i < N; ++i) w[i] = fminf(fmaxf(v[i] * inv, -127.f), 127.f);
#pragma unroll
        for (int i = 0; i < N / 4; ++i) q[i] = quant4<FMT>(w + 4 * i, 1.0f);
    } else {
#pragma unroll
        for (int i = 0; i < N / 4; ++i) q[i] = sb == 255 ? 0u : quant4<FMT>(v + 4 * i, inv);
    }
    Vec<T>::store_q(p.q + (row * halves + half) * p.width + c, q);
    if ((c & ((1 << p.group_shift) - 1)) == 0)
        p.s[(row * halves + half) * p.sgroups + (c >> p.group_shift)] = (uint8_t)sb;
}

// One vector of a checkpoint: fetched as bytes, widened later.
template <typename T>
struct Saved {
    uint32_t q[Vec<T>::N / 4], s;
    __device__ __forceinline__ void fetch(const Params &p, int64_t row, int half, int halves, int c) {
        Vec<T>::load_q(p.q_in + (row * halves + half) * p.width + c, q);
        s = p.s_in[(row * halves + half) * p.sgroups + (c >> p.group_shift)];
    }
    template <int FMT>
    __device__ __forceinline__ void widen(float (&v)[Vec<T>::N]) const {
        const float scale = scale_value(s);
#pragma unroll
        for (int i = 0; i < Vec<T>::N / 4; ++i) dequant4<FMT>(q[i], scale, v + 4 * i);
    }
};

template <typename T, int ACT, int FMT, int kUnroll>
__global__ void __launch_bounds__(kThreads) forward_kernel(const Params p) {
    pdl_enter();
    constexpr int N = Vec<T>::N, kHalves = ACT == SWIGLU ? 2 : 1;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t row = (int64_t)blockIdx.x * ((kThreads / 32) / p.row_warps) + warp / p.row_warps;
    if (row >= p.rows) return;
    const T *u = static_cast<const T *>(p.u) + row * p.ldu;
    const int stride = p.row_warps * 32 * N;
    for (int c0 = (warp % p.row_warps) * 32 * N; c0 < p.width; c0 += kUnroll * stride) {
        uint32_t ra[kUnroll][4] = {}, rb[kUnroll][4] = {};
#pragma unroll
        for (int k = 0; k < kUnroll; ++k) {
            const int c = c0 + k * stride + lane * N;
            if (c < p.width) {
                load16(u + c, ra[k]);
                if (ACT == SWIGLU) load16(u + p.width + c, rb[k]);
            }
        }
#pragma unroll
        for (int k = 0; k < kUnroll; ++k) {
            if (c0 + k * stride >= p.width) break;   // warp-uniform
            const int c = c0 + k * stride + lane * N;
            const bool in = c < p.width;
            float a[N], b[N], o[N];
            save_vec<T, FMT>(p, row, 0, kHalves, c, in, ra[k], a);
            if (ACT == SWIGLU) save_vec<T, FMT>(p, row, 1, kHalves, c, in, rb[k], b);
            if (ACT == NONE || !in) continue;
#pragma unroll
            for (int i = 0; i < N; ++i)
                o[i] = ACT == GELU ? a[i] * phi<T>(a[i], nullptr) : a[i] * sigmoid<T>(a[i]) * b[i];
            Vec<T>::store(static_cast<T *>(p.h) + row * p.ldh + c, o);
        }
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
            Saved<T> x;
            x.fetch(p, row, half, halves, c);
            x.template widen<FMT>(v);
            Vec<T>::store(static_cast<T *>(p.h) + row * p.ldh + (int64_t)half * p.width + c, v);
        }
}

// hw = w act(u^), du = w dh act'(u^), dw = <dh, act(u^)>; the row's sum is taken lane by lane, then
// over the lanes and warps of the row, in an order set by the sizes alone.
template <typename T, int ACT, int FMT, int kUnroll>
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
        const int stride = p.row_warps * 32 * N;
        for (int c0 = (warp % p.row_warps) * 32 * N; c0 < p.width; c0 += kUnroll * stride) {
            uint32_t rd[kUnroll][4] = {};
            Saved<T> xa[kUnroll], xb[kUnroll];
#pragma unroll
            for (int k = 0; k < kUnroll; ++k) {
                const int c = c0 + k * stride + lane * N;
                if (c < p.width) {
                    load16(dh + c, rd[k]);
                    xa[k].fetch(p, row, 0, kHalves, c);
                    if (ACT == SWIGLU) xb[k].fetch(p, row, 1, kHalves, c);
                }
            }
#pragma unroll
            for (int k = 0; k < kUnroll; ++k) {
                const int c = c0 + k * stride + lane * N;
                if (c >= p.width) break;
                float a[N], b[N], d[N], hv[N], da[N], db[N];
                Vec<T>::widen(rd[k], d);
                xa[k].template widen<FMT>(a);
                if (ACT == SWIGLU) xb[k].template widen<FMT>(b);
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    const float g = w * d[i];
                    if (ACT == GELU) {
                        float density;
                        const float ph = phi<T>(a[i], &density);
                        hv[i] = a[i] * ph;
                        da[i] = g * fmaf(a[i], density, ph);
                    } else {
                        const float sg = sigmoid<T>(a[i]), si = a[i] * sg;
                        hv[i] = si * b[i];
                        da[i] = g * b[i] * sg * (1.0f + a[i] * (1.0f - sg));
                        db[i] = g * si;
                    }
                    dot = fmaf(d[i], hv[i], dot);
                    hv[i] *= w;
                }
                Vec<T>::store(du + c, da);
                if (ACT == SWIGLU) Vec<T>::store(du + p.width + c, db);
                if (p.hw) Vec<T>::store(static_cast<T *>(p.hw) + row * p.ldh + c, hv);
            }
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
