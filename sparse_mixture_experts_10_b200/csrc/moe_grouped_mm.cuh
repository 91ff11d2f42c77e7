// moe_grouped_mm.cuh -- matrix products grouped by expert over ragged row segments.
//
// The rows of group g are [off[g], off[g+1]) of the row operands; weights are
// stored out x in (B[g] is n x k):
//   NT  C[r, :n]  = sum_i A[r, i] B[g, :, i]     an expert's linear on its rows
//   NN  C[r, :k]  = sum_i A[r, i] B[g, i, :]     the gradient of its input
//   TN  C[g, n, k] (+)= sum_r A[r, n] B[r, k]    the gradient of its weight
// Segments start anywhere and may be empty; rows outside every segment are
// neither read into a result nor written.
//
// This file: the segment table and the CUDA-core kernel (fp32 operands).
#pragma once

#include "moe_common.cuh"

namespace moe {
namespace gmm {

enum { NT = 0, NN = 1, TN = 2 };
constexpr int kMaxGroups = 1024;

// The offsets as a table in shared memory: off[0..G] clamped to [0, rows] and
// made non-decreasing (a table that breaks the rule sets MOE_STATUS_BOUNDS,
// and no access leaves the arrays), and cum[g] = tiles of `tile` rows before
// group g.  Executed by one whole warp.
__device__ __forceinline__ void load_segments(const int *__restrict__ row_offsets, int G, int64_t rows, int tile,
                                              int *off, int *cum) {
    const int lane = threadIdx.x & 31;
    int carry = 0, ctiles = 0;   // the previous offset; tiles of the groups before it
    bool bad = false;
    for (int i0 = 0; i0 <= G; i0 += 32) {
        const int i = i0 + lane;
        const int raw = i <= G ? row_offsets[i] : 0;
        int v = i <= G ? (int)min((int64_t)max(raw, 0), rows) : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {   // running maximum
            const int u = __shfl_up_sync(0xffffffffu, v, o);
            if (lane >= o) v = max(v, u);
        }
        v = max(v, carry);
        int prev = __shfl_up_sync(0xffffffffu, v, 1);
        if (lane == 0) prev = carry;
        const int t = (i == 0 || i > G) ? 0 : (int)(((int64_t)v - prev + tile - 1) / tile);   // tiles of group i - 1
        int incl = t;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += u;
        }
        if (i <= G) {
            off[i] = v;
            cum[i] = ctiles + incl;
            bad |= v != raw;
        }
        carry = __shfl_sync(0xffffffffu, v, 31);
        ctiles += __shfl_sync(0xffffffffu, incl, 31);
    }
    if (__any_sync(0xffffffffu, bad) && lane == 0) set_status(kStatusBounds);
}

// The group whose tiles hold tile i: the last g with cum[g] <= i.
__device__ __forceinline__ int group_of_tile(const int *cum, int G, int i) {
    int lo = 0, hi = G - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (cum[mid] <= i) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

struct Params {
    const void *A, *B;
    void *C;
    const int *row_offsets;   // [G+1]
    int64_t rows;             // rows of A (and of B in TN, of C in NT and NN)
    int64_t lda, ldb, ldc;    // row strides in elements
    int G, n, k;
    int accumulate;           // TN: add to C
    int m_tiles, n_tiles;     // TN: tiles of a group; NT, NN: n_tiles column tiles
    int total;                // TN: all tiles; NT, NN: at most so many (the count is known on the device)
    int m_chunks, n_chunks;   // tensor cores: an MN-major operand's map has chunks of 64 values as a dimension
    uint64_t timeout_ns;
};

template <typename T>
__device__ __forceinline__ float4 load4(const T *p);
template <>
__device__ __forceinline__ float4 load4<float>(const float *p) { return __ldg(reinterpret_cast<const float4 *>(p)); }
template <>
__device__ __forceinline__ float4 load4<__nv_bfloat16>(const __nv_bfloat16 *p) {
    const uint2 u = __ldg(reinterpret_cast<const uint2 *>(p));
    return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u), __uint_as_float(u.y << 16),
                       __uint_as_float(u.y & 0xffff0000u));
}
__device__ __forceinline__ float4 get4(const float *p) { return *reinterpret_cast<const float4 *>(p); }
__device__ __forceinline__ float4 get4(const __nv_bfloat16 *p) {
    const uint2 u = *reinterpret_cast<const uint2 *>(p);
    return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u), __uint_as_float(u.y << 16),
                       __uint_as_float(u.y & 0xffff0000u));
}
__device__ __forceinline__ void put4(float *p, float4 v) { *reinterpret_cast<float4 *>(p) = v; }
__device__ __forceinline__ void put4(__nv_bfloat16 *p, float4 v) {
    *reinterpret_cast<uint2 *>(p) = make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
}

// CUDA-core kernel: 64 x 64 tiles, slices of 16 along the contraction, 256
// threads with 4 x 4 results each, sums in fp32 in ascending order.
constexpr int kTile = 64, kSlice = 16;

template <typename T, typename TO, int KIND>
__global__ void __launch_bounds__(256) simt_kernel(const Params p) {
    pdl_enter();
    __shared__ __align__(16) float As[kSlice][kTile + 4];
    __shared__ __align__(16) float Bs[kSlice][kTile + 4];
    __shared__ int s_off[kMaxGroups + 1], s_cum[kMaxGroups + 1];
    const int tid = threadIdx.x;
    if (tid < 32) load_segments(p.row_offsets, p.G, p.rows, kTile, s_off, s_cum);
    __syncthreads();
    const T *A = static_cast<const T *>(p.A), *B = static_cast<const T *>(p.B);
    const int cols = KIND == NT ? p.n : p.k;   // columns of the result
    const int total = KIND == TN ? p.total : s_cum[p.G] * p.n_tiles;
    const int tx = tid & 15, ty = tid >> 4;
    // a K-major operand (rows of the tile contiguous along the contraction): thread -> row tid/4, 4 values from
    // (tid%4)*4; an MN-major one: thread -> contraction index tid/16, 4 values from (tid%16)*4
    const int kr = tid >> 2, kc = (tid & 3) * 4, mr = tid >> 4, mc = (tid & 15) * 4;
    for (int i = blockIdx.x; i < total; i += gridDim.x) {
        int g, m0, n0, m_hi, lo = 0, hi;   // rows (or A columns) m0..m_hi, result columns from n0, contraction lo..hi
        if (KIND == TN) {
            const int per = p.m_tiles * p.n_tiles;
            g = i / per;
            const int r = i - g * per;
            m0 = r / p.n_tiles * kTile;
            n0 = r % p.n_tiles * kTile;
            m_hi = p.n;
            lo = s_off[g];
            hi = s_off[g + 1];
        } else {
            const int mt = i / p.n_tiles;
            g = group_of_tile(s_cum, p.G, mt);
            m0 = s_off[g] + (mt - s_cum[g]) * kTile;
            n0 = (i - mt * p.n_tiles) * kTile;
            m_hi = s_off[g + 1];
            hi = KIND == NT ? p.k : p.n;
        }
        const T *Bg = KIND == TN ? B : B + (int64_t)g * p.n * p.ldb;
        float4 a, b;
        auto fetch = [&](int kk) {
            const float4 z = make_float4(0.f, 0.f, 0.f, 0.f);
            if (KIND == TN) a = kk + mr < hi && m0 + mc < m_hi ? load4(A + (kk + mr) * p.lda + m0 + mc) : z;
            else a = m0 + kr < m_hi && kk + kc < hi ? load4(A + (m0 + kr) * p.lda + kk + kc) : z;
            if (KIND == NT) b = n0 + kr < cols && kk + kc < hi ? load4(Bg + (int64_t)(n0 + kr) * p.ldb + kk + kc) : z;
            else b = kk + mr < hi && n0 + mc < cols ? load4(Bg + (int64_t)(kk + mr) * p.ldb + n0 + mc) : z;
        };
        float acc[4][4] = {};
        if (lo < hi) fetch(lo);
        for (int kk = lo; kk < hi; kk += kSlice) {
            if (KIND == TN) {
                *reinterpret_cast<float4 *>(&As[mr][mc]) = a;
            } else {
                As[kc][kr] = a.x; As[kc + 1][kr] = a.y; As[kc + 2][kr] = a.z; As[kc + 3][kr] = a.w;
            }
            if (KIND == NT) {
                Bs[kc][kr] = b.x; Bs[kc + 1][kr] = b.y; Bs[kc + 2][kr] = b.z; Bs[kc + 3][kr] = b.w;
            } else {
                *reinterpret_cast<float4 *>(&Bs[mr][mc]) = b;
            }
            __syncthreads();
            if (kk + kSlice < hi) fetch(kk + kSlice);
#pragma unroll
            for (int q = 0; q < kSlice; ++q) {
                const float4 av = *reinterpret_cast<const float4 *>(&As[q][ty * 4]);
                const float4 bv = *reinterpret_cast<const float4 *>(&Bs[q][tx * 4]);
                const float ar[4] = {av.x, av.y, av.z, av.w}, br[4] = {bv.x, bv.y, bv.z, bv.w};
#pragma unroll
                for (int x = 0; x < 4; ++x)
#pragma unroll
                    for (int y = 0; y < 4; ++y) acc[x][y] = fmaf(ar[x], br[y], acc[x][y]);
            }
            __syncthreads();
        }
        const int c = n0 + tx * 4;
        if (c >= cols) continue;
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            const int r = m0 + ty * 4 + x;
            if (r >= m_hi) continue;
            TO *dst = static_cast<TO *>(p.C) + ((KIND == TN ? (int64_t)g * p.n : 0) + r) * p.ldc + c;
            float4 v = make_float4(acc[x][0], acc[x][1], acc[x][2], acc[x][3]);
            if (KIND == TN && p.accumulate) {
                const float4 o = get4(dst);
                v = make_float4(o.x + v.x, o.y + v.y, o.z + v.z, o.w + v.w);
            }
            put4(dst, v);
        }
    }
}

}  // namespace gmm
}  // namespace moe
