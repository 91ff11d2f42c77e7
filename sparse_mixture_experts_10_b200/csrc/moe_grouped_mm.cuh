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

// CUDA-core kernel for fp32 operands: 64 x 64 tiles, slices of 32 along the
// contraction in two shared-memory buffers (the next two slices travel in
// registers meanwhile), two halves of 128 threads with 8 x 4 results each as pairs of rows
// (one f32x2 multiply-add for two); either half takes 16 of a slice's 32 steps,
// and their fp32 sums are added at the end.  12 floats are read from shared
// memory for 32 multiply-adds; the second half doubles the warps that hide
// the latencies where there are few tiles.  8 x 1024 x 256 over 1024 rows: 23 us;
// 4 x 1536 x 1536 over 2048 rows: 249 (NT), 242 (NN), 243 us (TN), 40 TFLOP/s of about
// 70; what is left is latency between slices (four warps a scheduler).
constexpr int kTile = 64, kSlice = 32, kSimtThreads = 256;

template <int KIND>
__global__ void __launch_bounds__(kSimtThreads) simt_kernel(const Params p) {
    pdl_enter();
    __shared__ __align__(16) float s_ab[2][2][kSlice][kTile + 4];   // [operand][buffer]
    auto &As = s_ab[0], &Bs = s_ab[1];
    __shared__ int s_off[kMaxGroups + 1], s_cum[kMaxGroups + 1];
    const int tid = threadIdx.x;
    if (tid < 32) load_segments(p.row_offsets, p.G, p.rows, kTile, s_off, s_cum);
    __syncthreads();
    const float *A = static_cast<const float *>(p.A), *B = static_cast<const float *>(p.B);
    const int cols = KIND == NT ? p.n : p.k;   // columns of the result
    const int total = KIND == TN ? p.total : s_cum[p.G] * p.n_tiles;
    const int half = tid >> 7, tx = tid & 15, ty = (tid & 127) >> 4;
    // a K-major operand (rows of the tile contiguous along the contraction): thread -> row tid/4, 8 values from
    // (tid%4)*8; an MN-major one: thread -> contraction index tid/8, 8 values from (tid%8)*8
    constexpr int kV = 2;   // 16-byte loads of each operand
    const int kr = tid >> 2, kc = (tid & 3) * 8, mr = tid >> 3, mc = (tid & 7) * 8;
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
        const float *Bg = KIND == TN ? B : B + (int64_t)g * p.n * p.ldb;
        float4 a0[kV], b0[kV], a1[kV], b1[kV];   // the next slice and the one after it, on their way
        auto fetch = [&](int kk, float4 (&a)[kV], float4 (&b)[kV]) {
#pragma unroll
            for (int h = 0; h < kV; ++h) {
                const float4 z = make_float4(0.f, 0.f, 0.f, 0.f);
                const int kh = kc + 4 * h, mh = mc + 4 * h;
                auto at = [](const float *q) { return __ldg(reinterpret_cast<const float4 *>(q)); };
                if (KIND == TN) a[h] = kk + mr < hi && m0 + mh < m_hi ? at(A + (kk + mr) * p.lda + m0 + mh) : z;
                else a[h] = m0 + kr < m_hi && kk + kh < hi ? at(A + (m0 + kr) * p.lda + kk + kh) : z;
                if (KIND == NT) b[h] = n0 + kr < cols && kk + kh < hi ? at(Bg + (n0 + kr) * p.ldb + kk + kh) : z;
                else b[h] = kk + mr < hi && n0 + mh < cols ? at(Bg + (kk + mr) * p.ldb + n0 + mh) : z;
            }
        };
        // Step k of a slice has its columns rotated by 8 (k / 8): a K-major operand is stored transposed, by lanes that hold
        // the steps 0, 8, 16 and 24 of 8 rows, and they then meet 32 different banks instead of 8 (283 -> 249 us).
        auto col = [](int k, int m) { return (m + (k & ~7)) & (kTile - 1); };
        auto put = [&](int buf, const float4 (&a)[kV], const float4 (&b)[kV]) {
#pragma unroll
            for (int h = 0; h < kV; ++h) {
                const int kh = kc + 4 * h, mh = mc + 4 * h;
                if (KIND == TN) {
                    *reinterpret_cast<float4 *>(&As[buf][mr][col(mr, mh)]) = a[h];
                } else {
                    const int c = col(kh, kr);   // kh .. kh + 3 are in one group of 8
                    As[buf][kh][c] = a[h].x; As[buf][kh + 1][c] = a[h].y;
                    As[buf][kh + 2][c] = a[h].z; As[buf][kh + 3][c] = a[h].w;
                }
                if (KIND == NT) {
                    const int c = col(kh, kr);
                    Bs[buf][kh][c] = b[h].x; Bs[buf][kh + 1][c] = b[h].y;
                    Bs[buf][kh + 2][c] = b[h].z; Bs[buf][kh + 3][c] = b[h].w;
                } else {
                    *reinterpret_cast<float4 *>(&Bs[buf][mr][col(mr, mh)]) = b[h];
                }
            }
        };
        uint64_t acc[4][4];   // [pair of rows][column]
#pragma unroll
        for (int x = 0; x < 4; ++x)
#pragma unroll
            for (int y = 0; y < 4; ++y) acc[x][y] = 0;
        auto multiply = [&](int buf) {
#pragma unroll
            for (int q0 = 0; q0 < kSlice / 2; ++q0) {
                const int q = half * (kSlice / 2) + q0;
                const int ca = col(q, ty * 8);
                const ulonglong2 av0 = *reinterpret_cast<const ulonglong2 *>(&As[buf][q][ca]);
                const ulonglong2 av1 = *reinterpret_cast<const ulonglong2 *>(&As[buf][q][ca + 4]);
                const float4 bv = *reinterpret_cast<const float4 *>(&Bs[buf][q][col(q, tx * 4)]);
                const uint64_t ar[4] = {av0.x, av0.y, av1.x, av1.y};
                const uint64_t br[4] = {f2_splat(bv.x), f2_splat(bv.y), f2_splat(bv.z), f2_splat(bv.w)};
#pragma unroll
                for (int x = 0; x < 4; ++x)
#pragma unroll
                    for (int y = 0; y < 4; ++y) acc[x][y] = f2_fma(ar[x], br[y], acc[x][y]);
            }
        };
        const bool active = m0 + ((tid & 127) >> 5) * 16 < m_hi;   // a warp whose 16 rows are past the segment's end rests
        if (lo < hi) fetch(lo, a0, b0);
        if (lo + kSlice < hi) fetch(lo + kSlice, a1, b1);
        for (int kk = lo; kk < hi; kk += 2 * kSlice) {   // two slices a turn, one per buffer and register set
            put(0, a0, b0);
            if (kk + 2 * kSlice < hi) fetch(kk + 2 * kSlice, a0, b0);
            __syncthreads();
            if (active) multiply(0);
            if (kk + kSlice >= hi) break;
            put(1, a1, b1);
            if (kk + 3 * kSlice < hi) fetch(kk + 3 * kSlice, a1, b1);
            __syncthreads();
            if (active) multiply(1);
        }
        __syncthreads();
        // the second half's sums, through the operands' buffers
        uint64_t *s_sum = reinterpret_cast<uint64_t *>(&s_ab[0][0][0][0]) + (tid & 127);
        if (half) {
#pragma unroll
            for (int x = 0; x < 16; ++x) s_sum[x * 128] = acc[x >> 2][x & 3];
        }
        __syncthreads();
        if (!half) {
#pragma unroll
            for (int x = 0; x < 16; ++x) acc[x >> 2][x & 3] = f2_add(acc[x >> 2][x & 3], s_sum[x * 128]);
        }
        __syncthreads();
        const int c = n0 + tx * 4;
        if (half || c >= cols) continue;
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            float v[2][4];
#pragma unroll
            for (int y = 0; y < 4; ++y) f2_unpack(acc[x][y], v[0][y], v[1][y]);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int r = m0 + ty * 8 + 2 * x + h;
                if (r >= m_hi) continue;
                float4 *dst = reinterpret_cast<float4 *>(static_cast<float *>(p.C) +
                                                         ((KIND == TN ? (int64_t)g * p.n : 0) + r) * p.ldc + c);
                float4 o = make_float4(v[h][0], v[h][1], v[h][2], v[h][3]);
                if (KIND == TN && p.accumulate) {
                    const float4 was = *dst;
                    o = make_float4(was.x + o.x, was.y + o.y, was.z + o.z, was.w + o.w);
                }
                *dst = o;
            }
        }
    }
}

}  // namespace gmm
}  // namespace moe
