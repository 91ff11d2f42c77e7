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

// ---------------------------------------------------------------- the products
// One warp per 16 rows of W[e] (SwiGLU: 8 gate rows and the 8 up rows beside
// them, so that a lane ends with both) and per share of k, against up to 16
// pairs of the expert as columns of m16n8k16 products (bf16 x bf16 -> fp32).
// A code is at most 4 bits, exact in bf16; the products of a group of 32 are
// summed in fp32 by the tensor core and enter the result with one fp32
// multiply-add by the group's scale, so nothing is rounded to fewer bits before
// the end.
//
// Bound by HBM (0.5 byte per weight).  Each warp streams its 16 rows itself, as
// boxes of 16 x 128 bytes (256 values of k) into a ring of its own: no block
// barrier in the loop, and 5 boxes x 16 warps = 160 KB per SM in flight.  The
// 128-byte swizzle lets the fragment reads (4 bytes per lane: 8 rows x 16
// bytes) hit 32 different banks.  Inside a group the order of k is free: lane t
// of a row takes the 8 codes of one 32-bit word, as pairs (i, i + 4) that one
// mask each extracts, and x is permuted the same way.
constexpr int kWarps = 4, kSlots = 5, kBoxBytes = 2048, kChunk = 256;
constexpr int kMaxPairs = 4096, kMaxExperts = 1024;

struct MatvecParams : Params {
    int act, y_f32;
    int tiles, ks;         // 16-row tiles of an expert; warps of a block that share a tile (split k)
    uint64_t timeout_ns;
};

// 8 codes as four bf16 pairs (i, i + 4), i = 0..3.
template <int FMT>
__device__ __forceinline__ void decode8(uint32_t w, uint32_t (&v)[4]) {
    if (FMT == INT4) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {   // 0x4300 | c is 128 + c; minus 136 exactly c - 8
            uint32_t u = ((w >> (4 * i)) & 0x000f000fu) | 0x43004300u;
            asm("sub.rn.bf16x2 %0, %0, %1;" : "+r"(u) : "r"(0x43084308u));
            v[i] = u;
        }
    } else {
        // exponent and mantissa bits at bf16's place read as value 2^-126 (subnormals included); times 2^126 exactly
        const uint32_t m[4] = {w << 6, w << 2, w >> 2, w >> 6}, s[4] = {w << 12, w << 8, w << 4, w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t u = (m[i] & 0x01c001c0u) | (s[i] & 0x80008000u);
            asm("mul.rn.bf16x2 %0, %0, %1;" : "+r"(u) : "r"(0x7e807e80u));
            v[i] = u;
        }
    }
}

// d = A B (first) or d += A B
__device__ __forceinline__ void mma16816_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                               uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, "
        "%10, %10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, "
        "%2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// What a lane holds of a chunk of k: the scales of the rows g and g + 8 for the 32-value pieces 2t and 2t + 1
// (one scale for both with groups of 64 and more; 0 past the last group).
template <int FMT, int SHIFT>
struct ScaleRows {
    static constexpr int kN = SHIFT == 5 ? 2 : 1;
    int64_t row0, row1;   // first scale of the row; row1 < 0: no such row
    __device__ __forceinline__ void load(const MatvecParams &p, int chunk, int t, float (&v)[2 * kN]) const {
#pragma unroll
        for (int j = 0; j < kN; ++j) {
            const int at = (chunk * kChunk + (2 * t + j) * 32) >> SHIFT;
            const bool in = at < p.groups;
            v[j] = in ? scale_of<FMT>(p.scales, row0 + at) : 0.f;
            v[kN + j] = in && row1 >= 0 ? scale_of<FMT>(p.scales, row1 + at) : 0.f;
        }
    }
};

// x of the columns g (+ 8 b) for four pieces of k from k0: 8 values per lane and piece, 0 from k on.
template <int NB>
__device__ __forceinline__ void load_x(const __nv_bfloat16 *const (&xr)[NB], int k0, int k, uint4 (&v)[NB][4]) {
    if (k0 + 128 <= k) {
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int c = 0; c < 4; ++c) v[b][c] = __ldg(reinterpret_cast<const uint4 *>(xr[b] + k0 + c * 32));
    } else {
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int c = 0; c < 4; ++c)
                v[b][c] = k0 + c * 32 < k ? __ldg(reinterpret_cast<const uint4 *>(xr[b] + k0 + c * 32))
                                          : make_uint4(0, 0, 0, 0);
    }
}

// One warp's share of k against columns of the expert's pairs (NB blocks of 8).
// acc[b]: rows g (0, 1) and g + 8 (2, 3), columns 2t and 2t + 1.  False if a wait ran out.
template <int FMT, int SHIFT, int NB>
__device__ __forceinline__ bool stream_rows(const MatvecParams &p, const CUtensorMap *map, uint8_t *ring, uint64_t *bars,
                                            uint32_t &phases, int box_row0, int box_row1, int64_t row0, int64_t row1,
                                            int c_lo, int c_hi, const uint16_t *list, int cnt, float (&acc)[NB][4]) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int n = c_hi - c_lo;
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[b][i] = 0.f;
    if (n <= 0) return true;
    auto issue = [&](int i, int slot) {   // box i of this share
        mbar_arrive_expect_tx(&bars[slot], kBoxBytes);
        tma_load_2d(map, &bars[slot], ring + slot * kBoxBytes, (c_lo + i) * (kChunk / 2), box_row0);
        tma_load_2d(map, &bars[slot], ring + slot * kBoxBytes + 1024, (c_lo + i) * (kChunk / 2), box_row1);
    };
    if (lane == 0)
        for (int i = 0; i < min(n, kSlots); ++i) issue(i, i);
    // scales three chunks ahead: they come straight from global memory
    using Rows = ScaleRows<FMT, SHIFT>;
    constexpr int kN = Rows::kN;
    const Rows rows{row0 * p.groups, row1 < 0 ? -1 : row1 * p.groups};
    float s0[2 * kN], s1[2 * kN] = {}, s2[2 * kN] = {};
    rows.load(p, c_lo, t, s0);
    if (n > 1) rows.load(p, c_lo + 1, t, s1);
    if (n > 2) rows.load(p, c_lo + 2, t, s2);
    // columns past the last pair repeat it; their results are not written
    const __nv_bfloat16 *xr[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b) xr[b] = p.x + (int64_t)(list[min(b * 8 + g, cnt - 1)] / p.x_div) * p.k + t * 8;
    constexpr int kPieces = 1 << (SHIFT - 5);   // per scale: their products are added up before it is applied
    // the word of piece c in the swizzled box: 16-byte unit c ^ g of row g; bits 4-6 of the rest are 0
    const uint32_t at = (uint32_t)(g * 128 + t * 4 + (g << 4));
    int slot = 0;
    for (int i = 0; i < n; ++i) {
        const int k0 = (c_lo + i) * kChunk;
        uint4 xa[NB][4], xb[NB][4];
        load_x<NB>(xr, k0, p.k, xa);
        if (!__all_sync(0xffffffffu, mbar_wait(&bars[slot], (phases >> slot) & 1u, p.timeout_ns))) {
            if (lane == 0)   // copies still in flight land before the block leaves
                for (int j = i; j < min(n, i + kSlots); ++j)
                    mbar_wait(&bars[j % kSlots], (phases >> (j % kSlots)) & 1u, p.timeout_ns);
            return false;
        }
        phases ^= 1u << slot;
        load_x<NB>(xr, k0 + 128, p.k, xb);
        const uint8_t *box = ring + slot * kBoxBytes;
        float d[NB][4];
#pragma unroll
        for (int c = 0; c < 8; ++c) {
            const uint8_t *w = box + (at ^ (uint32_t)(c << 4));
            uint32_t lo[4], hi[4];
            decode8<FMT>(*reinterpret_cast<const uint32_t *>(w), lo);
            decode8<FMT>(*reinterpret_cast<const uint32_t *>(w + 1024), hi);
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                const uint4 xv = c < 4 ? xa[b][c & 3] : xb[b][c & 3];
                const uint32_t b0 = __byte_perm(xv.x, xv.z, 0x5410), b1 = __byte_perm(xv.x, xv.z, 0x7632);
                const uint32_t b2 = __byte_perm(xv.y, xv.w, 0x5410), b3 = __byte_perm(xv.y, xv.w, 0x7632);
                if (c % kPieces == 0) mma16816_first(d[b], lo[0], hi[0], lo[1], hi[1], b0, b1);
                else mma16816(d[b], lo[0], hi[0], lo[1], hi[1], b0, b1);
                mma16816(d[b], lo[2], hi[2], lo[3], hi[3], b2, b3);
            }
            if (c % kPieces == kPieces - 1) {
                const float sa = __shfl_sync(0xffffffffu, s0[c % kN], (lane & ~3) | (c >> 1));
                const float sb = __shfl_sync(0xffffffffu, s0[kN + c % kN], (lane & ~3) | (c >> 1));
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    acc[b][0] = fmaf(sa, d[b][0], acc[b][0]);
                    acc[b][1] = fmaf(sa, d[b][1], acc[b][1]);
                    acc[b][2] = fmaf(sb, d[b][2], acc[b][2]);
                    acc[b][3] = fmaf(sb, d[b][3], acc[b][3]);
                }
            }
        }
        __syncwarp();
        if (lane == 0 && i + kSlots < n) issue(i + kSlots, slot);
#pragma unroll
        for (int j = 0; j < 2 * kN; ++j) {
            s0[j] = s1[j];
            s1[j] = s2[j];
        }
        if (i + 3 < n) rows.load(p, c_lo + i + 3, t, s2);
        if (++slot == kSlots) slot = 0;
    }
    return true;
}

// The expert's pairs list[0..cnt), at most 8 NB of them.
template <int FMT, int SHIFT, int NB>
__device__ __forceinline__ bool tile_columns(const MatvecParams &p, const CUtensorMap *map, uint8_t *ring, uint64_t *bars,
                                             uint32_t &phases, float (*part)[NB * 4][32], int e, int tile,
                                             const uint16_t *list, int cnt) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const bool swiglu = p.act == SWIGLU;
    const int share = warp % p.ks, cols = swiglu ? p.n / 2 : p.n;
    const int i0 = tile * (swiglu ? 8 : 16), i1 = swiglu ? cols + i0 : i0 + 8;   // first rows of the two halves
    const int64_t base = (int64_t)e * p.n;
    const int chunks = (p.k + kChunk - 1) / kChunk;
    float acc[NB][4];
    bool ok = true;
    if (tile < p.tiles)
        ok = stream_rows<FMT, SHIFT, NB>(p, map, ring, bars, phases, (int)(base + i0), (int)(base + i1), base + i0 + g,
                                         i1 + g < p.n ? base + i1 + g : -1, chunks * share / p.ks,
                                         chunks * (share + 1) / p.ks, list, cnt, acc);
    if (p.ks > 1) {   // the shares of k are added in their order
        if (share > 0)
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int i = 0; i < 4; ++i) part[warp][b * 4 + i][lane] = acc[b][i];
        __syncthreads();
        if (share == 0)
            for (int s = 1; s < p.ks; ++s)
#pragma unroll
                for (int b = 0; b < NB; ++b)
#pragma unroll
                    for (int i = 0; i < 4; ++i) acc[b][i] += part[warp + s][b * 4 + i][lane];
        __syncthreads();
    }
    if (!ok || share > 0 || tile >= p.tiles) return ok;
    auto put = [&](int64_t at, float v) {
        if (p.y_f32) static_cast<float *>(p.y)[at] = v;
        else static_cast<__nv_bfloat16 *>(p.y)[at] = __float2bfloat16(v);
    };
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int col = b * 8 + 2 * t + j;
            if (col >= cnt) continue;
            const int pr = list[col];
            const float w = p.gate ? p.gate[pr] : 1.0f;
            const int64_t y = (int64_t)pr * cols + i0 + g;
            float v0 = acc[b][j], v1 = acc[b][2 + j];
            if (swiglu) {
                put(y, w * (silu(v0) * v1));
            } else {
                if (p.act == GELU) {
                    v0 = gelu(v0);
                    v1 = gelu(v1);
                }
                put(y, w * v0);
                if (i1 + g < p.n) put(y + 8, w * v1);
            }
        }
    return ok;
}

// Grid (tile groups, live experts at most): block (x, y) takes kWarps / ks tiles of the y-th expert that has a pair.
template <int FMT, int SHIFT>
__global__ void __launch_bounds__(kWarps * 32, 4)
    matvec_kernel(const __grid_constant__ CUtensorMap map, const MatvecParams p) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *smem = align_smem_1024(smem_raw);
    __shared__ uint64_t s_bar[kWarps][kSlots];
    __shared__ uint32_t s_mask[kMaxExperts / 32];
    __shared__ int s_e, s_cnt, s_bad;
    __shared__ float s_part[kWarps][8][32];
    uint16_t *s_list = reinterpret_cast<uint16_t *>(smem + kWarps * kSlots * kBoxBytes);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x < kWarps * kSlots) mbar_init(&s_bar[threadIdx.x / kSlots][threadIdx.x % kSlots], 1);
    fence_mbar_init();
    if (threadIdx.x < kMaxExperts / 32) s_mask[threadIdx.x] = 0;
    if (threadIdx.x == 0) {
        s_e = -1;
        s_bad = 0;
        tma_prefetch_desc(&map);
    }
    __syncthreads();
    pdl_enter();
    const int pairs = (int)p.pairs;
    for (int i = threadIdx.x; i < pairs; i += kWarps * 32) {
        const int e = p.expert[i];
        if (e >= 0 && e < p.N) atomicOr(&s_mask[e >> 5], 1u << (e & 31));
        else s_bad = 1;
    }
    __syncthreads();
    if (warp == 0) {
        const uint32_t m = s_mask[lane];
        int incl = __popc(m);
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += u;
        }
        const int want = (int)blockIdx.y - (incl - __popc(m));   // this word's want-th live expert
        if (want >= 0 && want < __popc(m)) {
            uint32_t r = m;
            for (int i = 0; i < want; ++i) r &= r - 1;
            s_e = lane * 32 + __ffs(r) - 1;
        }
        __syncwarp();
        const int e = *(volatile int *)&s_e;
        int cnt = 0;
        if (e >= 0)
            for (int i0 = 0; i0 < pairs; i0 += 32) {   // the expert's pairs in order
                const bool mine = i0 + lane < pairs && p.expert[i0 + lane] == e;
                const uint32_t b = __ballot_sync(0xffffffffu, mine);
                if (mine) s_list[cnt + __popc(b & ((1u << lane) - 1))] = (uint16_t)(i0 + lane);
                cnt += __popc(b);
            }
        if (lane == 0) s_cnt = cnt;
    }
    __syncthreads();
    const int tiles_here = kWarps / p.ks, tile = blockIdx.x * tiles_here + warp / p.ks;
    if (s_bad && blockIdx.y == 0) {   // rows of pairs without an expert
        const int cols = p.act == SWIGLU ? p.n / 2 : p.n, per = (p.act == SWIGLU ? 8 : 16) * tiles_here;
        const int c0 = blockIdx.x * per, c1 = min(c0 + per, cols);
        for (int i = 0; i < pairs; ++i) {
            const int e = p.expert[i];
            if (e >= 0 && e < p.N) continue;
            if (e != -1 && blockIdx.x == 0 && threadIdx.x == 0) set_status(kStatusBounds);
            for (int c = c0 + threadIdx.x; c < c1; c += kWarps * 32) {
                if (p.y_f32) static_cast<float *>(p.y)[(int64_t)i * cols + c] = 0.f;
                else static_cast<__nv_bfloat16 *>(p.y)[(int64_t)i * cols + c] = __float2bfloat16(0.f);
            }
        }
    }
    const int e = s_e;
    if (e < 0) return;
    uint8_t *ring = smem + warp * kSlots * kBoxBytes;
    uint32_t phases = 0;
    // blocks of up to 16 pairs; the weights are read again (from L2) for each
    for (int c = 0; c < s_cnt; c += 16) {
        const int left = s_cnt - c;
        const bool ok = left <= 8 ? tile_columns<FMT, SHIFT, 1>(p, &map, ring, s_bar[warp], phases,
                                                                  reinterpret_cast<float(*)[4][32]>(s_part), e, tile,
                                                                  s_list + c, left)
                                  : tile_columns<FMT, SHIFT, 2>(p, &map, ring, s_bar[warp], phases,
                                                                  reinterpret_cast<float(*)[8][32]>(s_part), e, tile,
                                                                  s_list + c, min(left, 16));
        if (!__syncthreads_and(ok)) return;   // a wait ran out (status word); nothing is in flight any more
    }
}

constexpr size_t matvec_smem(int64_t pairs) { return 1024 + (size_t)kWarps * kSlots * kBoxBytes + (size_t)pairs * 2; }

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
