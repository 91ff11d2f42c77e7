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
__device__ __forceinline__ uint32_t raw_scale(const void *s, int64_t i) {
    return FMT == INT4 ? (uint32_t)__ldg(static_cast<const unsigned short *>(s) + i)
                       : (uint32_t)__ldg(static_cast<const unsigned char *>(s) + i);
}
template <int FMT>
__device__ __forceinline__ float wide_scale(uint32_t b) {
    if (FMT == INT4) return __uint_as_float(b << 16);
    return b == 255u ? __int_as_float(0x7fffffff) : b == 0u ? __int_as_float(0x00400000) : __int_as_float(b << 23);
}
template <int FMT>
__device__ __forceinline__ float scale_of(const void *s, int64_t i) { return wide_scale<FMT>(raw_scale<FMT>(s, i)); }

__device__ __forceinline__ float gelu(float v) { return 0.5f * v * (1.0f + erff(v * 0.70710678118654752f)); }
__device__ __forceinline__ float silu(float v) { return v / (1.0f + expf(-v)); }

// ---------------------------------------------------------------- the products
// One persistent block per SM takes an even share of the live experts' 16-row
// tiles of W[e] (SwiGLU: 8 gate rows and the 8 up rows beside them, so that a
// lane ends with both).  Its warps multiply tiles with up to 16 of the expert's
// pairs as columns of m16n8k16 products (bf16 x bf16 -> fp32); where there are
// few tiles, ks warps share a tile along k and their sums are added in order.
// A code is at most 4 bits, exact in bf16; the products of a group are summed
// in fp32 by the tensor core and enter the result with one fp32 multiply-add by
// the group's scale, so nothing is rounded to fewer bits before the end.
//
// HBM (0.5 byte per weight) is the floor; what is in the way of it is the
// instructions that unpack the codes (about 11 per 8 codes and lane).  Each warp
// streams its own boxes of 16 rows x 128 bytes (256 values of k) through a
// ring that runs on from tile to tile, without a block barrier.  The 128-byte
// swizzle lets the fragment reads (4 bytes per lane: 8 rows x 16 bytes) hit 32
// different banks.  Inside a group the order of k is free: lane t of a row takes
// the 8 codes of one 32-bit word, as pairs (i, i + 4) that one mask each
// extracts; the expert's rows of x are staged in shared memory in that order.
constexpr int kWarps = 16, kMaxSlots = 4, kBoxBytes = 2048, kChunk = 256;
constexpr int kMaxPairs = 4096, kMaxExperts = 1024, kMaxCols = 16;

struct MatvecParams : Params {
    int act, y_f32;
    int tiles, ks;         // 16-row tiles of an expert; warps that share a tile (split k)
    int slots;             // boxes of a warp's ring (3 or 4)
    int cols_pass;         // pairs staged at a time (at most kMaxCols)
    uint32_t x_stride;     // bytes between staged rows of x
    uint64_t timeout_ns;
};

// (a & b) | c in one instruction, the masks in registers: written in C++ it became two, and the integer
// instructions of the unpacking are what the kernel spends its time on.
__device__ __forceinline__ uint32_t and_or(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t d;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    return d;
}

// 8 codes as four bf16 pairs (i, i + 4), i = 0..3.
template <int FMT>
__device__ __forceinline__ void decode8(uint32_t w, uint32_t (&v)[4]) {
    if (FMT == INT4) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {   // 0x4300 | c is 128 + c; minus 136 exactly c - 8
            v[i] = and_or(w >> (4 * i), 0x000f000fu, 0x43004300u);
            asm("sub.rn.bf16x2 %0, %0, %1;" : "+r"(v[i]) : "r"(0x43084308u));
        }
    } else {
        // exponent and mantissa bits at bf16's place read as value 2^-126 (subnormals included); times 2^126 exactly
        const uint32_t m[4] = {w << 6, w << 2, w >> 2, w >> 6}, s[4] = {w << 12, w << 8, w << 4, w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[i] = and_or(m[i], 0x01c001c0u, s[i] & 0x80008000u);
            asm("mul.rn.bf16x2 %0, %0, %1;" : "+r"(v[i]) : "r"(0x7e807e80u));
        }
    }
}

__device__ __forceinline__ uint32_t lds32(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ uint4 lds128(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
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

// A warp's walk over its boxes: tiles tile, tile + step, ... (below end), in each the chunks lo..hi-1.
struct Walk {
    int tile, chunk, left;   // left: boxes not reached yet, this one included
    __device__ __forceinline__ void next(int lo, int hi, int step) {
        --left;
        if (++chunk == hi) {
            chunk = lo;
            tile += step;
        }
    }
};

__device__ __forceinline__ void group_sync(int id, int threads) {
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// One warp's tiles of expert e against the staged columns (NB blocks of 8; list[0..cnt) their pairs).
template <int FMT, int SHIFT, int NB>
__device__ __forceinline__ bool run_tiles(const MatvecParams &p, const CUtensorMap *map, uint8_t *ring, uint64_t *bars,
                                          uint32_t &phases, int &slot, const uint8_t *s_x, float (*part)[8][32], int e,
                                          int tile0, int tile1, const uint16_t *list, int cnt, bool ok) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const bool swiglu = p.act == SWIGLU;
    const int cols = swiglu ? p.n / 2 : p.n;
    const int share = warp % p.ks, step = kWarps / p.ks;
    const int chunks = (p.k + kChunk - 1) / kChunk;
    const int lo = chunks * share / p.ks, hi = chunks * (share + 1) / p.ks;
    const int first = tile0 + warp / p.ks, mine = first < tile1 ? (tile1 - first + step - 1) / step : 0;
    const int64_t base = (int64_t)e * p.n;
    const int half1 = swiglu ? cols : 8;   // distance of the tile's second 8 rows from its first
    const int rows_tile = swiglu ? 8 : 16;
    const int total = mine * (hi - lo);
    Walk in{first, lo, total}, sc{first, lo, total};
    // The scales of a tile's rows into L2, when its first box is issued: they are read one box ahead of their use, which
    // covers the latency of L2 but not of HBM.
    constexpr int kScaleBytes = FMT == INT4 ? 2 : 1;
    auto prefetch_scales = [&](int tile) {
        const int row = tile * rows_tile + (lane & 7) + (lane & 8 ? half1 : 0);
        if (row >= p.n) return;
        const char *s = static_cast<const char *>(p.scales) + (base + row) * p.groups * kScaleBytes;
        const int b1 = min((hi * kChunk) >> SHIFT, p.groups) * kScaleBytes;
        for (int b = ((lo * kChunk) >> SHIFT) * kScaleBytes + (lane >> 4) * 32; b < b1 + 31; b += 64)
            asm volatile("prefetch.global.L2 [%0];" ::"l"(s + min(b, b1 - 1)));
    };
    auto issue = [&](int sl) {   // lane 0: the next box into slot sl
        const int r = (int)base + in.tile * rows_tile;
        mbar_arrive_expect_tx(&bars[sl], kBoxBytes);
        tma_load_2d(map, &bars[sl], ring + sl * kBoxBytes, in.chunk * (kChunk / 2), r);
        tma_load_2d(map, &bars[sl], ring + sl * kBoxBytes + 1024, in.chunk * (kChunk / 2), r + half1);
    };
    int sl = slot, flying = 0;   // boxes issued and not waited for
    for (int i = 0; i < p.slots && in.left > 0 && ok; ++i) {
        if (in.chunk == lo) prefetch_scales(in.tile);
        if (lane == 0) issue(sl);
        ++flying;
        in.next(lo, hi, step);
        if (++sl == p.slots) sl = 0;
    }
    // What a lane holds of a box: the scales of the rows g and g + 8 for the 32-value pieces 2t and 2t + 1 (one scale
    // for both with groups of 64 and more; 0 past the last group).
    constexpr int kN = SHIFT == 5 ? 2 : 1;
    // They are loaded as they are and widened a box later, so that nothing waits for them in between.
    int64_t sr0 = 0, sr1 = 0;   // the rows' first scales (the second row may be no row of this expert: the first again)
    auto scale_rows = [&] {
        const int64_t r = base + sc.tile * rows_tile + g;
        sr0 = r * p.groups;
        sr1 = sc.tile * rows_tile + half1 + g < p.n ? (r + half1) * p.groups : sr0;
    };
    if (mine > 0) scale_rows();
    uint32_t next[2 * kN] = {}, next_in = 0;   // the next box's, and which of them are inside the row
    float s0[2 * kN] = {};
    auto load_scales = [&] {
        next_in = 0;
        if (sc.left <= 0) return;
#pragma unroll
        for (int j = 0; j < kN; ++j) {
            const int at = (sc.chunk * kChunk + (2 * t + j) * 32) >> SHIFT, in = min(at, p.groups - 1);
            next_in |= (at < p.groups ? 1u : 0u) << j;
            next[j] = raw_scale<FMT>(p.scales, sr0 + in);
            next[kN + j] = raw_scale<FMT>(p.scales, sr1 + in);
        }
        const int was = sc.tile;
        sc.next(lo, hi, step);
        if (sc.tile != was && sc.left > 0) scale_rows();
    };
    auto take_scales = [&] {
#pragma unroll
        for (int j = 0; j < 2 * kN; ++j) s0[j] = (next_in >> (j % kN)) & 1u ? wide_scale<FMT>(next[j]) : 0.f;
    };
    load_scales();
    take_scales();
    __syncthreads();   // x is staged
    constexpr int kPieces = 1 << (SHIFT - 5);   // per scale: their products are added up before it is applied
    // the word of piece c in the swizzled box: 16-byte unit c ^ g of row g; bits 4-6 of the rest are 0
    const uint32_t at = (uint32_t)(g * 128 + t * 4 + (g << 4));
    uint32_t xr[NB];   // columns past the last pair repeat it; their results are not written
#pragma unroll
    for (int b = 0; b < NB; ++b) xr[b] = smem_u32(s_x) + min(b * 8 + g, cnt - 1) * p.x_stride + t * 16;
    const uint32_t ring_at = smem_u32(ring) + at;
    for (int m = 0, tile = first; m < mine; ++m, tile += step) {
        float acc[NB][4];
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[b][i] = 0.f;
        for (int chunk = lo; chunk < hi && ok; ++chunk) {
            if (!__all_sync(0xffffffffu, mbar_wait(&bars[slot], (phases >> slot) & 1u, p.timeout_ns))) {
                ok = false;   // the copies still in flight land before the block leaves
                if (lane == 0)
                    for (int i = 1, q = slot; i < flying; ++i) {
                        if (++q == p.slots) q = 0;
                        mbar_wait(&bars[q], (phases >> q) & 1u, p.timeout_ns);
                    }
                break;
            }
            phases ^= 1u << slot;
            --flying;
            load_scales();
            const uint32_t box = ring_at + slot * kBoxBytes, x0 = chunk * (kChunk * 2);
            float d[NB][4];
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                const uint32_t w = box ^ (uint32_t)(c << 4);
                uint32_t lo4[4], hi4[4];
                decode8<FMT>(lds32(w), lo4);
                decode8<FMT>(lds32(w + 1024), hi4);
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    const uint4 xv = lds128(xr[b] + x0 + c * 64);
                    if (c % kPieces == 0) mma16816_first(d[b], lo4[0], hi4[0], lo4[1], hi4[1], xv.x, xv.y);
                    else mma16816(d[b], lo4[0], hi4[0], lo4[1], hi4[1], xv.x, xv.y);
                    mma16816(d[b], lo4[2], hi4[2], lo4[3], hi4[3], xv.z, xv.w);
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
            if (in.left > 0) {
                if (in.chunk == lo) prefetch_scales(in.tile);
                if (lane == 0) issue(slot);
                ++flying;
                in.next(lo, hi, step);
            }
            take_scales();
            if (++slot == p.slots) slot = 0;
        }
        if (p.ks > 1) {   // the shares of k are added in their order
            if (share > 0)
#pragma unroll
                for (int b = 0; b < NB; ++b)
#pragma unroll
                    for (int i = 0; i < 4; ++i) part[warp][b * 4 + i][lane] = acc[b][i];
            group_sync(1 + warp / p.ks, p.ks * 32);
            if (share == 0)
                for (int s = 1; s < p.ks; ++s)
#pragma unroll
                    for (int b = 0; b < NB; ++b)
#pragma unroll
                        for (int i = 0; i < 4; ++i) acc[b][i] += part[warp + s][b * 4 + i][lane];
            group_sync(1 + warp / p.ks, p.ks * 32);
            if (share > 0) continue;
        }
        if (!ok) continue;
        const int i0 = tile * rows_tile;
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int col = b * 8 + 2 * t + j;
                if (col >= cnt) continue;
                const int pr = list[col];
                const float w = p.gate ? p.gate[pr] : 1.0f;
                const int64_t y = (int64_t)pr * cols + i0 + g;
                auto put = [&](int64_t q, float v) {
                    if (p.y_f32) static_cast<float *>(p.y)[q] = v;
                    else static_cast<__nv_bfloat16 *>(p.y)[q] = __float2bfloat16(v);
                };
                float v0 = acc[b][j], v1 = acc[b][2 + j];
                if (swiglu) {
                    put(y, w * (silu(v0) * v1));
                } else {
                    if (p.act == GELU) {
                        v0 = gelu(v0);
                        v1 = gelu(v1);
                    }
                    put(y, w * v0);
                    if (i0 + 8 + g < p.n) put(y + 8, w * v1);
                }
            }
    }
    return ok;
}

template <int FMT, int SHIFT>
__global__ void __launch_bounds__(kWarps * 32, 1)
    matvec_kernel(const __grid_constant__ CUtensorMap map, const MatvecParams p) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *smem = align_smem_1024(smem_raw);
    __shared__ uint64_t s_bar[kWarps][kMaxSlots];
    __shared__ uint32_t s_mask[kMaxExperts / 32];
    __shared__ int s_live, s_cnt, s_bad;
    __shared__ float s_part[kWarps][8][32];
    __shared__ uint16_t s_experts[kMaxExperts];
    uint8_t *s_x = smem + kWarps * p.slots * kBoxBytes;
    uint16_t *s_list = reinterpret_cast<uint16_t *>(s_x + p.cols_pass * p.x_stride);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x < kWarps * kMaxSlots) mbar_init(&s_bar[threadIdx.x / kMaxSlots][threadIdx.x % kMaxSlots], 1);
    fence_mbar_init();
    if (threadIdx.x < kMaxExperts / 32) s_mask[threadIdx.x] = 0;
    if (threadIdx.x == 0) {
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
    if (warp == 0) {   // the experts that have a pair, ascending
        const uint32_t m = s_mask[lane];
        int incl = __popc(m);
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += u;
        }
        int at = incl - __popc(m);
        for (uint32_t r = m; r; r &= r - 1) s_experts[at++] = (uint16_t)(lane * 32 + __ffs(r) - 1);
        if (lane == 31) s_live = incl;
    }
    __syncthreads();
    if (s_bad) {   // rows of pairs without an expert, shared by the blocks
        const int cols = p.act == SWIGLU ? p.n / 2 : p.n;
        for (int i = blockIdx.x; i < pairs; i += gridDim.x) {
            const int e = p.expert[i];
            if (e >= 0 && e < p.N) continue;
            if (e != -1 && threadIdx.x == 0) set_status(kStatusBounds);
            for (int c = threadIdx.x; c < cols; c += kWarps * 32) {
                if (p.y_f32) static_cast<float *>(p.y)[(int64_t)i * cols + c] = 0.f;
                else static_cast<__nv_bfloat16 *>(p.y)[(int64_t)i * cols + c] = __float2bfloat16(0.f);
            }
        }
    }
    // this block's share of all live experts' tiles
    const int64_t all = (int64_t)s_live * p.tiles;
    const int64_t u0 = all * blockIdx.x / gridDim.x, u1 = all * (blockIdx.x + 1) / gridDim.x;
    uint8_t *ring = smem + warp * p.slots * kBoxBytes;
    uint32_t phases = 0;
    int slot = 0;
    bool ok = true;
    for (int64_t u = u0; u < u1;) {
        const int y = (int)(u / p.tiles), e = s_experts[y];
        const int tile0 = (int)(u - (int64_t)y * p.tiles), tile1 = (int)min((int64_t)p.tiles, tile0 + (u1 - u));
        __syncthreads();   // the last expert's list and rows of x have been used
        if (warp == 0) {
            int cnt = 0;
            for (int i0 = 0; i0 < pairs; i0 += 32) {   // the expert's pairs in order
                const bool mine = i0 + lane < pairs && p.expert[i0 + lane] == e;
                const uint32_t b = __ballot_sync(0xffffffffu, mine);
                if (mine) s_list[cnt + __popc(b & ((1u << lane) - 1))] = (uint16_t)(i0 + lane);
                cnt += __popc(b);
            }
            if (lane == 0) s_cnt = cnt;
        }
        __syncthreads();
        // as many pairs at a time as are staged; the weights are read again (from L2) for each lot
        for (int c = 0; c < s_cnt; c += p.cols_pass) {
            const int cnt = min(s_cnt - c, p.cols_pass);
            if (c > 0) __syncthreads();
            // x as 16-byte pieces (8 values of a lane), each as the pairs (0, 4), (1, 5), (2, 6), (3, 7); zeros from k
            // to the end of the last chunk
            const int pieces = (int)(p.x_stride / 16);
            for (int i = threadIdx.x; i < cnt * pieces; i += kWarps * 32) {
                const int col = i / pieces, q = i - col * pieces;
                uint4 v = make_uint4(0, 0, 0, 0);
                if (q * 8 < p.k)
                    v = __ldg(reinterpret_cast<const uint4 *>(p.x + (int64_t)(s_list[c + col] / p.x_div) * p.k) + q);
                *reinterpret_cast<uint4 *>(s_x + col * p.x_stride + q * 16) =
                    make_uint4(__byte_perm(v.x, v.z, 0x5410), __byte_perm(v.x, v.z, 0x7632),
                               __byte_perm(v.y, v.w, 0x5410), __byte_perm(v.y, v.w, 0x7632));
            }
            ok = cnt <= 8 ? run_tiles<FMT, SHIFT, 1>(p, &map, ring, s_bar[warp], phases, slot, s_x, s_part, e, tile0,
                                                     tile1, s_list + c, cnt, ok)
                          : run_tiles<FMT, SHIFT, 2>(p, &map, ring, s_bar[warp], phases, slot, s_x, s_part, e, tile0,
                                                     tile1, s_list + c, cnt, ok);
        }
        u += tile1 - tile0;
    }
}

// Bytes between staged rows of x: whole chunks of k, and an odd number of 64 bytes, so that the 16-byte reads
// of two rows hit different banks.
constexpr uint32_t x_stride(int k) { return (uint32_t)((k + kChunk - 1) / kChunk * kChunk * 2 + 64); }
constexpr size_t matvec_smem(int slots, int cols, int k, int64_t pairs) {
    return 1024 + (size_t)kWarps * slots * kBoxBytes + (size_t)cols * x_stride(k) + (size_t)pairs * 2;
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
