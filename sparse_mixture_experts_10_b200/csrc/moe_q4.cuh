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

#include <type_traits>

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

__device__ __forceinline__ float gelu(float v) { return v * normal_cdf(v); }
__device__ __forceinline__ float silu(float v) { return v / (1.0f + expf(-v)); }

// ---------------------------------------------------------------- the products
// One persistent block per SM takes an even share (by cost: tiles times lots of
// pairs) of the live experts' 16-row tiles of W[e] (SwiGLU: 8 gate rows and the
// 8 up rows beside them, so that a lane ends with both).  16 consumer warps
// multiply a tile each with up to 16 of the expert's pairs as columns of
// m16n8k16 products (bf16 x bf16 -> fp32); where there are few tiles, ks warps
// share a tile along k and their sums are added in order.  A code is at most
// 4 bits, exact in bf16; the products of a group are summed in fp32 by the
// tensor core and enter the result with one fp32 multiply-add by the group's
// scale, so nothing is rounded to fewer bits before the end.
//
// HBM (0.5 byte per weight) is the floor; what is in the way of it is the
// instructions that unpack the codes (about 11 per 8 codes and lane).  So one
// more warp does all the copies: slices of 256 values of k of 16 tiles (32 KB)
// go through a ring of 3 or 4 that runs on from tile to tile and from expert to
// expert.  The 128-byte swizzle lets the fragment reads (4 bytes per lane: 8
// rows x 16 bytes) hit 32 different banks.  Inside a group the order of k is
// free: lane t of a row takes the 8 codes of one 32-bit word, as pairs (i, i + 4)
// that one mask each extracts; the expert's rows of x are staged in shared
// memory in that order.
//
// Measured (32 experts, 5760 x 2880, int4): 64 tokens, top 4, groups of 32: 114 us,
// 2.6 TB/s of a floor of 46 us at the copy rate; the data in L2 already is no
// faster, it is the 60 instructions for each 16 rows of a group, issued at
// 2.4 a cycle.  One token: 18 us for 5.5 us of bytes, half of it start-up (the
// experts' list, x and the first slice are one latency after another).
constexpr int kWarps = 16, kThreadsMv = (kWarps + 1) * 32;
constexpr int kMaxSlots = 4, kSlotBytes = kWarps * 2048, kChunk = 256;
constexpr int kMaxPairs = 4096, kMaxExperts = 1024, kMaxCols = 16;

struct MatvecParams : Params {
    int act, y_f32;
    int tiles, ks;         // 16-row tiles of an expert; warps that share a tile (split k)
    int box_tiles;         // tiles of one copy (a tensor-map box of 128 bytes x 16 rows each)
    int slots;             // slices in the ring (3 or 4)
    int cols_pass;         // pairs staged at a time (at most kMaxCols)
    uint32_t x_stride;     // bytes between staged rows of x
    uint64_t timeout_ns;
};

// (a & b) | c in one instruction.  Written in C++ it became two: 41 integer instructions for 16 rows of a group
// against 28 now, and they are what the kernel spends its time on.
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
        for (int i = 0; i < 4; ++i) {   // 0x4300 | c is the bf16 128 + c; minus 136 exactly c - 8
            v[i] = and_or(w >> (4 * i), 0x000f000fu, 0x43004300u);
            asm("sub.rn.bf16x2 %0, %0, %1;" : "+r"(v[i]) : "r"(0x43084308u));
        }
    } else {
        // one multiplication puts the sign at bit 15 (2^12) and the other three bits at bf16's lowest exponent bits and
        // highest mantissa bit (2^6); what they read as is value 2^-126, subnormals included: times 2^126 exactly
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[i] = ((w >> (4 * i)) & 0x000f000fu) * 0x1040u & 0x81c081c0u;
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

__device__ __forceinline__ void group_sync(int id, int threads) {
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

__device__ __forceinline__ void tma_load_codes(const CUtensorMap *map, uint64_t *bar, void *dst, int c0, int c1, int e) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, %6}], "
        "[%2];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(0), "r"(e)
        : "memory");
}

// Where a consumer warp is in the ring.
struct Ring {
    uint32_t base;      // shared-memory address of the slots
    uint64_t *full, *empty;
    int slot = 0;
    uint32_t phase = 0;
    bool ok = true;     // false: a wait ran out (status word); nothing more is computed
};

// Tiles tile0..tile1-1 of expert e against the staged columns (NB blocks of 8; list[0..cnt) their pairs).
template <int FMT, int SHIFT, int NB>
__device__ __forceinline__ void run_tiles(const MatvecParams &p, Ring &ring, uint32_t s_x, float (*part)[8][32], int e,
                                          int tile0, int tile1, const uint16_t *list, int cnt) {
    using Raw = typename std::conditional<FMT == INT4, unsigned short, unsigned char>::type;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const bool swiglu = p.act == SWIGLU;
    const int cols = swiglu ? p.n / 2 : p.n;
    const int share = warp % p.ks, step = kWarps / p.ks, mine = warp / p.ks;
    const int chunks = (p.k + kChunk - 1) / kChunk, rounds = (chunks + p.ks - 1) / p.ks;
    const int rows_tile = swiglu ? 8 : 16, half1 = swiglu ? cols : 8;   // distance of a tile's second 8 rows
    const Raw *scales = static_cast<const Raw *>(p.scales) + (int64_t)e * p.n * p.groups;
    // the slot holds copies of box_tiles tiles; SwiGLU: their gate rows, then their up rows
    const int in_box = mine % p.box_tiles;
    const uint32_t box = (uint32_t)((share * (step / p.box_tiles) + mine / p.box_tiles) * p.box_tiles) * 2048u;
    // the word of piece c in the swizzled copy: 16-byte unit c ^ g of row g; bits 4-6 of the rest are 0
    const uint32_t at = ring.base + box + (uint32_t)(swiglu ? in_box * 1024 : in_box * 2048) +
                        (uint32_t)(g * 128 + t * 4 + (g << 4));
    const uint32_t second = swiglu ? (uint32_t)p.box_tiles * 1024u : 1024u;
    uint32_t xr[NB];   // columns past the last pair repeat it; their results are not written
#pragma unroll
    for (int b = 0; b < NB; ++b) xr[b] = s_x + min(b * 8 + g, cnt - 1) * p.x_stride + t * 16;

    // What a lane holds of a slice: the scales of the rows g and g + 8 for the 32-value pieces 2t and 2t + 1 (one scale
    // for both with groups of 64 and more).  They come straight from global memory, a slice ahead, and are widened
    // a slice later, so that nothing waits for them in between; their lines are brought into L2 a tile ahead.
    // Past the last group nothing is read (a finite value stands there): x is zero, and so are the sums.
    constexpr int kN = SHIFT == 5 ? 2 : 1, kPerChunk = kChunk >> SHIFT;
    const Raw *sp0 = scales, *sp1 = scales;
    uint32_t next[2 * kN] = {};
    float s0[2 * kN];
    auto scale_rows = [&](int tile) {
        const int r = tile * rows_tile + g;
        sp0 = scales + (int64_t)r * p.groups;
        sp1 = r + half1 < p.n ? sp0 + (int64_t)half1 * p.groups : sp0;
    };
    auto load_scales = [&](int chunk) {
#pragma unroll
        for (int j = 0; j < kN; ++j) {
            const int q = chunk * kPerChunk + (((2 * t + j) * 32) >> SHIFT);
            next[j] = next[kN + j] = 0;
            if (q < p.groups) {
                next[j] = __ldg(sp0 + q);
                next[kN + j] = __ldg(sp1 + q);
            }
        }
    };
    auto prefetch_scales = [&](int tile) {
        const int r = tile * rows_tile + (lane & 7) + (lane & 8 ? half1 : 0);
        if (tile >= tile1 || r >= p.n) return;
        const char *s = reinterpret_cast<const char *>(scales + (int64_t)r * p.groups);
        for (int b = (lane >> 4) * 32; b < p.groups * (int)sizeof(Raw) + 31; b += 64)
            asm volatile("prefetch.global.L2 [%0];" ::"l"(s + min(b, p.groups * (int)sizeof(Raw) - 1)));
    };
    if (tile0 + mine < tile1) {
        scale_rows(tile0 + mine);
        load_scales(share);
    }
    constexpr int kPieces = 1 << (SHIFT - 5);   // per scale: their products are added up before it is applied
    for (int tile = tile0 + mine; tile - mine < tile1; tile += step) {
        const bool have = tile < tile1;
        float acc[NB][4];
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[b][i] = 0.f;
        if (have) prefetch_scales(tile + step);
        for (int j = 0; j < rounds; ++j) {
            const int chunk = j * p.ks + share;
            if (ring.ok)
                ring.ok = __all_sync(0xffffffffu, mbar_wait(&ring.full[ring.slot], ring.phase, p.timeout_ns));
            if (have && chunk < chunks && ring.ok) {
#pragma unroll
                for (int i = 0; i < 2 * kN; ++i) s0[i] = wide_scale<FMT>(next[i]);
                if (chunk + p.ks < chunks) {
                    load_scales(chunk + p.ks);
                } else if (tile + step < tile1) {
                    scale_rows(tile + step);
                    load_scales(share);
                }
                const uint32_t w0 = at + (uint32_t)ring.slot * kSlotBytes, x0 = (uint32_t)chunk * (kChunk * 2);
                float d[NB][4];
                // the whole slice's codes and the next piece's x are read ahead of their use
                uint32_t wl[8], wh[8];
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    wl[c] = lds32(w0 ^ (uint32_t)(c << 4));
                    wh[c] = lds32((w0 ^ (uint32_t)(c << 4)) + second);
                }
                uint4 xn[NB];
#pragma unroll
                for (int b = 0; b < NB; ++b) xn[b] = lds128(xr[b] + x0);
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    uint32_t lo4[4], hi4[4];
                    decode8<FMT>(wl[c], lo4);
                    decode8<FMT>(wh[c], hi4);
#pragma unroll
                    for (int b = 0; b < NB; ++b) {
                        const uint4 xv = xn[b];
                        if (c < 7) xn[b] = lds128(xr[b] + x0 + (c + 1) * 64);
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
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&ring.empty[ring.slot]);
            if (++ring.slot == p.slots) {
                ring.slot = 0;
                ring.phase ^= 1;
            }
        }
        if (p.ks > 1) {   // the shares of k are added in their order
            if (share > 0)
#pragma unroll
                for (int b = 0; b < NB; ++b)
#pragma unroll
                    for (int i = 0; i < 4; ++i) part[warp][b * 4 + i][lane] = acc[b][i];
            group_sync(1 + mine, p.ks * 32);
            if (share == 0)
                for (int s = 1; s < p.ks; ++s)
#pragma unroll
                    for (int b = 0; b < NB; ++b)
#pragma unroll
                        for (int i = 0; i < 4; ++i) acc[b][i] += part[warp + s][b * 4 + i][lane];
            group_sync(1 + mine, p.ks * 32);
            if (share > 0) continue;
        }
        if (!have || !ring.ok) continue;
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
}

template <int FMT, int SHIFT>
__global__ void __launch_bounds__(kThreadsMv, 1)
    matvec_kernel(const __grid_constant__ CUtensorMap map, const MatvecParams p) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *smem = align_smem_1024(smem_raw);
    __shared__ uint64_t s_full[kMaxSlots], s_empty[kMaxSlots];
    __shared__ int s_count[kMaxExperts];             // pairs of each expert
    __shared__ uint16_t s_experts[kMaxExperts];      // the experts that have a pair, ascending
    __shared__ int s_cost0[kMaxExperts + 1];         // cost before each of them: all lots (at most 5120) times tiles
                                                     // (at most 65536) times 4 stay below 2^31
    __shared__ int s_live, s_bad;
    __shared__ float s_part[kWarps][8][32];
    uint8_t *s_x = smem + p.slots * kSlotBytes;
    uint16_t *s_list = reinterpret_cast<uint16_t *>(s_x + p.cols_pass * p.x_stride);
    int16_t *s_expert = reinterpret_cast<int16_t *>(s_list + p.pairs);   // each pair's expert, -1: none
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int i = threadIdx.x; i < kMaxExperts; i += kThreadsMv) s_count[i] = 0;
    if (threadIdx.x == 0) {
        for (int i = 0; i < kMaxSlots; ++i) {
            mbar_init(&s_full[i], 1);
            mbar_init(&s_empty[i], kWarps);
        }
        fence_mbar_init();
        s_bad = 0;
        tma_prefetch_desc(&map);
    }
    __syncthreads();
    pdl_enter();
    const int pairs = (int)p.pairs;
    for (int i = threadIdx.x; i < pairs; i += kThreadsMv) {
        const int e = p.expert[i];
        const bool good = e >= 0 && e < p.N;
        if (good) atomicAdd(&s_count[e], 1);
        else s_bad = 1;
        s_expert[i] = good ? (int16_t)e : (int16_t)-1;
    }
    __syncthreads();
    // An expert's pairs are staged in lots of cols_pass; its work is its tiles with the first lot, with the second and
    // so on.  A tile costs 3, with more than 8 pairs 4 (8 experts with 8 pairs each 49 us, with 16 each 70 us; a
    // batch of 64 tokens over 32 experts took 132 us with all tiles alike, 124 us so).  cost_of(e, u): that of the first u
    // of an expert's lots * tiles.
    auto cost_of = [&](int e, int u) {
        const int full = s_count[e] / p.cols_pass, rest = s_count[e] - full * p.cols_pass, f = min(u, full * p.tiles);
        return f * (p.cols_pass > 8 ? 4 : 3) + (u - f) * (rest > 8 ? 4 : 3);
    };
    auto lots = [&](int e) { return (s_count[e] + p.cols_pass - 1) / p.cols_pass; };
    if (warp == 0) {
        int live = 0;
        int cost = 0;
        for (int e0 = 0; e0 < p.N; e0 += 32) {
            const int e = e0 + lane;
            const bool has = e < p.N && s_count[e] > 0;
            const uint32_t m = __ballot_sync(0xffffffffu, has);
            if (m == 0) continue;
            int c = has ? cost_of(e, lots(e) * p.tiles) : 0, incl = c;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int u = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += u;
            }
            if (has) {
                const int at = live + __popc(m & ((1u << lane) - 1));
                s_experts[at] = (uint16_t)e;
                s_cost0[at] = cost + incl - c;
            }
            live += __popc(m);
            cost += __shfl_sync(0xffffffffu, incl, 31);
        }
        if (lane == 0) {
            s_live = live;
            s_cost0[live] = cost;
        }
    }
    __syncthreads();
    const int live = s_live;
    // this block's share: the work that starts in [x0, x1) of the cost
    const int even = s_cost0[live] / (int)gridDim.x, rest_all = s_cost0[live] - even * (int)gridDim.x;
    auto share_at = [&](int b) { return even * b + rest_all * b / (int)gridDim.x; };
    const int x0 = share_at(blockIdx.x), x1 = share_at(blockIdx.x + 1);
    int first = 0;
    for (int hi = live - 1; first < hi;) {   // the last expert that starts at or before x0
        const int mid = (first + hi + 1) >> 1;
        if (s_cost0[mid] <= x0) first = mid;
        else hi = mid - 1;
    }
    auto work_at = [&](int y, int x) {   // how much of the y-th live expert's work starts before x
        const int e = s_experts[y];
        const int full = s_count[e] / p.cols_pass, rest = s_count[e] - full * p.cols_pass, f = full * p.tiles;
        const int d = min(x, s_cost0[y + 1]) - s_cost0[y], wf = p.cols_pass > 8 ? 4 : 3, wr = rest > 8 ? 4 : 3;
        return d <= 0 ? 0 : d <= f * wf ? (d + wf - 1) / wf : f + (d - f * wf + wr - 1) / wr;
    };
    const int step = kWarps / p.ks, chunks = (p.k + kChunk - 1) / kChunk, rounds = (chunks + p.ks - 1) / p.ks;
    if (warp == kWarps) {
        // ------------------------------------------------------------ copies
        if (lane == 0) {
            const int rows_tile = p.act == SWIGLU ? 8 : 16, boxes = step / p.box_tiles;
            int slot = 0;
            uint32_t phase = 0;
            bool ok = true;
            IssuedSlots iss;
            for (int y = first; y < live && s_cost0[y] < x1 && ok; ++y) {
                const int e = s_experts[y];
                const int w1 = work_at(y, x1);
                for (int w = work_at(y, x0); w < w1 && ok;) {   // one lot at a time
                    const int tile0 = w % p.tiles, tile1 = min(p.tiles, tile0 + w1 - w);
                    w += tile1 - tile0;
                    for (int tile = tile0; tile < tile1 && ok; tile += step)
                        for (int j = 0; j < rounds; ++j) {
                            if (!mbar_wait(&s_empty[slot], phase ^ 1, p.timeout_ns)) {
                                ok = false;
                                break;
                            }
                            const int nb = min(boxes, (tile1 - tile + p.box_tiles - 1) / p.box_tiles);
                            const int nk = min(p.ks, chunks - j * p.ks);
                            mbar_arrive_expect_tx(&s_full[slot], (uint32_t)(nb * nk * p.box_tiles) * 2048u);
                            for (int h = 0; h < nk; ++h)
                                for (int b = 0; b < nb; ++b)
                                    tma_load_codes(&map, &s_full[slot],
                                                   smem + slot * kSlotBytes + (h * boxes + b) * p.box_tiles * 2048,
                                                   (j * p.ks + h) * (kChunk / 2), (tile + b * p.box_tiles) * rows_tile, e);
                            iss.note(slot, phase);
                            if (++slot == p.slots) {
                                slot = 0;
                                phase ^= 1;
                            }
                        }
                }
            }
            iss.drain(s_full, p.timeout_ns);   // every copy has landed before the block leaves
        }
        return;
    }
    // ---------------------------------------------------------------- products
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
    constexpr int kAll = 15;   // named barrier of the consumer warps; the groups of a tile use 1..8
    Ring ring;
    ring.base = smem_u32(smem);
    ring.full = s_full;
    ring.empty = s_empty;
    for (int y = first; y < live && s_cost0[y] < x1; ++y) {
        const int e = s_experts[y];
        const int w1 = work_at(y, x1);
        int w = work_at(y, x0);
        if (w >= w1) continue;
        if (y > first) group_sync(kAll, kWarps * 32);   // the last expert's list has been used
        if (warp == 0) {
            int cnt = 0;
            for (int i0 = 0; i0 < pairs; i0 += 32) {   // the expert's pairs in order
                const bool has = i0 + lane < pairs && s_expert[i0 + lane] == e;
                const uint32_t m = __ballot_sync(0xffffffffu, has);
                if (has) s_list[cnt + __popc(m & ((1u << lane) - 1))] = (uint16_t)(i0 + lane);
                cnt += __popc(m);
            }
        }
        while (w < w1) {   // one lot at a time; another lot reads the weights again (from L2)
            const int lot = w / p.tiles, c = lot * p.cols_pass, cnt = min(s_count[e] - c, p.cols_pass);
            const int tile0 = w - lot * p.tiles, tile1 = min(p.tiles, tile0 + w1 - w);
            w += tile1 - tile0;
            group_sync(kAll, kWarps * 32);   // the list is there; the rows of x before have been used
            // x as 16-byte pieces (8 values of a lane), each as the pairs (0, 4), (1, 5), (2, 6), (3, 7); zeros from k
            // to the end of the last slice
            const int pieces = (int)(p.x_stride / 16), total = cnt * pieces;
            constexpr int kAhead = 4;   // loads in flight per thread
            for (int i0 = threadIdx.x; i0 < total; i0 += kAhead * kWarps * 32) {
                uint4 v[kAhead];
                uint32_t dst[kAhead];
#pragma unroll
                for (int a = 0; a < kAhead; ++a) {
                    const int i = i0 + a * kWarps * 32, col = min(i, total - 1) / pieces, q = min(i, total - 1) - col * pieces;
                    dst[a] = col * p.x_stride + q * 16;
                    v[a] = make_uint4(0, 0, 0, 0);
                    if (i < total && q * 8 < p.k)
                        v[a] = __ldg(reinterpret_cast<const uint4 *>(p.x + (int64_t)(s_list[c + col] / p.x_div) * p.k) + q);
                }
#pragma unroll
                for (int a = 0; a < kAhead; ++a)
                    if (i0 + a * kWarps * 32 < total)
                        *reinterpret_cast<uint4 *>(s_x + dst[a]) =
                            make_uint4(__byte_perm(v[a].x, v[a].z, 0x5410), __byte_perm(v[a].x, v[a].z, 0x7632),
                                       __byte_perm(v[a].y, v[a].w, 0x5410), __byte_perm(v[a].y, v[a].w, 0x7632));
            }
            group_sync(kAll, kWarps * 32);
            if (cnt <= 8) run_tiles<FMT, SHIFT, 1>(p, ring, smem_u32(s_x), s_part, e, tile0, tile1, s_list + c, cnt);
            else run_tiles<FMT, SHIFT, 2>(p, ring, smem_u32(s_x), s_part, e, tile0, tile1, s_list + c, cnt);
        }
    }
}

// Bytes between staged rows of x: whole chunks of k, and an odd number of 64 bytes, so that the 16-byte reads
// of two rows hit different banks.
constexpr uint32_t x_stride(int k) { return (uint32_t)((k + kChunk - 1) / kChunk * kChunk * 2 + 64); }
constexpr size_t kRoom = 227 * 1024 - 32 * 1024;   // dynamic shared memory: 32 KB are left to the static one
constexpr size_t matvec_smem(int slots, int cols, int k, int64_t pairs) {
    return 1024 + (size_t)slots * kSlotBytes + (size_t)cols * x_stride(k) + (size_t)pairs * 4;
}

// Codes and scales of fp32 or bf16 weights: one warp per group of values.
//   int4  s = bf16(max|w| / 7), code = 8 + round(w / s) clamped to 0..15
//   e2m1  s = 2^e, e the smallest integer with max|w| <= 6 2^e; round(w / s) to
//         the nearest of 0, .5, 1, 1.5, 2, 3, 4, 6, ties to the even code
// A group with an infinity or a NaN gets a NaN scale.  Once per checkpoint, and as simple as that: 32 experts of
// 2880 x 2880 from bf16, int4 in groups of 32 1.58 ms, of 128 0.80 ms, e2m1 2.26 ms (0.3 to 0.8 TB/s: a warp's
// instructions for each group, half of its lanes idle while codes of 32 values are written).
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

// The values of codes and scales, rounded once to T.  The same weights to bf16: int4 145 us, 4.7 TB/s (four fifths of it
// writes), e2m1 198 us, 3.4 TB/s; to fp32 282 and 213 us, 4.3 and 5.7 TB/s.
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
