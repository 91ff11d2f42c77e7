// moe_grouped_mm_tc.cuh -- grouped products of bf16 operands on the tcgen05 tensor cores.
//
// Every kind is computed as  OUT[row, f] = sum_c M[f, c] N[row, c]  with the
// contiguous index f of the result on the accumulator's lanes (the M side of
// the instruction, fixed at 128 per CTA) and its rows on the accumulator's
// columns (the N side, any multiple of 16):
//          f      row            c         M operand          N operand
//   NT     n      token row      k         b[g] K-major       a K-major
//   NN     k      token row      n         b[g] MN-major      a K-major
//   TN     k      n              token row b MN-major         a MN-major
// The ragged length of a segment then sits on the side whose tile can have any
// size: a segment of L rows is cut into ceil(L / 256) nearly equal tiles of a
// multiple of 16 rows, and no tensor time goes into padding (with the rows on
// the 256-row side a segment of 520 rows would pay for 768).
//
// One persistent CTA per SM (kPair false: tiles of 128 x <=128), or a CTA pair
// per two (tiles of 256 x <=256, kWide <=512; each CTA of the pair loads its
// 128 f's and half of the rows):
//   epilogue   16 warps: tcgen05.ld; a lane holds one f,
//              so a warp writes 32 consecutive values of a row (bf16: two
//              rows of pairs after a lane exchange)
//   producer   one warp: TMA copies of 64-wide slices along c into a ring
//   issuer     one warp: tcgen05.mma into one of two accumulators
//   clearer    one warp, TN: clears the rows behind a segment's end in its last
//              slice, up to the next 16 (further steps of the slice are not
//              issued).  Those rows belong to another expert (or to nobody) and
//              may hold anything, NaN included, so both operands are cleared
// Slices past the end of n or k are zero-filled by TMA: the weights' tensor map
// has the group as its own dimension.
//
// What bounds it: large tiles, what L2 delivers to the SMs (about 61 to 74 GB/s
// to each, whatever the tile's shape; a slice of a 256 x 512 tile is 48 KB a CTA
// for 17 MFLOP, of a 256 x 256 one 32 KB for 8) beside the power cap; few rows, HBM.
// 32 experts of 512 rows each, n 4096, k 7168: 675 us, 1425 TFLOP/s with 256 x 512
// tiles, 714 us with 256 x 256, 963 us with single CTAs; of 512 +- 20 rows each 753 us
// in bf16, 815 us in fp32.  Weight gradients over
// 512 rows (18 of 4096 x 2048, fp32): 171 us, 3.5 TB/s written.
//
// Every wait is bounded; on expiry the waiting role stops issuing work, the
// status word records MOE_STATUS_TIMEOUT and the CTA drains and returns.
#pragma once

#include "moe_gemm_tc.cuh"
#include "moe_grouped_mm.cuh"

#include <type_traits>

namespace moe {
namespace gmm {

constexpr int kSl = 64;                 // slice along the contraction
constexpr int kOpBytes = 128 * kSl * 2; // 128 values of either side of a slice
// 16 epilogue warps: a weight gradient over few rows is mostly its epilogue (18 gradients of 4096 x 2048 over 512
// rows each: 208 us with 8 warps, 167 us with 16).
constexpr int kEpi = 16;
constexpr int kTcThreads = 32 * (kEpi + 3);
// The tensor core's fp32 accumulation drops bits, always towards zero: of each step's 16 products what is below 2^-25
// of the largest exponent in the sum, and of their sum what is below 2^-23 (seen with sums built of powers of two), so
// less than 16 * 2^-25 + 2^-23 = 5 * 2^-23 of the partial sum a step.  Measured against 64 bits, a result of terms of
// both signs comes out small by 8e-10 of itself for every term (4.4e-6 after 4096, 1.9e-5 after 16384), one of 2^23
// positive terms by 5%.  So a long contraction is cut into equal runs (kSums); the accumulator is read after each and
// added, rounded to nearest, to running sums in registers:
//   fp32 results  runs of at most 12 slices (768 terms: 6e-7, positive terms 1.3e-6)
//   bf16 results  runs of at most 256 slices (16384 terms: below 1024 * 5 * 2^-23 = 6.2e-4, beside up to 2^-8 of their
//                 own rounding); up to there they are read once and need no running sums
constexpr int kRunF32 = 12, kRunBf16 = 256;
template <bool kF32>
__device__ __forceinline__ int run_length(int nkb) {
    constexpr int kRun = kF32 ? kRunF32 : kRunBf16;
    if (nkb <= kRun) return nkb;
    const int runs = (nkb + kRun - 1) / kRun;
    return (nkb + runs - 1) / runs;
}

// Slices in the ring: 192 KB of shared memory, in TN with a buffer of their own for the last slices of segments.
// Those are copied when a tile begins and used when it ends, so that clearing them stays off the critical path
// (in the ring, 18 gradients of 4096 x 2048 took 213 us over 520 rows and 187 us over 528, which need no clearing).
__host__ __device__ constexpr int ring_stages(int kind, bool wide) { return wide ? 4 : kind == TN ? 5 : 6; }
__host__ __device__ constexpr size_t tc_smem_bytes(int groups) {
    return 1024 + (size_t)12 * kOpBytes + (2 * 6 + 8) * 8 + 16 + 12 * (size_t)(groups + 1);
}

// The N operand's tensor maps: K-major boxes of 16, 32, 64, 96 and 128 rows, so that a slice is one copy
// of nearly the tile's rows (192-row tiles in copies of 32 rows ran at 930 TFLOP/s, in one of 96 at 1166); TN uses
// the first.
struct NMaps {
    CUtensorMap m[5];
};
constexpr int box_rows(int i) { return i == 0 ? 16 : 32 * i; }

// cp.async.bulk.tensor of a 3-D box; kPair: completion on the leader CTA's barrier.
template <bool kPair>
__device__ __forceinline__ void tma_load_3d(const CUtensorMap *map, uint32_t bar, void *dst, int c0, int c1, int c2) {
    if (kPair)
        asm volatile(
            "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, "
            "%4, %5}], [%2];" ::"r"(smem_u32(dst)),
            "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2)
            : "memory");
    else
        asm volatile(
            "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, "
            "%5}], [%2];" ::"r"(smem_u32(dst)),
            "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2)
            : "memory");
}

// The same for a 4-D box (64-value chunks of an MN-major operand).
template <bool kPair>
__device__ __forceinline__ void tma_load_4d(const CUtensorMap *map, uint32_t bar, void *dst, int c0, int c1, int c2,
                                            int c3) {
    if (kPair)
        asm volatile(
            "cp.async.bulk.tensor.4d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, "
            "%4, %5, %6}], [%2];" ::"r"(smem_u32(dst)),
            "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
            : "memory");
    else
        asm volatile(
            "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, "
            "%5, %6}], [%2];" ::"r"(smem_u32(dst)),
            "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
            : "memory");
}
// 128 values x 64 c's of an MN-major operand: one copy of two 64-value chunks where the width is a
// multiple of 64 (the map then has the chunk as a dimension), else a copy for each.
template <bool kPair>
__device__ __forceinline__ void load_mn(const CUtensorMap *map, bool chunks, uint32_t bar, uint8_t *dst, int v, int c,
                                        int g) {
    if (chunks) {
        tma_load_4d<kPair>(map, bar, dst, 0, c, v >> 6, g);
    } else {
        tma_load_4d<kPair>(map, bar, dst, v, c, 0, g);
        tma_load_4d<kPair>(map, bar, dst + kOpBytes / 2, v + 64, c, 0, g);
    }
}

// Descriptor of an MN-major bf16 operand with 128-byte swizzle, written by TMA
// as boxes of 64 (c) rows x 64 values: along MN, chunks of 64 values are one
// box (8192 bytes) apart; along c, groups of 8 rows are 1024 bytes apart.
// Advancing by 16 c's adds 2048 bytes.
__device__ __forceinline__ uint64_t smem_desc_mn(uint32_t saddr) {
    uint64_t d = 0;
    d |= static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
    d |= static_cast<uint64_t>(8192u >> 4) << 16;
    d |= static_cast<uint64_t>(1024u >> 4) << 32;
    d |= static_cast<uint64_t>(1) << 46;
    d |= static_cast<uint64_t>(2) << 61;
    return d;
}

// Hands an accumulator back to the leader's MMA thread.  Nothing but the (completed) TMEM loads before the
// fence::before_thread_sync is ordered by it, so it is relaxed: a release at cluster scope would first wait for
// this warp's stores of the result.
__device__ __forceinline__ void mbar_arrive_remote_relaxed(uint32_t bar_cluster) {
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar_cluster) : "memory");
}

// One lane of the (converged) warp.  The issuing warps run their loops with all lanes and only the copies and
// tensor instructions under this predicate: their descriptors then stay in uniform registers.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\tselp.u32 %0, 1, 0, q;\n\t}" : "=r"(p));
    return p != 0;
}

// Rows of each of the tiles of a segment of len rows; unsigned, as the sum may pass 2^31.
__device__ __forceinline__ int tile_rows(int len, int tiles) { return (int)((unsigned)(len + (unsigned)tiles - 1) / tiles); }

struct Tile {
    int g, f0, r0, rows;        // first f and row of the result; valid rows
    int nh, nsub;               // N of one instruction, instructions side by side (kWide: up to two)
    int c0, nc;                 // contraction start and length
};

// The clearer's wait for a tile's last slice.  Tiles without one may lie before it, any number of them, so the limit
// is on the time in which the producer (`moving`: the tile that it is at) takes no step to another tile.
__device__ __forceinline__ bool wait_while_moving(uint64_t *bar, uint32_t parity, uint64_t timeout_ns,
                                                  const volatile int *moving) {
    if (mbar_try_wait(bar, parity)) return true;
    int seen = *moving;
    uint64_t t0 = globaltimer_ns();
    while (true) {
#pragma unroll 1
        for (int i = 0; i < 64; ++i)
            if (mbar_try_wait(bar, parity)) return true;
        if (globaltimer_ns() - t0 > timeout_ns) {
            const int now = *moving;
            if (now == seen) {
                set_status(kStatusTimeout);
                return false;
            }
            seen = now;
            t0 = globaltimer_ns();
        }
    }
}

// The order in which groups are worked on: those whose tiles take longest first, so that the blocks' last tiles are
// short ones (32 experts of 512 +- 22 rows, n 4096, k 7168: 945 us in the groups' own order, 896 us so).  ord[j] is the j-th
// group, cum its first tile.  By every thread of the block; s_off is complete.  Beyond kOrdered groups the tiles
// are many and small, and the groups keep their order.
constexpr int kOrdered = 128;
template <int KIND>
__device__ __forceinline__ void order_groups(const int *s_off, int G, int unit, int *cum, int *ord) {
    auto rows = [&](int g) { return s_off[g + 1] - s_off[g]; };
    auto tiles = [&](int g) { return (rows(g) + unit - 1) / unit; };
    auto weight = [&](int g) { return KIND == TN ? rows(g) : rows(g) == 0 ? 0 : tile_rows(rows(g), tiles(g)); };
    for (int g = threadIdx.x; g < G; g += kTcThreads) {
        int at = g;
        if (G <= kOrdered) {
            const int w = weight(g);
            at = 0;
            for (int h = 0; h < G; ++h) {
                const int v = weight(h);
                at += v > w || (v == w && h < g) ? 1 : 0;
            }
        }
        ord[at] = g;
    }
    __syncthreads();
    if (KIND != TN && threadIdx.x < 32) {
        int carry = 0;
        for (int j0 = 0; j0 <= G; j0 += 32) {
            const int j = j0 + threadIdx.x, t = j < G ? tiles(ord[j]) : 0;
            int incl = t;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int u = __shfl_up_sync(0xffffffffu, incl, o);
                if ((int)threadIdx.x >= o) incl += u;
            }
            if (j <= G) cum[j] = carry + incl - t;
            carry += __shfl_sync(0xffffffffu, incl, 31);
        }
    }
    __syncthreads();
}

template <int KIND, bool kPair, bool kWide>
__device__ __forceinline__ Tile tile_at(const Params &p, const int *s_off, const int *s_cum, const int *s_ord, int i) {
    constexpr int kM = kPair ? 256 : 128, kN = kPair ? 256 : 128;
    Tile t;
    t.nsub = 1;
    if (KIND == TN) {
        const int per = p.m_tiles * p.n_tiles;
        const int j = i / per, r = i - j * per;
        t.g = kPair ? s_ord[j] : j;
        t.f0 = r / p.n_tiles * kM;
        t.r0 = (r % p.n_tiles) * kN;
        t.rows = min(kN, p.n - t.r0);
        // an MN-major N operand is made of whole chunks of 64 per CTA
        t.nh = t.rows > kN / 2 ? kN : kN / 2;
        t.c0 = s_off[t.g];
        t.nc = s_off[t.g + 1] - t.c0;
    } else {
        // tile order: expert, then f tile, then row tile, so that the tiles in flight share weights
        int lo = 0, hi = p.G - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if ((int64_t)s_cum[mid] * p.m_tiles <= i) lo = mid;
            else hi = mid - 1;
        }
        t.g = kPair ? s_ord[lo] : lo;
        const int tiles = s_cum[lo + 1] - s_cum[lo];
        const int r = i - s_cum[lo] * p.m_tiles;
        t.f0 = r / tiles * kM;
        const int len = s_off[t.g + 1] - s_off[t.g], size = tile_rows(len, tiles);
        if (kWide && size > kN) t.nsub = 2;
        t.nh = ((size + t.nsub - 1) / t.nsub + 15) & ~15;
        const int at = r % tiles * t.nh * t.nsub;
        t.r0 = s_off[t.g] + at;
        // never empty: a tile has at most the unit of rows that the segment's number of tiles was taken with
        t.rows = min(t.nh * t.nsub, len - at);
        t.c0 = 0;
        t.nc = KIND == NT ? p.k : p.n;
    }
    return t;
}

// N accumulator columns (rows of the result) of this lane's f; rows: how many of them there are.
template <int N>
__device__ __forceinline__ void store_f32(float *dst, int64_t ldc, bool f_ok, const float (&v)[N], int rows,
                                          int accumulate) {
#pragma unroll
    for (int j = 0; j < N; ++j)
        if (j < rows && f_ok) dst[j * ldc] = accumulate ? dst[j * ldc] + v[j] : v[j];
}
template <int N>
__device__ __forceinline__ void store_bf16(__nv_bfloat16 *out, int64_t ldc, int f, bool f_ok, const float (&v)[N],
                                           int rows, int accumulate) {
    const int odd = threadIdx.x & 1;
    __nv_bfloat16 *dst = out + (f & ~1) + (odd ? ldc : 0);
#pragma unroll
    for (int j = 0; j < N; j += 2) {   // even lanes write row j, odd lanes row j + 1
        const float got = __shfl_xor_sync(0xffffffffu, odd ? v[j] : v[j + 1], 1);
        float lo = odd ? got : v[j], hi = odd ? v[j + 1] : got;
        if (j + odd < rows && f_ok) {
            uint32_t *q = reinterpret_cast<uint32_t *>(dst + j * ldc);
            if (accumulate) {
                const uint32_t o = *q;
                lo += __uint_as_float(o << 16);
                hi += __uint_as_float(o & 0xffff0000u);
            }
            *q = pack_bf16x2(lo, hi);
        }
    }
}

template <int KIND, typename TO, bool kPair, bool kWide, bool kSums>
__device__ __forceinline__ void tc_body(const CUtensorMap &tmM, const NMaps &tmN, const Params &p) {
    pdl_enter();
    constexpr bool kF32 = sizeof(TO) == 4;
    static_assert(kSums || !kF32, "fp32 results have running sums");
    static_assert(!kWide || (kPair && KIND != TN && !kSums), "wide tiles: CTA pairs, K-major N operand, one run");
    constexpr int kAccCols = kPair ? 256 : 128;
    constexpr int kStages = ring_stages(KIND, kWide), kNBytes = (kWide ? 2 : 1) * kOpBytes;
    constexpr bool kMmn = KIND != NT, kNmn = KIND == TN;   // MN-major operands
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *smem = align_smem_1024(smem_raw);
    uint8_t *sM = smem, *sN = smem + kStages * kOpBytes;
    uint8_t *sTail = sN + kStages * kNBytes;   // TN: a segment's last slice, the M operand and then the N operand
    uint64_t *full = reinterpret_cast<uint64_t *>(sTail + (KIND == TN ? 2 * kOpBytes : 0));
    uint64_t *empty = full + kStages;
    uint64_t *raw = empty + kStages;   // TN: the last slice has landed and is to be cleared
    uint64_t *fixed = raw + 1;         // ... has been, in every CTA of the pair
    uint64_t *used = fixed + 1;        // ... and has been used
    uint64_t *tfull = used + 1;        // an accumulator (kWide: [0], both) is complete
    uint64_t *tempty = tfull + 2;      // an accumulator has been read
    uint64_t *drain = tempty + 2;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(drain + 1);
    volatile int *s_at = reinterpret_cast<volatile int *>(tmem_slot + 1);   // TN: the producer's tile
    int *s_off = reinterpret_cast<int *>(tmem_slot + 4);
    int *s_cum = s_off + p.G + 1;
    int *s_ord = s_cum + p.G + 1;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = kPair ? tc::cluster_ctarank() : 0;
    const int first = kPair ? (int)tc::cluster_id_x() : (int)blockIdx.x;
    const int step = kPair ? (int)tc::nclusters_x() : (int)gridDim.x;

    if (warp == 0) load_segments(p.row_offsets, p.G, p.rows, (kWide ? 2 : 1) * kAccCols, s_off, s_cum);
    if (warp == kEpi && lane == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        mbar_init(raw, 1);
        mbar_init(fixed, kPair ? 2 : 1);
        mbar_init(used, 1);
        for (int a = 0; a < 2; ++a) {
            mbar_init(&tfull[a], 1);
            mbar_init(&tempty[a], (kPair ? 2 : 1) * kEpi);
        }
        mbar_init(drain, 1);
        fence_mbar_init();
        *s_at = -1;
        tma_prefetch_desc(&tmM);
        tma_prefetch_desc(&tmN.m[0]);
        if (!kNmn) tma_prefetch_desc(&tmN.m[4]);
    }
    if (warp == kEpi + 1) {
        if (kPair) tc::tmem_alloc2(tmem_slot, 2 * kAccCols);
        else tmem_alloc(tmem_slot, 2 * kAccCols);
    }
    if (kPair) {   // a single-CTA launch has about one tile per CTA, and 1 us more for this would show
        __syncthreads();
        order_groups<KIND>(s_off, p.G, (kWide ? 2 : 1) * kAccCols, s_cum, s_ord);
    }
    tc_fence_before();
    __syncthreads();
    if (kPair) tc::cluster_sync();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    const int total = KIND == TN ? p.total : s_cum[p.G] * p.m_tiles;
    auto tile = [&](int i) { return tile_at<KIND, kPair, kWide>(p, s_off, s_cum, s_ord, i); };

    if (warp == kEpi) {
        // ------------------------------------------------------------ TMA producer
        int stage = 0;
        uint32_t phase = 0;
        bool ok = true;
        IssuedSlots iss, iss_raw;
        uint32_t tail_phase = 0;
        for (int i = first; i < total && ok; i += step) {
            const Tile t = tile(i);
            if (KIND == TN && lane == 0) *s_at = i;
            const int f = t.f0 + (int)rank * 128;
            const int half = kPair ? t.nh / 2 : t.nh;   // N rows of an instruction that this CTA loads
            const int r = t.r0 + (int)rank * half;
            const int box = half <= 16 ? 0 : (half + 31) / 32;
            const uint32_t bytes = kOpBytes + (kNmn ? kOpBytes : t.nsub * (box == 0 ? 16 : box * 32) * (kSl * 2));
            const CUtensorMap *mapN = &tmN.m[kNmn ? 0 : box];
            auto loads = [&](auto pair, uint32_t bar, uint8_t *dM, uint8_t *dN, int c) {
                constexpr bool P = decltype(pair)::value;
                if (KIND == NT) tma_load_3d<P>(&tmM, bar, dM, c, f, t.g);
                else load_mn<P>(&tmM, p.m_chunks, bar, dM, f, c, KIND == NN ? t.g : 0);
                if (kNmn) {
                    load_mn<P>(mapN, p.n_chunks, bar, dN, r, c, 0);
                } else {
                    tma_load_3d<P>(mapN, bar, dN, c, r, 0);
                    if (kWide && t.nsub == 2) tma_load_3d<P>(mapN, bar, dN + kOpBytes, c, r + t.nh, 0);
                }
            };
            int nkb = (t.nc + kSl - 1) / kSl;   // slices through the ring
            const bool tail = KIND == TN && t.nc % 16 != 0;
            if (tail) --nkb;
            for (int kb = 0; kb <= nkb && ok; ++kb) {
                // the last slice goes out once the ring holds this tile's first ones: the tile before is then at its own
                // last slice, and this one is not needed before all the others
                if (tail && kb == min(nkb, kStages)) {
                    ok = __all_sync(0xffffffffu, mbar_wait(used, tail_phase ^ 1, p.timeout_ns));
                    if (!ok) break;
                    if (elect_one()) {
                        mbar_arrive_expect_tx(raw, bytes);
                        loads(std::false_type{}, smem_u32(raw), sTail, sTail + kOpBytes, t.c0 + nkb * kSl);
                    }
                    iss_raw.note(0, tail_phase);
                    tail_phase ^= 1;
                }
                if (kb == nkb) break;
                if (!__all_sync(0xffffffffu, mbar_wait(&empty[stage], phase ^ 1, p.timeout_ns))) {
                    ok = false;
                    break;
                }
                const uint32_t bar = smem_u32(&full[stage]);
                if (elect_one()) {
                    if (rank == 0) mbar_arrive_expect_tx(&full[stage], (kPair ? 2 : 1) * bytes);
                    loads(std::integral_constant<bool, kPair>{}, kPair ? tc::mapa_shared(bar, 0) : bar,
                          sM + stage * kOpBytes, sN + stage * kNBytes, t.c0 + kb * kSl);
                }
                iss.note(stage, phase);
                if (++stage == kStages) {
                    stage = 0;
                    phase ^= 1;
                }
            }
        }
        if (!ok) {   // copies in flight land before the CTA leaves (a pair's land on the leader's barriers)
            iss_raw.drain(raw, p.timeout_ns);
            if (rank == 0) iss.drain(full, p.timeout_ns);
        }
    } else if (warp == kEpi + 1) {
        // ------------------------------------------------------------ MMA issuer (leader CTA)
        if (rank == 0) {
            constexpr uint32_t kIdesc = idesc_bf16_f32(kPair ? 256 : 128, 0) | (kMmn ? 1u << 15 : 0u) |
                                        (kNmn ? 1u << 16 : 0u);
            int stage = 0;
            uint32_t phase = 0, tail_phase = 0, acc_phase = 3;   // acc_phase: parity of each accumulator's last release
            int local = 0;
            bool ok = true;
            for (int i = first; i < total && ok; i += step) {
                const Tile t = tile(i);
                if (KIND == TN && t.nc == 0) continue;
                const uint32_t idesc = kIdesc | (static_cast<uint32_t>(t.nh >> 3) << 17);
                const int nkb = (t.nc + kSl - 1) / kSl;
                const int run = kSums ? run_length<kF32>(nkb) : nkb;
                for (int kb = 0, end = 0; kb < nkb && ok;) {
                    end = min(nkb, kb + run);
                    const int a0 = kWide ? 0 : local & 1;
                    ++local;
                    const uint32_t d_tmem = tmem_base + a0 * kAccCols;
                    for (int a = a0; a < a0 + t.nsub && ok; ++a) {   // the accumulators have been read
                        const uint32_t ph = (acc_phase >> a) & 1u;
                        ok = __all_sync(0xffffffffu, kPair ? tc::mbar_wait_cluster(&tempty[a], ph, p.timeout_ns)
                                                           : mbar_wait(&tempty[a], ph, p.timeout_ns));
                        acc_phase ^= 1u << a;
                    }
                    uint32_t acc = 0;
                    for (; kb < end && ok; ++kb) {
                        const bool tail = KIND == TN && kb == nkb - 1 && t.nc % 16 != 0;
                        if (tail) {   // written by threads too, maybe the other CTA's
                            ok = __all_sync(0xffffffffu, kPair ? tc::mbar_wait_cluster(fixed, tail_phase, p.timeout_ns)
                                                               : mbar_wait(fixed, tail_phase, p.timeout_ns));
                            tail_phase ^= 1;
                        } else {
                            ok = __all_sync(0xffffffffu, mbar_wait(&full[stage], phase, p.timeout_ns));
                        }
                        if (!ok) break;
                        tc_fence_after();
                        const uint32_t aM = smem_u32(tail ? sTail : sM + stage * kOpBytes);
                        const uint32_t aN = smem_u32(tail ? sTail + kOpBytes : sN + stage * kNBytes);
                        const uint64_t dm = kMmn ? smem_desc_mn(aM) : smem_desc_sw128(aM);
                        const uint64_t dn = kNmn ? smem_desc_mn(aN) : smem_desc_sw128(aN);
                        const int steps = min(kSl, t.nc - kb * kSl + 15) / 16;   // 16 of the contraction each
                        if (elect_one()) {
#pragma unroll
                            for (int k = 0; k < kSl / 16; ++k) {
                                if (k >= steps) break;
                                const uint64_t m = dm + (kMmn ? 128 : 2) * k, n = dn + (kNmn ? 128 : 2) * k;
                                if (kPair) tc::tc_mma2_bf16(d_tmem, m, n, idesc, acc);
                                else tc_mma_bf16(d_tmem, m, n, idesc, acc);
                                // the two accumulators in turn, so that an instruction does not wait for the one before it
                                if (kWide && t.nsub == 2)
                                    tc::tc_mma2_bf16(d_tmem + kAccCols, m, n + (kOpBytes >> 4), idesc, acc);
                                acc = 1;
                            }
                            uint64_t *done = tail ? used : &empty[stage];
                            if (kPair) tc::tc_commit2_mc(done, 0x3);
                            else tc_commit(done);
                        }
                        acc = 1;
                        __syncwarp();
                        if (!tail && ++stage == kStages) {
                            stage = 0;
                            phase ^= 1;
                        }
                    }
                    if (ok && elect_one()) {
                        if (kPair) tc::tc_commit2_mc(&tfull[a0], 0x3);
                        else tc_commit(&tfull[a0]);
                    }
                    __syncwarp();
                }
            }
            if (!ok) {   // wait (bounded) for the MMAs already issued before TMEM is freed
                if (elect_one()) {
                    if (kPair) tc::tc_commit2(drain);
                    else tc_commit(drain);
                }
                __syncwarp();
                mbar_wait(drain, 0, p.timeout_ns);
            }
        }
    } else if (warp == kEpi + 2) {
        // ------------------------------------------------------------ TN: rows behind the segment's end
        if (KIND == TN) {
            uint32_t tail_phase = 0;
            for (int i = first; i < total; i += step) {
                const Tile t = tile(i);
                if (t.nc % 16 == 0) continue;
                if (!__all_sync(0xffffffffu, wait_while_moving(raw, tail_phase, p.timeout_ns, s_at))) break;
                tail_phase ^= 1;
                // up to the next 16: 16-byte pieces of the cleared rows in each chunk of 64 values
                const int left = t.nc % kSl, n16 = (16 - left % 16) * 8;
                for (int j = lane; j < 4 * n16; j += 32) {
                    const int b = j / n16;
                    reinterpret_cast<uint4 *>(sTail + b * (kOpBytes / 2))[left * 8 + j - b * n16] = make_uint4(0, 0, 0, 0);
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    if (kPair) tc::mbar_arrive_remote(tc::mapa_shared(smem_u32(fixed), 0));
                    else mbar_arrive(fixed);
                }
            }
        }
    } else {
        // ------------------------------------------------------------ epilogue
        const int q = warp & 3, part = warp >> 2;
        int local = 0;
        for (int i = first; i < total; i += step) {
            const Tile t = tile(i);
            const int f = t.f0 + (int)rank * 128 + q * 32 + lane;
            const bool f_ok = f < (KIND == NT ? p.n : p.k);
            TO *out = static_cast<TO *>(p.C) + ((KIND == TN ? (int64_t)t.g * p.n : 0) + t.r0) * p.ldc;
            if (KIND == TN && t.nc == 0) {   // an expert without rows: its gradient is zero
                if (!p.accumulate && f_ok)
                    for (int j = part; j < t.rows; j += kEpi / 4) out[j * p.ldc + f] = TO(0.0f);
                continue;
            }
            auto release = [&](int a) {   // the accumulator has been read
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    if (kPair) mbar_arrive_remote_relaxed(tc::mapa_shared(smem_u32(&tempty[a]), 0));
                    else mbar_arrive(&tempty[a]);
                }
            };
            const uint32_t lanes = tmem_base + (static_cast<uint32_t>(q * 32) << 16);
            if constexpr (kSums) {
                // running sums of this warp's columns
                constexpr int kCols = kAccCols / 4, kC16 = kCols / 16;
                const int c0 = part * kCols, nkb = (t.nc + kSl - 1) / kSl, run = run_length<kF32>(nkb);
                float sum[kC16][16];
#pragma unroll
                for (int c = 0; c < kC16; ++c)
#pragma unroll
                    for (int k = 0; k < 16; ++k) sum[c][k] = 0.f;
                bool ok = true;
                for (int kb = 0; kb < nkb && ok; kb += run) {
                    const int a = local & 1;
                    const uint32_t ph = (local >> 1) & 1;
                    ++local;
                    // warp-uniform decision: the TMEM loads below are warp-collective
                    ok = __all_sync(0xffffffffu, mbar_wait(&tfull[a], ph, p.timeout_ns));
                    if (!ok) break;
                    tc_fence_after();
#pragma unroll
                    for (int c = 0; c < kC16; ++c) {
                        if (c0 + c * 16 >= t.rows) break;   // warp-uniform
                        uint32_t r[16];
                        tc::tmem_ld_32x32b_x16(lanes + a * kAccCols + c0 + c * 16, r);
                        tc::tmem_ld_wait_regs(r);
#pragma unroll
                        for (int k = 0; k < 16; ++k) sum[c][k] += __uint_as_float(r[k]);
                    }
                    release(a);
                }
                if (!ok) break;
#pragma unroll
                for (int c = 0; c < kC16; ++c) {
                    TO *dst = out + (c0 + c * 16) * p.ldc;
                    const int rows = t.rows - c0 - c * 16, accumulate = KIND == TN ? p.accumulate : 0;
                    if constexpr (kF32) store_f32<16>(dst + f, p.ldc, f_ok, sum[c], rows, accumulate);
                    else store_bf16<16>(dst, p.ldc, f, f_ok, sum[c], rows, accumulate);
                }
            } else {
                const int a0 = kWide ? 0 : local & 1;
                const uint32_t ph = kWide ? local & 1 : (local >> 1) & 1;
                ++local;
                if (!__all_sync(0xffffffffu, mbar_wait(&tfull[a0], ph, p.timeout_ns))) break;
                tc_fence_after();
                for (int h = 0; h < t.nsub; ++h) {
                    const int rows = min(t.nh, t.rows - h * t.nh);
                    TO *dst = out + (int64_t)h * t.nh * p.ldc;
                    for (int c = part * 32; c < rows; c += 32 * (kEpi / 4)) {
                        uint32_t r[32];
                        tmem_ld_32x32b_x32(lanes + (a0 + h) * kAccCols + c, r);
                        tmem_ld_wait();
                        float v[32];
#pragma unroll
                        for (int k = 0; k < 32; ++k) v[k] = __uint_as_float(r[k]);
                        store_bf16<32>(dst + c * p.ldc, p.ldc, f, f_ok, v, rows - c, KIND == TN ? p.accumulate : 0);
                    }
                    release(a0 + h);
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (kPair) tc::cluster_sync();   // the leader's last MMAs read this CTA's shared memory and TMEM
    if (warp == kEpi + 1) {
        tc_fence_after();
        if (kPair) tc::tmem_dealloc2(tmem_base, 2 * kAccCols);
        else tmem_dealloc(tmem_base, 2 * kAccCols);
    }
}

template <int KIND, typename TO, bool kWide, bool kSums>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kTcThreads, 1)
    tc_pair_kernel(const __grid_constant__ CUtensorMap tmM, const __grid_constant__ NMaps tmN, const Params p) {
    tc_body<KIND, TO, true, kWide, kSums>(tmM, tmN, p);
}
template <int KIND, typename TO, bool kSums>
__global__ void __launch_bounds__(kTcThreads, 1)
    tc_single_kernel(const __grid_constant__ CUtensorMap tmM, const __grid_constant__ NMaps tmN, const Params p) {
    tc_body<KIND, TO, false, false, kSums>(tmM, tmN, p);
}

}  // namespace gmm
}  // namespace moe
