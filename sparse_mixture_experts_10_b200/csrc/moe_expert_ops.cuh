// moe_expert_ops.cuh -- host side of the expert operators beside the layer
// call: grouped products, 8-bit activation checkpoints, 4-bit expert products.
// Included by moe_api.cu after its helpers; argument checks come before any
// launch, nothing is allocated and no stream is synchronised.
#pragma once

namespace {

bool aligned4(const void *ptr) { return (reinterpret_cast<uintptr_t>(ptr) & 3u) == 0; }
bool dtype_ok(int32_t d) { return d == MOE_F32 || d == MOE_BF16; }
int64_t elem_size(int32_t d) { return d == MOE_F32 ? 4 : 2; }

// Row strides: 0 stands for a contiguous row; otherwise at least the row's
// length and a multiple of 16 bytes.
int take_stride(int64_t given, int64_t cols, int64_t es, int64_t *out) {
    *out = given == 0 ? cols : given;
    if (*out < cols || *out > (int64_t(1) << 32) || (*out * es) % 16 != 0) return MOE_ERR_INVALID_ARG;
    return MOE_OK;
}

// ---------------------------------------------------------------- grouped products
struct GmmPlan {
    gmm::Params p;
    int64_t a_cols, c_cols;
};

int make_gmm_plan(const moe_gmm *d, int64_t rows, GmmPlan *out) {
    if (!d || rows < 0 || rows > INT32_MAX - 1024) return MOE_ERR_INVALID_ARG;
    if (d->kind != MOE_GMM_NT && d->kind != MOE_GMM_NN && d->kind != MOE_GMM_TN) return MOE_ERR_INVALID_ARG;
    if (d->groups < 1 || d->groups > gmm::kMaxGroups || d->n < 1 || d->k < 1) return MOE_ERR_INVALID_ARG;
    // the kernels' 32-bit places step past the last one by a few slices, like those of rows
    if (d->n > INT32_MAX - 1024 || d->k > INT32_MAX - 1024) return MOE_ERR_UNSUPPORTED;
    if (!dtype_ok(d->dtype) || !dtype_ok(d->out_dtype)) return MOE_ERR_INVALID_ARG;
    if (d->dtype == MOE_F32 && d->out_dtype != MOE_F32) return MOE_ERR_UNSUPPORTED;
    if (d->accumulate != 0 && d->accumulate != 1) return MOE_ERR_INVALID_ARG;
    if (d->accumulate && d->kind != MOE_GMM_TN) return MOE_ERR_UNSUPPORTED;
    if (d->reserved != 0) return MOE_ERR_INVALID_ARG;
    const int64_t es = elem_size(d->dtype), os = elem_size(d->out_dtype);
    if (d->n % (16 / es) || d->k % (16 / es)) return MOE_ERR_INVALID_ARG;
    gmm::Params &p = out->p;
    p = gmm::Params{};
    out->a_cols = d->kind == MOE_GMM_NT ? d->k : d->n;
    out->c_cols = d->kind == MOE_GMM_NT ? d->n : d->k;
    MOE_TRY(take_stride(d->lda, out->a_cols, es, &p.lda));
    MOE_TRY(take_stride(d->ldb, d->k, es, &p.ldb));
    MOE_TRY(take_stride(d->ldc, out->c_cols, os, &p.ldc));
    // a tensor map's strides stay below 2^40 bytes: a group's weights are n rows of ldb (by division: their product may
    // pass 64 bits); the weight gradient's n rows of ldc keep to it too, so that no index of c does
    const int64_t most = (int64_t(1) << 40) - 1;
    if (d->kind == MOE_GMM_TN ? p.ldc > most / os / d->n : p.ldb > most / es / d->n) return MOE_ERR_UNSUPPORTED;
    p.rows = rows;
    p.G = d->groups;
    p.n = d->n;
    p.k = d->k;
    p.accumulate = d->accumulate;
    // a wait lasts at most one tile (the clearer's: one tile of the producer's): about half a microsecond for 64 of the
    // contraction, 2 allowed
    p.timeout_ns = kTimeoutNs + 32ull * (uint64_t)std::max<int64_t>(rows, std::max(d->n, d->k));
    return MOE_OK;
}

template <int KIND>
int launch_gmm_simt(gmm::Params p, const DeviceInfo &dev, cudaStream_t s) {
    const int64_t cols = KIND == gmm::NT ? p.n : p.k;
    p.n_tiles = (int)cdiv(cols, gmm::kTile);
    int64_t upper;
    if (KIND == gmm::TN) {
        p.m_tiles = (int)cdiv(p.n, gmm::kTile);
        upper = (int64_t)p.G * p.m_tiles * p.n_tiles;
    } else {
        upper = (cdiv(p.rows, gmm::kTile) + std::min<int64_t>(p.G, p.rows)) * p.n_tiles;
    }
    if (upper > INT32_MAX - 65536) return MOE_ERR_UNSUPPORTED;   // tile counters step past the last one
    p.total = (int)upper;
    const unsigned grid = (unsigned)std::min<int64_t>(upper, (int64_t)dev.sms * 6);
    return launch_pdl(gmm::simt_kernel<KIND>, dim3(grid), dim3(gmm::kSimtThreads), 0, s, p);
}

// bf16 tensor of up to four dimensions (d[0] contiguous, the others with strides of st elements), 128-byte swizzle.
int make_map_nd(CUtensorMap *m, int nd, const void *base, const int64_t *d, const int64_t *st, const int *box) {
    EncodeTiledFn enc = encode_fn();
    if (!enc) return MOE_ERR_CUDA;
    cuuint64_t dims[4], strides[3];
    cuuint32_t b[4], estr[4];
    for (int i = 0; i < nd; ++i) {
        dims[i] = (cuuint64_t)d[i];
        if (i) strides[i - 1] = (cuuint64_t)st[i - 1] * 2;
        b[i] = (cuuint32_t)box[i];
        estr[i] = 1;
    }
    const CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, (cuuint32_t)nd, const_cast<void *>(base), dims, strides,
                           b, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                           CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? MOE_OK : MOE_ERR_CUDA;
}
// K-major operand [G, rows, cols]: boxes of `box` rows x 64 columns.
int make_map_k(CUtensorMap *m, const void *base, int64_t G, int64_t rows, int64_t cols, int64_t ld, int box) {
    const int64_t d[3] = {cols, rows, G}, st[2] = {ld, G > 1 ? rows * ld : ld};
    const int b[3] = {64, box, 1};
    return make_map_nd(m, 3, base, d, st, b);
}
// MN-major operand [G, rows, cols]: boxes of 64 rows x two chunks of 64 columns where the width has whole
// chunks only (*chunks), else of 64 rows x 64 columns.
int make_map_mn(CUtensorMap *m, const void *base, int64_t G, int64_t rows, int64_t cols, int64_t ld, int *chunks) {
    *chunks = cols % 64 == 0;
    const int64_t gs = G > 1 ? rows * ld : ld;
    const int64_t d[4] = {*chunks ? 64 : cols, rows, *chunks ? cols / 64 : 1, G}, st[3] = {ld, 64, gs};
    const int b[4] = {64, 64, *chunks ? 2 : 1, 1};
    return make_map_nd(m, 4, base, d, st, b);
}

template <int KIND, typename TO, bool kSums>
int launch_gmm_tc(gmm::Params p, const DeviceInfo &dev, cudaStream_t s) {
    CUtensorMap mm;
    gmm::NMaps mn;
    if (KIND == gmm::NT) MOE_TRY(make_map_k(&mm, p.B, p.G, p.n, p.k, p.ldb, 128));
    else MOE_TRY(make_map_mn(&mm, p.B, KIND == gmm::NN ? p.G : 1, KIND == gmm::NN ? p.n : p.rows, p.k, p.ldb,
                             &p.m_chunks));
    if (KIND == gmm::TN) {
        MOE_TRY(make_map_mn(&mn.m[0], p.A, 1, p.rows, p.n, p.lda, &p.n_chunks));
        for (int i = 1; i < 5; ++i) mn.m[i] = mn.m[0];
    } else {
        for (int i = 0; i < 5; ++i)
            MOE_TRY(make_map_k(&mn.m[i], p.A, 1, p.rows, KIND == gmm::NT ? p.k : p.n, p.lda, gmm::box_rows(i)));
    }
    const int64_t F = KIND == gmm::NT ? p.n : p.k, live = std::min<int64_t>(p.G, p.rows);
    // Tile shapes, by the row tiles to be expected where every group has rows (segments are on the device; the host knows
    // their number and sum only).  Rows that crowd on one group make fewer tiles: 256 of them on one of 32 groups, n 4096,
    // k 1024, take pairs and 13.9 us, single CTAs 9.8 us; spread evenly, 54.6 us.  1500 on two of 8 groups 19.2 us, with
    // the two alone (wide pairs) 18.8 us.
    //  pairs (256 x 256) where they fill the machine: 32 x 4096 x 7168 over 512 rows each 714 us, single CTAs (128 x 128)
    //    963 us; 6 x 1536 x 768 over 34 rows 9.7 us, single CTAs 7.5 us (twice as many SMs read);
    //  wide pairs (256 x 512) where segments have more than 256 rows: 675 us against 714 us; 300 rows 482 against 556
    auto row_tiles = [&](int64_t unit) { return std::max(live, cdiv(p.rows, unit)); };
    const bool pair = (KIND == gmm::TN ? p.G * cdiv(p.n, 256) : row_tiles(256)) * cdiv(F, 256) >= dev.pair_clusters;
    // (they need both accumulators, and registers cannot hold the running sums of 512 rows)
    const bool wide = pair && KIND != gmm::TN && !kSums && p.rows > 256 * live &&
                      row_tiles(512) * cdiv(F, 256) >= dev.pair_clusters;
    const int unit = pair ? 256 : 128;
    p.m_tiles = (int)cdiv(F, unit);
    p.n_tiles = (int)cdiv(p.n, unit);
    const int64_t upper = KIND == gmm::TN ? (int64_t)p.G * p.m_tiles * p.n_tiles
                                          : (cdiv(p.rows, unit) + live) * p.m_tiles;
    if (upper > INT32_MAX - 65536) return MOE_ERR_UNSUPPORTED;   // tile counters step past the last one
    p.total = (int)upper;
    const size_t smem = gmm::tc_smem_bytes(p.G);
    if (pair) {
        const dim3 grid((unsigned)(2 * std::min<int64_t>(upper, dev.pair_clusters)));
        if constexpr (KIND != gmm::TN && !kSums)
            if (wide)
                return launch_pdl(gmm::tc_pair_kernel<KIND, TO, true, false>, grid, dim3(gmm::kTcThreads), smem, s, mm, mn,
                                  p);
        return launch_pdl(gmm::tc_pair_kernel<KIND, TO, false, kSums>, grid, dim3(gmm::kTcThreads), smem, s, mm, mn, p);
    }
    return launch_pdl(gmm::tc_single_kernel<KIND, TO, kSums>, dim3((unsigned)std::min<int64_t>(upper, dev.sms)),
                      dim3(gmm::kTcThreads), smem, s, mm, mn, p);
}

template <int KIND>
int launch_gmm(const moe_gmm *d, const gmm::Params &p, const DeviceInfo &dev, cudaStream_t s) {
    if (d->dtype == MOE_F32) return launch_gmm_simt<KIND>(p, dev, s);
    if (d->out_dtype == MOE_F32) return launch_gmm_tc<KIND, float, true>(p, dev, s);
    // running sums for a bf16 result where a contraction may be longer than a run (segments are known on the device only):
    // without them 32 weight gradients of 7168 x 2048 over 16448 rows take 450 us, with them 473 us; 8 of 2880 x 1000
    // over 16640 rows 87 and 89 us; 4 x 2048 x 16448 over 4096 rows 312 us either way
    const int64_t terms = KIND == gmm::NT ? p.k : KIND == gmm::NN ? p.n : p.rows;   // of a sum, at most
    if (terms > gmm::kRunBf16 * gmm::kSl) return launch_gmm_tc<KIND, __nv_bfloat16, true>(p, dev, s);
    return launch_gmm_tc<KIND, __nv_bfloat16, false>(p, dev, s);
}

// ---------------------------------------------------------------- 8-bit checkpoints
int make_ckpt_params(const moe_ckpt *d, int64_t rows, ckpt::Params *p) {
    if (!d || rows < 0 || rows > INT32_MAX) return MOE_ERR_INVALID_ARG;
    if (d->act != MOE_ACT_GELU && d->act != MOE_ACT_SWIGLU && d->act != MOE_ACT_NONE) return MOE_ERR_INVALID_ARG;
    if (!dtype_ok(d->dtype) || (d->format != MOE_CKPT_INT8 && d->format != MOE_CKPT_E4M3)) return MOE_ERR_INVALID_ARG;
    if (d->group != 32 && d->group != 64 && d->group != 128) return MOE_ERR_INVALID_ARG;
    if (d->reserved != 0) return MOE_ERR_INVALID_ARG;
    const int64_t es = elem_size(d->dtype);
    if (d->width < 1 || d->width % (16 / es) || d->width > (1 << 28)) return MOE_ERR_INVALID_ARG;
    *p = ckpt::Params{};
    MOE_TRY(take_stride(d->ldu, (d->act == MOE_ACT_SWIGLU ? 2 : 1) * (int64_t)d->width, es, &p->ldu));
    MOE_TRY(take_stride(d->ldh, d->width, es, &p->ldh));
    p->rows = rows;
    p->width = d->width;
    p->group_shift = d->group == 32 ? 5 : d->group == 64 ? 6 : 7;
    p->sgroups = (int)cdiv(d->width, d->group);
    return MOE_OK;
}

// Sets the warps of a block that share a row: as many as the row has pieces for (512 bytes a load, `unroll` loads at
// a time).
void set_row_warps(ckpt::Params *p, int64_t es, int unroll) {
    const int64_t pieces = cdiv((int64_t)p->width * es, 512 * unroll);
    p->row_warps = 1;
    while (p->row_warps < ckpt::kThreads / 32 && p->row_warps * 2 <= pieces) p->row_warps *= 2;
}

// One load at a time where all warps of the machine (64 an SM) have at most one piece each.
int ckpt_unroll(const ckpt::Params &p, int64_t es, const DeviceInfo &dev) {
    return p.rows * cdiv((int64_t)p.width * es, 512) <= (int64_t)dev.sms * 64 ? 1 : ckpt::kManyUnroll;
}

dim3 ckpt_grid(const ckpt::Params &p) {
    return dim3((unsigned)cdiv(p.rows, (ckpt::kThreads / 32) / p.row_warps));
}

template <typename T, int FMT, int U>
int launch_ckpt_forward_u(int act, ckpt::Params p, cudaStream_t s) {
    set_row_warps(&p, sizeof(T), U);
    auto *k = act == MOE_ACT_GELU     ? ckpt::forward_kernel<T, ckpt::GELU, FMT, U>
              : act == MOE_ACT_SWIGLU ? ckpt::forward_kernel<T, ckpt::SWIGLU, FMT, U>
                                      : ckpt::forward_kernel<T, ckpt::NONE, FMT, U>;
    return launch_pdl(k, ckpt_grid(p), dim3(ckpt::kThreads), 0, s, p);
}
template <typename T, int FMT>
int launch_ckpt_forward(int act, const ckpt::Params &p, cudaStream_t s) {
    DeviceInfo *dev = nullptr;
    MOE_TRY(device_info(&dev));
    return ckpt_unroll(p, sizeof(T), *dev) == 1 ? launch_ckpt_forward_u<T, FMT, 1>(act, p, s)
                                                : launch_ckpt_forward_u<T, FMT, ckpt::kManyUnroll>(act, p, s);
}
template <typename T, int FMT, int U>
int launch_ckpt_backward_u(int act, ckpt::Params p, cudaStream_t s) {
    set_row_warps(&p, sizeof(T), U);
    auto *k = act == MOE_ACT_GELU ? ckpt::backward_kernel<T, ckpt::GELU, FMT, U>
                                  : ckpt::backward_kernel<T, ckpt::SWIGLU, FMT, U>;
    return launch_pdl(k, ckpt_grid(p), dim3(ckpt::kThreads), 0, s, p);
}
template <typename T, int FMT>
int launch_ckpt_backward(int act, const ckpt::Params &p, cudaStream_t s) {
    DeviceInfo *dev = nullptr;
    MOE_TRY(device_info(&dev));
    return ckpt_unroll(p, sizeof(T), *dev) == 1 ? launch_ckpt_backward_u<T, FMT, 1>(act, p, s)
                                                : launch_ckpt_backward_u<T, FMT, ckpt::kManyUnroll>(act, p, s);
}

// ---------------------------------------------------------------- 4-bit weights
int make_q4_params(const moe_q4 *d, q4::Params *p) {
    if (!d || d->experts < 1 || d->experts > 1024) return MOE_ERR_INVALID_ARG;
    if (d->format != MOE_Q4_INT4 && d->format != MOE_Q4_E2M1) return MOE_ERR_INVALID_ARG;
    if (d->act != MOE_ACT_GELU && d->act != MOE_ACT_SWIGLU && d->act != MOE_ACT_NONE) return MOE_ERR_INVALID_ARG;
    if (d->group != 32 && d->group != 64 && d->group != 128) return MOE_ERR_INVALID_ARG;
    if (d->format == MOE_Q4_E2M1 && d->group != 32) return MOE_ERR_UNSUPPORTED;
    if (d->n < 1 || d->n % 8 || (d->act == MOE_ACT_SWIGLU && d->n % 16)) return MOE_ERR_INVALID_ARG;
    if (d->k < 1 || d->k % 32 || d->n > (1 << 20) || d->k > (1 << 20)) return MOE_ERR_INVALID_ARG;
    if ((int64_t)d->experts * d->n > INT32_MAX) return MOE_ERR_UNSUPPORTED;   // rows are tensor-map coordinates
    *p = q4::Params{};
    p->N = d->experts;
    p->n = d->n;
    p->k = d->k;
    p->group_shift = d->group == 32 ? 5 : d->group == 64 ? 6 : 7;
    p->groups = (int)cdiv(d->k, d->group);
    return MOE_OK;
}

// Codes [N, n, k / 2] as boxes of box_tiles tiles x 128 bytes, 128-byte swizzle: 16 rows a tile, or (halves) 8 rows of
// either half of the n rows.
int make_map_codes(CUtensorMap *m, const uint8_t *codes, int64_t N, int64_t n, int64_t row_bytes, bool halves,
                   int box_tiles) {
    EncodeTiledFn enc = encode_fn();
    if (!enc) return MOE_ERR_CUDA;
    const cuuint64_t rows = (cuuint64_t)(halves ? n / 2 : n), rb = (cuuint64_t)row_bytes;
    const cuuint64_t dims[4] = {rb, rows, halves ? 2u : 1u, (cuuint64_t)N}, strides[3] = {rb, rows * rb, (cuuint64_t)n * rb};
    const cuuint32_t box[4] = {128u, (cuuint32_t)(box_tiles * (halves ? 8 : 16)), halves ? 2u : 1u, 1u};
    const cuuint32_t estr[4] = {1u, 1u, 1u, 1u};
    const CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<uint8_t *>(codes), dims, strides, box, estr,
                           CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                           CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? MOE_OK : MOE_ERR_CUDA;
}

int launch_q4(int format, const q4::MatvecParams &p, const DeviceInfo &dev, cudaStream_t s) {
    const int64_t live = std::min<int64_t>(p.N, p.pairs);
    q4::MatvecParams q = p;
    q.tiles = (int)cdiv(p.n, 16);
    // warps that share a tile: the fewest rounds of boxes for a block's share of the tiles (a round more for
    // each tile's start and end); with few tiles a split of k keeps all warps streaming
    const int64_t chunks = cdiv(p.k, q4::kChunk), mine = cdiv(live * q.tiles, dev.sms);
    int64_t best = INT64_MAX;
    for (int ks = 1; ks <= q4::kWarps && ks <= chunks; ks *= 2) {
        const int64_t rounds = cdiv(mine, q4::kWarps / ks) * (cdiv(chunks, ks) + 1);
        if (rounds < best) {
            best = rounds;
            q.ks = ks;
        }
    }
    // pairs staged at a time and the ring's length: what shared memory holds
    q.x_stride = q4::x_stride(p.k);
    const size_t room = q4::kRoom;
    q.slots = 4;
    q.cols_pass = (int)std::min<int64_t>(p.pairs, q4::kMaxCols);
    if (q4::matvec_smem(4, q.cols_pass, p.k, p.pairs) > room) q.slots = 3;
    while (q.cols_pass > 1 && q4::matvec_smem(q.slots, q.cols_pass, p.k, p.pairs) > room) --q.cols_pass;
    const size_t smem = q4::matvec_smem(q.slots, q.cols_pass, p.k, p.pairs);   // one column fits: checked before
    // a copy is four tiles where a block's step has as many: a step at an expert's end then reads little too much
    q.box_tiles = std::min(4, q4::kWarps / q.ks);
    CUtensorMap map;
    MOE_TRY(make_map_codes(&map, q.codes, q.N, q.n, q.k / 2, q.act == MOE_ACT_SWIGLU, q.box_tiles));
    const int64_t lots = live + p.pairs / q.cols_pass;   // at most
    const dim3 grid((unsigned)std::min<int64_t>(dev.sms, lots * q.tiles));
    auto *k = format == MOE_Q4_E2M1      ? q4::matvec_kernel<q4::E2M1, 5>
              : p.group_shift == 5       ? q4::matvec_kernel<q4::INT4, 5>
              : p.group_shift == 6       ? q4::matvec_kernel<q4::INT4, 6>
                                         : q4::matvec_kernel<q4::INT4, 7>;
    return launch_pdl(k, grid, dim3(q4::kThreadsMv), smem, s, map, q);
}

// Attributes of this file's kernels, set once per device with the others'.
int expert_ops_attrs() {
#define MOE_GMM_ATTR(KIND)                                                     \
    MOE_TRY(allow_smem(gmm::tc_pair_kernel<KIND, float, false, true>));        \
    MOE_TRY(allow_smem(gmm::tc_single_kernel<KIND, float, true>));             \
    MOE_TRY(allow_smem(gmm::tc_pair_kernel<KIND, __nv_bfloat16, false, true>)); \
    MOE_TRY(allow_smem(gmm::tc_single_kernel<KIND, __nv_bfloat16, true>));     \
    MOE_TRY(allow_smem(gmm::tc_pair_kernel<KIND, __nv_bfloat16, false, false>)); \
    MOE_TRY(allow_smem(gmm::tc_single_kernel<KIND, __nv_bfloat16, false>))
    MOE_GMM_ATTR(gmm::NT);
    MOE_GMM_ATTR(gmm::NN);
    MOE_GMM_ATTR(gmm::TN);
    MOE_TRY(allow_smem(gmm::tc_pair_kernel<gmm::NT, __nv_bfloat16, true, false>));
    MOE_TRY(allow_smem(gmm::tc_pair_kernel<gmm::NN, __nv_bfloat16, true, false>));
#undef MOE_GMM_ATTR
    MOE_TRY(allow_smem(q4::matvec_kernel<q4::INT4, 5>));
    MOE_TRY(allow_smem(q4::matvec_kernel<q4::INT4, 6>));
    MOE_TRY(allow_smem(q4::matvec_kernel<q4::INT4, 7>));
    MOE_TRY(allow_smem(q4::matvec_kernel<q4::E2M1, 5>));
    return MOE_OK;
}

}  // namespace

extern "C" {

int moe_grouped_mm(const moe_gmm *d, const void *a, const void *b, void *c, const int32_t *row_offsets, int64_t rows,
                   moe_stream_t stream) {
    GmmPlan P;
    MOE_TRY(make_gmm_plan(d, rows, &P));
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const bool tn = d->kind == MOE_GMM_TN;
    if (rows == 0) {   // no segment has a row: the weight gradients are zero, the others have nothing to write
        if (!tn || d->accumulate) return MOE_OK;
        if (!c || !aligned16(c)) return MOE_ERR_INVALID_ARG;
        const size_t os = (size_t)elem_size(d->out_dtype);
        return cudaMemset2DAsync(c, (size_t)P.p.ldc * os, 0, (size_t)d->k * os, (size_t)d->groups * d->n, s) ==
                       cudaSuccess
                   ? MOE_OK
                   : MOE_ERR_CUDA;
    }
    if (!a || !b || !c || !row_offsets) return MOE_ERR_INVALID_ARG;
    if (!aligned16(a) || !aligned16(b) || !aligned16(c) || !aligned4(row_offsets)) return MOE_ERR_INVALID_ARG;
    DeviceInfo *dev = nullptr;
    MOE_TRY(device_info(&dev));
    P.p.A = a;
    P.p.B = b;
    P.p.C = c;
    P.p.row_offsets = row_offsets;
    if (tn) return launch_gmm<gmm::TN>(d, P.p, *dev, s);
    if (d->kind == MOE_GMM_NT) return launch_gmm<gmm::NT>(d, P.p, *dev, s);
    return launch_gmm<gmm::NN>(d, P.p, *dev, s);
}

int moe_ckpt_forward(const moe_ckpt *d, const void *u, int64_t rows, void *h, uint8_t *q, uint8_t *scales,
                     moe_stream_t stream) {
    ckpt::Params p;
    MOE_TRY(make_ckpt_params(d, rows, &p));
    if (rows == 0) return MOE_OK;
    if (!u || !q || !scales || (!h && d->act != MOE_ACT_NONE)) return MOE_ERR_INVALID_ARG;
    if (!aligned16(u) || !aligned16(q) || !aligned16(h)) return MOE_ERR_INVALID_ARG;
    p.u = u;
    p.h = h;
    p.q = q;
    p.s = scales;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (d->dtype == MOE_F32)
        return d->format == MOE_CKPT_INT8 ? launch_ckpt_forward<float, ckpt::INT8>(d->act, p, s)
                                          : launch_ckpt_forward<float, ckpt::E4M3>(d->act, p, s);
    return d->format == MOE_CKPT_INT8 ? launch_ckpt_forward<__nv_bfloat16, ckpt::INT8>(d->act, p, s)
                                      : launch_ckpt_forward<__nv_bfloat16, ckpt::E4M3>(d->act, p, s);
}

int moe_ckpt_load(const moe_ckpt *d, const uint8_t *q, const uint8_t *scales, int64_t rows, void *u,
                  moe_stream_t stream) {
    ckpt::Params p;
    MOE_TRY(make_ckpt_params(d, rows, &p));
    if (rows == 0) return MOE_OK;
    if (!u || !q || !scales || !aligned16(u) || !aligned16(q)) return MOE_ERR_INVALID_ARG;
    p.q_in = q;
    p.s_in = scales;
    p.h = u;
    p.ldh = p.ldu;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const int halves = d->act == MOE_ACT_SWIGLU ? 2 : 1;
    set_row_warps(&p, elem_size(d->dtype), 1);
    auto *k = d->dtype == MOE_F32
                  ? (d->format == MOE_CKPT_INT8 ? ckpt::load_kernel<float, ckpt::INT8>
                                                : ckpt::load_kernel<float, ckpt::E4M3>)
                  : (d->format == MOE_CKPT_INT8 ? ckpt::load_kernel<__nv_bfloat16, ckpt::INT8>
                                                : ckpt::load_kernel<__nv_bfloat16, ckpt::E4M3>);
    return launch_pdl(k, ckpt_grid(p), dim3(ckpt::kThreads), 0, s, p, halves);
}

int moe_ckpt_backward(const moe_ckpt *d, const uint8_t *q, const uint8_t *scales, int64_t rows, const void *dh,
                      const float *w, void *du, void *hw, float *dw, moe_stream_t stream) {
    ckpt::Params p;
    MOE_TRY(make_ckpt_params(d, rows, &p));
    if (d->act == MOE_ACT_NONE) return MOE_ERR_INVALID_ARG;
    if (rows == 0) return MOE_OK;
    if (!q || !scales || !dh || !du) return MOE_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(dh) || !aligned16(du) || !aligned16(hw) || !aligned4(w) || !aligned4(dw))
        return MOE_ERR_INVALID_ARG;
    p.q_in = q;
    p.s_in = scales;
    p.dh = dh;
    p.w = w;
    p.du = du;
    p.hw = hw;
    p.dw = dw;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (d->dtype == MOE_F32)
        return d->format == MOE_CKPT_INT8 ? launch_ckpt_backward<float, ckpt::INT8>(d->act, p, s)
                                          : launch_ckpt_backward<float, ckpt::E4M3>(d->act, p, s);
    return d->format == MOE_CKPT_INT8 ? launch_ckpt_backward<__nv_bfloat16, ckpt::INT8>(d->act, p, s)
                                      : launch_ckpt_backward<__nv_bfloat16, ckpt::E4M3>(d->act, p, s);
}

int moe_q4_quantize(const moe_q4 *d, const void *W, int32_t w_dtype, uint8_t *codes, void *scales,
                    moe_stream_t stream) {
    q4::Params p;
    MOE_TRY(make_q4_params(d, &p));
    if (!dtype_ok(w_dtype)) return MOE_ERR_INVALID_ARG;
    if (!W || !codes || !scales || !aligned16(W) || !aligned16(codes) || !aligned16(scales)) return MOE_ERR_INVALID_ARG;
    DeviceInfo *dev = nullptr;
    MOE_TRY(device_info(&dev));
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const int64_t rows = (int64_t)p.N * p.n;
    const dim3 grid((unsigned)std::min<int64_t>(cdiv(rows * p.groups, q4::kThreads / 32), (int64_t)dev->sms * 32));
    if (w_dtype == MOE_F32) {
        auto *k = d->format == MOE_Q4_INT4 ? q4::quantize_kernel<q4::INT4, float> : q4::quantize_kernel<q4::E2M1, float>;
        return launch_pdl(k, grid, dim3(q4::kThreads), 0, s, static_cast<const float *>(W), rows, p.k, p.group_shift,
                          p.groups, codes, scales);
    }
    auto *k = d->format == MOE_Q4_INT4 ? q4::quantize_kernel<q4::INT4, __nv_bfloat16>
                                       : q4::quantize_kernel<q4::E2M1, __nv_bfloat16>;
    return launch_pdl(k, grid, dim3(q4::kThreads), 0, s, static_cast<const __nv_bfloat16 *>(W), rows, p.k,
                      p.group_shift, p.groups, codes, scales);
}

int moe_q4_dequantize(const moe_q4 *d, const uint8_t *codes, const void *scales, void *W, int32_t w_dtype,
                      moe_stream_t stream) {
    q4::Params p;
    MOE_TRY(make_q4_params(d, &p));
    if (!dtype_ok(w_dtype)) return MOE_ERR_INVALID_ARG;
    if (!W || !codes || !scales || !aligned16(W) || !aligned16(codes) || !aligned16(scales)) return MOE_ERR_INVALID_ARG;
    DeviceInfo *dev = nullptr;
    MOE_TRY(device_info(&dev));
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const int64_t rows = (int64_t)p.N * p.n;
    const dim3 grid((unsigned)std::min<int64_t>(cdiv(rows * (p.k / 8), q4::kThreads), (int64_t)dev->sms * 32));
    if (w_dtype == MOE_F32) {
        auto *k = d->format == MOE_Q4_INT4 ? q4::dequantize_kernel<q4::INT4, float>
                                           : q4::dequantize_kernel<q4::E2M1, float>;
        return launch_pdl(k, grid, dim3(q4::kThreads), 0, s, codes, scales, rows, p.k, p.group_shift, p.groups,
                          static_cast<float *>(W));
    }
    auto *k = d->format == MOE_Q4_INT4 ? q4::dequantize_kernel<q4::INT4, __nv_bfloat16>
                                       : q4::dequantize_kernel<q4::E2M1, __nv_bfloat16>;
    return launch_pdl(k, grid, dim3(q4::kThreads), 0, s, codes, scales, rows, p.k, p.group_shift, p.groups,
                      static_cast<__nv_bfloat16 *>(W));
}

int moe_q4_matvec(const moe_q4 *d, const void *x, int64_t pairs, int32_t x_div, const int32_t *expert,
                  const uint8_t *codes, const void *scales, const float *gate, void *y, int32_t y_dtype,
                  moe_stream_t stream) {
    q4::MatvecParams p{};
    MOE_TRY(make_q4_params(d, &p));
    if (pairs < 0 || x_div < 1 || !dtype_ok(y_dtype)) return MOE_ERR_INVALID_ARG;
    if (pairs > q4::kMaxPairs) return MOE_ERR_UNSUPPORTED;
    if (pairs == 0) return MOE_OK;
    if (q4::matvec_smem(3, 1, p.k, pairs) > q4::kRoom) return MOE_ERR_UNSUPPORTED;
    if (!x || !expert || !codes || !scales || !y) return MOE_ERR_INVALID_ARG;
    if (!aligned16(x) || !aligned16(codes) || !aligned16(scales) || !aligned16(y) || !aligned4(expert) || !aligned4(gate))
        return MOE_ERR_INVALID_ARG;
    p.x = static_cast<const __nv_bfloat16 *>(x);
    p.pairs = pairs;
    p.x_div = x_div;
    p.expert = expert;
    p.codes = codes;
    p.scales = scales;
    p.gate = gate;
    p.y = y;
    p.timeout_ns = kTimeoutNs;
    DeviceInfo *dev = nullptr;
    MOE_TRY(device_info(&dev));
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    p.act = d->act;
    p.y_f32 = y_dtype == MOE_F32;
    return launch_q4(d->format, p, *dev, s);
}

}  // extern "C"
