// pqg_kv_attention: argument checks, the plan of a call and its launches.
#include "pqg_attention.cuh"

#include <algorithm>
#include <cmath>

#include "pqg_cache_host.cuh"

namespace pqg {

int sm_count(int device);  // cached cudaDevAttrMultiProcessorCount

namespace {

// How a call is cut: 8-row tiles of a block, units per key/value head, blocks.
struct Plan {
    int64_t rows, n_tiles, row_tiles, units, shares, workspace;
    bool split;                // whether a unit may be divided among blocks
};

int make_plan(const CacheView &c, int64_t max_pages, int64_t B, int64_t q_len, int64_t q_heads,
              int64_t max_len, Plan *plan) {
    if (B < 0 || B > kMaxSequences || q_len < 1 || q_len > kMaxQueryTokens || q_heads < 1 ||
        q_heads % c.heads != 0 || q_heads > kMaxQueryHeads || max_pages < 1 ||
        max_pages > kMaxStride)
        return PQG_ERR_INVALID_ARG;
    plan->rows = q_len * (q_heads / c.heads);
    // 16 rows to a block where there are more than 8 (not for a head of 256: registers)
    plan->n_tiles = plan->rows > kTileRows && c.head_dim < 256 ? 2 : 1;
    const int64_t rows = kTileRows * plan->n_tiles;
    plan->row_tiles = (plan->rows + rows - 1) / rows;
    plan->units = B * c.heads * plan->row_tiles;
    // one wave of blocks, or fewer where the keys do not give each a piece
    const int64_t cap = max_pages << c.page_shift;
    const int64_t len = max_len > 0 && max_len < cap ? max_len : cap;
    const int64_t pieces = (len + kPieceKeys - 1) / kPieceKeys;
    int device = 0;
    if (cudaGetDevice(&device) != cudaSuccess) device = 0;
    const int64_t wave = static_cast<int64_t>(sm_count(device)) *
                         (c.head_dim == 64    ? attention_blocks(64, plan->n_tiles)
                          : c.head_dim == 128 ? attention_blocks(128, plan->n_tiles)
                                              : attention_blocks(256, plan->n_tiles));
    plan->shares = plan->units >= wave || pieces >= wave ? wave
                                                         : std::min(wave, plan->units * pieces);
    plan->split = cap > kPieceKeys;
    // rows of the join are counted in 31 bits (so units are, and the product below fits 64),
    // pieces in 32
    if (B * c.heads * plan->rows >= (int64_t{1} << 31) - 4 ||
        plan->units * ((cap + kPieceKeys - 1) / kPieceKeys) >= (int64_t{1} << 32))
        return PQG_ERR_INVALID_ARG;
    plan->workspace = 0;
    if (plan->split && B > 0)
        plan->workspace = plan->shares * 2 * rows * (c.head_dim + 2) * 4 + plan->units * 8;
    return PQG_OK;
}

// Query rows from which the join takes a warp per row rather than a block (32 query and 8 key
// heads of 128, MXFP4; us of the whole call with a block and with a warp, for sequences of up
// to 600, 2000 and 16384 keys: 128 rows 7.5 / 7.2, 7.9 / 8.1, 18.7 / 19.7; 256 rows 8.1 / 7.7,
// 9.1 / 9.2, 26.0 / 26.2; 512 rows 9.9 / 8.9, 13.5 / 12.3, 46.6 / 45.8; 2048 rows 20.7 / 16.3,
// 33.1 / 28.4, 139.5 / 133.7; 64 rows of 131072 keys 36.6 / 42.0).
constexpr int64_t kManyJoins = 512;

template <typename In, int G, int D, int NT>
cudaError_t launch_rows(const AttentionParams &p, const Plan &plan, cudaStream_t stream,
                        int *kernels) {
    *kernels = 1;
    auto kernel = attention_kernel<In, G, D, NT, false>;
    if constexpr (G == 32)
        if (p.q_len > 1u) kernel = attention_kernel<In, G, D, NT, true>;
    const cudaError_t err = launch(kernel, plan.shares, attention_warps(D) * 32, 0, stream, p);
    if (err != cudaSuccess || !plan.split) return err;
    *kernels = 2;
    const int64_t rows = static_cast<int64_t>(p.B) * p.c.heads * p.rows;
    if (rows < kManyJoins)
        return launch(attention_join_kernel<In, G, D, NT, 1>, rows, join_warps(1) * 32, 0,
                      stream, p);
    return launch(attention_join_kernel<In, G, D, NT, 4>, (rows + 3) / 4, join_warps(4) * 32, 0,
                  stream, p);
}

template <typename In, int G, int D>
cudaError_t launch_attention(const AttentionParams &p, const Plan &plan, cudaStream_t stream,
                             int *kernels) {
    if constexpr (D < 256)
        if (plan.n_tiles == 2) return launch_rows<In, G, D, 2>(p, plan, stream, kernels);
    return launch_rows<In, G, D, 1>(p, plan, stream, kernels);
}

template <typename In, int G>
cudaError_t launch_head_dim(const AttentionParams &p, const Plan &plan, cudaStream_t stream,
                            int *kernels) {
    switch (p.c.head_dim) {
        case 64: return launch_attention<In, G, 64>(p, plan, stream, kernels);
        case 128: return launch_attention<In, G, 128>(p, plan, stream, kernels);
        case 256: return launch_attention<In, G, 256>(p, plan, stream, kernels);
    }
    return cudaErrorInvalidValue;
}

}  // namespace
}  // namespace pqg

extern "C" {

int64_t pqg_kv_attention_workspace(const pqg_kv_cache *cache, int64_t max_pages, int64_t B,
                                   int64_t q_len, int64_t q_heads, int64_t max_len) {
    using namespace pqg;
    CacheView c;
    const int st = check_cache(cache, &c);
    if (st != PQG_OK) return st;
    Plan plan;
    const int ps = make_plan(c, max_pages, B, q_len, q_heads, max_len, &plan);
    return ps != PQG_OK ? ps : plan.workspace;
}

int pqg_kv_attention(const pqg_kv_cache *cache, const void *q, int64_t q_stride,
                     const int32_t *page_table, int64_t table_stride, int64_t max_pages,
                     const int32_t *seq_lens, int64_t B, int64_t q_len, int64_t q_heads,
                     float sm_scale, int64_t max_len, void *out, float *lse, void *workspace,
                     int64_t workspace_bytes, int in_dtype, pqg_stream_t stream) {
    using namespace pqg;
    AttentionParams p;
    const int st = check_cache(cache, &p.c);
    if (st != PQG_OK) return st;
    if (in_dtype != PQG_BF16 && in_dtype != PQG_FP16) return PQG_ERR_INVALID_ARG;
    const int ts = check_table(B, table_stride, max_pages);
    if (ts != PQG_OK) return ts;
    Plan plan;
    const int ps = make_plan(p.c, max_pages, B, q_len, q_heads, max_len, &plan);
    if (ps != PQG_OK) return ps;
    const int64_t D = cache->head_dim, row = q_heads * D;
    if (!std::isfinite(sm_scale) || q_stride < row || q_stride > kMaxStride)
        return PQG_ERR_INVALID_ARG;
    if (B == 0) return PQG_OK;
    if (q == nullptr || page_table == nullptr || seq_lens == nullptr || out == nullptr)
        return PQG_ERR_INVALID_ARG;
    if (plan.workspace > 0 && (workspace == nullptr || workspace_bytes < plan.workspace))
        return PQG_ERR_INVALID_ARG;
    if (!aligned(q, 16) || q_stride % 8 != 0 || !aligned(out, 16) || !aligned(lse, 4) ||
        !aligned(page_table, 4) || !aligned(seq_lens, 4) ||
        (plan.workspace > 0 && !aligned(workspace, 16)))
        return PQG_ERR_ALIGNMENT;

    const int64_t T = B * q_len;
    struct Buffer { const void *p; int64_t n; };
    const Buffer reads[] = {{q, ((T - 1) * q_stride + row) * 2},
                            {page_table, ((B - 1) * table_stride + max_pages) * 4},
                            {seq_lens, B * 4}};
    const Buffer writes[] = {{out, T * row * 2}, {lse, lse != nullptr ? T * q_heads * 4 : 0},
                             {workspace, plan.workspace}};
    for (int i = 0; i < 3; ++i) {
        if (writes[i].n == 0) continue;
        if (overlaps_cache(cache, writes[i].p, writes[i].n)) return PQG_ERR_INVALID_ARG;
        for (const Buffer &r : reads)
            if (overlaps(writes[i].p, writes[i].n, r.p, r.n)) return PQG_ERR_INVALID_ARG;
        for (int j = 0; j < i; ++j)
            if (writes[j].n > 0 && overlaps(writes[i].p, writes[i].n, writes[j].p, writes[j].n))
                return PQG_ERR_INVALID_ARG;
    }

    p.q = static_cast<const uint8_t *>(q);
    p.out = static_cast<uint8_t *>(out);
    p.lse = lse;
    p.part = static_cast<float *>(workspace);
    p.stat = nullptr;
    p.joins = nullptr;
    if (plan.workspace > 0) {
        const int64_t places = plan.shares * 2 * kTileRows * plan.n_tiles;
        p.stat = reinterpret_cast<float2 *>(p.part + places * D);
        p.joins = reinterpret_cast<uint2 *>(p.stat + places);
    }
    p.table = page_table;
    p.seq_lens = seq_lens;
    p.q_stride = static_cast<uint64_t>(q_stride);
    p.table_stride = static_cast<uint64_t>(table_stride);
    // a negative scale goes to the queries, so that larger products are larger scores
    p.scale_log2 =
        static_cast<float>(std::fabs(static_cast<double>(sm_scale)) * 1.4426950408889634);
    p.sign = sm_scale < 0.0f ? -1.0f : 1.0f;
    p.max_pages = static_cast<uint32_t>(max_pages);
    p.B = static_cast<uint32_t>(B);
    p.q_len = static_cast<uint32_t>(q_len);
    p.group = static_cast<uint32_t>(q_heads / p.c.heads);
    p.rows = static_cast<uint32_t>(plan.rows);
    p.row_tiles = static_cast<uint32_t>(plan.row_tiles);
    p.shares = static_cast<uint32_t>(plan.shares);
    const bool nv = cache->format == PQG_KV_NVFP4;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    int kernels = 0;
    cudaError_t err;
    if (in_dtype == PQG_BF16)
        err = nv ? launch_head_dim<__nv_bfloat16, 16>(p, plan, s, &kernels)
                 : launch_head_dim<__nv_bfloat16, 32>(p, plan, s, &kernels);
    else
        err = nv ? launch_head_dim<__half, 16>(p, plan, s, &kernels)
                 : launch_head_dim<__half, 32>(p, plan, s, &kernels);
    return launched(err, kernels);
}

}  // extern "C"
