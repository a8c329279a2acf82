// pqg_kv_write and pqg_kv_read: argument checks and launch.
#include "pqg_cache.cuh"
#include "pqg_cache_host.cuh"

namespace pqg {

void segs_divider(uint32_t segs, uint32_t *magic, uint32_t *shift);   // pqg_api.cu
int sm_count(int device);  // cached cudaDevAttrMultiProcessorCount

int check_cache(const pqg_kv_cache *cache, CacheView *view) {
    if (cache == nullptr) return PQG_ERR_INVALID_ARG;
    if (cache->format != PQG_KV_MXFP4 && cache->format != PQG_KV_NVFP4) return PQG_ERR_INVALID_ARG;
    const bool nvfp4 = cache->format == PQG_KV_NVFP4;
    const int P = cache->page_size, D = cache->head_dim;
    if (P <= 0 || D <= 0) return PQG_ERR_INVALID_ARG;
    if (P != 16 && P != 32 && P != 64 && P != 128 && P != 256) return PQG_ERR_UNSUPPORTED;
    if (D != 64 && D != 128 && D != 256) return PQG_ERR_UNSUPPORTED;
    if (cache->kv_heads < 1 || cache->kv_heads > kMaxKvHeads) return PQG_ERR_INVALID_ARG;
    if (cache->num_pages < 1 || cache->num_pages > ((int64_t{1} << 31) - 1) / P)
        return PQG_ERR_INVALID_ARG;
    if (cache->k_codes == nullptr || cache->v_codes == nullptr || cache->k_scales == nullptr ||
        cache->v_scales == nullptr || nvfp4 != (cache->global_scale != nullptr))
        return PQG_ERR_INVALID_ARG;
    if (!aligned(cache->k_codes, 16) || !aligned(cache->v_codes, 16) ||
        !aligned(cache->k_scales, 16) || !aligned(cache->v_scales, 16) ||
        !aligned(cache->global_scale, 4))
        return PQG_ERR_ALIGNMENT;
    view->codes[0] = static_cast<uint8_t *>(cache->k_codes);
    view->codes[1] = static_cast<uint8_t *>(cache->v_codes);
    view->scales[0] = static_cast<uint8_t *>(cache->k_scales);
    view->scales[1] = static_cast<uint8_t *>(cache->v_scales);
    view->gscale = cache->global_scale;
    view->num_pages = static_cast<uint32_t>(cache->num_pages);
    view->heads = static_cast<uint32_t>(cache->kv_heads);
    view->head_dim = static_cast<uint32_t>(D);
    segs_divider(view->heads, &view->heads_magic, &view->heads_shift);
    view->page_shift = 4;
    while ((1 << view->page_shift) < P) ++view->page_shift;
    // the four buffers, and the global scales, lie apart
    const int64_t rows = cache->num_pages * cache->kv_heads * P;
    const int64_t n[5] = {rows * (D / 2), rows * (D / 2), rows * (D / (nvfp4 ? 16 : 32)),
                          rows * (D / (nvfp4 ? 16 : 32)), nvfp4 ? 8 : 0};
    const void *at[5] = {cache->k_codes, cache->v_codes, cache->k_scales, cache->v_scales,
                         cache->global_scale};
    for (int i = 0; i < 5; ++i)
        for (int j = 0; j < i; ++j)
            if (n[i] > 0 && overlaps(at[i], n[i], at[j], n[j])) return PQG_ERR_INVALID_ARG;
    return PQG_OK;
}

bool overlaps_cache(const pqg_kv_cache *cache, const void *p, int64_t bytes) {
    if (p == nullptr || bytes <= 0) return false;
    const int64_t rows = cache->num_pages * cache->kv_heads * cache->page_size;
    const int64_t codes = rows * (cache->head_dim / 2);
    const int64_t scales = rows * (cache->head_dim / (cache->format == PQG_KV_NVFP4 ? 16 : 32));
    return overlaps(p, bytes, cache->k_codes, codes) || overlaps(p, bytes, cache->v_codes, codes) ||
           overlaps(p, bytes, cache->k_scales, scales) ||
           overlaps(p, bytes, cache->v_scales, scales) ||
           (cache->global_scale != nullptr && overlaps(p, bytes, cache->global_scale, 8));
}

}  // namespace pqg


extern "C" {

int pqg_kv_write(const pqg_kv_cache *cache, const void *k, const void *v, const int32_t *slots,
                 int64_t T, int64_t k_stride, int64_t v_stride, int in_dtype,
                 pqg_stream_t stream) {
    using namespace pqg;
    WriteParams p;
    const int st = check_cache(cache, &p.c);
    if (st != PQG_OK) return st;
    if (in_dtype != PQG_BF16 && in_dtype != PQG_FP16) return PQG_ERR_INVALID_ARG;
    const int64_t row = static_cast<int64_t>(cache->kv_heads) * cache->head_dim;
    if (T < 0 || T >= (int64_t{1} << 31) || k_stride < row || v_stride < row ||
        k_stride > kMaxStride || v_stride > kMaxStride)
        return PQG_ERR_INVALID_ARG;
    const uint32_t tokens_per_warp = 32u / (p.c.head_dim / 16u);
    const int64_t warps = (T + tokens_per_warp - 1) / tokens_per_warp * cache->kv_heads;
    const int64_t blocks = (warps * 32 + kCacheThreads - 1) / kCacheThreads;
    if (warps > (int64_t{1} << 31) - kCacheThreads) return PQG_ERR_INVALID_ARG;
    if (T == 0) return PQG_OK;
    if (k == nullptr || v == nullptr || slots == nullptr) return PQG_ERR_INVALID_ARG;
    if (!aligned(k, 32) || !aligned(v, 32) || !aligned(slots, 4) || k_stride % 16 != 0 ||
        v_stride % 16 != 0)
        return PQG_ERR_ALIGNMENT;
    if (overlaps_cache(cache, k, ((T - 1) * k_stride + row) * 2) ||
        overlaps_cache(cache, v, ((T - 1) * v_stride + row) * 2) ||
        overlaps_cache(cache, slots, T * 4))
        return PQG_ERR_INVALID_ARG;
    p.src[0] = static_cast<const uint8_t *>(k);
    p.src[1] = static_cast<const uint8_t *>(v);
    p.stride[0] = static_cast<uint64_t>(k_stride) * 2u;
    p.stride[1] = static_cast<uint64_t>(v_stride) * 2u;
    p.slots = slots;
    p.T = static_cast<uint32_t>(T);
    const bool nv = cache->format == PQG_KV_NVFP4, bf = in_dtype == PQG_BF16;
    auto kernel = bf ? (nv ? kv_write_kernel<__nv_bfloat16, 16> : kv_write_kernel<__nv_bfloat16, 32>)
                     : (nv ? kv_write_kernel<__half, 16> : kv_write_kernel<__half, 32>);
    return launched(launch(kernel, blocks, kCacheThreads, 0,
                           reinterpret_cast<cudaStream_t>(stream), p), 1);
}

int pqg_kv_read(const pqg_kv_cache *cache, const int32_t *page_table, int64_t table_stride,
                int64_t max_pages, const int32_t *indptr, int64_t B, void *k_out, void *v_out,
                int64_t M, int out_dtype, pqg_stream_t stream) {
    using namespace pqg;
    ReadParams p;
    const int st = check_cache(cache, &p.c);
    if (st != PQG_OK) return st;
    if (out_dtype != PQG_BF16 && out_dtype != PQG_FP16) return PQG_ERR_INVALID_ARG;
    const int ts = check_table(B, table_stride, max_pages);
    if (ts != PQG_OK) return ts;
    const int64_t row = static_cast<int64_t>(cache->kv_heads) * cache->head_dim;
    if (M < 0 || M >= (int64_t{1} << 31)) return PQG_ERR_INVALID_ARG;
    // Four rows a thread where that still gives the SMs two waves of 2048 threads (MXFP4 and
    // NVFP4, 8 heads of 128, us with one and with four: 3350 tokens 4.1 / 5.1 and 4.3 / 5.8,
    // 21500 20.6 / 20.5 and 21.6 / 21.7, 46300 40.4 / 40.7 and 42.4 / 42.0, 70000 60.1 / 59.6
    // and 63.2 / 61.0).
    int device = 0;
    if (cudaGetDevice(&device) != cudaSuccess) device = 0;
    const bool many = M * row / 16 >= int64_t{4} * 2 * 2048 * sm_count(device);
    const int64_t rowheads = (M + (many ? 3 : 0)) / (many ? 4 : 1) * cache->kv_heads;
    const int64_t blocks = (rowheads * (cache->head_dim / 16) + kCacheThreads - 1) / kCacheThreads;
    if (rowheads > (int64_t{1} << 31) - kCacheThreads) return PQG_ERR_INVALID_ARG;
    if (M == 0 || B == 0) return PQG_OK;
    if (page_table == nullptr || indptr == nullptr || k_out == nullptr || v_out == nullptr)
        return PQG_ERR_INVALID_ARG;
    if (!aligned(page_table, 4) || !aligned(indptr, 4) || !aligned(k_out, 32) ||
        !aligned(v_out, 32))
        return PQG_ERR_ALIGNMENT;
    const int64_t bytes = M * row * 2, table = ((B - 1) * table_stride + max_pages) * 4;
    for (void *out : {k_out, v_out})
        if (overlaps_cache(cache, out, bytes) || overlaps(out, bytes, page_table, table) ||
            overlaps(out, bytes, indptr, (B + 1) * 4))
            return PQG_ERR_INVALID_ARG;
    if (overlaps(k_out, bytes, v_out, bytes)) return PQG_ERR_INVALID_ARG;
    p.table = page_table;
    p.indptr = indptr;
    p.dst[0] = static_cast<uint8_t *>(k_out);
    p.dst[1] = static_cast<uint8_t *>(v_out);
    p.table_stride = static_cast<uint64_t>(table_stride);
    p.max_pages = static_cast<uint32_t>(max_pages);
    p.B = static_cast<uint32_t>(B);
    p.M = static_cast<uint32_t>(M);
    const bool nv = cache->format == PQG_KV_NVFP4, bf = out_dtype == PQG_BF16;
    auto kernel = many ? (bf ? (nv ? kv_read_kernel<__nv_bfloat16, 16, 4>
                                   : kv_read_kernel<__nv_bfloat16, 32, 4>)
                             : (nv ? kv_read_kernel<__half, 16, 4> : kv_read_kernel<__half, 32, 4>))
                       : (bf ? (nv ? kv_read_kernel<__nv_bfloat16, 16, 1>
                                   : kv_read_kernel<__nv_bfloat16, 32, 1>)
                             : (nv ? kv_read_kernel<__half, 16, 1>
                                    : kv_read_kernel<__half, 32, 1>));
    return launched(launch(kernel, blocks, kCacheThreads, 0,
                           reinterpret_cast<cudaStream_t>(stream), p), 1);
}

}  // extern "C"
