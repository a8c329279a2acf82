// Host-side checks shared by the cache's entry points (defined in pqg_cache.cu).
#pragma once

#include "pqg.h"
#include "pqg_cache.cuh"
#include "pqg_host.cuh"

namespace pqg {

constexpr int64_t kMaxKvHeads = 1024;
constexpr int64_t kMaxStride = int64_t{1} << 30;      // elements between tokens or table rows
constexpr int64_t kMaxSequences = int64_t{1} << 20;
constexpr int64_t kMaxQueryTokens = 1024;             // q_len
constexpr int64_t kMaxQueryHeads = 16384;

// Checks the cache's description and fills in the kernels' view of it.
int check_cache(const pqg_kv_cache *cache, CacheView *view);

// Whether `bytes` bytes at p meet any of the cache's buffers.
bool overlaps_cache(const pqg_kv_cache *cache, const void *p, int64_t bytes);

// A page table's shape: B rows of max_pages entries, table_stride apart.
inline int check_table(int64_t B, int64_t table_stride, int64_t max_pages) {
    if (B < 0 || B > kMaxSequences || max_pages < 1 || table_stride < max_pages ||
        table_stride > kMaxStride)
        return PQG_ERR_INVALID_ARG;
    return PQG_OK;
}

}  // namespace pqg
