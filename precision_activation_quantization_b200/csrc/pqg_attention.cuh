// Attention over the paged 4-bit cache, for sm_100a.
//
// The keys of a sequence are cut into chunks; a block computes one chunk for the
// query rows of one key/value head (row r = t * group + h: token t, query head h
// of the head's group) with a running maximum and sum, and leaves (max, sum,
// weighted values) in the workspace; a second kernel joins the chunks in their
// order.  A sequence that fits in one chunk is written out at once.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "pqg_cache.cuh"

namespace pqg {

struct AttentionParams {
    CacheView c;
    const uint8_t *q;
    uint8_t *out;
    float *lse;                // or null
    float *part;               // [B][heads][chunks][rows][D] weighted values, then
    float2 *stat;              // [B][heads][chunks][rows] (max in log2 units, sum)
    const int32_t *table;
    const int32_t *seq_lens;
    uint64_t q_stride;         // elements between tokens
    uint64_t table_stride;
    float scale_log2;          // sm_scale * log2(e)
    uint32_t max_pages;
    uint32_t B;
    uint32_t q_len;
    uint32_t group;            // query heads per key/value head
    uint32_t rows;             // q_len * group
    uint32_t row_tiles;
    uint32_t chunk;            // keys per chunk
    uint32_t chunks;           // chunks a sequence is dealt to (it may have more keys: they wrap)
};

constexpr float kLn2 = 0.6931471805599453f;
constexpr float kNoMax = -1e30f;   // the running maximum before any key

// Keys of sequence b that the cache can hold.
__device__ __forceinline__ uint32_t sequence_length(const AttentionParams &p, uint32_t b) {
    const uint64_t cap = static_cast<uint64_t>(p.max_pages) << p.c.page_shift;
    const int n = max(__ldg(p.seq_lens + b), 0);
    return static_cast<uint64_t>(n) < cap ? static_cast<uint32_t>(n) : static_cast<uint32_t>(cap);
}
// Chunks that hold keys (0 or 1: the block writes the result itself).
__device__ __forceinline__ uint32_t used_chunks(const AttentionParams &p, uint32_t n) {
    return min((n + p.chunk - 1u) / p.chunk, p.chunks);
}

template <typename T>
__device__ __forceinline__ float to_float(T v) {
    if constexpr (std::is_same<T, __nv_bfloat16>::value) return __bfloat162float(v);
    else return __half2float(v);
}

// An E2M1 code's value: its exponent and mantissa bits are the middle bits of a
// binary16 number that is 2^14 times smaller (code 1, a half, is subnormal there
// too).
__device__ __forceinline__ float e2m1_value(uint32_t c) {
    const uint16_t h = static_cast<uint16_t>(((c & 8u) << 12) | ((c & 7u) << 9));
    return __half2float(__ushort_as_half(h)) * 16384.0f;
}

constexpr int kAttentionThreads = 128;

// One warp per query row; a lane holds D / 32 elements.
template <typename In, int G, int D>
__global__ void __launch_bounds__(kAttentionThreads)
    attention_kernel(const __grid_constant__ AttentionParams p) {
    constexpr int E = D / 32;
    wait_for_producer();
    const uint32_t lane = threadIdx.x & 31u, warp = threadIdx.x >> 5;
    uint32_t at = blockIdx.x;
    const uint32_t chunk = at % p.chunks;
    at /= p.chunks;
    const uint32_t tile = at % p.row_tiles;
    at /= p.row_tiles;
    const uint32_t head = at % p.c.heads, b = at / p.c.heads;
    const uint32_t r = tile * (kAttentionThreads / 32) + warp;
    const uint32_t n = sequence_length(p, b);
    const uint32_t used = used_chunks(p, n);
    if (r < p.rows && (chunk < used || (chunk == 0u && used == 0u))) {
        const uint32_t t = r / p.group, qh = head * p.group + (r - t * p.group);
        const uint64_t token = static_cast<uint64_t>(b) * p.q_len + t;
        const In *q = reinterpret_cast<const In *>(p.q) + token * p.q_stride +
                      static_cast<uint64_t>(qh) * D + lane * E;
        float qv[E], acc[E];
#pragma unroll
        for (int i = 0; i < E; ++i) {
            qv[i] = to_float(q[i]);
            acc[i] = 0.0f;
        }
        const int seen = static_cast<int>(n) - static_cast<int>(p.q_len - 1u - t);
        const float inv_k = G == 16 ? __frcp_rn(__ldg(p.c.gscale)) : 1.0f;
        const float inv_v = G == 16 ? __frcp_rn(__ldg(p.c.gscale + 1)) : 1.0f;
        float m = kNoMax, l = 0.0f;
        for (uint64_t first = static_cast<uint64_t>(chunk) * p.chunk;
             static_cast<int64_t>(first) < seen;
             first += static_cast<uint64_t>(p.chunk) * p.chunks) {
            const int last = static_cast<int>(min(first + p.chunk, static_cast<uint64_t>(seen)));
            for (int j = static_cast<int>(first); j < last; ++j) {
                const int page = __ldg(p.table + static_cast<uint64_t>(b) * p.table_stride +
                                       (static_cast<uint32_t>(j) >> p.c.page_shift));
                if (page < 0 || static_cast<uint32_t>(page) >= p.c.num_pages) continue;
                const uint32_t off = static_cast<uint32_t>(j) & ((1u << p.c.page_shift) - 1u);
                float kv[2][E];
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const uint8_t *code =
                        p.c.codes[x] + code_offset(p.c, page, head, off) + lane * E / 2;
                    const uint32_t e =
                        p.c.scales[x][scale_offset<G>(p.c, page, head, lane * E / G, off)];
                    const float s = G == 16 ? e4m3_code_value(e & 0x7Fu) : ue8m0_value(e);
#pragma unroll
                    for (int i = 0; i < E; i += 2) {
                        const float2 f = make_float2(e2m1_value(code[i / 2] & 15u),
                                                     e2m1_value(code[i / 2] >> 4));
                        kv[x][i] = f.x * s;
                        kv[x][i + 1] = f.y * s;
                    }
                }
                float s = 0.0f;
#pragma unroll
                for (int i = 0; i < E; ++i) s = fmaf(qv[i], kv[0][i], s);
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
                s *= inv_k * p.scale_log2;
                const float m2 = fmaxf(m, s);
                const float f = exp2f(m - m2), w = exp2f(s - m2);
                l = l * f + w;
#pragma unroll
                for (int i = 0; i < E; ++i) acc[i] = acc[i] * f + w * kv[1][i];
                m = m2;
            }
        }
        if (used <= 1u) {
            const float norm = l > 0.0f ? inv_v / l : 0.0f;
            uint8_t *dst = p.out + ((token * p.c.heads * p.group + qh) * D + lane * E) * 2u;
#pragma unroll
            for (int i = 0; i < E; i += 2)
                *reinterpret_cast<uint32_t *>(dst + 2 * i) =
                    narrow2<In>(acc[i] * norm, acc[i + 1] * norm);
            if (lane == 0 && p.lse != nullptr)
                p.lse[token * p.c.heads * p.group + qh] =
                    l > 0.0f ? (m + log2f(l)) * kLn2 : -INFINITY;
        } else {
            const uint64_t slot =
                ((static_cast<uint64_t>(b) * p.c.heads + head) * p.chunks + chunk) * p.rows + r;
#pragma unroll
            for (int i = 0; i < E; ++i) p.part[slot * D + lane * E + i] = acc[i];
            if (lane == 0) p.stat[slot] = make_float2(m, l);
        }
    }
    release_dependents();
}

// Joins the chunks of one (sequence, query row): a warp per row.
template <typename In, int G, int D>
__global__ void __launch_bounds__(kAttentionThreads)
    attention_join_kernel(const __grid_constant__ AttentionParams p) {
    constexpr int E = D / 32;
    wait_for_producer();
    const uint32_t lane = threadIdx.x & 31u;
    const uint64_t unit =
        static_cast<uint64_t>(blockIdx.x) * (kAttentionThreads / 32) + (threadIdx.x >> 5);
    const uint64_t bh = unit / p.rows;
    const uint32_t r = static_cast<uint32_t>(unit - bh * p.rows);
    const uint64_t b = bh / p.c.heads;
    const uint32_t head = static_cast<uint32_t>(bh - b * p.c.heads);
    if (b < p.B) {
        const uint32_t used = used_chunks(p, sequence_length(p, static_cast<uint32_t>(b)));
        if (used > 1u) {
            const uint32_t t = r / p.group, qh = head * p.group + (r - t * p.group);
            const uint64_t row = (b * p.q_len + t) * p.c.heads * p.group + qh;
            const float inv_v = G == 16 ? __frcp_rn(__ldg(p.c.gscale + 1)) : 1.0f;
            float m = kNoMax, l = 0.0f, acc[E];
#pragma unroll
            for (int i = 0; i < E; ++i) acc[i] = 0.0f;
            for (uint32_t c = 0; c < used; ++c) m = fmaxf(m, p.stat[(bh * p.chunks + c) * p.rows + r].x);
            for (uint32_t c = 0; c < used; ++c) {
                const uint64_t slot = (bh * p.chunks + c) * p.rows + r;
                const float2 st = p.stat[slot];
                const float f = exp2f(st.x - m);
                l = fmaf(st.y, f, l);
#pragma unroll
                for (int i = 0; i < E; ++i) acc[i] = fmaf(p.part[slot * D + lane * E + i], f, acc[i]);
            }
            const float norm = l > 0.0f ? inv_v / l : 0.0f;
            uint8_t *dst = p.out + (row * D + lane * E) * 2u;
#pragma unroll
            for (int i = 0; i < E; i += 2)
                *reinterpret_cast<uint32_t *>(dst + 2 * i) =
                    narrow2<In>(acc[i] * norm, acc[i + 1] * norm);
            if (lane == 0 && p.lse != nullptr)
                p.lse[row] = l > 0.0f ? (m + log2f(l)) * kLn2 : -INFINITY;
        }
    }
    release_dependents();
}

}  // namespace pqg
