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

constexpr int kAttentionWarps = 4;
constexpr int kAttentionThreads = kAttentionWarps * 32;
constexpr int kTileKeys = 32;      // keys a warp takes at a time
constexpr int kTileRows = 8;       // query rows of one matrix product (its N)

// ---------------------------------------------------------------------------
// Matrix fragments
// ---------------------------------------------------------------------------

// c += a b: a 16 x 16, b 16 x 8 in binary16, c in fp32.
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The transpose of an 8 x 8 binary16 matrix held two columns of a row per lane.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}

// The eight E2M1 codes of a word as binary16 pairs, byte j in h[j].
__device__ __forceinline__ void decode_e2m1x8(uint32_t w, uint32_t (&h)[4]) {
    asm("{\n\t.reg .b8 p, q, s, t;\n\t"
        "mov.b32 {p, q, s, t}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, p;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, q;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, s;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, t;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3]) : "r"(w));
}
// The four E4M3 bytes of a word as two binary16 pairs.
__device__ __forceinline__ void decode_e4m3x4(uint32_t w, uint32_t (&h)[2]) {
    asm("{\n\t.reg .b16 p, q;\n\t"
        "mov.b32 {p, q}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, p;\n\t"
        "cvt.rn.f16x2.e4m3x2 %1, q;\n\t}"
        : "=r"(h[0]), "=r"(h[1]) : "r"(w));
}
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// N consecutive words of read-only global memory, N in {1, 2, 4, 8}.
template <int N>
__device__ __forceinline__ void load_words(const uint8_t *p, uint32_t (&w)[N]) {
    if constexpr (N == 1) {
        asm volatile("ld.global.nc.b32 %0, [%1];" : "=r"(w[0]) : "l"(p));
    } else if constexpr (N == 2) {
        asm volatile("ld.global.nc.v2.b32 {%0,%1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "l"(p));
    } else {
#pragma unroll
        for (int i = 0; i < N; i += 4)
            asm volatile("ld.global.nc.v4.b32 {%0,%1,%2,%3}, [%4];"
                         : "=r"(w[i]), "=r"(w[i + 1]), "=r"(w[i + 2]), "=r"(w[i + 3])
                         : "l"(p + 4 * i));
    }
}

// The largest of the four bytes of each word.
template <int N>
__device__ __forceinline__ uint32_t max_byte(const uint32_t (&w)[N]) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < N; ++i)
        m = __vimax3_u16x2(m, w[i] & 0x00FF00FFu, (w[i] >> 8) & 0x00FF00FFu);
    return max(m & 0xFFFFu, m >> 16);
}

// 2^(e - ref + 12) in binary16 for two UE8M0 bytes (in bits 0-7 and 16-23) that
// are at most ref; 0 where the power is below 2^-14.
__device__ __forceinline__ uint32_t relative_power2(uint32_t e2, uint32_t ref) {
    const uint32_t shift = (27u - ref) & 0xFFFFu;
    return __viaddmax_s16x2(e2, shift | (shift << 16), 0u) << 10;
}

// A word's bytes [from, from + 4) of a tile, those at or past `end` zeroed.
__device__ __forceinline__ uint32_t keep_bytes(uint32_t w, int from, int end) {
    const int n = min(max(end - from, 0), 4);
    return n == 4 ? w : w & ((1u << (8 * n)) - 1u);
}

// ---------------------------------------------------------------------------
// One chunk
// ---------------------------------------------------------------------------
//
// Mathematics.  With c_jd the 4-bit code of key j, s_jg its scale and q the
// query, score_j = sum_g sum_{d in g} q_d (c_jd s_jg); out = sum_j p_j (c_jd
// s_jg) / sum_j p_j.  Both products run on the tensor cores in binary16 with
// fp32 sums, and their operands are exact: a code has 2 significant bits and an
// E4M3 scale 4, so their product is a binary16 number.  A UE8M0 scale has a
// wider range than binary16, so it is taken relative to the largest scale of the
// tile's keys, or, for the values, the largest so far of the lane's elements
// (12 binades above 1; scales 2^-26 below the largest count as zero).  A query
// row is scaled by a power of two into [2^14, 2^15).  Only the weights p are
// rounded, to binary16's 11 bits, at 2^7 times their size so that small ones keep
// their bits.
//
// Layout.  A warp takes 32 keys at a time; tokens are M of the first product, so
// that 8 query rows (N) cost no more tensor work than one.  The order of a sum's
// terms is free, so every lane reads what is contiguous in the cache: of the
// keys, D / 4 neighbouring elements of keys 4 gid .. 4 gid + 3 (gid = lane / 4,
// tig = lane % 4); of the values, D / 8 neighbouring elements of keys 8 tig ..
// 8 tig + 7; and one word (two) of scales of 4 (8) neighbouring keys.  The second
// product wants pairs of keys in a register while the cache holds pairs of
// elements: two words of two keys are interleaved by nibbles, two operations for
// eight pairs.  The weights change from the first product's layout to the
// second's by an 8 x 8 transpose.  No shared memory until the warps of a block
// join: loads go to registers, those of the next tile are issued as soon as this
// tile's registers are free.
//
// The running maximum moves only when a score exceeds it by 2^8 (binary16 has
// the room), so most tiles neither reduce it across lanes nor rescale.

// A row of the first product's M, i.e. a lane's token of the tile:
//   m-tile mt, rows gid and gid + 8  ->  tokens 4 gid + 2 mt and 4 gid + 2 mt + 1.
template <typename In, int G, int D, int NT>
__global__ void __launch_bounds__(kAttentionThreads)
    attention_kernel(const __grid_constant__ AttentionParams p) {
    constexpr int KW = D / 32;                 // words of a lane's part of a key
    constexpr int VW = D / 64;                 // words of a lane's part of a value
    constexpr int KG = D / 4 > G ? D / 4 / G : 1;   // groups a lane's part spans
    constexpr int VG = D / 8 > G ? D / 8 / G : 1;
    constexpr int MT = D / 16;                 // m-tiles of the second product
    constexpr int R = NT * kTileRows;          // query rows of the block
    constexpr int kPad = D + 4;
    __shared__ float joined[kAttentionWarps][R][kPad];
    __shared__ float stats[kAttentionWarps][R][2];

    wait_for_producer();
    const uint32_t lane = threadIdx.x & 31u, warp = threadIdx.x >> 5;
    const uint32_t gid = lane >> 2, tig = lane & 3u;
    uint32_t at = blockIdx.x;
    const uint32_t tile = at % p.row_tiles;
    at /= p.row_tiles;
    const uint32_t chunk = at % p.chunks;
    at /= p.chunks;
    const uint32_t head = at % p.c.heads, b = at / p.c.heads;
    const uint32_t n = sequence_length(p, b);
    const uint32_t used = used_chunks(p, n);
    if (chunk >= max(used, 1u)) {
        release_dependents();
        return;
    }

    // -- the query rows, normalised, as the first product's B operand -----------
    uint32_t q[NT][MT][2];
    float head_scale[NT][2];                   // of this lane's columns 2 tig, 2 tig + 1
    int limit[NT][2];                          // keys they see
    const float inv_k = G == 16 ? __frcp_rn(__ldg(p.c.gscale)) : 1.0f;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const uint32_t r = tile * R + nt * kTileRows + gid;
        uint32_t raw[D / 8];
#pragma unroll
        for (int i = 0; i < D / 8; ++i) raw[i] = 0u;
        if (r < p.rows) {
            const uint32_t t = r / p.group, qh = head * p.group + (r - t * p.group);
            const uint64_t token = static_cast<uint64_t>(b) * p.q_len + t;
            load_words(p.q + (token * p.q_stride + static_cast<uint64_t>(qh) * D + tig * (D / 4)) * 2u,
                       raw);
        }
        float top = 0.0f;
#pragma unroll
        for (int i = 0; i < D / 8; ++i) {
            float lo, hi;
            widen2<In>(raw[i], lo, hi);
            top = fmaxf(top, fmaxf(fabsf(lo), fabsf(hi)));
        }
        top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
        // 2^(14 - exponent), at most 2^126 (so that its reciprocal is normal)
        const int e = static_cast<int>(__float_as_uint(top) >> 23);
        const int up = min(max(268 - e, 14), 253);
        const float grow = __uint_as_float(static_cast<uint32_t>(up) << 23);
        const float shrink = __uint_as_float(static_cast<uint32_t>(254 - up) << 23);
#pragma unroll
        for (int i = 0; i < MT; ++i) {
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                float lo, hi;
                widen2<In>(raw[2 * i + k], lo, hi);
                q[nt][i][k] = narrow2<__half>(lo * grow, hi * grow);
            }
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const uint32_t col = 2u * tig + k;
            head_scale[nt][k] = __shfl_sync(0xFFFFFFFFu, shrink, col * 4u) * (p.scale_log2 * inv_k);
            const uint32_t rc = tile * R + nt * kTileRows + col;
            limit[nt][k] = static_cast<int>(n) - static_cast<int>(p.q_len - 1u) +
                           static_cast<int>(min(rc / p.group, p.q_len - 1u));
        }
    }

    float acc[MT][NT][4], m[NT][2], l[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            m[nt][k] = kNoMax;
            l[nt][k] = 0.0f;
        }
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int k = 0; k < 4; ++k) acc[i][nt][k] = 0.0f;
    }
    uint32_t vref = 0u;                        // MXFP4: the values' reference exponent

    // -- where a lane reads ------------------------------------------------------
    const uint32_t page_mask = (1u << p.c.page_shift) - 1u;
    const uint32_t code_page = (p.c.heads << p.c.page_shift) * (D / 2);
    const uint32_t scale_page = (p.c.heads << p.c.page_shift) * (D / G);
    const uint32_t k_first = 4u * gid, v_first = 8u * tig;   // this lane's tokens of a tile
    const uint8_t *k_code = p.c.codes[0] + (static_cast<uint64_t>(head) << p.c.page_shift) * (D / 2) +
                            tig * (D / 8);
    const uint8_t *v_code = p.c.codes[1] + (static_cast<uint64_t>(head) << p.c.page_shift) * (D / 2) +
                            gid * (D / 16);
    const uint8_t *k_scale = p.c.scales[0] + ((static_cast<uint64_t>(head) * (D / G) +
                                               tig * (D / 4) / G) << p.c.page_shift);
    const uint8_t *v_scale = p.c.scales[1] + ((static_cast<uint64_t>(head) * (D / G) +
                                               gid * (D / 8) / G) << p.c.page_shift);
    const int32_t *table = p.table + static_cast<uint64_t>(b) * p.table_stride;

    // pages of this lane's keys and of its values in the tile at j (-1: none)
    auto pages = [&](uint32_t j, int &kp, int &vp) {
        kp = vp = -1;
        if (j + (k_first & 16u) < n) kp = __ldg(table + ((j + (k_first & 16u)) >> p.c.page_shift));
        if (j + (v_first & 16u) < n) vp = __ldg(table + ((j + (v_first & 16u)) >> p.c.page_shift));
        if (static_cast<uint32_t>(kp) >= p.c.num_pages) kp = -1;
        if (static_cast<uint32_t>(vp) >= p.c.num_pages) vp = -1;
    };
    uint32_t kraw[4][KW], vraw[8][VW], ksc[KG], vsc[VG][2];
    auto load_keys = [&](uint32_t j, int page) {
        const uint64_t pg = static_cast<uint32_t>(max(page, 0));
        const uint32_t off = (j + k_first) & page_mask;
        const uint8_t *c = k_code + pg * code_page + off * (D / 2);
#pragma unroll
        for (int x = 0; x < 4; ++x) load_words(c + x * (D / 2), kraw[x]);
        const uint8_t *s = k_scale + pg * scale_page + off;
#pragma unroll
        for (int g = 0; g < KG; ++g) {
            uint32_t w[1];
            load_words(s + (g << p.c.page_shift), w);
            ksc[g] = w[0];
        }
    };
    auto load_values = [&](uint32_t j, int page) {
        const uint64_t pg = static_cast<uint32_t>(max(page, 0));
        const uint32_t off = (j + v_first) & page_mask;
        const uint8_t *c = v_code + pg * code_page + off * (D / 2);
#pragma unroll
        for (int x = 0; x < 8; ++x) load_words(c + x * (D / 2), vraw[x]);
        const uint8_t *s = v_scale + pg * scale_page + off;
#pragma unroll
        for (int g = 0; g < VG; ++g) load_words(s + (g << p.c.page_shift), vsc[g]);
    };

    // -- the warp's tiles: every 4th of the chunk, and of the chunks that wrap ----
    const uint64_t lap = static_cast<uint64_t>(p.chunk) * p.chunks;
    uint64_t first = static_cast<uint64_t>(chunk) * p.chunk;
    uint32_t in_chunk = warp * kTileKeys;
    auto next_tile = [&]() {                   // the tile after this one
        in_chunk += kAttentionWarps * kTileKeys;
        if (in_chunk >= p.chunk) {
            in_chunk = warp * kTileKeys;
            first += lap;
        }
    };
    uint64_t j64 = first + in_chunk;
    int kp = -1, vp = -1, kp_next = -1, vp_next = -1;
    bool more = in_chunk < p.chunk && j64 < n;
    if (more) {
        pages(static_cast<uint32_t>(j64), kp, vp);
        load_keys(static_cast<uint32_t>(j64), kp);
        load_values(static_cast<uint32_t>(j64), vp);
    }
    while (more) {
        const uint32_t j = static_cast<uint32_t>(j64);
        next_tile();
        j64 = first + in_chunk;
        more = j64 < n;
        if (more) pages(static_cast<uint32_t>(j64), kp_next, vp_next);

        // a tile some of whose keys some row does not see (warp-uniform)
        const bool edge = static_cast<int>(j + kTileKeys) > static_cast<int>(n - (p.q_len - 1u)) ||
                          __any_sync(0xFFFFFFFFu, kp < 0);
        const int live = static_cast<int>(n - j);          // tokens of the tile in the sequence
        const int k_end = kp < 0 ? 0 : live, v_end = vp < 0 ? 0 : live;
        if (edge) {                            // scales of keys that are not there may be anything
#pragma unroll
            for (int g = 0; g < KG; ++g) ksc[g] = keep_bytes(ksc[g], k_first, k_end);
#pragma unroll
            for (int g = 0; g < VG; ++g) {
                vsc[g][0] = keep_bytes(vsc[g][0], v_first, v_end);
                vsc[g][1] = keep_bytes(vsc[g][1], v_first + 4, v_end);
            }
        }

        // -- scores: 32 tokens x rows ----------------------------------------------
        float tile_scale = 1.0f;
        uint32_t ks[KG][4];                    // a token's scale, twice
        if constexpr (G == 16) {
#pragma unroll
            for (int g = 0; g < KG; ++g) {
                uint32_t h[2];
                decode_e4m3x4(ksc[g], h);
#pragma unroll
                for (int x = 0; x < 4; ++x) ks[g][x] = __byte_perm(h[x >> 1], 0, x & 1 ? 0x3232 : 0x1010);
            }
        } else {
            const uint32_t kref = __reduce_max_sync(0xFFFFFFFFu, max_byte(ksc));
#pragma unroll
            for (int g = 0; g < KG; ++g) {
                const uint32_t even = relative_power2(ksc[g] & 0x00FF00FFu, kref);
                const uint32_t odd = relative_power2((ksc[g] >> 8) & 0x00FF00FFu, kref);
#pragma unroll
                for (int x = 0; x < 4; ++x)
                    ks[g][x] = __byte_perm(x & 1 ? odd : even, 0, x & 2 ? 0x3232 : 0x1010);
            }
            // 2^(kref - 127 - 12); below 2^-126 the scores are nothing
            tile_scale = kref > 12u ? __uint_as_float((kref - 12u) << 23) : 0.0f;
        }
        float c[2][NT][4];
#pragma unroll
        for (int mt = 0; mt < 2; ++mt)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int k = 0; k < 4; ++k) c[mt][nt][k] = 0.0f;
#pragma unroll
        for (int w = 0; w < KW; ++w) {
#pragma unroll
            for (int mt = 0; mt < 2; ++mt) {
                uint32_t a[4], a8[4];
                decode_e2m1x8(kraw[2 * mt][w], a);
                decode_e2m1x8(kraw[2 * mt + 1][w], a8);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    a[i] = hmul2(a[i], ks[8 * w / G][2 * mt]);
                    a8[i] = hmul2(a8[i], ks[8 * w / G][2 * mt + 1]);
                }
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    mma16816(c[mt][nt], a[0], a8[0], a[1], a8[1], q[nt][2 * w][0], q[nt][2 * w][1]);
                    mma16816(c[mt][nt], a[2], a8[2], a[3], a8[3], q[nt][2 * w + 1][0],
                             q[nt][2 * w + 1][1]);
                }
            }
        }
        if (more) load_keys(static_cast<uint32_t>(j64), kp_next);

        // -- weights ------------------------------------------------------------------
        uint32_t weights[NT][4];               // B operand: [2 * k-step + half]
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const float f[2] = {head_scale[nt][0] * tile_scale, head_scale[nt][1] * tile_scale};
            float s[4][2];                     // [token][column]
#pragma unroll
            for (int x = 0; x < 4; ++x)
#pragma unroll
                for (int k = 0; k < 2; ++k) s[x][k] = c[x >> 1][nt][2 * (x & 1) + k] * f[k];
            if (edge) {
#pragma unroll
                for (int x = 0; x < 4; ++x)
#pragma unroll
                    for (int k = 0; k < 2; ++k)
                        if (kp < 0 || static_cast<int>(j + k_first + x) >= limit[nt][k])
                            s[x][k] = -INFINITY;
            }
            float top[2];
#pragma unroll
            for (int k = 0; k < 2; ++k)
                top[k] = fmaxf(fmaxf(s[0][k], s[1][k]), fmaxf(s[2][k], s[3][k]));
            if (__any_sync(0xFFFFFFFFu, top[0] > m[nt][0] + 8.0f || top[1] > m[nt][1] + 8.0f)) {
#pragma unroll
                for (int k = 0; k < 2; ++k) {
#pragma unroll
                    for (int o = 4; o < 32; o <<= 1)
                        top[k] = fmaxf(top[k], __shfl_xor_sync(0xFFFFFFFFu, top[k], o));
                    const float next = fmaxf(m[nt][k], top[k]);
                    const float fade = ex2_approx(m[nt][k] - next);
                    m[nt][k] = next;
                    l[nt][k] *= fade;
#pragma unroll
                    for (int i = 0; i < MT; ++i) {
                        acc[i][nt][k] *= fade;
                        acc[i][nt][k + 2] *= fade;
                    }
                }
            }
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const float w0 = ex2_approx(s[x][0] - (m[nt][0] - 7.0f));
                const float w1 = ex2_approx(s[x][1] - (m[nt][1] - 7.0f));
                l[nt][0] += w0;
                l[nt][1] += w1;
                weights[nt][x] = transpose8x8(narrow2<__half>(w0, w1));
            }
        }

        // -- weighted values ------------------------------------------------------------
        uint32_t vs[VG][4];                    // scales of tokens x and x + 4 of this lane's 8
        if constexpr (G == 16) {
#pragma unroll
            for (int g = 0; g < VG; ++g) {
                uint32_t h[2];
                decode_e4m3x4(__byte_perm(vsc[g][0], vsc[g][1], 0x5140), h);
                vs[g][0] = h[0];
                vs[g][1] = h[1];
                decode_e4m3x4(__byte_perm(vsc[g][0], vsc[g][1], 0x7362), h);
                vs[g][2] = h[0];
                vs[g][3] = h[1];
            }
        } else {
            static_assert(G == 16 || VG == 1, "one reference exponent per lane");
            uint32_t top = max_byte(vsc[0]);
            top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
            top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
            if (__any_sync(0xFFFFFFFFu, top > vref)) {
                const uint32_t next = max(vref, top);
                const float fade = ex2_approx(-static_cast<float>(next - vref));
                vref = next;
#pragma unroll
                for (int i = 0; i < MT; ++i)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int k = 0; k < 4; ++k) acc[i][nt][k] *= fade;
            }
#pragma unroll
            for (int x = 0; x < 4; ++x)
                vs[0][x] = relative_power2(
                    __byte_perm(vsc[0][0], vsc[0][1], (x + 4) << 8 | x) & 0x00FF00FFu, vref);
        }
#pragma unroll
        for (int w = 0; w < VW; ++w) {
#pragma unroll
            for (int ks2 = 0; ks2 < 2; ++ks2) {
                // even and odd elements of token pairs (x, x + 4), x = 2 ks2 and 2 ks2 + 1
                uint32_t even[2][4], odd[2][4];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint32_t x = vraw[2 * ks2 + h][w], y = vraw[2 * ks2 + h + 4][w];
                    decode_e2m1x8((x & 0x0F0F0F0Fu) | ((y << 4) & 0xF0F0F0F0u), even[h]);
                    decode_e2m1x8(((x >> 4) & 0x0F0F0F0Fu) | (y & 0xF0F0F0F0u), odd[h]);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        even[h][i] = hmul2(even[h][i], vs[8 * w / G][2 * ks2 + h]);
                        odd[h][i] = hmul2(odd[h][i], vs[8 * w / G][2 * ks2 + h]);
                    }
                }
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
                        mma16816(acc[4 * w + i][nt], even[0][i], odd[0][i], even[1][i], odd[1][i],
                                 weights[nt][2 * ks2], weights[nt][2 * ks2 + 1]);
            }
        }
        if (more) load_values(static_cast<uint32_t>(j64), vp_next);
        kp = kp_next;
        vp = vp_next;
    }

    // -- join the block's warps ----------------------------------------------------------
    const float unit = G == 16 ? 1.0f : exp2f(static_cast<float>(vref) - 139.0f);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) l[nt][k] += __shfl_xor_sync(0xFFFFFFFFu, l[nt][k], o);
            const uint32_t r = nt * kTileRows + 2u * tig + k;
            if (gid == 0) {
                stats[warp][r][0] = m[nt][k];
                stats[warp][r][1] = l[nt][k];
            }
#pragma unroll
            for (int i = 0; i < MT; ++i)
                *reinterpret_cast<float2 *>(&joined[warp][r][gid * (D / 8) + 2 * i]) =
                    make_float2(acc[i][nt][k] * unit, acc[i][nt][k + 2] * unit);
        }
    }
    __syncthreads();
    const float inv_v = G == 16 ? __frcp_rn(__ldg(p.c.gscale + 1)) : 1.0f;
    for (uint32_t i = threadIdx.x; i < R * (D / 2); i += kAttentionThreads) {
        const uint32_t r = i / (D / 2), d = i % (D / 2) * 2u, row = tile * R + r;
        if (row >= p.rows) break;
        float top = kNoMax, sum = 0.0f, x = 0.0f, y = 0.0f;
#pragma unroll
        for (int w = 0; w < kAttentionWarps; ++w) top = fmaxf(top, stats[w][r][0]);
#pragma unroll
        for (int w = 0; w < kAttentionWarps; ++w) {
            const float f = ex2_approx(stats[w][r][0] - top);
            const float2 o = *reinterpret_cast<const float2 *>(&joined[w][r][d]);
            sum = fmaf(stats[w][r][1], f, sum);
            x = fmaf(o.x, f, x);
            y = fmaf(o.y, f, y);
        }
        if (used <= 1u) {
            const uint32_t t = row / p.group, qh = head * p.group + (row - t * p.group);
            const uint64_t slot =
                (static_cast<uint64_t>(b) * p.q_len + t) * p.c.heads * p.group + qh;
            const float norm = sum > 0.0f ? inv_v / sum : 0.0f;
            *reinterpret_cast<uint32_t *>(p.out + (slot * D + d) * 2u) =
                narrow2<In>(x * norm, y * norm);
            if (d == 0u && p.lse != nullptr)
                p.lse[slot] = sum > 0.0f ? (top - 7.0f + log2f(sum)) * kLn2 : -INFINITY;
        } else {
            const uint64_t slot =
                ((static_cast<uint64_t>(b) * p.c.heads + head) * p.chunks + chunk) * p.rows + row;
            *reinterpret_cast<float2 *>(p.part + slot * D + d) = make_float2(x, y);
            if (d == 0u) p.stat[slot] = make_float2(top, sum);
        }
    }
    release_dependents();
}

// Joins the chunks of one (sequence, query row): a block per row, whose warps
// take every fourth chunk each.  The order of the sums is fixed.
template <typename In, int G, int D>
__global__ void __launch_bounds__(kAttentionThreads)
    attention_join_kernel(const __grid_constant__ AttentionParams p) {
    constexpr int E = D / 32;                  // elements a lane sums
    __shared__ float sums[kAttentionWarps][D];
    wait_for_producer();
    const uint32_t lane = threadIdx.x & 31u, warp = threadIdx.x >> 5;
    const uint32_t r = blockIdx.x % p.rows, bh = blockIdx.x / p.rows;
    const uint32_t head = bh % p.c.heads, b = bh / p.c.heads;
    const uint32_t used = used_chunks(p, sequence_length(p, b));
    if (used > 1u) {
        const uint64_t slot = static_cast<uint64_t>(bh) * p.chunks * p.rows + r;
        float m = kNoMax, l = 0.0f, acc[E];
#pragma unroll
        for (int i = 0; i < E; ++i) acc[i] = 0.0f;
        for (uint32_t c = lane; c < used; c += 32u)
            m = fmaxf(m, p.stat[slot + static_cast<uint64_t>(c) * p.rows].x);
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
        // 32 chunks at a time: a lane holds one chunk's factor, and every warp
        // adds the values of 8 of them
        for (uint32_t c0 = 0; c0 < used; c0 += 32u) {
            float f = 0.0f;
            if (c0 + lane < used) {
                const float2 st = p.stat[slot + static_cast<uint64_t>(c0 + lane) * p.rows];
                f = ex2_approx(st.x - m);
                l = fmaf(st.y, f, l);
            }
#pragma unroll
            for (uint32_t i = 0; i < 32u / kAttentionWarps; ++i) {
                const uint32_t c = c0 + i * kAttentionWarps + warp;
                const float fc = __shfl_sync(0xFFFFFFFFu, f, i * kAttentionWarps + warp);
                if (c < used) {                // warp-uniform
                    uint32_t v[E];
                    load_words(reinterpret_cast<const uint8_t *>(
                                   p.part + (slot + static_cast<uint64_t>(c) * p.rows) * D + lane * E),
                               v);
#pragma unroll
                    for (int k = 0; k < E; ++k) acc[k] = fmaf(__uint_as_float(v[k]), fc, acc[k]);
                }
            }
        }
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) l += __shfl_xor_sync(0xFFFFFFFFu, l, o);
#pragma unroll
        for (int k = 0; k < E; ++k) sums[warp][lane * E + k] = acc[k];
        __syncthreads();
        const float inv_v = G == 16 ? __frcp_rn(__ldg(p.c.gscale + 1)) : 1.0f;
        const float norm = l > 0.0f ? inv_v / l : 0.0f;
        const uint32_t t = r / p.group, qh = head * p.group + (r - t * p.group);
        const uint64_t row = (static_cast<uint64_t>(b) * p.q_len + t) * p.c.heads * p.group + qh;
        for (uint32_t d = 2u * threadIdx.x; d < D; d += 2u * kAttentionThreads) {
            float x = 0.0f, y = 0.0f;
#pragma unroll
            for (int w = 0; w < kAttentionWarps; ++w) {
                x += sums[w][d];
                y += sums[w][d + 1];
            }
            *reinterpret_cast<uint32_t *>(p.out + (row * D + d) * 2u) =
                narrow2<In>(x * norm, y * norm);
        }
        if (threadIdx.x == 0u && p.lse != nullptr)
            p.lse[row] = l > 0.0f ? (m - 7.0f + log2f(l)) * kLn2 : -INFINITY;
    }
    release_dependents();
}

}  // namespace pqg
