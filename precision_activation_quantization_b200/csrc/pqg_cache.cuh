// The paged 4-bit key/value cache: geometry, quantizing writes and the read-back.
//
// Layout (a page of P tokens, one key/value head):
//   codes  [page][head][P][D / 2]      E2M1, two per byte, element 2i low
//   scales [page][head][D / G][P]      one byte per (group, token)
// The codes of a (page, head) are contiguous for bulk reading; the scales are
// group-major, so that a reader of one group takes those of 4 or 8 neighbouring
// tokens with one load.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "pqg_kernel.cuh"
#include "pqg_memory.cuh"

namespace pqg {

struct CacheView {
    uint8_t *codes[2];         // keys, values
    uint8_t *scales[2];
    const float *gscale;       // NVFP4: g of keys and of values
    uint32_t num_pages;
    uint32_t page_shift;       // log2(page size)
    uint32_t heads;
    uint32_t head_dim;
    uint32_t heads_magic;      // x / heads = umulhi(x, heads_magic) >> heads_shift for
    uint32_t heads_shift;      // x < 2^31 (div_segs' rule; magic 0: one head)
};

__device__ __forceinline__ uint32_t div_heads(const CacheView &c, uint32_t x) {
    return c.heads_magic == 0u ? x : __umulhi(x, c.heads_magic) >> c.heads_shift;
}

// First byte of the codes of (page, head, offset) and of the scale bytes of
// (page, head, group 0, offset); 64-bit: a cache passes 4 GB.
__device__ __forceinline__ uint64_t code_offset(const CacheView &c, uint32_t page, uint32_t head,
                                                uint32_t off) {
    const uint64_t row = ((static_cast<uint64_t>(page) * c.heads + head) << c.page_shift) + off;
    return row * (c.head_dim / 2u);
}
template <int G>
__device__ __forceinline__ uint64_t scale_offset(const CacheView &c, uint32_t page, uint32_t head,
                                                 uint32_t group, uint32_t off) {
    const uint32_t ng = c.head_dim / G;
    return (((static_cast<uint64_t>(page) * c.heads + head) * ng + group) << c.page_shift) + off;
}

constexpr int kCacheThreads = 256;

struct WriteParams {
    CacheView c;
    const uint8_t *src[2];     // k, v
    uint64_t stride[2];        // bytes between tokens
    const int32_t *slots;
    uint32_t T;
};

// One lane quantizes 16 elements of a key row and the same 16 of the value row;
// a (token, head) row is D / 16 neighbouring lanes, a warp holds neighbouring
// tokens of one head (their scale bytes are neighbours), and the heads of those
// tokens go to neighbouring warps (their input is contiguous).  Bound by the
// 16-bit input: 115 MB in 21.0 us (5.5 TB/s); 23.7 us when the rows waited for the
// slot.
template <typename In, int G>
__global__ void __launch_bounds__(kCacheThreads)
    kv_write_kernel(const __grid_constant__ WriteParams p) {
    constexpr Kind KIND = G == 16 ? Kind::E2M1_E4M3 : Kind::E2M1_UE8M0;
    constexpr uint32_t L = G / 16;              // lanes per group
    wait_for_producer();
    const uint32_t lanes = p.c.head_dim / 16u;  // lanes per row: 4, 8 or 16
    const uint32_t rpw = 32u / lanes;           // tokens per warp
    const uint32_t lane = threadIdx.x & 31u;
    const uint32_t sub = lane / lanes, col = (lane - sub * lanes) * 16u;
    const uint32_t warp = blockIdx.x * (kCacheThreads / 32) + (threadIdx.x >> 5);
    const uint32_t block = div_heads(p.c, warp), head = warp - block * p.c.heads;
    const uint64_t token = static_cast<uint64_t>(block) * rpw + sub;
    // the rows are loaded while the slot is in flight: a padding token's row is read too
    const bool some = token < p.T;
    int slot = -1;
    if (some) slot = __ldg(p.slots + token);
    uint32_t x[2][8];
#pragma unroll
    for (int n = 0; n < 2; ++n) {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[n][i] = 0u;
        if (some)
            load32B(p.src[n] + token * p.stride[n] +
                        (static_cast<uint64_t>(head) * p.c.head_dim + col) * 2u, x[n]);
    }
    const bool live = slot >= 0 && (static_cast<uint32_t>(slot) >> p.c.page_shift) < p.c.num_pages;
    const uint32_t page = static_cast<uint32_t>(slot) >> p.c.page_shift;
    const uint32_t off = static_cast<uint32_t>(slot) & ((1u << p.c.page_shift) - 1u);
#pragma unroll
    for (int n = 0; n < 2; ++n) {
        float v[16];
#pragma unroll
        for (int i = 0; i < 8; ++i) widen2<In>(x[n][i], v[2 * i], v[2 * i + 1]);
        float amax = absmax16(v);
#pragma unroll
        for (uint32_t o = 1; o < L; o <<= 1)
            amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, o));
        GroupScale gs;
        if constexpr (G == 16) {
            // pqg_quant_nvfp4's rule with this row's g
            const float g = __ldg(p.c.gscale + n);
            const float r = __fmul_rn(div_by_const(fmaxf(amax, 1e-10f), 6.0f, kRcp6), g);
            gs.e8 = e4m3x2(r, 0.0f) & 0xFFu;
            const float sf = e4m3_code_value(gs.e8 & 0x7Fu);
            gs.mult = sf == 0.0f ? 0.0f : __fdiv_rn(g, sf);
        } else {
            gs = make_scale<KIND>(amax);
        }
        uint32_t w[4];
        encode16<KIND>(v, gs, w);
        if (live) {
            store8B(p.c.codes[n] + code_offset(p.c, page, head, off) + col / 2u, w[0], w[1]);
            if ((lane & (L - 1u)) == 0u)
                p.c.scales[n][scale_offset<G>(p.c, page, head, col / G, off)] =
                    static_cast<uint8_t>(gs.e8);
        }
    }
    release_dependents();
}

struct ReadParams {
    CacheView c;
    const int32_t *table;
    const int32_t *indptr;
    uint8_t *dst[2];           // k_out, v_out
    uint64_t table_stride;
    uint32_t max_pages;
    uint32_t B;
    uint32_t M;
};

// The sequence of packed row `row`: the last b with indptr[b] <= row, or -1
// where no sequence holds the row.  indptr does not decrease.
__device__ __forceinline__ int find_sequence(const int32_t *indptr, uint32_t B, int row,
                                             int *first) {
    uint32_t lo = 0, hi = B;                    // indptr[lo] <= row < indptr[hi], if in any
    while (hi - lo > 1u) {
        const uint32_t mid = (lo + hi) >> 1;
        if (__ldg(indptr + mid) <= row) lo = mid; else hi = mid;
    }
    *first = __ldg(indptr + lo);
    return *first <= row && row < __ldg(indptr + lo + 1) ? static_cast<int>(lo) : -1;
}

// Eight codes of a packed word, times `s` (and, NVFP4, `inv`), each rounded once to
// 16 bits: four packed words.  code * scale is exact in fp32.
template <typename Out, bool INV>
__device__ __forceinline__ void decode8(uint32_t codes, float s, float inv, uint32_t *w) {
    uint32_t h[4];
    asm("{\n\t.reg .b8 p, q, s, t;\n\t"
        "mov.b32 {p, q, s, t}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, p;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, q;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, s;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, t;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3]) : "r"(codes));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float2 v = __fmul2_rn(__half22float2(*reinterpret_cast<__half2 *>(&h[i])),
                              make_float2(s, s));
        if constexpr (INV) v = __fmul2_rn(v, make_float2(inv, inv));
        w[i] = narrow2<Out>(v.x, v.y);
    }
}

// 2^(e - 127) for a UE8M0 byte (e = 0: 2^-127, a subnormal).
__device__ __forceinline__ float ue8m0_value(uint32_t e) {
    return e == 0u ? __uint_as_float(0x00400000u) : __uint_as_float(e << 23);
}

// One lane decodes 16 elements of the key rows and of the value rows of ROWS
// neighbouring output rows: 4 where there are many, so that finding the sequence is
// shared and eight loads of codes are in flight, 1 where the rows would not fill the
// SMs otherwise (7 sequences of up to 300 tokens: 2.1 us against 4.4).  The pages of all
// rows are asked for before any code.  Bound by the 16-bit output: 363 MB in 59.5 us
// (6.1 TB/s, 0.93 of the copy rate); 67 us when a row's codes were asked for before the
// next row's page.
template <typename Out, int G, int ROWS>
__global__ void __launch_bounds__(kCacheThreads)
    kv_read_kernel(const __grid_constant__ ReadParams p) {
    wait_for_producer();
    const uint32_t lane_shift = p.c.head_dim == 64u ? 2u : p.c.head_dim == 128u ? 3u : 4u;
    const uint64_t unit = static_cast<uint64_t>(blockIdx.x) * kCacheThreads + threadIdx.x;
    const uint32_t col = (static_cast<uint32_t>(unit) & ((1u << lane_shift) - 1u)) * 16u;
    const uint32_t rowhead = static_cast<uint32_t>(unit >> lane_shift);   // < 2^31
    const uint32_t group = div_heads(p.c, rowhead), head = rowhead - group * p.c.heads;
    const uint64_t row0 = static_cast<uint64_t>(group) * ROWS;
    if (row0 < p.M) {
        const float inv[2] = {G == 16 ? __frcp_rn(__ldg(p.c.gscale)) : 1.0f,
                              G == 16 ? __frcp_rn(__ldg(p.c.gscale + 1)) : 1.0f};
        uint2 codes[ROWS][2];
        uint32_t scale[ROWS][2], at[ROWS];     // at: token of its sequence
        int page[ROWS];
        bool held[ROWS];
        int b = -1, first = 0, last = INT32_MIN;    // the sequence and its rows [first, last)
#pragma unroll
        for (uint32_t i = 0; i < ROWS; ++i) {
            const uint64_t row = row0 + i;
            held[i] = false;
            page[i] = -1;
            at[i] = 0u;
            if (row < p.M) {
                if (static_cast<int>(row) >= last) {
                    b = find_sequence(p.indptr, p.B, static_cast<int>(row), &first);
                    last = b >= 0 ? __ldg(p.indptr + b + 1) : static_cast<int>(row) + 1;
                }
                at[i] = static_cast<uint32_t>(row) - static_cast<uint32_t>(first);
                held[i] = b >= 0 && (at[i] >> p.c.page_shift) < p.max_pages;
                if (held[i])
                    page[i] = __ldg(p.table + static_cast<uint64_t>(b) * p.table_stride +
                                    (at[i] >> p.c.page_shift));
            }
        }
#pragma unroll
        for (uint32_t i = 0; i < ROWS; ++i) {
            if (static_cast<uint32_t>(page[i]) >= p.c.num_pages) page[i] = -1;
            if (page[i] >= 0) {
                const uint32_t off = at[i] & ((1u << p.c.page_shift) - 1u);
                const uint64_t code = code_offset(p.c, page[i], head, off) + col / 2u;
                const uint64_t sc = scale_offset<G>(p.c, page[i], head, col / G, off);
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                    codes[i][n] = __ldg(reinterpret_cast<const uint2 *>(p.c.codes[n] + code));
                    scale[i][n] = __ldg(p.c.scales[n] + sc);
                }
            }
        }
#pragma unroll
        for (uint32_t i = 0; i < ROWS; ++i) {
            if (!held[i]) continue;
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                uint32_t w[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) w[k] = 0u;
                if (page[i] >= 0) {
                    const float s = G == 16 ? e4m3_code_value(scale[i][n] & 0x7Fu)
                                            : ue8m0_value(scale[i][n]);
                    decode8<Out, G == 16>(codes[i][n].x, s, inv[n], w);
                    decode8<Out, G == 16>(codes[i][n].y, s, inv[n], w + 4);
                }
                store32B(p.dst[n] + (((row0 + i) * p.c.heads + head) * p.c.head_dim + col) * 2u,
                         w);
            }
        }
    }
    release_dependents();
}

}  // namespace pqg
