// Residual addition, root-mean-square norm and quantization in one pass, for
// sm_100a.
//
// Mathematics.  h = x + r (rounded to the input type), inv = 1 / sqrt(mean(h^2)
// + eps), y = (h inv) w, and y is quantized by groups as in pqg_kernel.cuh.
// The sum of squares is kept in 64 bits: the order of its terms then moves inv, an
// fp32 number, only where it lies within some 2^-50 of the middle between two of
// them, about one row in 10^8.  All other rows have the same codes whatever the launch
// shape, and an independent implementation meets them bit for bit.  One conversion and one 64-bit FMA per element fit
// beside the memory traffic (an SM streams about 3.5 elements per clock here,
// and its 64-bit pipe takes many more).
//
// A row stays in registers between the statistic and the quantization, so x and
// r are read once and h and the codes are written once: 7 bytes per element
// with a residual (bf16 in, one-byte codes), which HBM bounds.  A block takes rows
// in turn; as soon as a row is in registers, the next one's asynchronous copies into
// shared memory begin, each warp copying what it reads itself.
//
// [8192, 7168] bf16 with a residual, E4M3 + fp32 scales per 128: 67 us, 6.2 TB/s, 0.94
// of the copy rate.  On the way there: loads to registers 91.9 us (latency: 24 warps
// on an SM, one row in flight per block); next row prefetched to L2, weights kept in
// L1 78.6; two buffers in shared memory 73.7; blocks of just the warps that a row
// fills (7 of 8 here) and packed additions 71.0; one buffer, so more blocks, 67.  What
// is left is issue: 21 instructions per element at 57 % of the issue slots.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "pqg_kernel.cuh"
#include "pqg_memory.cuh"

namespace pqg {

struct NormParams {
    const uint8_t *in;
    const uint8_t *residual;   // or null
    const uint8_t *weight;
    uint8_t *residual_out;     // or null
    uint8_t *out;
    uint8_t *scales;
    const float *gscale;       // NVFP4 only
    double eps;
    double per_k;              // 1 / K
    uint32_t M;
    uint32_t K;
    uint32_t out_row_bytes;
    uint32_t ng;               // groups per row
    uint32_t group_lanes;      // 16-element slots per group: 1, 2, 4, 8 (not per token)
    uint32_t group_shift;      // log2(group_lanes)
    uint32_t mpad;
    uint32_t layout;
};

constexpr int kNormThreads = 256;      // of a block, at most: 1 to 8 warps share a row

// 32-byte load that stays in L1: the weights, which every row reads again.
__device__ __forceinline__ void load32B_cached(const void *p, uint32_t (&r)[8]) {
    asm volatile("ld.global.nc.L1::evict_last.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]),
                   "=r"(r[6]), "=r"(r[7])
                 : "l"(p));
}

// x + r for two packed pairs, each sum rounded once to the type.  (One rounding to
// fp32 and one to the type give the same: where the fp32 sum is not exact the
// smaller term is below 2^-13 of the larger, less than half a step of the type.)
template <typename T>
__device__ __forceinline__ uint32_t add2(uint32_t a, uint32_t b) {
    uint32_t r;
    if constexpr (std::is_same<T, __nv_bfloat16>::value)
        asm("add.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    else
        asm("add.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// A group's scale.  The fp32 scales are amax times the fp32 constant nearest 1 /
// FMAX, as this entry point defines them: one rounding, and at most an ulp from the
// quotient that pqg_quant stores (make_scale).  The codes are the rounding of
// fp32(y / s) for that s.  The other kinds as in make_scale.
template <Kind KIND>
__device__ __forceinline__ GroupScale make_norm_scale(float amax, const float *nv) {
    if constexpr (KIND == Kind::E4M3_FP32 || KIND == Kind::INT8_FP32) {
        GroupScale gs;
        gs.s = __fmul_rn(fmaxf(amax, 1e-10f), KIND == Kind::INT8_FP32 ? kRcp127 : kRcp448);
        gs.mult = __frcp_rn(gs.s);
        gs.neg_s = -gs.s;
        gs.e8 = 0;
        return gs;
    } else {
        return make_scale<KIND>(amax, nv);
    }
}

// 1 / sqrt(v) rounded to fp32, for a normal v > 0: v is scaled by an even power of
// two into [1, 4), and two Newton steps d (3 - m d^2) / 2 in 64 bits take the 22
// good bits of the hardware's approximation to 44 and then to the last bit or two
// of 53.  A 64-bit division and square root cost four times the instructions, in
// every thread of every row ([8192, 7168] 78.6 -> 76.7 us).
__device__ __forceinline__ float inverse_root(double v) {
    const int hi = __double2hiint(v), k = ((hi >> 20) - 1023) & ~1;
    const double m = __hiloint2double(hi - (k << 20), __double2loint(v));
    float d0;
    asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(d0) : "f"(static_cast<float>(m)));
    double d = d0;
    const double half = -0.5 * m;
#pragma unroll
    for (int i = 0; i < 2; ++i) d = fma(d, fma(half * d, d, 0.5), d);
    const float r = static_cast<float>(
        __hiloint2double(__double2hiint(d) - ((k / 2) << 20), __double2loint(d)));
    return v == v ? r : __int_as_float(0x7FFFFFFF);   // a NaN of either sign; infinity gives 0
}

// Store the scale of group g of a row (the slot's first lane calls it; for the
// word layouts `word` holds the exponents of groups 4j..4j+3).
template <Kind KIND>
__device__ __forceinline__ void store_norm_scale(const NormParams &p, uint32_t row, uint32_t g,
                                                 const GroupScale &gs, uint32_t word) {
    if (p.layout == kPacked) {
        if ((g & 3u) == 0u)
            reinterpret_cast<uint32_t *>(p.scales)[static_cast<uint64_t>(g >> 2) * p.mpad + row] =
                word;
    } else if (p.layout == kTiled128x4) {
        store_tiled(p.scales, row, g, p.ng, gs.e8);
    } else {
        const uint64_t idx = p.layout == kRowMajor ? static_cast<uint64_t>(row) * p.ng + g
                                                   : static_cast<uint64_t>(g) * p.mpad + row;
        if constexpr (byte_scale(KIND))
            p.scales[idx] = static_cast<uint8_t>(gs.e8);
        else
            reinterpret_cast<float *>(p.scales)[idx] = gs.s;
    }
}

// A row is shared by the block's warps; a thread holds SLOTS slots of 16 consecutive
// elements, neighbouring lanes holding neighbouring slots, so that a group is
// 1 to 8 neighbouring lanes (or, per token, the whole row).
//
// Shared memory: [SLOTS][x, r][warp][1 KB], x alone without a residual.
__host__ __device__ constexpr uint32_t norm_smem(int slots, int warps, bool residual) {
    return slots * (residual ? 2u : 1u) * warps * 1024u;
}

template <typename In, Kind KIND, int SLOTS, bool PER_TOKEN>
__global__ void __launch_bounds__(kNormThreads)
    rmsnorm_quant_kernel(const __grid_constant__ NormParams p) {
    extern __shared__ __align__(128) uint8_t rows[];
    __shared__ double sums[2][kNormThreads / 32];
    __shared__ float maxima[PER_TOKEN ? 2 : 1][kNormThreads / 32];
    __shared__ float nv[KIND == Kind::E2M1_E4M3 ? kNvTable : 1];

    wait_for_producer();                        // before the first global access
    if constexpr (KIND == Kind::E2M1_E4M3) {
        // build_nvfp4_table for a block of any size
        const float g = __ldg(p.gscale);
        for (uint32_t c = threadIdx.x; c < 128u; c += blockDim.x) {
            const float d = e4m3_code_value(c);
            nv[c] = d == 0.0f ? 0.0f : __fdiv_rn(g, d);
        }
        if (threadIdx.x == 0u) nv[128] = g;
        __syncthreads();
    }
    const uint32_t lane = threadIdx.x & 31u;
    const uint32_t warp = threadIdx.x >> 5;
    const uint32_t tid = threadIdx.x, tpr = blockDim.x, warps = blockDim.x >> 5;
    const uint32_t nslots = p.K / 16u;
    const uint64_t row_bytes = static_cast<uint64_t>(p.K) * 2u;

    const uint32_t inputs = p.residual != nullptr ? 2u : 1u;
    const uint32_t rows_at = static_cast<uint32_t>(__cvta_generic_to_shared(rows)) + warp * 1024u;
    const uint32_t part = tpr * 32u;                    // bytes of one slot of all threads
    // Part c (16 bytes) of a warp's 1 KB goes to place c ^ ((c >> 3) & 1): lanes copy
    // neighbouring parts, then read parts 2 lane and 2 lane + 1, both without conflicts.
    const uint32_t place = (lane ^ ((lane >> 3) & 1u)) * 16u;
    const uint32_t flip = (lane >> 2) & 1u;             // of parts 2 lane and 2 lane + 1
    auto copy_row = [&](uint32_t row) {
        if (row < p.M) {
#pragma unroll
            for (int j = 0; j < SLOTS; ++j) {
                const uint32_t slot = (tid & ~31u) + j * tpr;   // the warp's first
                const uint64_t from = row * row_bytes + slot * 32u + lane * 16u;
                const uint32_t to = rows_at + j * inputs * part + place;
#pragma unroll
                for (uint32_t half = 0; half < 2; ++half) {
                    if (slot + half * 16u + lane / 2u >= nslots) continue;
                    copy16(to + half * 512u, p.in + from + half * 512u);
                    if (inputs == 2u)
                        copy16(to + part + half * 512u, p.residual + from + half * 512u);
                }
            }
        }
        commit_copies();
    };
    auto read_slot = [&](uint32_t at, uint32_t (&v)[8]) {
        const uint8_t *mine = rows + at + warp * 1024u + lane * 32u;
        const uint4 a = *reinterpret_cast<const uint4 *>(mine + flip * 16u);
        const uint4 b = *reinterpret_cast<const uint4 *>(mine + (flip ^ 1u) * 16u);
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
        v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    };

    uint32_t parity = 0;
    copy_row(blockIdx.x);
    for (uint32_t row = blockIdx.x; row < p.M; row += gridDim.x, parity ^= 1u) {
        wait_copies<0>();
        __syncwarp();

        // -- h = x + r; the next row's copies start as soon as the buffer is read ------
        uint32_t h[SLOTS][8];
#pragma unroll
        for (int j = 0; j < SLOTS; ++j) {
            const uint32_t slot = tid + j * tpr;
#pragma unroll
            for (int i = 0; i < 8; ++i) h[j][i] = 0u;
            if (slot < nslots) {
                const uint32_t at = j * inputs * part;
                read_slot(at, h[j]);
                if (inputs == 2u) {
                    uint32_t r[8];
                    read_slot(at + part, r);
#pragma unroll
                    for (int i = 0; i < 8; ++i) h[j][i] = add2<In>(h[j][i], r[i]);
                }
                if (p.residual_out != nullptr)
                    store32B(p.residual_out + row * row_bytes + slot * 32u, h[j]);
            }
        }
        __syncwarp();                           // the warp has read its buffer
        copy_row(row + gridDim.x);
        double ss = 0.0;
#pragma unroll
        for (int j = 0; j < SLOTS; ++j) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                float a0, a1;
                widen2<In>(h[j][i], a0, a1);
                ss = fma(static_cast<double>(a0), static_cast<double>(a0), ss);
                ss = fma(static_cast<double>(a1), static_cast<double>(a1), ss);
            }
        }
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, o);
        if (warps > 1u) {
            if (lane == 0) sums[parity][warp] = ss;
            __syncthreads();
            ss = 0.0;
            for (uint32_t w = 0; w < warps; ++w) ss += sums[parity][w];
        }
        const float inv = inverse_root(fma(ss, p.per_k, p.eps));

        // -- y, its groups' absmax, scales and codes ------------------------------
        auto norm_slot = [&](int j, uint32_t slot, float (&y)[16]) {
            uint32_t w[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) w[i] = 0u;
            if (slot < nslots) load32B_cached(p.weight + slot * 32u, w);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                float a0, a1, w0, w1;
                widen2<In>(h[j][i], a0, a1);
                widen2<In>(w[i], w0, w1);
                const float2 v = __fmul2_rn(
                    __fmul2_rn(make_float2(a0, a1), make_float2(inv, inv)), make_float2(w0, w1));
                y[2 * i] = v.x;
                y[2 * i + 1] = v.y;
            }
        };
        // per token: the whole row's absmax first, y kept in registers
        float kept[PER_TOKEN ? SLOTS : 1][16], row_max = 0.0f;
        if constexpr (PER_TOKEN) {
#pragma unroll
            for (int j = 0; j < SLOTS; ++j) {
                norm_slot(j, tid + j * tpr, kept[j]);
                row_max = fmaxf(row_max, absmax16(kept[j]));
            }
#pragma unroll
            for (int o = 1; o < 32; o <<= 1)
                row_max = fmaxf(row_max, __shfl_xor_sync(0xFFFFFFFFu, row_max, o));
            if (warps > 1u) {
                if (lane == 0) maxima[parity][warp] = row_max;
                __syncthreads();
                for (uint32_t w = 0; w < warps; ++w) row_max = fmaxf(row_max, maxima[parity][w]);
            }
        }
#pragma unroll
        for (int j = 0; j < SLOTS; ++j) {
            const uint32_t slot = tid + j * tpr;
            const bool ok = slot < nslots;
            float y[16];
            float amax = row_max;
            if constexpr (PER_TOKEN) {
#pragma unroll
                for (int i = 0; i < 16; ++i) y[i] = kept[j][i];
            } else {
                norm_slot(j, slot, y);
                amax = absmax16(y);
                for (uint32_t o = 1; o < p.group_lanes; o <<= 1)
                    amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, o));
            }
            const GroupScale gs = make_norm_scale<KIND>(amax, nv);
            uint32_t code[4];
            // two quotient corrections: y has all 24 bits, and the one-correction
            // quotient is proved for 16-bit inputs only
            encode16<KIND, 2>(y, gs, code);

            const uint32_t g = PER_TOKEN ? 0u : slot >> p.group_shift;
            uint32_t word = gs.e8;              // per token: bytes 1..3 are 0
            if (!PER_TOKEN && p.layout == kPacked) {
                // exponents of groups 4j..4j+3, from the 4 groups' lanes
                word = ok ? gs.e8 << (8u * (g & 3u)) : 0u;
                word |= __shfl_xor_sync(0xFFFFFFFFu, word, p.group_lanes);
                word |= __shfl_xor_sync(0xFFFFFFFFu, word, 2u * p.group_lanes);
            }
            if (!ok) continue;
            uint8_t *dst = p.out + static_cast<uint64_t>(row) * p.out_row_bytes;
            if constexpr (is_e2m1(KIND))
                store8B(dst + slot * 8u, code[0], code[1]);
            else
                store16B(dst + slot * 16u, code[0], code[1], code[2], code[3]);
            const bool first = PER_TOKEN ? slot == 0u : (slot & (p.group_lanes - 1u)) == 0u;
            if (first) store_norm_scale<KIND>(p, row, g, gs, word);
        }
    }
    release_dependents();
}

}  // namespace pqg
