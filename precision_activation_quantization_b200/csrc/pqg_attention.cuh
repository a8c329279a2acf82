// Attention over the paged 4-bit cache, for sm_100a.
//
// A unit of work is one (sequence, key/value head, tile of 8 or 16 query rows); row
// r = t * group + h is token t and query head h of the head's group.  Its keys
// are cut into pieces of 128, and all pieces of all units, in order, are dealt
// to one wave of blocks in equal shares, so that ragged lengths leave no block
// behind.  A block computes a unit's pieces in its share with a running maximum
// and sum; it writes a whole unit's result itself and leaves (maximum, sum,
// weighted values) of a part of a unit in the workspace, where a second kernel
// joins the parts in their order.
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
    float *part;               // [2 shares][query rows of a unit][D] weighted values
    float2 *stat;              // [2 shares][query rows of a unit] (max in log2 units, sum)
    uint2 *joins;              // [units] (first part's place, parts); 0 parts: written
    const int32_t *table;
    const int32_t *seq_lens;
    uint64_t q_stride;         // elements between tokens
    uint64_t table_stride;
    float scale_log2;          // |sm_scale| * log2(e)
    float sign;                // of sm_scale
    uint32_t max_pages;
    uint32_t B;
    uint32_t q_len;
    uint32_t group;            // query heads per key/value head
    uint32_t rows;             // q_len * group
    uint32_t row_tiles;
    uint32_t shares;           // blocks
};

constexpr float kLn2 = 0.6931471805599453f;
constexpr float kNoMax = -3e38f;   // a row's reference before any key (finite: differences are)

// Keys of sequence b that the cache can hold.
__device__ __forceinline__ uint32_t sequence_length(const AttentionParams &p, uint32_t b) {
    const uint64_t cap = static_cast<uint64_t>(p.max_pages) << p.c.page_shift;
    const int n = max(__ldg(p.seq_lens + b), 0);
    return static_cast<uint64_t>(n) < cap ? static_cast<uint32_t>(n) : static_cast<uint32_t>(cap);
}
// Pieces of a unit of n keys; one without keys is a piece too, which writes zeros.
constexpr uint32_t kPieceKeys = 128;
__device__ __forceinline__ uint32_t pieces_of(uint32_t n) {
    return max((n + kPieceKeys - 1u) / kPieceKeys, 1u);
}

// A block's share [at, end) of the pieces, and the sequence that holds piece
// `at`, whose own pieces begin at `first`.  P pieces (the host keeps P below 2^32)
// are dealt to s = min(blocks, P) shares: P / s each, and one more to the first P % s.
struct Share {
    uint32_t at, end, first, b;
    uint32_t size, longer;     // pieces of a share, and how many shares have one more
    __device__ __forceinline__ void deal(uint32_t pieces, uint32_t blocks) {
        const uint32_t shares = min(blocks, pieces);
        size = pieces / shares;
        longer = pieces - size * shares;
        const uint32_t i = min(blockIdx.x, shares);
        at = i * size + min(i, longer);
        end = i < shares ? at + size + (i < longer ? 1u : 0u) : at;
    }
    // The share that holds piece x.
    __device__ __forceinline__ uint32_t of(uint32_t x) const {
        const uint32_t in_longer = longer * (size + 1u);
        return x < in_longer ? x / (size + 1u) : longer + (x - in_longer) / size;
    }
};
// Every thread of the block calls it.  Each sums the pieces of neighbouring
// sequences, a prefix sum over the block finds the thread that holds `at`, and
// that one walks to the sequence.
template <int THREADS>
__device__ __forceinline__ Share find_share(const AttentionParams &p, uint32_t units_per_sequence) {
    Share s;
    s.b = 0;
    s.first = 0;
    if (p.B == 1u) {
        s.deal(pieces_of(sequence_length(p, 0)) * units_per_sequence, p.shares);
        return s;
    }
    __shared__ uint32_t sums[THREADS / 32], found_b, found_first;
    const uint32_t lane = threadIdx.x & 31u, warp = threadIdx.x >> 5;
    const uint32_t per = (p.B + THREADS - 1u) / THREADS;
    const uint32_t lo = min(threadIdx.x * per, p.B), hi = min(lo + per, p.B);
    uint32_t own = 0;
    for (uint32_t b = lo; b < hi; ++b) own += pieces_of(sequence_length(p, b));
    uint32_t incl = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t v = __shfl_up_sync(0xFFFFFFFFu, incl, o);
        if (lane >= static_cast<uint32_t>(o)) incl += v;
    }
    if (lane == 31u) sums[warp] = incl;
    __syncthreads();
    uint32_t before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) {
        if (w < static_cast<int>(warp)) before += sums[w];
        all += sums[w];
    }
    s.deal(all * units_per_sequence, p.shares);
    uint32_t first = (before + incl - own) * units_per_sequence;
    if (first <= s.at && s.at - first < own * units_per_sequence) {
        uint32_t b = lo;
        for (; b + 1u < hi; ++b) {
            const uint32_t n = pieces_of(sequence_length(p, b)) * units_per_sequence;
            if (s.at - first < n) break;
            first += n;
        }
        found_b = b;
        found_first = first;
    }
    __syncthreads();
    s.b = found_b;
    s.first = found_first;
    return s;
}

// Warps of a block (a head of 256 takes more shared memory per warp).
__host__ __device__ constexpr int attention_warps(int D) { return D < 256 ? 4 : 2; }
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
// The low (high) half of a pair, twice.
__device__ __forceinline__ uint32_t both_halves(uint32_t v, bool high) {
    const __half2 h = *reinterpret_cast<const __half2 *>(&v);
    const __half2 r = high ? __high2half2(h) : __low2half2(h);
    return *reinterpret_cast<const uint32_t *>(&r);
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

// N consecutive words, N a multiple of 2, that another kernel of the call has written.
template <int N>
__device__ __forceinline__ void load_written(const float *p, float (&v)[N]) {
    if constexpr (N == 2) {
        asm volatile("ld.global.cg.v2.f32 {%0,%1}, [%2];" : "=f"(v[0]), "=f"(v[1]) : "l"(p));
    } else {
#pragma unroll
        for (int i = 0; i < N; i += 4)
            asm volatile("ld.global.cg.v4.f32 {%0,%1,%2,%3}, [%4];"
                         : "=f"(v[i]), "=f"(v[i + 1]), "=f"(v[i + 2]), "=f"(v[i + 3])
                         : "l"(p + i));
    }
}

// N consecutive words of shared memory.
template <int N>
__device__ __forceinline__ void load_shared(const uint8_t *p, uint32_t (&w)[N]) {
    if constexpr (N == 1) {
        w[0] = *reinterpret_cast<const uint32_t *>(p);
    } else if constexpr (N == 2) {
        const uint2 v = *reinterpret_cast<const uint2 *>(p);
        w[0] = v.x, w[1] = v.y;
    } else {
#pragma unroll
        for (int i = 0; i < N; i += 4) {
            const uint4 v = *reinterpret_cast<const uint4 *>(p + 4 * i);
            w[i] = v.x, w[i + 1] = v.y, w[i + 2] = v.z, w[i + 3] = v.w;
        }
    }
}

// The larger half of a pair of 16-bit numbers.
__device__ __forceinline__ uint32_t larger_half(uint32_t v) { return max(v & 0xFFFFu, v >> 16); }

// The smallest of eight 16-bit numbers that is not 0 (0x10000 where all are).
__device__ __forceinline__ uint32_t smallest_half(const uint32_t (&e)[4]) {
    uint32_t low = 0xFFFFFFFFu;                // of e - 1, which 0 wraps around
#pragma unroll
    for (int x = 0; x < 4; ++x) low = __viaddmin_u16x2(e[x], 0xFFFFFFFFu, low);
    return min(low & 0xFFFFu, low >> 16) + 1u;
}

// 2^(e - ref + 12) in binary16 for two UE8M0 bytes (in bits 0-7 and 16-23) that
// are at most ref, which comes as reference2(ref); 0 where the power is below 2^-14.
__device__ __forceinline__ uint32_t relative_power2(uint32_t e2, uint32_t ref2) {
    return __viaddmax_s16x2(e2, ref2, 0u) << 10;
}
// The second argument for a reference exponent.
__device__ __forceinline__ uint32_t reference2(uint32_t ref) {
    return ((27u - ref) & 0xFFFFu) * 0x00010001u;
}

// 2^(e - 127) / kKeyShift for a UE8M0 byte of a key's group, 0 for byte 0.  The sum over
// a group of queries below 2^15 times codes may reach 2^23, so that fp32 sums would
// overflow with scales from 2^102 on; divided, from 2^118.
constexpr float kKeyShift = 65536.0f;
__device__ __forceinline__ float key_power(uint32_t e) {
    return __uint_as_float(e << 23) * (1.0f / kKeyShift);
}

// A row's reference when set, below its maximum, and where it rises (2^kHigh fits binary16).
constexpr float kBelow = 11.0f, kHigh = 15.0f;

// A warp's values are summed under weights that sum to l, up to 2^46 over many keys: with
// values from 2^82 on such sums overflow where the mean, which is wanted, does not.  A warp
// that has met scales of 2^kHugeScale moves a power of two from its sums to m, which rounds
// nothing: l is in [2^-14, 2^-13) then, so that the sums of below 2^11 parts of 4 warps are
// below the largest value.  m is a whole number; one from 2^23 on cannot take the power, so
// there the sums stay as they are.  Returns the power.
constexpr uint32_t kHugeScale = 50;
__device__ __forceinline__ float move_power(float &m, float &l) {
    if (!(fabsf(m) < 8388608.0f) || l == 0.0f) return 1.0f;
    const int e = static_cast<int>(__float_as_uint(l) >> 23 & 0xFFu) - 113;
    const float f = __uint_as_float(static_cast<uint32_t>(max(127 - e, 1)) << 23);
    m += static_cast<float>(e);
    l *= f;
    return f;
}

// A word's bytes [from, from + 4) of a tile, those at or past `end` zeroed.
__device__ __forceinline__ uint32_t keep_bytes(uint32_t w, int from, int end) {
    const int n = min(max(end - from, 0), 4);
    return n == 4 ? w : w & ((1u << (8 * n)) - 1u);
}

// ---------------------------------------------------------------------------
// A block's share
// ---------------------------------------------------------------------------
//
// Mathematics.  With c_jd the 4-bit code of key j, s_jg its scale and q the
// query, score_j = sum_g sum_{d in g} q_d (c_jd s_jg); out = sum_j p_j (c_jd
// s_jg) / sum_j p_j.  Both products run on the tensor cores in binary16 with
// fp32 sums.  Keys and values are exact there: a code has 2 significant bits and an
// E4M3 scale 4, so their product is a binary16 number.  A UE8M0 scale has a
// wider range than binary16.  Keys: the codes alone are multiplied, a group (two steps
// of 16 elements) at a time, and fp32 sums take the group's sum times its power: one
// fp32 FMA per key and row in place of a multiplication of each pair of elements
// (82.6 -> 82.0 us for the 64 sequences below).  Values: a sum runs over keys of
// different scales, so they are taken relative to a reference, 12 binades above 1: the
// largest scale so far of the lane's elements.  A group whose scale is 2^-27 of the
// reference or less counts as zero.  With several new tokens some rows do not see the keys
// of the last tiles, nor then any newer ones, and must not lose theirs to a large scale
// there: such a tile adds its groups by rising scale, the reference raised by up to 26 in
// between.  (In a kernel of its own: the loop, though not run, costs the others 1 to 4 %.)
// A query row is scaled by a power of two so that its largest element is in [2^14, 2^15):
// elements of 2^-14 and more are exact, smaller ones off by 2^-25 at most, 2^-39 of the
// largest.  The weights p are rounded to binary16's 11 bits, or by 2^-36 of the row's largest
// where that is more (see the reference m below).
//
// Layout.  A warp takes 32 keys at a time; tokens are M of the first product, so
// that 8 query rows (N) cost no more tensor work than one.  The order of a sum's
// terms is free, so every lane reads what is contiguous in the cache: of the
// keys, D / 4 neighbouring elements (MXFP4: 8 of every group) of keys 4 gid .. 4 gid + 3
// (gid = lane / 4, tig = lane % 4); of the values, D / 8 neighbouring elements of keys 8 tig ..
// 8 tig + 7; and one word (two) of scales of 4 (8) neighbouring keys.  The second
// product wants pairs of keys in a register while the cache holds pairs of
// elements: two words of two keys are interleaved by nibbles, two operations for
// eight pairs.  The weights change from the first product's layout to the
// second's by an 8 x 8 transpose.
//
// Every warp copies its own tiles into its own two buffers of shared memory
// (asynchronous 16-byte copies, the next tile's in flight while one is computed),
// so warps never wait on one another before the join.  A tile's rows are laid out
// so that the lanes of one load meet 32 different banks (row_at below).
//
// The reference m of a row's weights 2^(score - m) is a whole number, kBelow to kBelow + 1
// below a maximum when it is set, and rises when a score exceeds it by kHigh, so that most
// tiles neither reduce a maximum across lanes nor rescale.  Weights below 2^-14 lose bits in
// binary16, those below 2^-25 all of them: the error is 2^-25 at most where the row's largest
// weight is 2^11 or more, 2^-36 of it.  A larger kBelow would reach further down but rise
// more often: 13 costs the 64 sequences below 0.6 % and 131072 keys 0.8 %, 11 0.3 and 0.3 %,
// against 7.
//
// Measured.  64 ragged sequences of up to 8192 keys, 32 query and 8 key heads of 128:
// 348 MB of MXFP4 in 79.4 us (4.4 TB/s), 367 MB of NVFP4 in 75.5 us (4.9); one sequence
// of 131072 keys, 151 MB, in 36.5 us.  HBM would take 53, 56 and 23.  No pipe is full: of
// the first call 62 % of the issue slots, 53 % of the ALU and 26 % of the tensor pipe are
// busy, at 4 warps per scheduler.  A tile of 32 MXFP4 keys takes 616 warp instructions, of
// which 128 convert codes, 64 multiply values by scales and 32 are products; the larger part
// is addresses, reads of shared memory, interleaving, softmax and the loop.  A loop of one
// product, four conversions and four multiplications alone takes 5 clocks of an SM (each kind
// alone 2), which is half of what the long sequence takes.  With the copies left out the 64
// sequences take 70 us: weighted values 27, scores 21, softmax, loop and start 23; copies and
// softmax alone take 60.  Blocks of 12 or 20 warps an SM are slower than 16, and moving the
// shifts to the multiplier changes nothing.
//
// Every 8 or 16 query rows read and decode the keys again, so that many new tokens run at
// some 200 TFLOP/s (512 over 8192 keys, MXFP4: 332 us).

// (A lane's tokens as rows of the first product's M: m-tile mt, rows gid and gid + 8
// are tokens 4 gid + 2 mt and 4 gid + 2 mt + 1.)

// Where 16-byte part c of token r's codes lies in a tile of keys (values).
// Lanes of one load differ in r / 4 (keys, read by gid) or r / 8 (values, read by
// tig); those bits choose among the places of equal banks.  MXFP4 keys are read a
// word of one part at a time by all gid, so there the bits choose the part's place
// in its row too.
template <int G, int D>
__device__ __forceinline__ uint32_t row_at(bool values, uint32_t r, uint32_t c) {
    const uint32_t g = values ? r >> 3 : r >> 2;
    if constexpr (D == 64) {      // 4 rows of 2 parts per 128 bytes
        if (!values && G == 32) c ^= (g >> 2) & 1u;
        return (r & ~3u) * 32u + ((r ^ g) & 3u) * 32u + c * 16u;
    } else if constexpr (D == 128) {   // 2 rows of 4 parts
        c ^= values ? g & 2u : G == 32 ? (g >> 1) & 3u : 0u;
        return (r & ~1u) * 64u + ((r ^ g) & 1u) * 64u + c * 16u;
    } else {                      // a row of 8 parts
        c ^= values ? (g << 1) & 6u : G == 32 ? g & 7u : g & 1u;
        return r * 128u + c * 16u;
    }
}

template <int G, int D, int NT>
struct AttentionShape {
    static constexpr int kWarps = attention_warps(D);
    static constexpr int kThreads = kWarps * 32;
    static constexpr int kRows = NT * kTileRows;            // query rows of the block
    static constexpr int kCodes = kTileKeys * (D / 2);      // bytes of a tile's keys
    static constexpr int kScales = kTileKeys * (D / G);
    static constexpr int kTile = 2 * (kCodes + kScales);    // keys, values, their scales
    static constexpr int kPad = D + 4;                      // floats of a row in the join
    static constexpr int kJoin = kRows * kPad * 4;
    static constexpr int kWarpBytes = 2 * kTile > kJoin ? 2 * kTile : kJoin;
    struct Shared {
        alignas(128) uint8_t ring[kWarps][kWarpBytes];
        uint2 queries[NT][D / 16][32];                      // the first product's B, per lane
        float4 key_scales[G == 32 ? kWarps : 1][kTileKeys][G == 32 ? (D + 64) / 128 : 1];
        float stats[kWarps][kRows][2];
        float shrinks[kRows];
    };
};

// Resident blocks per SM, which the registers are held to and a wave counts on: at 4
// blocks the kernels take 119 to 128 registers; 5 blocks spill or lose more to the
// schedule than the warps bring (64 sequences up to 8192 keys, 84.8 against 90.6 us),
// 3 are slower too (87.3).  16 rows of a head of 128 need 3 (32 sequences with 16 query
// heads per key head: 86.3 -> 79.4 us against 2).  16 rows of a head of 64 need 4 (64 sequences
// up to 8192 keys with 16 query heads per key head: 48.4 -> 47.3 us MXFP4, 45.2 -> 44.5 NVFP4
// against 3; 16 up to 2000 keys: 11.3 -> 9.7).
__host__ __device__ constexpr int attention_blocks(int D, int NT) {
    return D == 128 && NT == 2 ? 3 : 4;
}

// Query rows [tile * R, + R) of (sequence b, key/value head) over keys [k_begin, k_end)
// of its n: written out when `whole`, else left at `place` of the workspace.
template <typename In, int G, int D, int NT, bool MULTI>
__device__ __forceinline__ void attend(const AttentionParams &p,
                                       typename AttentionShape<G, D, NT>::Shared &smem, uint32_t b,
                                       uint32_t head, uint32_t tile, uint32_t n, uint32_t k_begin,
                                       uint32_t k_end, bool whole, uint32_t place) {
    using Shape = AttentionShape<G, D, NT>;
    constexpr int W = Shape::kWarps;
    constexpr int KW = D / 32;                 // words of a lane's part of a key
    constexpr int VW = D / 64;                 // words of a lane's part of a value
    constexpr int KG = D / 4 > G ? D / 4 / G : 1;   // groups a lane's part spans
    constexpr int VG = D / 8 > G ? D / 8 / G : 1;
    constexpr int MT = D / 16;                 // m-tiles of the second product
    constexpr int R = Shape::kRows;
    static_assert(NT <= W, "a warp prepares 8 query rows");
    const uint32_t lane = threadIdx.x & 31u, warp = threadIdx.x >> 5;
    const uint32_t gid = lane >> 2, tig = lane & 3u;

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
    uint32_t vref = 0u;                        // MXFP4: reference exponent of this lane's values

    // -- copying a tile -----------------------------------------------------------
    const uint32_t page_mask = (1u << p.c.page_shift) - 1u;
    const uint32_t code_page = (p.c.heads << p.c.page_shift) * (D / 2);
    const uint32_t scale_page = (p.c.heads << p.c.page_shift) * (D / G);
    const int32_t *table = p.table + static_cast<uint64_t>(b) * p.table_stride;
    uint8_t *const mine = smem.ring[warp];
    const uint32_t mine_at = static_cast<uint32_t>(__cvta_generic_to_shared(mine));
    // this lane's 16-byte part of the first rows, in the cache and in the tile; a
    // copy takes kRowsPerCopy rows, and row_at's choice of place for later rows is
    // that of row0 with a bit or two flipped
    constexpr uint32_t kParts = D / 32, kRowsPerCopy = 32 / kParts;
    const uint32_t row0 = lane / kParts, part = lane % kParts;
    const uint32_t code_at = ((head << p.c.page_shift) + row0) * (D / 2) + part * 16u;
    const uint32_t to_k = row_at<G, D>(false, row0, part), to_v = row_at<G, D>(true, row0, part);
    // this lane's part of the scales: 16 tokens of one group, keys' groups first
    constexpr uint32_t kScaleParts = 4u * (D / G);
    const uint32_t scale_half = lane & 1u;
    const uint8_t *scale_src[(kScaleParts + 31) / 32];
#pragma unroll
    for (uint32_t i = 0; i < kScaleParts; i += 32u) {
        const uint32_t at = (i + lane) % kScaleParts, g = (at >> 1) % (D / G);
        scale_src[i / 32u] = p.c.scales[at / (2u * (D / G))] +
                             ((static_cast<uint64_t>(head) * (D / G) + g) << p.c.page_shift);
    }

    // Pages of 32 tokens and more hold a whole tile: one page, and the second half's
    // places are the first half's a constant later (81.9 -> 80.4 us for the 64 sequences
    // above, against the addresses of two pages for every tile).
    const bool one_page = p.c.page_shift >= 5u;
    const uint32_t scale_later = one_page ? 16u * scale_half : 0u;

    // pages of the two halves of the tile at j (-1: none)
    auto pages = [&](uint32_t j, int (&pg)[2]) {
        pg[0] = __ldg(table + (j >> p.c.page_shift));
        pg[1] = pg[0];
        if (!one_page) {
            pg[1] = -1;
            if (j + 16u < n) pg[1] = __ldg(table + ((j + 16u) >> p.c.page_shift));
        }
    };
    // 16 tokens (half h) of the keys' or values' codes
    auto copy_half = [&](uint32_t to, const uint8_t *src, int h, bool values) {
#pragma unroll
        for (uint32_t r = 0; r < 16; r += kRowsPerCopy) {
            const uint32_t row = 16u * h + r;
            // the bits that row changes in row_at(row + row0) beyond its own place
            const uint32_t flip = row_at<G, D>(values, row, 0) ^ (row * (D / 2));
            copy16(to + row * (D / 2) + ((values ? to_v : to_k) ^ flip), src + r * (D / 2));
        }
    };
    auto copy_tile = [&](uint32_t j, int (&pg)[2], uint32_t buffer) {
        const uint32_t to = mine_at + buffer * Shape::kTile, off = j & page_mask;
        if (static_cast<uint32_t>(pg[0]) >= p.c.num_pages) pg[0] = -1;
        const uint32_t page0 = static_cast<uint32_t>(max(pg[0], 0));
        const uint64_t code0 = static_cast<uint64_t>(page0) * code_page + (code_at + off * (D / 2));
        const uint8_t *k = p.c.codes[0] + code0, *v = p.c.codes[1] + code0;
        uint64_t scale = static_cast<uint64_t>(page0) * scale_page + (off + scale_later);
        copy_half(to, k, 0, false);
        copy_half(to + Shape::kCodes, v, 0, true);
        if (one_page) {
            pg[1] = pg[0];
            copy_half(to, k + 16 * (D / 2), 1, false);
            copy_half(to + Shape::kCodes, v + 16 * (D / 2), 1, true);
        } else {                               // the second half begins a page
            if (static_cast<uint32_t>(pg[1]) >= p.c.num_pages) pg[1] = -1;
            const uint32_t page1 = static_cast<uint32_t>(max(pg[1], 0));
            const uint64_t code1 = static_cast<uint64_t>(page1) * code_page + code_at;
            copy_half(to, p.c.codes[0] + code1, 1, false);
            copy_half(to + Shape::kCodes, p.c.codes[1] + code1, 1, true);
            if (scale_half) scale = static_cast<uint64_t>(page1) * scale_page;
        }
#pragma unroll
        for (uint32_t i = 0; i < kScaleParts; i += 32u)
            if (i + lane < kScaleParts)
                copy16(to + 2 * Shape::kCodes + (i + lane) * 16u, scale_src[i / 32u] + scale);
    };

    // -- the warp's tiles: every W-th ----------------------------------------------
    // pages are read a tile before the copies that need them
    uint32_t j = k_begin + warp * kTileKeys;
    int pg[2] = {-1, -1}, pg_next[2] = {-1, -1};
    if (j < k_end) {
        pages(j, pg);
        if (j + W * kTileKeys < k_end) pages(j + W * kTileKeys, pg_next);
        copy_tile(j, pg, 0u);                  // (a page outside the cache becomes -1)
    }
    commit_copies();
    // -- the query rows, normalised: a warp each for 8 of them, while tiles come ---
    if (warp < NT) {
        const uint32_t r = tile * R + warp * kTileRows + gid;
        uint32_t raw[D / 8];
#pragma unroll
        for (int i = 0; i < D / 8; ++i) raw[i] = 0u;
        if (r < p.rows) {
            const uint32_t t = r / p.group, qh = head * p.group + (r - t * p.group);
            const uint64_t token = static_cast<uint64_t>(b) * p.q_len + t;
            const uint8_t *q = p.q + (token * p.q_stride + static_cast<uint64_t>(qh) * D) * 2u;
            if constexpr (G == 16) {           // the elements of this lane's part of a key
                load_words(q + tig * (D / 2), raw);
            } else {
#pragma unroll
                for (int g = 0; g < D / 32; ++g) {
                    uint32_t w[4];
                    load_words(q + g * 64 + tig * 16, w);
#pragma unroll
                    for (int i = 0; i < 4; ++i) raw[4 * g + i] = w[i];
                }
            }
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
        const float grow = p.sign * __uint_as_float(static_cast<uint32_t>(up) << 23);
        if (tig == 0u)
            smem.shrinks[warp * kTileRows + gid] =
                __uint_as_float(static_cast<uint32_t>(254 - up) << 23);
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            float x0, x1, x2, x3;
            widen2<In>(raw[2 * i], x0, x1);
            widen2<In>(raw[2 * i + 1], x2, x3);
            smem.queries[warp][i][lane] = make_uint2(narrow2<__half>(x0 * grow, x1 * grow),
                                                     narrow2<__half>(x2 * grow, x3 * grow));
        }
    }
    __syncthreads();
    float scale[NT][2];                        // factors of a score, columns 2 tig, 2 tig + 1
    int limit[NT][2];                          // keys they see
    const float inv_k =
        G == 16 ? __frcp_rn(__ldg(p.c.gscale)) : kKeyShift;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const uint32_t col = nt * kTileRows + 2u * tig + k;
            scale[nt][k] = smem.shrinks[col] * (p.scale_log2 * inv_k);
            limit[nt][k] = static_cast<int>(n) - static_cast<int>(p.q_len - 1u) +
                           static_cast<int>(min((tile * R + col) / p.group, p.q_len - 1u));
        }
    }

    const uint32_t k_first = 4u * gid, v_first = 8u * tig;   // this lane's tokens of a tile
    // this lane's codes of its even and odd keys, and of its even and odd values (rows
    // four, or two, apart lie that many rows apart: see the reads below)
    const uint8_t *const scales_at = mine + 2 * Shape::kCodes;
    const uint32_t k_scale_at = tig * (D / 4) / G * kTileKeys + k_first;
    const uint32_t v_scale_at = Shape::kScales + gid * (D / 8) / G * kTileKeys + v_first;
    constexpr uint32_t kCycle = D == 64 ? 4 : D == 128 ? 2 : 1;   // rows per 128 bytes
    uint32_t k_at[kCycle], v_at[kCycle];
#pragma unroll
    for (uint32_t x = 0; x < kCycle; ++x) {
        k_at[x] = G == 16 ? row_at<G, D>(false, k_first + x, tig * (D / 8) / 16u) +
                                (tig * (D / 8)) % 16u
                          : row_at<G, D>(false, k_first + x, 0u) + tig * 4u;
        v_at[x] = Shape::kCodes + row_at<G, D>(true, v_first + x, gid * (D / 16) / 16u) +
                  (gid * (D / 16)) % 16u;
    }
    uint32_t buffer = 0;
    for (; j < k_end; j += W * kTileKeys) {
        const int now[2] = {pg[0], pg[1]};
        // the other buffer's tile is done with (the loop ends in __syncwarp)
        const uint32_t next = j + W * kTileKeys;
        pg[0] = pg_next[0];
        pg[1] = pg_next[1];
        if (next < k_end) {
            copy_tile(next, pg, buffer ^ 1u);
            if (next + W * kTileKeys < k_end) pages(next + W * kTileKeys, pg_next);
        }
        commit_copies();
        wait_copies<1>();
        __syncwarp();
        const uint32_t tile_at = buffer * Shape::kTile;
        // a tile some of whose keys some row does not see (warp-uniform; two copies of
        // the body, so that the others carry no test of it)
        const int live = static_cast<int>(n - j);          // tokens of the tile in the sequence
        const bool edge = live < kTileKeys + static_cast<int>(p.q_len - 1u) || now[0] < 0 ||
                          now[1] < 0;
        auto body = [&](auto edge_tag) {
            constexpr bool EDGE = decltype(edge_tag)::value;
            constexpr bool PASSES = EDGE && MULTI && G == 32;
            uint32_t vsc[VG][2];
#pragma unroll
            for (int g = 0; g < VG; ++g)
                load_shared(scales_at + tile_at + v_scale_at + g * kTileKeys, vsc[g]);
            if constexpr (EDGE) {      // scales of values that are not there may be anything
                const int v_live = (tig < 2u ? now[0] : now[1]) < 0 ? 0 : live;
#pragma unroll
                for (int g = 0; g < VG; ++g) {
                    vsc[g][0] = keep_bytes(vsc[g][0], v_first, v_live);
                    vsc[g][1] = keep_bytes(vsc[g][1], v_first + 4, v_live);
                }
            }

            // -- scores: 32 tokens x rows (of keys that are not there: anything) ------------
            float c[2][NT][4];
#pragma unroll
            for (int mt = 0; mt < 2; ++mt)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int k = 0; k < 4; ++k) c[mt][nt][k] = 0.0f;
            if constexpr (G == 16) {
                uint32_t ks[KG][4];                // a token's scale, twice
#pragma unroll
                for (int g = 0; g < KG; ++g) {
                    uint32_t h[2];
                    uint32_t w[1];
                    load_shared(scales_at + tile_at + k_scale_at + g * kTileKeys, w);
                    decode_e4m3x4(w[0], h);
#pragma unroll
                    for (int x = 0; x < 4; ++x) ks[g][x] = both_halves(h[x >> 1], x & 1);
                }
                uint32_t kraw[4][KW];
#pragma unroll
                for (uint32_t x = 0; x < 4; ++x) {
                    const uint8_t *at = mine + tile_at + k_at[x % kCycle] + x / kCycle * 128u;
                    if constexpr (D == 256) {      // two 16-byte parts, which row_at may swap
                        uint32_t lo[4], hi[4];
                        load_shared(at, lo);
                        load_shared(mine + tile_at + (k_at[0] ^ 16u) + x * 128u, hi);
#pragma unroll
                        for (int i = 0; i < 4; ++i) kraw[x][i] = lo[i], kraw[x][i + 4] = hi[i];
                    } else {
                        load_shared(at, kraw[x]);
                    }
                }
#pragma unroll
                for (int w = 0; w < KW; ++w) {
                    uint2 q[NT][2];
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        q[nt][0] = smem.queries[nt][2 * w][lane];
                        q[nt][1] = smem.queries[nt][2 * w + 1][lane];
                    }
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
                            mma16816(c[mt][nt], a[0], a8[0], a[1], a8[1], q[nt][0].x, q[nt][0].y);
                            mma16816(c[mt][nt], a[2], a8[2], a[3], a8[3], q[nt][1].x, q[nt][1].y);
                        }
                    }
                }
            } else {
                // a lane turns one token's scale bytes into fp32 powers for all
                float4 *const mine_scales = smem.key_scales[warp][0];
                constexpr int NG = D / 32, NV = (NG + 3) / 4;
#pragma unroll
                for (int v = 0; v < NV; ++v) {
                    float f[4];
#pragma unroll
                    for (int g = 0; g < 4; ++g)
                        f[g] = 4 * v + g < NG
                                   ? key_power(scales_at[tile_at + (4 * v + g) * kTileKeys + lane])
                                   : 0.0f;
                    mine_scales[lane * NV + v] = make_float4(f[0], f[1], f[2], f[3]);
                }
                __syncwarp();
                float ks[4][4 * NV];
#pragma unroll
                for (int x = 0; x < 4; ++x)
#pragma unroll
                    for (int v = 0; v < NV; ++v) {
                        const float4 f = mine_scales[(k_first + x) * NV + v];
                        ks[x][4 * v] = f.x, ks[x][4 * v + 1] = f.y;
                        ks[x][4 * v + 2] = f.z, ks[x][4 * v + 3] = f.w;
                    }
#pragma unroll
                for (int g = 0; g < NG; ++g) {     // one group: two k-steps, then its scales
                    uint2 q[NT][2];
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        q[nt][0] = smem.queries[nt][2 * g][lane];
                        q[nt][1] = smem.queries[nt][2 * g + 1][lane];
                    }
#pragma unroll
                    for (int mt = 0; mt < 2; ++mt) {
                        uint32_t w[2][1], a[4], a8[4];
#pragma unroll
                        for (uint32_t h = 0; h < 2; ++h) {
                            const uint32_t x = 2u * mt + h;
                            load_shared(mine + tile_at + (k_at[x % kCycle] ^ (g * 16u)) +
                                            x / kCycle * 128u, w[h]);
                        }
                        decode_e2m1x8(w[0][0], a);
                        decode_e2m1x8(w[1][0], a8);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            float part[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                            mma16816(part, a[0], a8[0], a[1], a8[1], q[nt][0].x, q[nt][0].y);
                            mma16816(part, a[2], a8[2], a[3], a8[3], q[nt][1].x, q[nt][1].y);
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                c[mt][nt][k] =
                                    fmaf(part[k], ks[2 * mt + (k >> 1)][g], c[mt][nt][k]);
                        }
                    }
                }
            }

            // -- weights ------------------------------------------------------------------
            uint32_t weights[NT][4];               // B operand: [2 * k-step + half]
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                // Scores of token x, columns 2 tig and 2 tig + 1, rounded before anything is
                // subtracted: the largest of them is then the reference's own number (a fused
                // c scale - m would differ from it by up to half an ulp of a huge score).
                float2 score[4];
                bool seen[4][2];
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    score[x] = __fmul2_rn(make_float2(c[x >> 1][nt][2 * (x & 1)],
                                                      c[x >> 1][nt][2 * (x & 1) + 1]),
                                          make_float2(scale[nt][0], scale[nt][1]));
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        seen[x][k] = true;
                        if constexpr (EDGE)
                            seen[x][k] = (gid < 4u ? now[0] : now[1]) >= 0 &&
                                         static_cast<int>(k_first + x + j) < limit[nt][k];
                    }
                    if (EDGE && !seen[x][0]) score[x].x = -INFINITY;
                    if (EDGE && !seen[x][1]) score[x].y = -INFINITY;
                }
                float top[2];
                top[0] = fmaxf(fmaxf(score[0].x, score[1].x), fmaxf(score[2].x, score[3].x));
                top[1] = fmaxf(fmaxf(score[0].y, score[1].y), fmaxf(score[2].y, score[3].y));
                // (the difference, which is exact for near numbers: m + 15 is not for a huge m)
                if (__any_sync(0xFFFFFFFFu,
                               top[0] - m[nt][0] > kHigh || top[1] - m[nt][1] > kHigh)) {
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
#pragma unroll
                        for (int o = 4; o < 32; o <<= 1)
                            top[k] = fmaxf(top[k], __shfl_xor_sync(0xFFFFFFFFu, top[k], o));
                        // (rounded up: a huge top's neighbours may be 16 apart)
                        const float next = fmaxf(m[nt][k], __fadd_ru(floorf(top[k]), -kBelow));
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
                    const float2 e = __fadd2_rn(score[x], make_float2(-m[nt][0], -m[nt][1]));
                    float w[2] = {ex2_approx(e.x), ex2_approx(e.y)};
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        if (EDGE && !seen[x][k]) w[k] = 0.0f;
                        l[nt][k] += w[k];
                    }
                    weights[nt][x] = transpose8x8(narrow2<__half>(w[0], w[1]));
                }
            }

            // -- weighted values ------------------------------------------------------------
            uint32_t vs[VG][4];                    // scales of tokens x and x + 4 of this lane's 8
            uint32_t e[4];                         // MXFP4: their exponents, 16 bits each
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
                // scales of tokens x and x + 4, 16 bits each
                const uint32_t first = __byte_perm(vsc[0][0], vsc[0][1], 0x5410);
                const uint32_t last = __byte_perm(vsc[0][0], vsc[0][1], 0x7632);
                e[0] = first & 0x00FF00FFu, e[1] = (first >> 8) & 0x00FF00FFu;
                e[2] = last & 0x00FF00FFu, e[3] = (last >> 8) & 0x00FF00FFu;
            }
            // once, or (PASSES) until no scale is left above the reference
            bool again = false;
            do {
                if constexpr (G == 32) {
                    uint32_t top = __vimax3_u16x2(e[0], e[1], vref * 0x00010001u);
                    top = __vimax3_u16x2(e[2], e[3], top);
                    if (__any_sync(0xFFFFFFFFu, top != vref * 0x00010001u)) {
                        uint32_t next = larger_half(top);
                        next = max(next, __shfl_xor_sync(0xFFFFFFFFu, next, 1));
                        next = max(next, __shfl_xor_sync(0xFFFFFFFFu, next, 2));
                        if constexpr (PASSES) {    // by no more than keeps the smallest scale
                            uint32_t low = smallest_half(e);
                            low = min(low, __shfl_xor_sync(0xFFFFFFFFu, low, 1));
                            low = min(low, __shfl_xor_sync(0xFFFFFFFFu, low, 2));
                            next = min(next, max(low + 26u, vref));
                        }
                        const uint32_t up = next - vref;
                        vref = next;
                        // PASSES: in two steps, since no factor below 2^-126 is normal
                        const float fade = ex2_approx(-static_cast<float>(PASSES ? up / 2u : up));
                        const float rest =
                            PASSES ? ex2_approx(-static_cast<float>(up - up / 2u)) : 1.0f;
#pragma unroll
                        for (int i = 0; i < MT; ++i)
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                                for (int k = 0; k < 4; ++k) {
                                    acc[i][nt][k] *= fade;
                                    if constexpr (PASSES) acc[i][nt][k] *= rest;
                                }
                    }
                    if constexpr (PASSES) {
#pragma unroll
                        for (int x = 0; x < 4; ++x) {
                            const uint32_t taken = e[x] & __vcmpleu2(e[x], vref * 0x00010001u);
                            vs[0][x] = relative_power2(taken, reference2(vref));
                            e[x] ^= taken;         // those above the reference wait
                        }
                        again = __any_sync(0xFFFFFFFFu, (e[0] | e[1] | e[2] | e[3]) != 0u);
                    } else {
#pragma unroll
                        for (int x = 0; x < 4; ++x)
                            vs[0][x] = relative_power2(e[x], reference2(vref));
                    }
                }
                uint32_t vraw[8][VW];
#pragma unroll
                for (uint32_t x = 0; x < 8; ++x)
                    load_shared(mine + tile_at + v_at[x % kCycle] + x / kCycle * 128u, vraw[x]);
#pragma unroll
                for (int w = 0; w < VW; ++w) {
#pragma unroll
                    for (int ks2 = 0; ks2 < 2; ++ks2) {
                        // even and odd elements of token pairs (x, x + 4), x = 2 ks2, 2 ks2 + 1
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
                                mma16816(acc[4 * w + i][nt], even[0][i], odd[0][i], even[1][i],
                                         odd[1][i], weights[nt][2 * ks2], weights[nt][2 * ks2 + 1]);
                    }
                }
            } while (PASSES && again);
        };
        if (edge) body(std::true_type{});
        else body(std::false_type{});
        __syncwarp();
        buffer ^= 1u;
    }
    wait_copies<0>();
    __syncwarp();                              // the buffers are free for the join

    // -- join the block's warps ----------------------------------------------------------
    float grain = G == 16 ? 1.0f : exp2f(static_cast<float>(vref) - 139.0f);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) l[nt][k] += __shfl_xor_sync(0xFFFFFFFFu, l[nt][k], o);
    if (G == 32 && __any_sync(0xFFFFFFFFu, vref >= 127u + kHugeScale)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                // (with grain at once: sums of values far below the reference are small)
                const float f = move_power(m[nt][k], l[nt][k]) * grain;
#pragma unroll
                for (int i = 0; i < MT; ++i) {
                    acc[i][nt][k] *= f;
                    acc[i][nt][k + 2] *= f;
                }
            }
        grain = 1.0f;
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const uint32_t r = nt * kTileRows + 2u * tig + k;
            if (gid == 0) {
                smem.stats[warp][r][0] = m[nt][k];
                smem.stats[warp][r][1] = l[nt][k];
            }
#pragma unroll
            for (int i = 0; i < MT; ++i)
                *reinterpret_cast<float2 *>(mine + (r * Shape::kPad + gid * (D / 8) + 2 * i) * 4) =
                    make_float2(acc[i][nt][k] * grain, acc[i][nt][k + 2] * grain);
        }
    }
    __syncthreads();
    const float inv_v = G == 16 ? __frcp_rn(__ldg(p.c.gscale + 1)) : 1.0f;
    for (uint32_t i = threadIdx.x; i < R * (D / 2); i += Shape::kThreads) {
        const uint32_t r = i / (D / 2), d = i % (D / 2) * 2u, row = tile * R + r;
        if (row >= p.rows) break;
        float top = kNoMax, sum = 0.0f, x = 0.0f, y = 0.0f;
#pragma unroll
        for (int w = 0; w < W; ++w) top = fmaxf(top, smem.stats[w][r][0]);
#pragma unroll
        for (int w = 0; w < W; ++w) {
            const float f = ex2_approx(smem.stats[w][r][0] - top);
            const float2 o =
                *reinterpret_cast<const float2 *>(smem.ring[w] + (r * Shape::kPad + d) * 4);
            sum = fmaf(smem.stats[w][r][1], f, sum);
            x = fmaf(o.x, f, x);
            y = fmaf(o.y, f, y);
        }
        if (whole) {
            const uint32_t t = row / p.group, qh = head * p.group + (row - t * p.group);
            const uint64_t slot =
                (static_cast<uint64_t>(b) * p.q_len + t) * p.c.heads * p.group + qh;
            const float norm = sum != 0.0f ? inv_v / sum : 0.0f;   // 0: no key was seen
            *reinterpret_cast<uint32_t *>(p.out + (slot * D + d) * 2u) =
                narrow2<In>(x * norm, y * norm);
            if (d == 0u && p.lse != nullptr)
                p.lse[slot] = sum != 0.0f ? (top + log2f(sum)) * kLn2 : -INFINITY;
        } else {
            const uint64_t at = static_cast<uint64_t>(place) * R + r;
            *reinterpret_cast<float2 *>(p.part + at * D + d) = make_float2(x, y);
            if (d == 0u) p.stat[at] = make_float2(top, sum);
        }
    }
}

// MULTI: several new tokens of a sequence (it makes a difference with MXFP4 alone).
template <typename In, int G, int D, int NT, bool MULTI>
__global__ void __launch_bounds__(attention_warps(D) * 32, attention_blocks(D, NT))
    attention_kernel(const __grid_constant__ AttentionParams p) {
    using Shape = AttentionShape<G, D, NT>;
    __shared__ typename Shape::Shared smem;
    wait_for_producer();
    const uint32_t units = p.c.heads * p.row_tiles;          // of a sequence
    Share share = find_share<Shape::kThreads>(p, units);
    for (const uint32_t first = share.at; share.at < share.end;) {
        // the unit that holds piece `at`, and its pieces in the share
        const uint32_t n = sequence_length(p, share.b), pieces = pieces_of(n);
        const uint32_t within = share.at - share.first;
        const uint32_t unit = within / pieces, piece = within - unit * pieces;
        const uint32_t taken = min(pieces - piece, share.end - share.at);
        // a share's first unit may have begun in another share, its last may end in one
        const uint32_t place = 2u * blockIdx.x + (share.at == first ? 0u : 1u);
        const uint32_t head = unit / p.row_tiles;
        attend<In, G, D, NT, MULTI>(p, smem, share.b, head, unit - head * p.row_tiles, n,
                                    piece * kPieceKeys, min(n, (piece + taken) * kPieceKeys),
                                    taken == pieces, place);
        // the block that holds a unit's first piece says where its parts are: its own
        // place, then one in every share up to the last that begins before the unit's end
        if (piece == 0u && threadIdx.x == 0u && p.joins != nullptr) {
            p.joins[static_cast<uint64_t>(share.b) * units + unit] = make_uint2(
                place, taken == pieces ? 0u : share.of(share.at + pieces - 1u) - blockIdx.x + 1u);
        }
        share.at += taken;
        if (piece + taken == pieces && unit + 1u == units) {
            ++share.b;
            share.first = share.at;
        }
        __syncthreads();                       // the next unit reuses the buffers
    }
    release_dependents();
}

// Warps of a block of the join, by its rows.  64 rows of 74 parts take 0.6 us less
// with 8 warps than with 4.
__host__ __device__ constexpr int join_warps(int rows) { return rows == 1 ? 8 : 4; }

// Joins the parts of query rows' units.  A block takes ROWS rows: one, whose parts its
// warps share (few rows, of many parts), or four, a warp each (many rows, of which
// most have no more than a few parts).  The order of a row's sums is fixed.
template <typename In, int G, int D, int NT, int ROWS>
__global__ void __launch_bounds__(join_warps(ROWS) * 32)
    attention_join_kernel(const __grid_constant__ AttentionParams p) {
    constexpr int kWarps = join_warps(ROWS);
    static_assert(ROWS == 1 || ROWS == kWarps, "a row per block or per warp");
    constexpr int E = D / 32;                  // elements a lane sums
    constexpr uint32_t R = NT * kTileRows;
    constexpr uint32_t kSharing = kWarps / ROWS;          // warps of a row
    // parts a warp has in flight: 32 registers of them, within a round of 32 parts (17
    // sequences of 4 tokens and up to 2000 keys, head 64: 10.6 -> 9.8 us of the whole call
    // against 4)
    constexpr uint32_t kLoads = ROWS == 1 ? 32u / kSharing : 32u / E;
    static_assert(kLoads * kSharing <= 32u, "a factor's lane is its part's place in the round");
    __shared__ float sums[ROWS == 1 ? kWarps : 1][D];
    wait_for_producer();
    const uint32_t lane = threadIdx.x & 31u, warp = threadIdx.x >> 5;
    const uint32_t turn = ROWS == 1 ? warp : 0u;              // of the warps of a row
    const uint32_t unit_row = blockIdx.x * ROWS + (ROWS == 1 ? 0u : warp);   // < 2^31 + 4
    const uint32_t bh = unit_row / p.rows, r = unit_row - bh * p.rows;
    const uint32_t b = bh / p.c.heads, head = bh - b * p.c.heads;
    uint2 join = make_uint2(0u, 0u);
    if (b < p.B) join = __ldcg(p.joins + static_cast<uint64_t>(bh) * p.row_tiles + r / R);
    const uint32_t used = join.y;              // the same in all warps of a row
    if (used > 1u) {
        // part 0, then the first place of each later share
        auto part_at = [&](uint32_t c) {
            return static_cast<uint64_t>(c == 0u ? join.x : (join.x / 2u + c) * 2u) * R + r % R;
        };
        // values of parts c + turn, c + kSharing + turn, ..; past the last one zeros.  The
        // first are on their way before the maxima that weight them.
        float v[kLoads][E];
        auto fetch = [&](uint32_t c) {
#pragma unroll
            for (uint32_t k = 0; k < kLoads; ++k) {
                const uint32_t mine = c + k * kSharing + turn;
#pragma unroll
                for (int x = 0; x < E; ++x) v[k][x] = 0.0f;
                if (mine < used) load_written(p.part + lane * E + part_at(mine) * D, v[k]);
            }
        };
        float m, l = 0.0f, acc[E];
#pragma unroll
        for (int i = 0; i < E; ++i) acc[i] = 0.0f;
        // a lane's share of 32 (few rows: 128) parts' statistics, read together and kept
        // (131072 keys, 74 parts: 37.8 -> 36.4 us; many rows lose 0.2 us by it)
        constexpr uint32_t kHeld = ROWS == 1 ? 4u : 1u;
        float2 st[kHeld];
        auto stats = [&](uint32_t c0) {
#pragma unroll
            for (uint32_t h = 0; h < kHeld; ++h) {
                const uint32_t c = c0 + 32u * h + lane;
                st[h] = make_float2(kNoMax, 0.0f);
                if (c < used) st[h] = __ldcg(p.stat + part_at(c));
            }
        };
        stats(0u);
        fetch(0u);
        m = st[0].x;
#pragma unroll
        for (uint32_t h = 1; h < kHeld; ++h) m = fmaxf(m, st[h].x);
        for (uint32_t c = 32u * kHeld + lane; c < used; c += 32u)
            m = fmaxf(m, __ldcg(p.stat + part_at(c)).x);
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
        // 32 parts at a time: a lane holds one part's factor, and every warp of the
        // row adds the values of its turns
        for (uint32_t first = 0; first < used; first += 32u * kHeld) {
            if (first > 0u) stats(first);
#pragma unroll
            for (uint32_t h = 0; h < kHeld; ++h) {
                const uint32_t c0 = first + 32u * h;
                if (c0 >= used) break;
                const float f = ex2_approx(st[h].x - m);
                l = fmaf(st[h].y, f, l);
                for (uint32_t i = 0; i < 32u && c0 + i < used; i += kLoads * kSharing) {
                    if (c0 + i > 0u) fetch(c0 + i);
#pragma unroll
                    for (uint32_t k = 0; k < kLoads; ++k) {
                        const uint32_t from = (i + k * kSharing + turn) & 31u;
                        const float fc = __shfl_sync(0xFFFFFFFFu, f, from);
#pragma unroll
                        for (int x = 0; x < E; ++x) acc[x] = fmaf(v[k][x], fc, acc[x]);
                    }
                }
            }
        }
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) l += __shfl_xor_sync(0xFFFFFFFFu, l, o);
        const float inv_v = G == 16 ? __frcp_rn(__ldg(p.c.gscale + 1)) : 1.0f;
        const float norm = l != 0.0f ? inv_v / l : 0.0f;
        const uint32_t t = r / p.group, qh = head * p.group + (r - t * p.group);
        const uint64_t row = (static_cast<uint64_t>(b) * p.q_len + t) * p.c.heads * p.group + qh;
        if constexpr (ROWS == 1) {
#pragma unroll
            for (int k = 0; k < E; ++k) sums[warp][lane * E + k] = acc[k];
            __syncthreads();
            for (uint32_t d = 2u * threadIdx.x; d < D; d += 2u * 32u * kWarps) {
                float x = 0.0f, y = 0.0f;
#pragma unroll
                for (int w = 0; w < kWarps; ++w) {
                    x += sums[w][d];
                    y += sums[w][d + 1];
                }
                *reinterpret_cast<uint32_t *>(p.out + (row * D + d) * 2u) =
                    narrow2<In>(x * norm, y * norm);
            }
        } else {
#pragma unroll
            for (int k = 0; k < E; k += 2)
                *reinterpret_cast<uint32_t *>(p.out + (row * D + lane * E + k) * 2u) =
                    narrow2<In>(acc[k] * norm, acc[k + 1] * norm);
        }
        if (lane == 0u && turn == 0u && p.lse != nullptr)
            p.lse[row] = l != 0.0f ? (m + log2f(l)) * kLn2 : -INFINITY;
    }
    release_dependents();
}

}  // namespace pqg
