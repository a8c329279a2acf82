// pqg_rmsnorm_quant: argument checks and launch.
#include <algorithm>
#include <cmath>

#include "pqg.h"
#include "pqg_host.cuh"
#include "pqg_launch.cuh"
#include "pqg_norm.cuh"

namespace pqg {
namespace {

template <typename In, Kind KIND, int SLOTS, bool PER_TOKEN>
cudaError_t launch_norm_variant(const NormParams &p, int warps, cudaStream_t stream) {
    auto kernel = rmsnorm_quant_kernel<In, KIND, SLOTS, PER_TOKEN>;
    int device = 0;
    cudaError_t err = cudaGetDevice(&device);
    if (err != cudaSuccess) return err;
    // resident blocks by warps and residual, cached per device; the shared-memory
    // limit is that of the largest
    static OccupancyCache cache[kNormThreads / 32];
    const int which = p.residual != nullptr ? 1 : 0;
    const uint32_t smem = norm_smem(SLOTS, warps, which != 0);
    const bool cached = device >= 0 && device < kOccDevices;
    std::atomic<int> &known = cache[warps - 1].n[cached ? device : 0][which];
    int bps = cached ? known.load(std::memory_order_relaxed) : 0;
    if (bps <= 0) {
        err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                   static_cast<int>(norm_smem(SLOTS, kNormThreads / 32, true)));
        if (err != cudaSuccess) return err;
        if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&bps, kernel, warps * 32, smem) !=
                cudaSuccess || bps < 1)
            bps = 1;
        if (cached) known.store(bps, std::memory_order_relaxed);
    }
    const int64_t ctas = std::min<int64_t>(p.M, static_cast<int64_t>(sm_count(device)) * bps);
    return launch(kernel, ctas, warps * 32, smem, stream, p);
}

// Whether a per-token call of rows of 2 to 8 units takes half the warps with twice the
// elements: a row's two reductions take less then, but fewer loads are in flight.  INT8, us
// with all and with half the warps:
//                     without a residual              with one
//   8 units (K 4096)  512 rows 3.6 / 3.4 (128: 2.6 /  768 rows 5.0 / 4.8, 1024 6.5 / 5.9, 2048
//                     2.8), 2048 9.4 / 7.5, 12288     12.8 / 12.7, 2560 14.6 / 15.2, 8192
//                     47.6 / 39.9                     39.6 / 41.7
//   4, 5 units        1536 rows 4.1 / 4.3, 2048 5.0 / 1024 rows 3.6 / 4.0, 2048 6.1 / 6.1,
//   (K 2048)          5.0, 2560 6.2 / 5.7             6144 15.9 / 17.0
//   2 units (K 1024)  1024 rows 3.0 / 3.3, 4096       1024 rows 3.1 / 3.4, 6144 9.6 / 12.0
//                     6.0 / 7.0
// With groups there is one reduction, and all warps are as fast or faster ([8192, 4096]
// 40.3 / 40.9).
bool half_the_warps(int units, uint32_t M, bool residual) {
    if (units >= 7) return M >= 768 && (!residual || M < 2048);
    return units >= 4 && M >= 2048 && !residual;
}

template <typename In, Kind KIND, bool PER_TOKEN>
cudaError_t launch_norm_slots(const NormParams &p, cudaStream_t stream) {
    // a row is units of 32 lanes x 16 elements; a warp takes 1, 2 or 4 of them, so that
    // 8 warps are enough and as few of them as may be idle (K = 7168: 7 warps x 2)
    const int units = static_cast<int>((p.K / 16u + 31u) / 32u);
    if (PER_TOKEN && units <= 8 && half_the_warps(units, p.M, p.residual != nullptr))
        return launch_norm_variant<In, KIND, 2, PER_TOKEN>(p, (units + 1) / 2, stream);
    if (units <= 8) return launch_norm_variant<In, KIND, 1, PER_TOKEN>(p, units, stream);
    if (units <= 16)
        return launch_norm_variant<In, KIND, 2, PER_TOKEN>(p, (units + 1) / 2, stream);
    return launch_norm_variant<In, KIND, 4, PER_TOKEN>(p, (units + 3) / 4, stream);
}

template <typename In, Kind KIND>
cudaError_t launch_norm_kind(const NormParams &p, cudaStream_t stream) {
    if constexpr (!is_e2m1(KIND))   // FP4 codes have groups of 16 to 128
        if (p.group_lanes == 0u) return launch_norm_slots<In, KIND, true>(p, stream);
    return launch_norm_slots<In, KIND, false>(p, stream);
}

template <typename In>
cudaError_t launch_norm(const NormParams &p, Kind kind, cudaStream_t stream) {
    switch (kind) {
        case Kind::E4M3_FP32: return launch_norm_kind<In, Kind::E4M3_FP32>(p, stream);
        case Kind::E4M3_UE8M0: return launch_norm_kind<In, Kind::E4M3_UE8M0>(p, stream);
        case Kind::INT8_FP32: return launch_norm_kind<In, Kind::INT8_FP32>(p, stream);
        case Kind::E2M1_UE8M0: return launch_norm_kind<In, Kind::E2M1_UE8M0>(p, stream);
        case Kind::E2M1_E4M3: return launch_norm_kind<In, Kind::E2M1_E4M3>(p, stream);
    }
    return cudaErrorInvalidValue;
}

}  // namespace
}  // namespace pqg

extern "C" int pqg_rmsnorm_quant(const void *in, const void *residual, const void *weight,
                                 void *residual_out, void *out, void *scales,
                                 const float *global_scale, int64_t M, int64_t K, int group,
                                 double eps, int in_dtype, int out_dtype, int scale_fmt,
                                 int scale_layout, pqg_stream_t stream) {
    using namespace pqg;
    if (in_dtype != PQG_BF16 && in_dtype != PQG_FP16) return PQG_ERR_INVALID_ARG;
    if (out_dtype != PQG_E4M3 && out_dtype != PQG_INT8 && out_dtype != PQG_E2M1)
        return PQG_ERR_INVALID_ARG;
    if (!(eps >= 0.0) || !std::isfinite(eps)) return PQG_ERR_INVALID_ARG;
    const bool nvfp4 = scale_fmt == PQG_SCALE_E4M3;
    if (nvfp4 != (global_scale != nullptr)) return PQG_ERR_INVALID_ARG;
    int64_t plane = 0;
    const int st = check_geometry(1, M, K, group, scale_fmt, scale_layout, &plane);
    if (st != PQG_OK) return st;
    if (nvfp4 && out_dtype != PQG_E2M1) return PQG_ERR_UNSUPPORTED;
    if (scale_fmt == PQG_SCALE_UE8M0 && out_dtype == PQG_INT8) return PQG_ERR_UNSUPPORTED;
    if (out_dtype == PQG_E2M1 && !nvfp4 &&
        (scale_fmt != PQG_SCALE_UE8M0 || (group != 32 && group != 64 && group != 128)))
        return PQG_ERR_UNSUPPORTED;
    if (K % 16 != 0 || K > kMaxPerTokenK) return PQG_ERR_UNSUPPORTED;   // a row stays in registers
    if (M == 0) return PQG_OK;

    if (in == nullptr || weight == nullptr || out == nullptr || scales == nullptr)
        return PQG_ERR_INVALID_ARG;
    if (!aligned(in, 32) || !aligned(residual, 32) || !aligned(weight, 32) ||
        !aligned(residual_out, 32) || !aligned(out, 16) || !aligned(global_scale, 4))
        return PQG_ERR_ALIGNMENT;
    if ((scale_fmt == PQG_SCALE_FP32 || scale_layout == PQG_UE8M0_PACKED ||
         scale_layout == PQG_UE8M0_TILED_128x4) && !aligned(scales, 4))
        return PQG_ERR_ALIGNMENT;

    const int64_t rows = M * K * 2, weights = K * 2;
    const int64_t out_row = out_dtype == PQG_E2M1 ? K / 2 : K, codes = M * out_row;
    // every output against every input and against the other outputs
    struct Buffer { const void *p; int64_t n; };
    const Buffer reads[] = {{in, rows}, {residual, residual != nullptr ? rows : 0},
                            {weight, weights}, {global_scale, nvfp4 ? 4 : 0}};
    const Buffer writes[] = {{out, codes}, {scales, plane},
                             {residual_out, residual_out != nullptr ? rows : 0}};
    for (const Buffer &w : writes)
        for (const Buffer &r : reads)
            if (r.n > 0 && w.n > 0 && overlaps(w.p, w.n, r.p, r.n) &&
                !(w.p == residual_out && w.p == r.p && r.n == rows && r.p != weight))
                return PQG_ERR_INVALID_ARG;
    for (int i = 0; i < 3; ++i)
        for (int j = 0; j < i; ++j)
            if (writes[i].n > 0 && writes[j].n > 0 &&
                overlaps(writes[i].p, writes[i].n, writes[j].p, writes[j].n))
                return PQG_ERR_INVALID_ARG;

    NormParams p;
    p.in = static_cast<const uint8_t *>(in);
    p.residual = static_cast<const uint8_t *>(residual);
    p.weight = static_cast<const uint8_t *>(weight);
    p.residual_out = static_cast<uint8_t *>(residual_out);
    p.out = static_cast<uint8_t *>(out);
    p.scales = static_cast<uint8_t *>(scales);
    p.gscale = global_scale;
    p.eps = eps;
    p.per_k = 1.0 / static_cast<double>(K);
    p.M = static_cast<uint32_t>(M);
    p.K = static_cast<uint32_t>(K);
    p.out_row_bytes = static_cast<uint32_t>(out_row);
    p.ng = static_cast<uint32_t>(K / group);
    // a group of 16, 32, 64 or 128 is 1, 2, 4 or 8 lanes; any other is the row (0)
    const bool lanes = group == 16 || group == 32 || group == 64 || group == 128;
    p.group_lanes = lanes ? static_cast<uint32_t>(group) / 16u : 0u;
    p.group_shift = 0;
    while (lanes && (1u << p.group_shift) < p.group_lanes) ++p.group_shift;
    p.mpad = static_cast<uint32_t>((M + 3) / 4 * 4);
    p.layout = static_cast<uint32_t>(scale_layout);
    const Kind kind = nvfp4                            ? Kind::E2M1_E4M3
                      : out_dtype == PQG_E2M1          ? Kind::E2M1_UE8M0
                      : scale_fmt == PQG_SCALE_UE8M0 ? Kind::E4M3_UE8M0
                      : out_dtype == PQG_INT8        ? Kind::INT8_FP32
                                                     : Kind::E4M3_FP32;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return launched(in_dtype == PQG_BF16 ? launch_norm<__nv_bfloat16>(p, kind, s)
                                         : launch_norm<__half>(p, kind, s), 1);
}
