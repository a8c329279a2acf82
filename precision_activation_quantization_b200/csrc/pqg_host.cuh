// Host-side pieces shared by the C entry points: argument checks, the
// process-wide PDL switch and the launch bookkeeping (defined in pqg_api.cu).
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

namespace pqg {

constexpr int64_t kMaxPerTokenK = 16384;

inline bool aligned(const void *p, uintptr_t a) {
    return (reinterpret_cast<uintptr_t>(p) % a) == 0;
}

inline bool overlaps(const void *a, int64_t na, const void *b, int64_t nb) {
    const uintptr_t a0 = reinterpret_cast<uintptr_t>(a), b0 = reinterpret_cast<uintptr_t>(b);
    return a0 < b0 + static_cast<uintptr_t>(nb) && b0 < a0 + static_cast<uintptr_t>(na);
}

// Checks the enum values and sizes shared by the quantizing entry points and
// pqg_scales_bytes, and returns the bytes of one expert's scale plane through
// *plane.
int check_geometry(int64_t num_experts, int64_t M, int64_t K, int group, int scale_fmt,
                   int scale_layout, int64_t *plane);

// Whether launches carry the programmatic-dependent-launch attribute.
bool pdl_enabled();

// The status of a call whose launches ended with `err`: records the error, or
// counts `kernels` launches.
int launched(cudaError_t err, int kernels);

// Launches `kernel` over `blocks` blocks on `stream`, with the PDL attribute
// when it is enabled.
template <typename... Params, typename... Args>
cudaError_t launch(void (*kernel)(Params...), int64_t blocks, int threads, size_t smem,
                   cudaStream_t stream, Args &&...args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(blocks), 1, 1);
    cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl_enabled() ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<Args &&>(args)...);
}

}  // namespace pqg
