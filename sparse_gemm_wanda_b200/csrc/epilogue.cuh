// The epilogue of a hybrid product, computed on its fp32 sums before the one
// rounding to the output type (see patch_hybrid_linear in include/patch.h).
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "patch_internal.h"

namespace patchk {

// The activations in fp32, through CUDA's own math functions.
__device__ __forceinline__ float activate(float v, int act) {
    switch (act) {
        case kActRelu: return v < 0.0f ? 0.0f : v;  // NaN stays NaN
        case kActGelu: return 0.5f * v * (1.0f + erff(v * 0.70710678f));
        case kActGeluTanh: return 0.5f * v * (1.0f + tanhf(0.79788456f * (v + 0.044715f * v * v * v)));
        case kActSilu: return v / (1.0f + expf(-v));
        default: return v;
    }
}

__device__ __forceinline__ float load_real(const void *p, int64_t i, int fp32) {
    return fp32 ? static_cast<const float *>(p)[i] : __bfloat162float(static_cast<const __nv_bfloat16 *>(p)[i]);
}

__device__ __forceinline__ void store_real(void *p, int64_t i, float v, int fp32) {
    if (fp32)
        static_cast<float *>(p)[i] = v;
    else
        static_cast<__nv_bfloat16 *>(p)[i] = __float2bfloat16_rn(v);
}

}  // namespace patchk
