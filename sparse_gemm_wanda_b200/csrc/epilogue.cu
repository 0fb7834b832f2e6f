// Epilogues as a pass of their own over fp32 sums (sm_100a).
//
//     linear:  Y[m,n] = residual[m,n] + alpha * act(sum[m,n] + bias[n])
//     gated:   Y[m,n] = act(gate[m,n] + bias_gate[n]) * (up[m,n] + bias_up[n])
//
// Bound by memory: 4 bytes of sums (twice for the gated pair), the residual
// and the output per element.
#include <cuda_runtime.h>
#include <stdint.h>

#include "epilogue.cuh"
#include "patch_common.cuh"
#include "patch_internal.h"

namespace patchk {

namespace {

constexpr int kEpiThreads = 128;  // one band of columns

__global__ void __launch_bounds__(kEpiThreads)
epilogue_kernel(const float *sum, const float *up, void *Y, int y_fp32, int64_t N, int64_t M,
                const __grid_constant__ Epilogue e) {
    if (threadIdx.x == 0) pdl_trigger();
    pdl_wait();
    const int64_t n = static_cast<int64_t>(blockIdx.x) * kEpiThreads + threadIdx.x;
    const float b = e.bias ? load_real(e.bias, n, e.bias_fp32) : 0.0f;
    const float b2 = e.bias2 ? load_real(e.bias2, n, e.bias_fp32) : 0.0f;
    for (int64_t m = blockIdx.y; m < M; m += gridDim.y) {
        float v = activate(sum[m * N + n] + b, e.act);
        if (up) {
            v *= up[m * N + n] + b2;
        } else {
            v *= e.alpha;
            if (e.residual) v += load_real(e.residual, m * e.ldr + n, e.res_fp32);
        }
        store_real(Y, m * e.ldy + n, v, y_fp32);
    }
}

}  // namespace

void preload_epilogue_kernels() {
    cudaFuncAttributes a;
    (void)cudaFuncGetAttributes(&a, epilogue_kernel);
}

cudaError_t launch_epilogue(const float *sum, const float *up, void *Y, int y_fp32, int64_t N, int64_t M,
                            const Epilogue &e, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(N / kEpiThreads), static_cast<unsigned>(M < 65535 ? M : 65535));
    cfg.blockDim = dim3(kEpiThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t err = cudaLaunchKernelEx(&cfg, epilogue_kernel, sum, up, Y, y_fp32, N, M, e);
    if (err == cudaSuccess) note_launches(1);
    return err;
}

}  // namespace patchk
