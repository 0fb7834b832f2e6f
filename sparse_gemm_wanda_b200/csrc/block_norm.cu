// The boundary between two sublayers (sm_100a):
//     h = residual + scale * gate * norm_post(branch),   z = norm_pre(h)
// with RMS or layer norms, all in fp32 (see patch_block_norm in
// include/patch.h).
//
// One block per row; the row is held in shared memory as fp32, so every input
// is read once.  A layer norm's variance is the mean of squared distances
// from the mean, not a difference of two large sums.
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "epilogue.cuh"
#include "patch_common.cuh"
#include "patch_internal.h"

namespace patchk {

namespace {

constexpr int kNormThreads = 256;

__device__ __forceinline__ float block_sum(float v, float *red) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    __syncthreads();  // `red` may still be read from the sum before
    if (threadIdx.x % 32 == 0) red[threadIdx.x / 32] = v;
    __syncthreads();
    float s = 0.0f;
    for (int w = 0; w < kNormThreads / 32; ++w) s += red[w];
    return s;
}

__device__ __forceinline__ float block_amax(float v, float *red) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
    __syncthreads();
    if (threadIdx.x % 32 == 0) red[threadIdx.x / 32] = v;
    __syncthreads();
    float s = 0.0f;
    for (int w = 0; w < kNormThreads / 32; ++w) s = fmaxf(s, red[w]);
    return s;
}

// the row in `row` normed in place
__device__ __forceinline__ void norm_row(const NormSpec &n, float *row, int C, float *red) {
    if (n.kind == kNormNone) return;
    float mean = 0.0f;
    if (n.kind == kNormLayer) {
        float s = 0.0f;
        for (int c = threadIdx.x; c < C; c += kNormThreads) s += row[c];
        mean = block_sum(s, red) / static_cast<float>(C);
    }
    float s = 0.0f;
    for (int c = threadIdx.x; c < C; c += kNormThreads) s += (row[c] - mean) * (row[c] - mean);
    const float inv = 1.0f / sqrtf(block_sum(s, red) / static_cast<float>(C) + n.eps);
    for (int c = threadIdx.x; c < C; c += kNormThreads) {
        float v = (row[c] - mean) * inv;
        if (n.weight) v *= load_real(n.weight, c, n.fp32);
        if (n.bias) v += load_real(n.bias, c, n.fp32);
        row[c] = v;
    }
}

__global__ void __launch_bounds__(kNormThreads)
block_norm_kernel(const __grid_constant__ BlockNormParams p) {
    extern __shared__ float row[];
    __shared__ float red[kNormThreads / 32];
    if (threadIdx.x == 0) pdl_trigger();
    pdl_wait();
    const int64_t m = blockIdx.x;
    const int C = p.C;
    for (int c = threadIdx.x; c < C; c += kNormThreads)
        row[c] = load_real(p.branch, m * p.branch_stride + c, p.branch_fp32);
    norm_row(p.post, row, C, red);
    const int64_t g0 = p.gate ? (m / p.gate_tokens) * p.gate_stride : 0;
    for (int c = threadIdx.x; c < C; c += kNormThreads) {
        float v = row[c] * p.scale;
        if (p.gate) v *= load_real(p.gate, g0 + c, p.gate_fp32);
        if (p.residual) v += load_real(p.residual, m * p.residual_stride + c, p.residual_fp32);
        if (p.h) store_real(p.h, m * p.h_stride + c, v, p.h_fp32);
        row[c] = v;
    }
    if (p.z_type == kZNone) return;
    norm_row(p.pre, row, C, red);
    float s = 1.0f;
    if (p.z_type == kZE4m3) {
        float amax = 0.0f;
        for (int c = threadIdx.x; c < C; c += kNormThreads) amax = fmaxf(amax, fabsf(row[c]));
        amax = block_amax(amax, red);
        s = amax > 0.0f ? __fdiv_rn(amax, 448.0f) : 1.0f;
        if (threadIdx.x == 0) p.z_scales[m] = s;
    }
    for (int c = threadIdx.x; c < C; c += kNormThreads) {
        const int64_t i = m * p.z_stride + c;
        if (p.z_type == kZE4m3)
            static_cast<uint8_t *>(p.z)[i] = __nv_cvt_float_to_fp8(__fdiv_rn(row[c], s), __NV_SATFINITE, __NV_E4M3);
        else
            store_real(p.z, i, row[c], p.z_type == kZFp32);
    }
}

cudaError_t norm_attributes() {
    // per device: a 128 KB row needs the opt-in limit
    return cudaFuncSetAttribute(block_norm_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kNormMaxC * 4);
}

}  // namespace

cudaError_t launch_block_norm(const BlockNormParams &p, cudaStream_t stream) {
    cudaError_t err = norm_attributes();
    if (err != cudaSuccess) return err;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(p.M));
    cfg.blockDim = dim3(kNormThreads);
    cfg.dynamicSmemBytes = sizeof(float) * static_cast<size_t>(p.C);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    err = cudaLaunchKernelEx(&cfg, block_norm_kernel, p);
    if (err == cudaSuccess) note_launches(1);
    return err;
}

}  // namespace patchk
