// The epilogue of a hybrid product, computed in fp32 on its sums before the one
// rounding to the output type (see patch_hybrid_linear in include/patch.h).
//
// A product's last kernel (the GEMM, or the fix-up that joins its partials)
// holds every sum in a register of the thread that stores it, so the epilogue
// costs one read of the residual and no pass of its own (4096x11008, M = 512,
// residual: 56 us, against 67.5 with a kernel of its own over fp32 sums and
// 48-50 for the product alone).
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "patch_common.cuh"
#include "patch_internal.h"

namespace patchk {

// What the last kernel of a product does with its sums.
enum EpiMode { kEpiPlain = 0, kEpiLinear = 1, kEpiGated = 2 };

// The activations, through CUDA's own math functions.
__device__ __forceinline__ float act_relu(float v) { return v < 0.0f ? 0.0f : v; }  // NaN stays NaN
// off by 3 |v| 2^-24: far below zero 1 + erf, and so the result, keeps few digits
// (erfcf keeps them: 4096 tokens, 4096x1024 45 -> 62 us)
__device__ __forceinline__ float act_gelu(float v) { return 0.5f * v * (1.0f + erff(v * 0.70710678f)); }
// x / (1 + exp(-y)) by the hardware's exponential and reciprocal.  __expf is
// documented at 2 + floor(|1.173 y|) ulp and __fdividef at 2: with the sum's
// rounding (10 + 2.4 |y|) 2^-24 of the result (0 below y = -87.3, where the result
// is under 2^-118).  A bf16 output rounds by 2^-9; an fp32 output's sums are off
// by more than that from some tens of terms on (2^-23 for every 16 added).
// Eight warps finish an accumulator, so a short K is bound by these instructions
// (FP8, 2478 tokens, 7168x256 gated: 66 us, 77 with tanhf; 4096 tokens, 4096x1024
// gated, fp32 output: 53 us, 81 by expf and a full division, 62 by an exponential
// with its argument's rounding corrected).
__device__ __forceinline__ float over_one_plus_exp(float x, float y) { return __fdividef(x, 1.0f + __expf(-y)); }
// (1 + tanh(u)) / 2 = 1 / (1 + exp(-y)), y = 2 u; y's own roundings add 5 |y| 2^-24
__device__ __forceinline__ float act_gelu_tanh(float v) {
    return over_one_plus_exp(v, v * fmaf(0.07135481f * v, v, 1.59576912f));
}
__device__ __forceinline__ float act_silu(float v) { return over_one_plus_exp(v, v); }

// `act` is the same for the whole launch: one uniform branch per NV values.
template <int NV>
__device__ __forceinline__ void activate(float (&v)[NV], int act) {
    if (act == kActSilu) {
#pragma unroll
        for (int q = 0; q < NV; ++q) v[q] = act_silu(v[q]);
    } else if (act == kActGelu) {
#pragma unroll
        for (int q = 0; q < NV; ++q) v[q] = act_gelu(v[q]);
    } else if (act == kActGeluTanh) {
#pragma unroll
        for (int q = 0; q < NV; ++q) v[q] = act_gelu_tanh(v[q]);
    } else if (act == kActRelu) {
#pragma unroll
        for (int q = 0; q < NV; ++q) v[q] = act_relu(v[q]);
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

__device__ __forceinline__ float epi_bias(const Epilogue &e, int64_t n) {
    return e.bias ? load_real(e.bias, n, e.bias_fp32) : 0.0f;
}

// NV values of type T to or from consecutive rows of a column, `ld` elements
// apart, the first `count` of them (whole chunks without predicates).
template <class T, int NV, class Put>
__device__ __forceinline__ void for_column(T *y, int64_t ld, int count, const Put &put) {
    if (count >= NV) {
#pragma unroll
        for (int q = 0; q < NV; ++q) put(y[q * ld], q);
    } else {
#pragma unroll
        for (int q = 0; q < NV; ++q)
            if (q < count) put(y[q * ld], q);
    }
}

template <int NV>
__device__ __forceinline__ void store_column(void *Y, int64_t i, int64_t ld, int count, const float (&v)[NV],
                                             int fp32) {
    if (fp32)
        for_column<float, NV>(static_cast<float *>(Y) + i, ld, count, [&](float &y, int q) { y = v[q]; });
    else
        for_column<__nv_bfloat16, NV>(static_cast<__nv_bfloat16 *>(Y) + i, ld, count,
                                      [&](__nv_bfloat16 &y, int q) { y = __float2bfloat16_rn(v[q]); });
}

// NV consecutive tokens m0 .. m0 + count - 1 (count <= NV) of output column n.
// epi_fetch reads what the epilogue adds (or multiplies by), as stored, and is
// called before the sums are ready; epi_store finishes and stores them.  The
// values are converted only there: a conversion right behind its load would
// make every load wait for the one before it.
template <int NV>
__device__ __forceinline__ void epi_fetch(const Epilogue &e, int64_t N, int64_t m0, int64_t n, int count,
                                          uint32_t (&r)[NV]) {
    if (e.mul)
        for_column<const float, NV>(e.mul + m0 * N + n, N, count,
                                    [&](const float &x, int q) { r[q] = __float_as_uint(x); });
    else if (e.residual && e.res_fp32)
        for_column<const float, NV>(static_cast<const float *>(e.residual) + m0 * e.ldr + n, e.ldr, count,
                                    [&](const float &x, int q) { r[q] = __float_as_uint(x); });
    else if (e.residual)
        for_column<const uint16_t, NV>(static_cast<const uint16_t *>(e.residual) + m0 * e.ldr + n, e.ldr, count,
                                       [&](const uint16_t &x, int q) { r[q] = x; });
}

template <int NV>
__device__ __forceinline__ void epi_store(const Epilogue &e, void *Y, int y_fp32, int64_t m0, int64_t n, int count,
                                          float bias, float (&v)[NV], const uint32_t (&r)[NV]) {
#pragma unroll
    for (int q = 0; q < NV; ++q) v[q] += bias;
    activate(v, e.act);
    if (e.mul) {
#pragma unroll
        for (int q = 0; q < NV; ++q) v[q] *= __uint_as_float(r[q]);
    } else if (e.residual) {
        const int shift = e.res_fp32 ? 0 : 16;
#pragma unroll
        for (int q = 0; q < NV; ++q) v[q] = fmaf(e.alpha, v[q], __uint_as_float(r[q] << shift));
    } else {
#pragma unroll
        for (int q = 0; q < NV; ++q) v[q] *= e.alpha;
    }
    store_column(Y, m0 * e.ldy + n, e.ldy, count, v, y_fp32);
}

// The chunks c, c + step, ... of an accumulator finished and stored; `sums(c, v)`
// reads 16 sums, `add` holds what epi_fetch gave for the first chunk.  The next
// chunk's residual is on its way while a chunk is stored.
template <class Sums>
__device__ __forceinline__ void epi_drain(const Epilogue &e, void *Y, int y_fp32, int64_t N, int c, int step,
                                          int64_t m_base, int m_valid, int64_t n, float bias, uint32_t (&add)[16],
                                          const Sums &sums) {
    const bool reads = e.mul || e.residual;
#pragma unroll 1
    for (; c < m_valid; c += step) {
        float v[16];
        uint32_t next[16];
        sums(c, v);
        if (reads) epi_fetch(e, N, m_base + c + step, n, m_valid - c - step, next);
        epi_store(e, Y, y_fp32, m_base + c, n, m_valid - c, bias, v, add);
        if (reads) {
#pragma unroll
            for (int q = 0; q < 16; ++q) add[q] = next[q];
        }
    }
}

// One piece of a gated item in a kernel of whole tiles: this thread's output column n
// (TMEM lane) for the 16-token chunks 16 * grp + 32 j of an accumulator at
// tensor-memory address `acc`; `sums(c0, v)` reads a chunk's sums.
//   gate (mi = 0): act(sum + bias), written back in place chunk by chunk (one
//     copy of the activation code), then held in 16 J registers (J chunks cover
//     the tile) so that the accumulator is free while the up projection runs;
//   up (mi = 1): (sum + bias) * the held gate, stored.
template <int J, class Sums>
__device__ __forceinline__ void gated_piece(const Epilogue &e, void *Y, int y_fp32, int mi, uint32_t acc, int grp,
                                            int64_t m_base, int m_valid, int64_t n, float bias,
                                            uint32_t (&held)[J][16], const Sums &sums) {
    if (mi == 0) {
#pragma unroll 1
        for (int c0 = 16 * grp; c0 < m_valid; c0 += 32) {
            float v[16];
            uint32_t r[16];
            sums(c0, v);
#pragma unroll
            for (int q = 0; q < 16; ++q) v[q] += bias;
            activate(v, e.act);
#pragma unroll
            for (int q = 0; q < 16; ++q) r[q] = __float_as_uint(v[q]);
            tmem_st_32x32b_x16(acc + static_cast<uint32_t>(c0), r);
        }
        tmem_st_wait();
#pragma unroll
        for (int j = 0; j < J; ++j)
            if (16 * grp + 32 * j < m_valid)
                tmem_ld_32x32b_x16(acc + static_cast<uint32_t>(16 * grp + 32 * j), held[j]);
#pragma unroll
        for (int j = 0; j < J; ++j) tmem_ld_wait(held[j]);
    } else {
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const int c0 = 16 * grp + 32 * j;
            if (c0 < m_valid) {
                float v[16];
                sums(c0, v);
#pragma unroll
                for (int q = 0; q < 16; ++q) v[q] = (v[q] + bias) * __uint_as_float(held[j][q]);
                store_column(Y, (m_base + c0) * e.ldy + n, e.ldy, m_valid - c0, v, y_fp32);
            }
        }
    }
}

}  // namespace patchk
