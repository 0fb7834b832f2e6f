// FP8 hybrid GEMM on the sm_100a tensor cores: Y = diag(sx) (QX QW^T) diag(sw).
//
// FP8 values inside dense and 2:4 tiles ("SparseGPT vs Wanda: one-shot LLM
// pruning without retraining", FAQ: prune first, then quantise; the tile
// scheme of "PATCH: Learnable Tile-level Hybrid Sparsity for LLMs", section
// 2): dense k-steps issue tcgen05.mma kind::f8f6f4 (4 x M128 N=BN K32 per
// 128-column k-step), 2:4 k-steps tcgen05.mma.sp kind::f8f6f4 (2 x M128 N=BN
// K64, after one tcgen05.cp of the k-step's metadata block into 4 TMEM
// columns; the metadata of sparse MMA q sits at TMEM column 2q with selector
// 0).  Both e4m3, fp32 accumulation in tensor memory; the epilogue multiplies
// by the token's and the output row's fp32 scales and rounds once.
//
// Work: an output tile is one 128-row band x BN tokens; persistent CTAs take
// tiles c, c + P, ...; two accumulators alternate so one tile's epilogue
// overlaps the next tile's main loop.  With at most half as many tiles as SMs
// (decode token counts on smaller matrices) each tile's k-steps are cut into
// `ksplit` equal ranges, the
// work items are (tile, range), each item leaves its fp32 accumulator in its
// own slot, and a fix-up kernel adds a tile's slots in range order and
// applies the scales, so the result does not depend on timing.  A stage is one k-step: one bulk copy of
// its packed bytes (16 KB dense, or 2 KB metadata + 8 KB kept codes) and one
// TMA load of the BN x 128-byte X tile (128-byte swizzle, rows past M zero).
// Roles (224 threads): warp 0 lane 0 weight producer, warp 6 lane 0 X
// producer (the copies one thread issues are processed largely one after
// another, so the two streams go through two threads), warp 1 lane 0 MMA
// (warp 1 also allocates tensor memory), warps 2..5 (with an epilogue also
// 7..10) the accumulators.  Every mbarrier
// wait is bounded by %globaltimer; a wait that runs out raises the handle's
// status.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <cmath>
#include <mutex>

#include "epilogue.cuh"
#include "patch_common.cuh"
#include "patch_internal.h"

namespace patchk {

namespace {

constexpr int kF8Threads = 224;
// products with an epilogue: + a second group of four epilogue warps (7-10),
// the two taking alternate 16-column chunks (a short K is bound by them)
template <bool EPI>
constexpr int kF8Block = kF8Threads + (EPI ? 128 : 0);
constexpr int kF8Step = 128;                 // columns (bytes of codes) per k-step
constexpr int kF8Aslot = kDenseStepBytes;    // 16 KB: a dense k-step, or metadata + kept codes
constexpr int kF8SmemLimit = 232448;
constexpr int kF8MaxStages = 8;
constexpr uint64_t kF8WaitLimitNs = 2000000000ull;

struct F8Params {
    const uint8_t *packed;
    const uint64_t *table;   // [bands][K/128]
    const float *sw;         // [N] weight row scales
    const float *sx;         // [M] token scales
    int64_t N, K, M;
    int steps, bands, ttiles, tiles;
    int ksplit;      // k-step ranges per tile (1: no split)
    int kper;        // k-steps per range (the last range may hold fewer)
    int items;       // tiles * ksplit
    float *partial;  // ksplit > 1: [items][BN][128] fp32, unscaled
    void *Y;
    int y_fp32;
    uint32_t *status;
    Epilogue epi;
    // gated pairs: the up projection's (p.packed, .. are the gate's)
    const uint8_t *up_packed;
    const uint64_t *up_table;
    const float *up_sw;
    uint32_t *up_status;
    Epilogue up_epi;
    int chain;  // kChainLead, or kChainFollow and kChainLast, with an epilogue only
    uint32_t *chain_flag;
};

// Work item w: tile w / ksplit, k-steps [c0, c1) of it.
__device__ __forceinline__ void f8_item(const F8Params &p, int w, int &tile, int &c0, int &c1) {
    tile = w / p.ksplit;
    c0 = (w % p.ksplit) * p.kper;
    c1 = min(p.steps, c0 + p.kper);
}

__device__ __forceinline__ void store_y(const F8Params &p, int64_t idx, float v) {
    if (p.y_fp32)
        static_cast<float *>(p.Y)[idx] = v;
    else
        static_cast<__nv_bfloat16 *>(p.Y)[idx] = __float2bfloat16_rn(v);
}

template <int BN>
struct F8Cfg {
    static constexpr int kXBytes = BN * kF8Step;
    static constexpr int kStageBytes = kF8Aslot + kXBytes;
    static constexpr int kTail = 1024 + 512;
    static constexpr int kStages = std::min(kF8MaxStages, (kF8SmemLimit - kTail) / kStageBytes);
    static constexpr int kSmem = kStages * kStageBytes + kTail;
    static constexpr int kCols = 2 * BN + 4;
    static constexpr int kTmemCols = kCols <= 128 ? 128 : (kCols <= 256 ? 256 : 512);
    static_assert(kStages >= 2, "at least two stages");
    static_assert(kXBytes % 1024 == 0, "stage regions stay 1024-B aligned");
    static_assert(kCols <= 512, "tensor memory holds 512 columns");
};

template <bool GATED>
__device__ __forceinline__ void raise_timeout(const F8Params &p) {
    atomicOr(p.status, kStatusTimeout);
    if (GATED) atomicOr(p.up_status, kStatusTimeout);
}

// GATED: whole tiles, piece 2q of a CTA a tile of the gate and 2q + 1 the same
// tile of the up projection.
template <int BN, bool EPI, bool GATED>
__global__ void __launch_bounds__(kF8Block<EPI>, 1)
fp8_gemm_kernel(const __grid_constant__ CUtensorMap tmap_x, const __grid_constant__ F8Params p) {
    using C = F8Cfg<BN>;
    constexpr int S = C::kStages;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + S * C::kStageBytes);
    uint64_t *empty = full + S;
    uint64_t *acc_full = empty + S;   // [2]
    uint64_t *acc_empty = acc_full + 2;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(acc_empty + 2);
    volatile uint32_t *abort_flag = tmem_slot + 1;
    volatile uint32_t *never_flag = tmem_slot + 2;
    volatile uint32_t *early_flag = tmem_slot + 3;  // a follower that may run ahead of its wait
    uint64_t *stage_info = reinterpret_cast<uint64_t *>(tmem_slot + 4);  // [S]

    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int cta = blockIdx.x, P = gridDim.x;

    const int chain = EPI ? p.chain : 0;
    if (threadIdx.x == 0) {
        if (!(chain & kChainLead)) pdl_trigger();  // the fix-up (or the next kernel) may start its prologue
        for (int s = 0; s < S; ++s) {
            mbar_init(&full[s], 2);  // the weight and X producers
            mbar_init(&empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&acc_full[b], 1);
            mbar_init(&acc_empty[b], EPI ? 8 : 4);  // epilogue warps
        }
        *never_flag = 0u;
        // X, the weights, the residual and the bias are then complete and visible
        *early_flag = (chain & kChainFollow) && ld_acquire_gpu(p.chain_flag) != 0u ? 1u : 0u;
        uint32_t raised = *reinterpret_cast<volatile uint32_t *>(p.status);
        if (GATED) raised |= *reinterpret_cast<volatile uint32_t *>(p.up_status);
        *abort_flag = (raised & kStatusTimeout) ? 1u : 0u;
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc(tmem_slot, C::kTmemCols);
        tmem_relinquish();
    }
    if (warp == 0 && lane == 0) prefetch_tmap(&tmap_x);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    const bool skip = *abort_flag != 0;
    const bool early = EPI && *early_flag != 0;
    if (threadIdx.x == 64 && ((chain & kChainLead) || (chain && skip))) {  // an epilogue thread
        pdl_wait();
        if (chain & kChainLead) {
            if (cta == 0) raise_chain_flag(p.chain_flag);
            pdl_trigger();
        }
    }

    if (warp == 0) {
        if (lane == 0 && !skip) {
            // ------------------------------------------------------ producer
            // launched as a programmatic dependent: global memory after the wait
            // (early: behind the wait of the chain's first product)
            if (early) fence_async_global();
            else pdl_wait();
            int it = 0;
            bool ok = true;
            for (int i = 0; ok; ++i) {
                const int w = cta + (GATED ? i >> 1 : i) * P;
                if (w >= p.items) break;
                int tile, c0, c1;
                f8_item(p, w, tile, c0, c1);
                const int band = tile / p.ttiles;
                const bool up = GATED && (i & 1);
                const uint64_t *tab = (up ? p.up_table : p.table) + static_cast<int64_t>(band) * p.steps;
                const uint8_t *packed = up ? p.up_packed : p.packed;
                for (int c = c0; c < c1; ++c) {
                    const int s = it % S;
                    const uint32_t ph = (it / S) & 1u;
                    if (it >= S && !mbar_wait_bounded(&empty[s], ph ^ 1u, abort_flag, kF8WaitLimitNs)) {
                        ok = false;
                        break;
                    }
                    const uint64_t e = __ldg(tab + c);
                    const bool sp = (e & kEntrySparse) != 0;
                    const uint64_t first = (e & kEntryOffsetMask) - (sp ? kMetaBlockBytes : 0);
                    const uint32_t bytes = sp ? kMetaBlockBytes + kSparseStepBytes : kDenseStepBytes;
                    stage_info[s] = e;
                    ++it;
                    uint8_t *st = smem + s * C::kStageBytes;
                    mbar_arrive_expect_tx(&full[s], bytes);
                    bulk_g2s(st, packed + first, bytes, &full[s]);
                }
            }
            if (!ok) {
                *abort_flag = 1u;
                raise_timeout<GATED>(p);
            }
            // the last phase issued on every stage lands before the CTA exits
            for (int q = (it > S ? it - S : 0); q < it; ++q)
                mbar_wait_bounded(&full[q % S], (q / S) & 1u, never_flag, kF8WaitLimitNs / 4);
        }
    } else if (warp == 6) {
        if (lane == 0 && !skip) {
            // ---------------------------------------------------- X producer
            // the codes are written by the kernel just before
            if (early) fence_async_global();
            else pdl_wait();
            int it = 0;
            bool ok = true;
            for (int i = 0; ok; ++i) {
                const int w = cta + (GATED ? i >> 1 : i) * P;
                if (w >= p.items) break;
                int tile, c0, c1;
                f8_item(p, w, tile, c0, c1);
                const int tt = tile % p.ttiles;
                for (int c = c0; c < c1; ++c) {
                    const int s = it % S;
                    const uint32_t ph = (it / S) & 1u;
                    if (it >= S && !mbar_wait_bounded(&empty[s], ph ^ 1u, abort_flag, kF8WaitLimitNs)) {
                        ok = false;
                        break;
                    }
                    ++it;
                    mbar_arrive_expect_tx(&full[s], C::kXBytes);
                    tma_load_2d(smem + s * C::kStageBytes + kF8Aslot, &tmap_x, c * kF8Step, tt * BN, &full[s]);
                }
            }
            if (!ok) {
                *abort_flag = 1u;
                raise_timeout<GATED>(p);
            }
        }
    } else if (warp == 1) {
        if (lane == 0 && !skip) {
            // ---------------------------------------------------------- MMA
            const uint32_t e_tmem = tmem_base + static_cast<uint32_t>(2 * BN);
            constexpr uint32_t kIdDense = idesc_e4m3(BN, false);
            constexpr uint32_t kIdSparse = idesc_e4m3(BN, true);
            int it = 0;
            bool ok = true;
            for (int i = 0; ok; ++i) {
                const int w = cta + (GATED ? i >> 1 : i) * P;
                if (w >= p.items) break;
                int tile, c0, c1;
                f8_item(p, w, tile, c0, c1);
                const int buf = i & 1;
                if (i >= 2 &&
                    !mbar_wait_bounded(&acc_empty[buf], ((i >> 1) & 1u) ^ 1u, abort_flag, kF8WaitLimitNs)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(buf * BN);
                for (int c = c0; c < c1; ++c, ++it) {
                    const int s = it % S;
                    const uint32_t ph = (it / S) & 1u;
                    if (!mbar_wait_bounded(&full[s], ph, abort_flag, kF8WaitLimitNs)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t slot = smem_u32(smem + s * C::kStageBytes);
                    const uint32_t b_addr = slot + kF8Aslot;
                    if (stage_info[s] & kEntrySparse) {
                        tmem_cp_128x128b(e_tmem, smem_desc(slot, 16, 128, kSwizzleNone));
#pragma unroll
                        for (int q = 0; q < 2; ++q) {
                            const uint64_t ad = smem_desc(slot + kMetaBlockBytes + q * 32, 16, 512, kSwizzle64B);
                            const uint64_t bd = smem_desc(b_addr + q * 64, 16, 1024, kSwizzle128B);
                            mma_f8_sparse(d_tmem, ad, bd, e_tmem + 2 * q, kIdSparse, (c == c0 && q == 0) ? 0u : 1u);
                        }
                    } else {
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            const uint64_t ad = smem_desc(slot + q * 32, 16, 1024, kSwizzle128B);
                            const uint64_t bd = smem_desc(b_addr + q * 32, 16, 1024, kSwizzle128B);
                            mma_f8(d_tmem, ad, bd, kIdDense, (c == c0 && q == 0) ? 0u : 1u);
                        }
                    }
                    tc_commit(&empty[s]);
                }
                // fires once every MMA of the tile has completed (also after a
                // failure, so the epilogue never frees TMEM under a running MMA)
                tc_commit(&acc_full[buf]);
            }
            if (!ok) {
                *abort_flag = 1u;
                raise_timeout<GATED>(p);
            }
        }
    } else if (!skip) {
        // ------------------------------------------------------- epilogue
        // Y and the partial slots may still be used by earlier kernels
        const bool late = early && p.ksplit == 1 && !p.epi.mul;
        if (!late) pdl_wait();
        const int quad = warp % 4;
        const int c_first = EPI && warp >= 7 ? 16 : 0;  // the second group's first chunk
        constexpr int kChunkStep = EPI ? 32 : 16;
        const int row = quad * 32 + lane;
        const uint32_t lane_base = tmem_base + (static_cast<uint32_t>(quad * 32) << 16);
        // gated: the gate's activated values, held from a tile's first piece to its second
        [[maybe_unused]] uint32_t held[(BN + 31) / 32][16];
        for (int i = 0;; ++i) {
            const int w = cta + (GATED ? i >> 1 : i) * P;
            if (w >= p.items) break;
            const int tile = w / p.ksplit;
            const int buf = i & 1;
            const bool ok = mbar_wait_bounded(&acc_full[buf], (i >> 1) & 1u, never_flag, kF8WaitLimitNs);
            tc_fence_after();
            if (!ok) {
                *abort_flag = 1u;
                raise_timeout<GATED>(p);
                break;
            }
            const int band = tile / p.ttiles, tt = tile % p.ttiles;
            const int64_t n = static_cast<int64_t>(band) * kBand + row;
            const int64_t m_base = static_cast<int64_t>(tt) * BN;
            const int m_valid = static_cast<int>(min(static_cast<int64_t>(BN), p.M - m_base));
            // (scales by plain loads: the read-only path takes no part in a follower's acquire)
            const float swn = (GATED && buf ? p.up_sw : p.sw)[n];
            if (*abort_flag == 0 && p.ksplit > 1) {
                // this range's accumulator, unscaled, into the item's slot
                float *part = p.partial + static_cast<int64_t>(w) * BN * kBand + row;
#pragma unroll 1
                for (int c0 = c_first; c0 < m_valid; c0 += kChunkStep) {
                    uint32_t r[16];
                    tmem_ld_32x32b_x16(lane_base + static_cast<uint32_t>(buf * BN + c0), r);
                    tmem_ld_wait(r);
#pragma unroll
                    for (int q = 0; q < 16; ++q)
                        if (c0 + q < m_valid) part[(c0 + q) * kBand] = __uint_as_float(r[q]);
                }
            } else if (*abort_flag != 0) {
            } else if constexpr (EPI) {
                [[maybe_unused]] uint32_t add[16];
                if constexpr (!GATED) epi_fetch(p.epi, p.N, m_base + c_first, n, m_valid - c_first, add);
                auto scaled = [&](int c0, float(&v)[16]) {
                    uint32_t r[16];
                    tmem_ld_32x32b_x16(lane_base + static_cast<uint32_t>(buf * BN + c0), r);
                    // token scales of the chunk: lane l holds column l % 16's
                    const int ml = c0 + (lane & 15);
                    const float sxl = ml < m_valid ? p.sx[m_base + ml] : 0.0f;
                    tmem_ld_wait(r);
#pragma unroll
                    for (int q = 0; q < 16; ++q)
                        v[q] = __uint_as_float(r[q]) * swn * __shfl_sync(0xFFFFFFFFu, sxl, q);
                };
                if constexpr (GATED)
                    gated_piece(p.epi, p.Y, p.y_fp32, buf, lane_base + static_cast<uint32_t>(buf * BN), c_first / 16,
                                m_base, m_valid, n, epi_bias(buf ? p.up_epi : p.epi, n), held, scaled);
                else
                    epi_drain(p.epi, p.Y, p.y_fp32, p.N, c_first, kChunkStep, m_base, m_valid, n, epi_bias(p.epi, n),
                              add, scaled);
            } else {
#pragma unroll 1
                for (int c0 = c_first; c0 < m_valid; c0 += kChunkStep) {
                    uint32_t r[16];
                    tmem_ld_32x32b_x16(lane_base + static_cast<uint32_t>(buf * BN + c0), r);
                    tmem_ld_wait(r);
#pragma unroll
                    for (int q = 0; q < 16; ++q)
                        if (c0 + q < m_valid) {
                            const int64_t m = m_base + c0 + q;
                            store_y(p, m * p.N + n, __uint_as_float(r[q]) * swn * __ldg(p.sx + m));
                        }
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&acc_empty[buf]);
        }
        if (late) pdl_wait();  // done only when the product before is
    }
    if (threadIdx.x == 64 && (chain & kChainLast) && cta == 0) *p.chain_flag = 0u;  // past its wait
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem_base, C::kTmemCols);
}

// Split-K fix-up: Y[m, n] = (the tile's range accumulators added in range
// order, from zero) * sw[n] * sx[m].  Block (tile, token of the tile), one
// thread per row of the band.  Launched as a programmatic dependent of the
// GEMM; waits for it.
template <int BN, bool EPI>
__global__ void __launch_bounds__(kBand)
fp8_splitk_reduce_kernel(const __grid_constant__ F8Params p) {
    if (threadIdx.x == 0) pdl_trigger();
    pdl_wait();
    const int tile = blockIdx.x, ml = blockIdx.y, row = threadIdx.x;
    const int band = tile / p.ttiles, tt = tile % p.ttiles;
    const int64_t m = static_cast<int64_t>(tt) * BN + ml;
    if (m >= p.M) return;
    const float *src = p.partial + (static_cast<int64_t>(tile) * p.ksplit * BN + ml) * kBand + row;
    const int64_t n = static_cast<int64_t>(band) * kBand + row;
    [[maybe_unused]] uint32_t add[1];
    [[maybe_unused]] float bias = 0.0f;
    if constexpr (EPI) {
        epi_fetch(p.epi, p.N, m, n, 1, add);
        bias = epi_bias(p.epi, n);
    }
    float acc = 0.0f;
    for (int k0 = 0; k0 < p.ksplit; k0 += 8) {
        float v[8];
#pragma unroll
        for (int q = 0; q < 8; ++q)
            v[q] = (k0 + q < p.ksplit) ? __ldcg(src + static_cast<int64_t>(k0 + q) * BN * kBand) : 0.0f;
#pragma unroll
        for (int q = 0; q < 8; ++q)
            if (k0 + q < p.ksplit) acc = __fadd_rn(acc, v[q]);
    }
    acc = acc * __ldg(p.sw + n) * __ldg(p.sx + m);
    if constexpr (EPI) {
        float v[1] = {acc};
        epi_store(p.epi, p.Y, p.y_fp32, m, n, 1, bias, v, add);
    } else {
        store_y(p, m * p.N + n, acc);
    }
}

using EncodeTiledFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                   const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                   const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
    static EncodeTiledFn fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void *ptr = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &ptr, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiledFn>(ptr);
    });
    return fn;
}

// At most half as many tiles as SMs: split each tile's k-steps so that about
// two work items fall on every SM (ranges of equal length, none empty); with
// more tiles the partials and the fix-up cost more than the idle SMs (measured
// on 11008x4096: 86 tiles, 22.3 us split against 17.3).
void split_tiles(const Fp8Launch &g, int tiles, int steps, int peers, int *ksplit, int *kper) {
    *ksplit = 1;
    *kper = steps;
    if (2 * tiles <= g.num_sms && g.pool) {
        const int want = std::min(steps, std::min(16, (2 * g.num_sms + tiles - 1) / tiles));
        if (want > 1) {
            *kper = (steps + want - 1) / want;
            *ksplit = (steps + *kper - 1) / *kper;
        }
    }
    if (!g.epi_on || *ksplit == 1) return;
    // With an epilogue: whole tiles all the same where the fix-up is estimated
    // to cost more than the k-steps it shares out.  Fitted to calls in a graph
    // on B200, f = 0.5 (us, split / whole): 1152x256 M = 16 5.1 / 4.0, M = 1000
    // 16.6 / 10.5, 2432x1024 M = 300 18.0 / 12.4, 1152x1024 M = 129 7.7 / 9.7,
    // 384x2048 M = 16 5.6 / 8.2, M = 1000 13.0 / 14.8.
    const double mn = 1e-6 * static_cast<double>(g.M) * static_cast<double>(g.N);
    const double cols = static_cast<double>(std::min<int64_t>(g.M, g.M <= 64 ? 64 : g.M <= 128 ? 128 : 240));
    const int rounds = (tiles * *ksplit + g.num_sms - 1) / g.num_sms;
    const double whole = 3.0 + 0.03 * cols + 0.31 * steps;
    const double split = 4.4 + 0.009 * cols + 0.3 * *kper + 1.6 * (rounds - 1) + mn * (8.5 + 0.67 * *ksplit);
    // peers side by side: whole tiles next to each other, splits one by one
    const int waves = (peers * tiles + g.num_sms - 1) / g.num_sms;
    if (waves * whole + 2.0 * (peers - 1) <= peers * split) {
        *ksplit = 1;
        *kper = steps;
    }
}

template <int BN, bool EPI, bool GATED = false>
cudaError_t run_fp8_mode(const Fp8Launch *gs, cudaStream_t stream) {
    const Fp8Launch &g = gs[0];
    using C = F8Cfg<BN>;
    const cudaError_t attr_err = allow_smem<fp8_gemm_kernel<BN, EPI, GATED>>(C::kSmem);
    if (attr_err != cudaSuccess) return attr_err;
    EncodeTiledFn enc = encode_fn();
    if (!enc) return cudaErrorInvalidValue;
    // X codes [M, K] uint8 row-major: box = 128 bytes x BN rows, 128-byte
    // swizzle, rows past M read as zero
    CUtensorMap map;
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(g.K), static_cast<cuuint64_t>(g.M)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(g.K)};
    const cuuint32_t box[2] = {static_cast<cuuint32_t>(kF8Step), static_cast<cuuint32_t>(BN)};
    const cuuint32_t estr[2] = {1, 1};
    if (enc(&map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t *>(g.xq), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
        return cudaErrorInvalidValue;
    F8Params p;
    p.packed = g.packed;
    p.table = g.table;
    p.sw = g.sw;
    p.sx = g.sx;
    p.N = g.N;
    p.K = g.K;
    p.M = g.M;
    p.steps = static_cast<int>(g.K / kF8Step);
    p.bands = static_cast<int>(g.N / kBand);
    p.ttiles = static_cast<int>((g.M + BN - 1) / BN);
    p.tiles = p.bands * p.ttiles;
    p.Y = g.Y;
    p.y_fp32 = g.y_fp32;
    p.status = g.status;
    p.epi = g.epi;
    p.chain = g.chain;
    p.chain_flag = g.chain_flag;
    const Fp8Launch &up = gs[GATED ? 1 : 0];
    p.up_packed = up.packed;
    p.up_table = up.table;
    p.up_sw = up.sw;
    p.up_status = up.status;
    p.up_epi = up.epi;
    p.ksplit = 1;
    p.kper = p.steps;
    if (!GATED) split_tiles(g, p.tiles, p.steps, g.peers, &p.ksplit, &p.kper);
    p.items = p.tiles * p.ksplit;
    p.partial = nullptr;
    float *ws = nullptr;
    if (p.ksplit > 1) {
        const size_t bytes = sizeof(float) * static_cast<size_t>(p.items) * BN * kBand;
        const cudaError_t e = cudaMallocFromPoolAsync(reinterpret_cast<void **>(&ws), bytes, g.pool, stream);
        if (e != cudaSuccess) return e;
        p.partial = ws;
    }
    const int grid = std::min(g.num_sms, p.items);
    // programmatic dependent of the X quantisation before it (see the roles)
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t kcfg = {};
    kcfg.gridDim = dim3(static_cast<unsigned>(grid));
    kcfg.blockDim = dim3(kF8Block<EPI>);
    kcfg.dynamicSmemBytes = C::kSmem;
    kcfg.stream = stream;
    kcfg.attrs = attr;
    kcfg.numAttrs = 1;
    cudaError_t err = cudaLaunchKernelEx(&kcfg, fp8_gemm_kernel<BN, EPI, GATED>, map, p);
    if (err == cudaSuccess) note_launches(1);
    if (err == cudaSuccess && p.ksplit > 1) {
        cudaLaunchConfig_t cfg = {};
        // blocks only for the tokens a tile holds
        cfg.gridDim = dim3(static_cast<unsigned>(p.tiles), static_cast<unsigned>(std::min<int64_t>(BN, g.M)));
        cfg.blockDim = dim3(kBand);
        cfg.stream = stream;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        err = cudaLaunchKernelEx(&cfg, fp8_splitk_reduce_kernel<BN, EPI>, p);
        if (err == cudaSuccess) note_launches(1);
    }
    if (ws) {
        const cudaError_t e2 = cudaFreeAsync(ws, stream);
        if (err == cudaSuccess) err = e2;
    }
    return err;
}

template <int BN>
cudaError_t run_fp8(const Fp8Launch &g, cudaStream_t stream) {
    return g.epi_on ? run_fp8_mode<BN, true>(&g, stream) : run_fp8_mode<BN, false>(&g, stream);
}

template <int BN, bool EPI>
void preload_fp8() {
    cudaFuncAttributes a;
    (void)cudaFuncGetAttributes(&a, fp8_gemm_kernel<BN, EPI, false>);
    if (EPI) (void)cudaFuncGetAttributes(&a, fp8_gemm_kernel<BN, true, true>);
    (void)cudaFuncGetAttributes(&a, fp8_splitk_reduce_kernel<BN, EPI>);
}

}  // namespace

void preload_fp8_gemm_kernels() {
    preload_fp8<64, false>();
    preload_fp8<128, false>();
    preload_fp8<240, false>();
    preload_fp8<64, true>();
    preload_fp8<128, true>();
    preload_fp8<240, true>();
}

namespace {

// the two-SM kernel: the bands pair up (prefill table), an even k-step count
bool duo_fits(const Fp8Launch &g) {
    return g.ptable && (g.N / kBand) % 2 == 0 && (g.K / kF8Step) % 2 == 0 && g.K / kF8Step <= 224 &&
           g.force_kernel != 1;
}

// Estimated time (us) of one product of more than 64 tokens with an epilogue
// on the one-band kernel with its partials; duo_fp8_us the two-SM kernel's
// (`pieces` of it a work item).  Fitted to calls in a graph on B200, f = 0.5,
// X quantised (us, one-band / two-SM): 256x8192 M = 129 10.6 / 25, 1024x8192
// M = 300 18 / 27.6, 512x4096 M = 512 15.9 / 20.2, 4096x4096 M = 300 33.7 /
// 18.7, M = 512 22.4 / 20.2.
double one_band_fp8_us(const Fp8Launch &g) {
    const int bn = g.M <= 128 ? 128 : 240;
    const int64_t tiles = (g.N / kBand) * ((g.M + bn - 1) / bn);
    if (tiles > 1 << 24) return 1e9;
    int ksplit, kper;
    split_tiles(g, static_cast<int>(tiles), static_cast<int>(g.K / kF8Step), 1, &ksplit, &kper);
    const int64_t rounds = (tiles * ksplit + g.num_sms - 1) / g.num_sms;
    const double partial_mb = ksplit > 1 ? 4e-6 * static_cast<double>(g.M) * static_cast<double>(g.N) * ksplit : 0.0;
    // unsplit, a tile's own epilogue of bn columns
    const double store = ksplit > 1 ? 0.0 : static_cast<double>(rounds * bn) / 60.0;
    return 8.5 + 0.45 * static_cast<double>(rounds * kper) + partial_mb / 3.0 + store;
}

}  // namespace

double duo_fp8_us(const Fp8Launch &g, const DuoFp8Plan &dp, int pieces) {
    return 10.4 + pieces * dp.cost * static_cast<double>(g.K / kF8Step) / 1750.0;
}

bool takes_duo_fp8(const Fp8Launch &g) {
    if (!duo_fits(g)) return false;
    if (g.force_kernel == 3) return true;
    // plain products: whenever there is more than one token tile
    if (!g.epi_on) return g.M > 128;
    if (g.M <= 64) return false;
    const DuoFp8Plan dp = plan_duo_fp8(g.N, g.M, g.num_sms, g.all_sparse != 0);
    return dp.bn > 0 && duo_fp8_us(g, dp, 1) <= one_band_fp8_us(g);
}

double fp8_us(const Fp8Launch &g) {
    const double one = one_band_fp8_us(g);
    if (!duo_fits(g)) return one;
    const DuoFp8Plan dp = plan_duo_fp8(g.N, g.M, g.num_sms, g.all_sparse != 0);
    return dp.bn > 0 ? std::min(one, duo_fp8_us(g, dp, 1)) : one;
}

bool takes_duo_fp8_gated(const Fp8Launch *gs) {
    const Fp8Launch &g = gs[0];
    if (!duo_fits(gs[0]) || !duo_fits(gs[1])) return false;
    if (g.force_kernel == 3) return true;
    if (g.M <= 64) return false;
    const DuoFp8Plan dp = plan_duo_fp8(g.N, g.M, g.num_sms, gs[0].all_sparse && gs[1].all_sparse);
    return dp.bn > 0 && duo_fp8_us(g, dp, 2) <= fp8_us(gs[0]) + fp8_us(gs[1]);
}

// The gated pair on the one-band kernel: whole tiles of both matrices, against two
// products and their fp32 scratch by the fitted estimates (us, two / one launch:
// X quantised: 2432x256 M = 324 22.3 / 14.9, 1664x1024 M = 209 20.9 / 17.1).
bool takes_one_band_gated_fp8(const Fp8Launch *gs) {
    const Fp8Launch &g = gs[0];
    if (g.force_kernel != 0 && g.force_kernel != 1) return false;
    const int bn = g.M <= 64 ? 64 : g.M <= 128 ? 128 : 240;
    const double cols = static_cast<double>(std::min<int64_t>(g.M, bn));
    const double tiles = static_cast<double>((g.N / kBand) * ((g.M + bn - 1) / bn));
    const double waves = std::ceil(tiles / g.num_sms), steps = static_cast<double>(g.K / kF8Step);
    const double own = 3.0 + waves * (0.045 * cols + 2 * 0.31 * steps);
    const double two = fp8_us(gs[0]) + fp8_us(gs[1]) - 2.0 +
                       2.5e-6 * static_cast<double>(g.M) * static_cast<double>(g.N);
    return g.force_kernel == 1 || own <= two;
}

cudaError_t launch_one_band_gated_fp8(const Fp8Launch *gs, cudaStream_t stream) {
    const Fp8Launch &g = gs[0];
    if (g.K % kF8Step != 0 || g.N % kBand != 0 || g.M < 1) return cudaErrorInvalidValue;
    if (g.M <= 64) return run_fp8_mode<64, true, true>(gs, stream);
    if (g.M <= 128) return run_fp8_mode<128, true, true>(gs, stream);
    return run_fp8_mode<240, true, true>(gs, stream);
}

bool fp8_chains(const Fp8Launch &g) { return g.epi_on && !takes_duo_fp8(g); }

cudaError_t launch_fp8_gemm(const Fp8Launch &g, cudaStream_t stream) {
    if (g.K % kF8Step != 0 || g.N % kBand != 0 || g.M < 1) return cudaErrorInvalidValue;
    if (g.chain && (!g.chain_flag || !fp8_chains(g))) return cudaErrorInvalidValue;
    if (takes_duo_fp8(g)) {
        const DuoFp8Plan dp = plan_duo_fp8(g.N, g.M, g.num_sms, g.all_sparse != 0);
        if (dp.bn > 0) return launch_duo_fp8(g, dp, stream);
    }
    if (g.M <= 64) return run_fp8<64>(g, stream);
    if (g.M <= 128) return run_fp8<128>(g, stream);
    return run_fp8<240>(g, stream);
}

}  // namespace patchk
