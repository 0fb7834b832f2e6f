// The boundary between two sublayers (sm_100a):
//     h = residual + scale * gate * norm_post(branch),   z = norm_pre(h)
// with RMS or layer norms, all in fp32 (see patch_block_norm in
// include/patch.h).
//
// Bound by memory: the branch and the residual are read once, h and z written
// once; gate and weights come from L2 after the first rows.  A row belongs to
// T threads (a block, or a warp with four rows to the block) that hold it in
// registers, NV chunks of 8 consecutive values a thread, from the first load
// to the last store; the norms cost one reduction each (a layer norm two: the
// variance is the mean of squared distances from the mean, not a difference
// of two large sums).  A reduction is shuffles, one barrier and a sum over the
// warps, in an order that depends on the shapes alone.
//
// All loads of a row are issued before the first value is used (PREFETCH; with
// four chunks a thread the residual is read late, for registers).  Rows whose width,
// addresses or strides do not allow 16-byte accesses take the same kernel with
// one value per access, neighbouring threads on neighbouring values.
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "epilogue.cuh"
#include "patch_common.cuh"
#include "patch_internal.h"

namespace patchk {

namespace {

__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    return make_float2(fmaf(a.x, b.x, c.x), fmaf(a.y, b.y, c.y));
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) { return make_float2(a.x * b.x, a.y * b.y); }
__device__ __forceinline__ float2 add2(float2 a, float2 b) { return make_float2(a.x + b.x, a.y + b.y); }
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

// Element types fixed at compile time (kRun: by the call's flags): with every
// flag at run time the conversions' branches and addresses made 46
// instructions a value and bound the kernel.
enum { kBf16 = 0, kFp32 = 1, kRun = 2 };
template <int B, int R, int W>
struct Types {  // of the branch; the residual and h; the weights, biases and gate
    static __device__ __forceinline__ int branch(const BlockNormParams &p) { return B == kRun ? p.branch_fp32 : B; }
    static __device__ __forceinline__ int residual(const BlockNormParams &p) { return R == kRun ? p.residual_fp32 : R; }
    static __device__ __forceinline__ int h(const BlockNormParams &p) { return R == kRun ? p.h_fp32 : R; }
    static __device__ __forceinline__ int gate(const BlockNormParams &p) { return W == kRun ? p.gate_fp32 : W; }
    static __device__ __forceinline__ int weight(const NormSpec &n) { return W == kRun ? n.fp32 : W; }
    static bool fit(const BlockNormParams &p) {
        if (B == kRun) return true;
        auto norm = [](const NormSpec &n) { return (!n.weight && !n.bias) || n.fp32 == W; };
        return p.branch_fp32 == B && (!p.residual || p.residual_fp32 == R) && (!p.h || p.h_fp32 == R) &&
               (!p.gate || p.gate_fp32 == W) && norm(p.post) && norm(p.pre);
    }
};
using AllBf16 = Types<kBf16, kBf16, kBf16>;
using Fp32Stream = Types<kBf16, kFp32, kBf16>;  // a residual stream held in fp32
using AnyTypes = Types<kRun, kRun, kRun>;

// Thread t's place in a row of C values: chunk i holds the 8 values from at(i)
// on (VEC), or at(i), at(i) + 32, ...: a warp's 8 accesses then cover 256
// consecutive values at offsets known at compile time (with offsets in
// multiples of the team's threads 1541x8585 took 51.6 us in place of 37.7,
// 777x1001 with two layer norms 9.1 in place of 7.1).
template <bool VEC>
struct Place {
    int t, threads, C;
    static constexpr int step = VEC ? 1 : 32;
    __device__ __forceinline__ int at(int i) const {
        return VEC ? (i * threads + t) * 8 : (i * threads + (t & ~31)) * 8 + (t & 31);
    }
    __device__ __forceinline__ bool has(int i) const { return at(i) < C; }
    __device__ __forceinline__ bool in(int i, int k) const { return VEC ? has(i) : at(i) + k * step < C; }
    // whether all 8 values lie inside the row
    __device__ __forceinline__ bool full(int i) const { return VEC ? has(i) : at(i) + 7 * step < C; }
};

// 8 values as stored: fp32 one a word; bf16 two a word (VEC) or one
struct Raw {
    uint32_t w[8];
};

// zeros outside the row
template <class T>
__device__ __forceinline__ void load_singles(const T *q, const Place<false> &a, int i, Raw &r) {
    if (a.full(i)) {
#pragma unroll
        for (int k = 0; k < 8; ++k) r.w[k] = q[k * a.step];
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) r.w[k] = a.in(i, k) ? q[k * a.step] : 0u;
    }
}

template <bool VEC>
__device__ __forceinline__ void load8(const void *p, int64_t base, const Place<VEC> &a, int i, int fp32, Raw &r) {
    const int64_t at = base + a.at(i);
    if constexpr (VEC) {
        if (fp32) {
            asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                         : "=r"(r.w[0]), "=r"(r.w[1]), "=r"(r.w[2]), "=r"(r.w[3]), "=r"(r.w[4]), "=r"(r.w[5]),
                           "=r"(r.w[6]), "=r"(r.w[7])
                         : "l"(static_cast<const float *>(p) + at));
        } else {
            const uint4 v = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p) + at);
            r.w[0] = v.x, r.w[1] = v.y, r.w[2] = v.z, r.w[3] = v.w;
        }
    } else if (fp32) {
        load_singles(static_cast<const uint32_t *>(p) + at, a, i, r);
    } else {
        load_singles(static_cast<const uint16_t *>(p) + at, a, i, r);
    }
}

template <bool VEC>
__device__ __forceinline__ void unpack8(const Raw &r, int fp32, float2 (&f)[4]) {
    if (fp32) {
#pragma unroll
        for (int k = 0; k < 4; ++k)
            f[k] = make_float2(__uint_as_float(r.w[2 * k]), __uint_as_float(r.w[2 * k + 1]));
    } else if constexpr (VEC) {
#pragma unroll
        for (int k = 0; k < 4; ++k)
            f[k] = make_float2(__uint_as_float(r.w[k] << 16), __uint_as_float(r.w[k] & 0xFFFF0000u));
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
            f[k] = make_float2(__uint_as_float(r.w[2 * k] << 16), __uint_as_float(r.w[2 * k + 1] << 16));
    }
}

template <class T, class Convert>
__device__ __forceinline__ void store_singles(T *q, const Place<false> &a, int i, const float2 (&f)[4],
                                              const Convert &convert) {
    auto value = [&](int k) { return convert(k & 1 ? f[k / 2].y : f[k / 2].x); };
    if (a.full(i)) {
#pragma unroll
        for (int k = 0; k < 8; ++k) q[k * a.step] = value(k);
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (a.in(i, k)) q[k * a.step] = value(k);
    }
}

template <bool VEC>
__device__ __forceinline__ void store8(void *p, int64_t base, const Place<VEC> &a, int i, int fp32,
                                       const float2 (&f)[4]) {
    const int64_t at = base + a.at(i);
    if constexpr (VEC) {
        if (fp32) {
            asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(static_cast<float *>(p) + at),
                         "f"(f[0].x), "f"(f[0].y), "f"(f[1].x), "f"(f[1].y), "f"(f[2].x), "f"(f[2].y), "f"(f[3].x),
                         "f"(f[3].y)
                         : "memory");
        } else {
            uint32_t w[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const __nv_bfloat162 two = __float22bfloat162_rn(f[k]);
                w[k] = *reinterpret_cast<const uint32_t *>(&two);
            }
            *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p) + at) = make_uint4(w[0], w[1], w[2], w[3]);
        }
    } else if (fp32) {
        store_singles(static_cast<float *>(p) + at, a, i, f, [](float v) { return v; });
    } else {
        store_singles(static_cast<__nv_bfloat16 *>(p) + at, a, i, f, [](float v) { return __float2bfloat16_rn(v); });
    }
}

// The sum or maximum over the threads of a row.  `red` holds two sets of 32
// words, zeroed at the start and used in turn, so one barrier a reduction is
// enough.
struct Team {
    float *red;
    int threads, t;
    int bar;  // the team's named barrier
    int turn = 0;

    template <class Op>
    __device__ __forceinline__ float reduce(float v, Op op) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v = op(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
        if (threads == 32) return v;
        float *slot = red + 32 * turn;
        turn ^= 1;
        if (t % 32 == 0) slot[t / 32] = v;
        asm volatile("bar.sync %0, %1;" ::"r"(bar), "r"(threads) : "memory");
        if (threads <= 256) {
            const float4 a = reinterpret_cast<const float4 *>(slot)[0], b = reinterpret_cast<const float4 *>(slot)[1];
            return op(op(op(a.x, a.y), op(a.z, a.w)), op(op(b.x, b.y), op(b.z, b.w)));
        }
        v = slot[t % 32];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v = op(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
        return v;
    }
    __device__ __forceinline__ float sum(float v) {
        return reduce(v, [](float a, float b) { return a + b; });
    }
    __device__ __forceinline__ float amax(float v) {  // of values >= 0; NaN is passed over
        return reduce(v, [](float a, float b) { return fmaxf(a, b); });
    }
};

// The row normed in place, times `scale`.  Values behind the row are zero
// before and after.
template <class TY, int NV, bool VEC>
__device__ __forceinline__ void norm_row(const NormSpec &n, float scale, const Place<VEC> &at, Team &team,
                                         float2 (&v)[NV][4]) {
    const float inv_c = 1.0f / static_cast<float>(at.C);
    const int fp32 = TY::weight(n);
    if (n.kind == kNormLayer) {
        float2 s = both(0.0f);
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int k = 0; k < 4; ++k) s = add2(s, v[i][k]);
        const float mean = team.sum(s.x + s.y) * inv_c;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (at.full(i)) {
#pragma unroll
                for (int k = 0; k < 4; ++k) v[i][k] = add2(v[i][k], both(-mean));
            } else {
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    if (at.in(i, 2 * k)) v[i][k].x -= mean;
                    if (at.in(i, 2 * k + 1)) v[i][k].y -= mean;
                }
            }
        }
    }
    // the weights are on their way during the reduction
    Raw w[NV];
    if (n.weight) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (at.has(i)) load8(n.weight, 0, at, i, fp32, w[i]);
    }
    float2 s = both(0.0f);
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k) s = fma2(v[i][k], v[i][k], s);
    const float inv = scale / sqrtf(team.sum(s.x + s.y) * inv_c + n.eps);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        if (!at.has(i)) continue;
        float2 f[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) v[i][k] = mul2(v[i][k], both(inv));
        if (n.weight) {
            unpack8<VEC>(w[i], fp32, f);
#pragma unroll
            for (int k = 0; k < 4; ++k) v[i][k] = mul2(v[i][k], f[k]);
        }
        if (n.bias) {
            Raw b;
            load8(n.bias, 0, at, i, fp32, b);
            unpack8<VEC>(b, fp32, f);
#pragma unroll
            for (int k = 0; k < 4; ++k) v[i][k] = fma2(both(scale), f[k], v[i][k]);
        }
    }
}

// The row's e4m3 codes and scale.  A quotient is Markstein's: with r the
// correctly rounded reciprocal of s, q = z r and q + (z - q s) r is the
// correctly rounded z / s (P. Markstein, "Computation of elementary functions
// on the IBM RISC System/6000 processor", 1990) wherever nothing underflows;
// scales outside 2^-60 .. 2^60 take the division.
template <int NV, bool VEC>
__device__ __forceinline__ void store_codes(const BlockNormParams &p, int64_t m, const Place<VEC> &at, Team &team,
                                            const float2 (&v)[NV][4]) {
    float amax = 0.0f;  // values behind the row are zero
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k) amax = fmaxf(amax, fmaxf(fabsf(v[i][k].x), fabsf(v[i][k].y)));
    amax = team.amax(amax);
    const float s = amax > 0.0f ? __fdiv_rn(amax, 448.0f) : 1.0f;
    if (at.t == 0) p.z_scales[m] = s;
    uint8_t *z = static_cast<uint8_t *>(p.z) + m * p.z_stride;
    const bool direct = !(s > 8.7e-19f && s < 1.1e18f);
    const float r = __frcp_rn(s);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        if (!at.has(i)) continue;
        uint32_t c[4];  // two codes each
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            float2 q = mul2(v[i][k], both(r));
            if (direct)
                q = make_float2(__fdiv_rn(v[i][k].x, s), __fdiv_rn(v[i][k].y, s));
            else
                q = fma2(fma2(q, both(-s), v[i][k]), both(r), q);
            c[k] = __nv_cvt_float2_to_fp8x2(q, __NV_SATFINITE, __NV_E4M3);
        }
        if constexpr (VEC) {
            *reinterpret_cast<uint2 *>(z + at.at(i)) = make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (at.in(i, k)) z[at.at(i) + k * at.step] = static_cast<uint8_t>(c[k / 2] >> (8 * (k & 1)));
        }
    }
}

// From the branch's values to the stores; `res(i, f)` gives the residual's chunk i.
template <class TY, int NV, bool VEC, class Res>
__device__ __forceinline__ void finish_row(const BlockNormParams &p, int64_t m, const Place<VEC> &at, Team &team,
                                           float2 (&v)[NV][4], const Res &res) {
    // the scale rides on the post norm's factor, or on the sum with the residual
    const float scale = p.post.kind == kNormNone ? p.scale : 1.0f;
    if (p.post.kind != kNormNone) norm_row<TY>(p.post, p.scale, at, team, v);

    const int64_t g0 = p.gate ? (m / p.gate_tokens) * p.gate_stride : 0;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        if (!at.has(i)) continue;
        float2 f[4];
        if (p.gate) {
            Raw g;
            load8(p.gate, g0, at, i, TY::gate(p), g);
            unpack8<VEC>(g, TY::gate(p), f);
#pragma unroll
            for (int k = 0; k < 4; ++k) v[i][k] = mul2(v[i][k], f[k]);
        }
        if (p.residual) {
            res(i, f);
#pragma unroll
            for (int k = 0; k < 4; ++k) v[i][k] = fma2(both(scale), v[i][k], f[k]);
        } else {
#pragma unroll
            for (int k = 0; k < 4; ++k) v[i][k] = mul2(v[i][k], both(scale));
        }
        if (p.h) store8(p.h, m * p.h_stride, at, i, TY::h(p), v[i]);
    }
    if (p.z_type == kZNone) return;
    if (p.pre.kind != kNormNone) norm_row<TY>(p.pre, 1.0f, at, team, v);
    if (p.z_type == kZE4m3) {
        store_codes(p, m, at, team, v);
    } else {
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (at.has(i)) store8(p.z, m * p.z_stride, at, i, p.z_type == kZFp32, v[i]);
    }
}

template <class TY, int NV, int MAXT, int MINB, bool PREFETCH, bool VEC>
__global__ void __launch_bounds__(MAXT, MINB)
block_norm_kernel(const __grid_constant__ BlockNormParams p, int threads) {
    __shared__ __align__(16) float red[64];
    if (threads > 32) {
        if (threadIdx.x < 64) red[threadIdx.x] = 0.0f;
        __syncthreads();
    }
    // The next kernel starts early where it can be a product of these rows (its
    // weights then stream meanwhile: 1 x 4096 and the product 9.7 us in place of
    // 11.4); other widths' next rows start later but side by side sooner
    // (777x1001, two layer norms, 5.5 in place of 7.1 a call).
    if (threadIdx.x == 0 && p.C % 128 == 0) pdl_trigger();
    pdl_wait();
    const int t = threadIdx.x % threads;
    const int64_t m = static_cast<int64_t>(blockIdx.x) * (blockDim.x / threads) + threadIdx.x / threads;
    if (m >= p.M) return;  // whole warps: several rows to the block only where a row is one warp
    Team team{red, threads, t, 1};  // a row of several warps is alone in its block
    const Place<VEC> at{t, threads, p.C};

    const int64_t r0 = m * p.residual_stride;
    Raw res[NV];
    float2 v[NV][4];
    {
        Raw raw[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (at.has(i)) load8(p.branch, m * p.branch_stride, at, i, TY::branch(p), raw[i]);
        if (PREFETCH && p.residual) {
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (at.has(i)) load8(p.residual, r0, at, i, TY::residual(p), res[i]);
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (at.has(i)) {
                unpack8<VEC>(raw[i], TY::branch(p), v[i]);
            } else {
#pragma unroll
                for (int k = 0; k < 4; ++k) v[i][k] = both(0.0f);
            }
        }
    }
    finish_row<TY>(p, m, at, team, v, [&](int i, float2(&f)[4]) {
        if (!PREFETCH) load8(p.residual, r0, at, i, TY::residual(p), res[i]);
        unpack8<VEC>(res[i], TY::residual(p), f);
    });
}

__device__ __forceinline__ void copy16(uint32_t dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
template <int N>
__device__ __forceinline__ void copies_left() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// The same for many all-bf16 rows of RMS norms without biases and at most a gate
// per channel (the shapes of a prefill): the blocks stay, one to an SM, and every
// team of threads runs down its rows with the next one on its way into shared
// memory.  A thread copies exactly the bytes it will read, so a row needs no
// barrier before its values are used, and no register waits for a value.
// The weights are held in shared memory as fp32, post weight, gate and scale
// multiplied once: per value that is one load and one product in place of two
// or three loads, conversions and products.
// Shared memory: [post C] [pre C] fp32, then [2][teams][planes][NV * threads]
// of 16 bytes, a plane for the branch and one for the residual.
template <int NV, int MAXT>
__global__ void __launch_bounds__(MAXT, 1)
block_norm_stream_kernel(const __grid_constant__ BlockNormParams p, int threads) {
    extern __shared__ uint4 ring_raw[];
    __shared__ __align__(16) float red[(MAXT / 32) * 64];
    for (int i = threadIdx.x; i < (MAXT / 32) * 64; i += blockDim.x) red[i] = 0.0f;
    if (threadIdx.x == 0) pdl_trigger();
    pdl_wait();
    const int C = p.C;
    const bool has_a = p.gate || p.post.weight, has_b = p.pre.weight;
    float *wa = reinterpret_cast<float *>(ring_raw);
    float *wb = wa + (has_a ? C : 0);
    uint4 *ring = reinterpret_cast<uint4 *>(wb + (has_b ? C : 0));

    const int teams = blockDim.x / threads, j = threadIdx.x / threads, t = threadIdx.x % threads;
    Team team{red + 64 * j, threads, t, 1 + j};
    const Place<true> at{t, threads, C};
    const int plane = NV * threads;
    const int planes = p.residual ? 2 : 1;
    const int slot_stride = teams * planes * plane;
    const uint4 *mine = ring + j * planes * plane + t;
    const int64_t step = static_cast<int64_t>(gridDim.x) * teams;
    const int64_t first = static_cast<int64_t>(blockIdx.x) * teams + j;

    auto fetch = [&](int64_t m, int slot) {
        if (m < p.M) {
            const uint32_t dst = smem_u32(mine + slot * slot_stride);
            const uint16_t *b = static_cast<const uint16_t *>(p.branch) + m * p.branch_stride + t * 8;
            const uint16_t *r = static_cast<const uint16_t *>(p.residual) + m * p.residual_stride + t * 8;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                if (!at.has(i)) continue;
                const uint32_t d = dst + 16u * static_cast<uint32_t>(i * threads);
                copy16(d, b + i * threads * 8);
                if (p.residual) copy16(d + 16u * plane, r + i * threads * 8);
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    auto take = [&](int slot, int from, int i, float2(&f)[4]) {
        const uint4 a = mine[slot * slot_stride + from * plane + i * threads];
        unpack8<true>(Raw{{a.x, a.y, a.z, a.w}}, 0, f);
    };
    // v *= the 8 weights of chunk i
    auto times = [&](const float *w, int i, float2(&v)[4]) {
        const float4 a = *reinterpret_cast<const float4 *>(w + at.at(i));
        const float4 b = *reinterpret_cast<const float4 *>(w + at.at(i) + 4);
        v[0] = mul2(v[0], make_float2(a.x, a.y));
        v[1] = mul2(v[1], make_float2(a.z, a.w));
        v[2] = mul2(v[2], make_float2(b.x, b.y));
        v[3] = mul2(v[3], make_float2(b.z, b.w));
    };
    auto inverse_rms = [&](const float2(&v)[NV][4], float eps) {
        float2 s = both(0.0f);
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int k = 0; k < 4; ++k) s = fma2(v[i][k], v[i][k], s);
        return 1.0f / sqrtf(team.sum(s.x + s.y) / static_cast<float>(C) + eps);
    };

    fetch(first, 0);
    for (int c = threadIdx.x; c < C; c += blockDim.x) {
        if (has_a) {
            float a = p.scale;
            if (p.post.weight) a *= load_real(p.post.weight, c, 0);
            if (p.gate) a *= load_real(p.gate, c, 0);
            wa[c] = a;
        }
        if (has_b) wb[c] = load_real(p.pre.weight, c, 0);
    }
    __syncthreads();
    const float scale = has_a ? 1.0f : p.scale;
    int slot = 0;
#pragma unroll 1
    for (int64_t m = first; m < p.M; m += step) {
        fetch(m + step, slot ^ 1);  // the other slot was read to the end in the last pass
        copies_left<1>();           // one group a row, in order: this row's has landed
        float2 v[NV][4];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (at.has(i)) {
                take(slot, 0, i, v[i]);
            } else {
#pragma unroll
                for (int k = 0; k < 4; ++k) v[i][k] = both(0.0f);
            }
        }
        float f = scale;
        if (p.post.kind != kNormNone) f *= inverse_rms(v, p.post.eps);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (!at.has(i)) continue;
            if (has_a) times(wa, i, v[i]);
            if (p.residual) {
                float2 r[4];
                take(slot, 1, i, r);
#pragma unroll
                for (int k = 0; k < 4; ++k) v[i][k] = fma2(both(f), v[i][k], r[k]);
            } else {
#pragma unroll
                for (int k = 0; k < 4; ++k) v[i][k] = mul2(v[i][k], both(f));
            }
            if (p.h) store8(p.h, m * p.h_stride, at, i, 0, v[i]);
        }
        slot ^= 1;
        if (p.z_type == kZNone) continue;
        if (p.pre.kind != kNormNone) {
            const float g = inverse_rms(v, p.pre.eps);
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                if (!at.has(i)) continue;
#pragma unroll
                for (int k = 0; k < 4; ++k) v[i][k] = mul2(v[i][k], both(g));
                if (has_b) times(wb, i, v[i]);
            }
        }
        if (p.z_type == kZE4m3) {
            store_codes(p, m, at, team, v);
        } else {
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (at.has(i)) store8(p.z, m * p.z_stride, at, i, p.z_type == kZFp32, v[i]);
        }
    }
    copies_left<0>();
}

template <class TY, int NV, int MAXT, int MINB, bool PREFETCH, bool VEC>
cudaError_t run_types(const BlockNormParams &p, cudaStream_t stream) {
    const int threads = ((p.C + 8 * NV - 1) / (8 * NV) + 31) / 32 * 32;
    if (threads > MAXT) return cudaErrorInvalidValue;
    const int rows = threads == 32 ? 4 : 1;  // rows to the block
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>((p.M + rows - 1) / rows));
    cfg.blockDim = dim3(static_cast<unsigned>(threads * rows));
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t err = cudaLaunchKernelEx(&cfg, block_norm_kernel<TY, NV, MAXT, MINB, PREFETCH, VEC>, p, threads);
    if (err == cudaSuccess) note_launches(1);
    return err;
}

template <int NV, int MAXT, int MINB, bool PREFETCH>
cudaError_t run(const BlockNormParams &p, bool vec, cudaStream_t stream) {
    if (!vec) return run_types<AnyTypes, NV, MAXT, MINB, PREFETCH, false>(p, stream);
    if (AllBf16::fit(p)) return run_types<AllBf16, NV, MAXT, MINB, PREFETCH, true>(p, stream);
    if (Fp32Stream::fit(p)) return run_types<Fp32Stream, NV, MAXT, MINB, PREFETCH, true>(p, stream);
    return run_types<AnyTypes, NV, MAXT, MINB, PREFETCH, true>(p, stream);
}

constexpr int kNormSmem = 216 * 1024;

// The stream kernel's teams to a block for this call, of all-bf16 rows with a
// residual or without; 0 where it does not take the call.
template <int NV, int MAXT>
int stream_teams(const BlockNormParams &p, int *threads, int *smem) {
    for (const NormSpec *n : {&p.post, &p.pre})
        if (n->kind == kNormLayer || (n->kind != kNormNone && n->bias)) return 0;
    if (p.gate && p.gate_tokens < p.M) return 0;
    *threads = ((p.C + 8 * NV - 1) / (8 * NV) + 31) / 32 * 32;
    if (*threads > MAXT) return 0;
    const int row = 2 * (p.residual ? 2 : 1) * NV * *threads * 16;
    const int weights = 4 * p.C * ((p.gate || p.post.weight ? 1 : 0) + (p.pre.weight ? 1 : 0));
    const int teams = std::min(std::min(MAXT / *threads, 15), (kNormSmem - weights) / row);
    *smem = weights + row * teams;
    return std::max(teams, 0);
}

template <int NV, int MAXT>
cudaError_t run_stream(const BlockNormParams &p, cudaStream_t stream) {
    int threads = 0, smem = 0;
    const int teams = stream_teams<NV, MAXT>(p, &threads, &smem);
    if (teams < 1) return cudaErrorInvalidValue;
    const cudaError_t attr_err = allow_smem<block_norm_stream_kernel<NV, MAXT>>(kNormSmem);
    if (attr_err != cudaSuccess) return attr_err;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(std::min<int64_t>(p.num_sms, (p.M + teams - 1) / teams)));
    cfg.blockDim = dim3(static_cast<unsigned>(threads * teams));
    cfg.dynamicSmemBytes = static_cast<size_t>(smem);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t err = cudaLaunchKernelEx(&cfg, block_norm_stream_kernel<NV, MAXT>, p, threads);
    if (err == cudaSuccess) note_launches(1);
    return err;
}

// whether rows of p (null: absent) start on `align` bytes, whatever the row
bool rows_aligned(const void *p, int64_t stride, int elem, int align) {
    return !p || (reinterpret_cast<uintptr_t>(p) % align == 0 && stride * elem % align == 0);
}

}  // namespace

cudaError_t launch_block_norm(const BlockNormParams &p, cudaStream_t stream) {
    // bf16 chunks are accessed as 16 bytes, fp32 ones as 32, codes as 8
    auto fits = [](const void *q, int64_t stride, int fp32) {
        return rows_aligned(q, stride, fp32 ? 4 : 2, fp32 ? 32 : 16);
    };
    bool vec = p.C % 8 == 0 && fits(p.branch, p.branch_stride, p.branch_fp32) &&
               fits(p.residual, p.residual_stride, p.residual_fp32) && fits(p.gate, p.gate_stride, p.gate_fp32) &&
               fits(p.h, p.h_stride, p.h_fp32) &&
               (p.z_type == kZE4m3 ? rows_aligned(p.z, p.z_stride, 1, 8) : fits(p.z, p.z_stride, p.z_type == kZFp32));
    for (const NormSpec *n : {&p.post, &p.pre}) vec = vec && fits(n->weight, 0, n->fp32) && fits(n->bias, 0, n->fp32);
    const int64_t values = p.M * p.C;
    // Measured on B200, calls in a graph over inputs beyond L2, us a call:
    // - few rows: one chunk a thread, a row's chain of loads, reductions and
    //   stores is then shortest (1 x 4096 2.1 against 2.4 and 3.4 with two and
    //   four chunks; 256 x 5120 with two norms 4.2, 5.0, 7.3);
    // - more: two chunks (512 x 4096 4.4 against 5.5 and 6.5), then four with
    //   two blocks to an SM and the residual read late (2048 x 4096 13.3
    //   against 14.3 and 13.8; 4096 x 5120, two norms, 42 against 53 and 47);
    // - many bf16 rows: the streaming kernel (4096 x 4096 22.3 against 28.3,
    //   two norms on 4096 x 5120 35.5 against 42; but 1024 x 8192 16.1 against
    //   13.8, the rows being too few for its start), with two norms on four
    //   chunks a thread, so more rows are under way (35.5 against 38.1).
    int threads, smem;
    if (vec && AllBf16::fit(p) && p.C >= 1024 && values >= 10000000) {
        if (p.post.kind != kNormNone && stream_teams<4, 768>(p, &threads, &smem) > 1)
            return run_stream<4, 768>(p, stream);
        if (stream_teams<2, 1024>(p, &threads, &smem) > 0) return run_stream<2, 1024>(p, stream);
    }
    if (p.C > 16384) return run<4, 1024, 1, false>(p, vec, stream);
    // Where types are known at run time only (and where accesses are single),
    // two chunks at most: the conversions leave no registers for four (4096 x
    // 4096, fp32 weights, a layer norm 31.6 against 40.8, two with a gate 46.7
    // against 59.8, fp32 rows 39.6 against 52.9), and wide ones are worth it
    // earlier (300 x 4096 4.4 against 5.4).
    const bool any = !vec || !(AllBf16::fit(p) || Fp32Stream::fit(p));
    // An fp32 stream keeps two with one norm (4096 x 4096 33.3 against 34.9, e4m3
    // 34.7 against 36.9; two norms on 4096 x 5120 53 against 49).
    const int64_t one = any && vec ? 500000 : 1500000;
    const int64_t two = any ? 2000000 : Fp32Stream::fit(p) && p.post.kind == kNormNone ? INT64_MAX : 8000000;
    if (p.C <= 256 || (p.C <= 8192 && values <= one)) return run<1, 1024, 1, true>(p, vec, stream);
    if (p.C <= 8192 && (p.C <= 512 || values < two)) return run<2, 512, 1, true>(p, vec, stream);
    if (any && p.C <= 8192)
        return vec ? run_types<AnyTypes, 2, 512, 2, true, true>(p, stream)
                   : run_types<AnyTypes, 2, 512, 2, true, false>(p, stream);
    // (1500 x 12000, a layer norm, 48.2 against 59.3; single accesses, whose
    // 1541 x 8585 takes 46.6 this way, keep four: 37.7)
    if (any)
        return vec ? run_types<AnyTypes, 2, 1024, 1, true, true>(p, stream)
                   : run_types<AnyTypes, 4, 512, 2, false, false>(p, stream);
    return AllBf16::fit(p) ? run_types<AllBf16, 4, 512, 2, false, true>(p, stream)
                           : run_types<Fp32Stream, 4, 512, 2, false, true>(p, stream);
}

}  // namespace patchk
