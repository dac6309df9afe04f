// AdamW over many tensors in one launch.
//
//   m = b1 m + (1 - b1) g,  v = b2 v + (1 - b2) g^2,
//   p = p (1 - lr wd) - (m / (sqrt(v) / sqrt(1 - b2^t) + eps)) lr / (1 - b1^t)
//
// Every element is independent, so the step is bound by memory: 28 bytes an element in fp32
// (22 with bf16 parameters and gradients, 56 in fp64), 16.06 and 10.06 with 8-bit moments.
// One launch covers up to kAdamwTensors tensors: their addresses travel in the kernel
// arguments, so nothing is copied to the device first, and a workgroup finds its tensor by
// bisection over the tensors' first workgroups.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "hqml_ops.hpp"

namespace hqml {
namespace {

constexpr int kThreadsA = 256;
constexpr int kChunk = 4096;   // elements of a workgroup: 16 a thread, or 4 blocks of 256 a wave

struct AdamwTensor {
    void *p;
    const void *g;
    void *m, *v;
    float *ms, *vs;
    long long n;
};

struct AdamwBatch {
    int count;
    unsigned first[kAdamwTensors];   // first workgroup of each tensor
    AdamwTensor t[kAdamwTensors];
};
static_assert(sizeof(AdamwBatch) + sizeof(AdamwScalars) <= 4096, "kernel arguments");

struct bf16 {
    uint16_t u;
};

__device__ __forceinline__ float widen(float x) { return x; }
__device__ __forceinline__ double widen(double x) { return x; }
__device__ __forceinline__ float widen(bf16 x) { return __builtin_bit_cast(float, (uint32_t)x.u << 16); }
__device__ __forceinline__ void narrow(float x, float &o) { o = x; }
__device__ __forceinline__ void narrow(double x, double &o) { o = x; }
// round to nearest even; a NaN stays one
__device__ __forceinline__ void narrow(float x, bf16 &o) { o.u = __builtin_bit_cast(uint16_t, (__bf16)x); }

// n neighbouring values, 16 bytes or fewer at a time and at any alignment of the element: the hardware
// takes them so.
template <int n, typename T>
__device__ __forceinline__ void get(T (&to)[n], const T *from)
{
    struct __attribute__((packed)) All {
        T t[n];
    };
    const All a = *(const All *)from;
#pragma unroll
    for (int k = 0; k < n; ++k) to[k] = a.t[k];
}

template <int n, typename T>
__device__ __forceinline__ void put(T *to, const T (&from)[n])
{
    struct __attribute__((packed)) All {
        T t[n];
    };
    All a;
#pragma unroll
    for (int k = 0; k < n; ++k) a.t[k] = from[k];
    *(All *)to = a;
}

template <typename R>
struct Coef {
    R less, b1, c1, b2, c2, inv_root, eps, size;
    __device__ __forceinline__ explicit Coef(const AdamwScalars &k)
        : less((R)-k.decay), b1((R)k.b1), c1((R)k.c1), b2((R)k.b2), c2((R)k.c2), inv_root((R)k.inv_root),
          eps((R)k.eps), size((R)k.size)
    {
    }
};

// One element.  No contraction: an e4m3 code is decided by the last bit of what it rounds,
// and each product and sum here rounds by itself, as written.
template <typename R>
__device__ __forceinline__ void element(const Coef<R> &k, R &p, R g, R &m, R v, R &v_new, R &root)
{
#pragma clang fp contract(off)
    m = m * k.b1 + g * k.c1;
    v_new = v * k.b2 + (g * g) * k.c2;
    root = sqrt(v_new);
    // one rounding for the decayed parameter: 1 - lr wd, held in R, would add its own
    p = fma(p, k.less, p) - (m / (root * k.inv_root + k.eps)) * k.size;
}

__device__ __forceinline__ int tensor_of(const AdamwBatch &b, unsigned wg)
{
    int lo = 0, hi = b.count - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (b.first[mid] <= wg) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

// `end` elements of a tensor by the workgroup: a thread takes kN neighbours at a time, kAt times before the
// first is computed; the last ones of a tensor (not WHOLE) one at a time.
template <bool WHOLE, typename P, typename G, typename R>
__device__ __forceinline__ void run_chunk(const Coef<R> &k, P *p, const G *g, R *m, R *v, int end)
{
    constexpr int kN = sizeof(R) == 8 ? 2 : 4, kAt = 2;
#pragma unroll 1
    for (int i = threadIdx.x * kN; i < end; i += kThreadsA * kN * kAt) {
        P pe[kAt][kN];
        G ge[kAt][kN];
        R me[kAt][kN], ve[kAt][kN];
#pragma unroll
        for (int a = 0; a < kAt; ++a) {
            const int at = i + a * kThreadsA * kN;
            if (WHOLE || at + kN <= end) get(pe[a], p + at), get(ge[a], g + at), get(me[a], m + at), get(ve[a], v + at);
        }
#pragma unroll
        for (int a = 0; a < kAt; ++a) {
            const int at = i + a * kThreadsA * kN;
            if (WHOLE || at + kN <= end) {
#pragma unroll
                for (int e = 0; e < kN; ++e) {
                    R x = widen(pe[a][e]), vn, root;
                    element<R>(k, x, (R)widen(ge[a][e]), me[a][e], ve[a][e], vn, root);
                    narrow(x, pe[a][e]);
                    ve[a][e] = vn;
                }
                put(p + at, pe[a]), put(m + at, me[a]), put(v + at, ve[a]);
            } else {
                for (int j = at; j < end; ++j) {
                    R x = widen(p[j]), mj = m[j], vn, root;
                    element<R>(k, x, (R)widen(g[j]), mj, v[j], vn, root);
                    narrow(x, p[j]);
                    m[j] = mj;
                    v[j] = vn;
                }
            }
        }
    }
}

// Moments in 32 bits (fp64 for fp64 parameters).  12 tensors with 20 M elements in fp32: 112 us, 5.0 TB/s, what a copy
// reaches; four small ones 4.6 us.
template <typename P, typename G, typename R>
__global__ __launch_bounds__(kThreadsA) void k_adamw(AdamwBatch batch, AdamwScalars sc)
{
    const int ti = tensor_of(batch, blockIdx.x);
    const AdamwTensor t = batch.t[ti];
    const long long base = (long long)(blockIdx.x - batch.first[ti]) * kChunk, left = t.n - base;
    const Coef<R> k(sc);
    P *p = (P *)t.p + base;
    const G *g = (const G *)t.g + base;
    R *m = (R *)t.m + base, *v = (R *)t.v + base;
    if (left >= kChunk) run_chunk<true>(k, p, g, m, v, kChunk);
    else run_chunk<false>(k, p, g, m, v, (int)left);
}

using f32x2 = __attribute__((ext_vector_type(2))) float;

// Largest magnitude of a half wave, as bits: magnitudes order as integers and a NaN is above them
// all, so it is kept.  Within sixteen lanes by DPP, then once across.
__device__ __forceinline__ uint32_t half_wave_max(uint32_t b)
{
    auto with = [&](uint32_t other) { b = b > other ? b : other; };
    with((uint32_t)__builtin_amdgcn_update_dpp(0, (int)b, 0xB1, 0xF, 0xF, true));    // lane ^ 1
    with((uint32_t)__builtin_amdgcn_update_dpp(0, (int)b, 0x4E, 0xF, 0xF, true));    // lane ^ 2
    with((uint32_t)__builtin_amdgcn_update_dpp(0, (int)b, 0x141, 0xF, 0xF, true));   // mirrored in eight
    with((uint32_t)__builtin_amdgcn_update_dpp(0, (int)b, 0x140, 0xF, 0xF, true));   // mirrored in sixteen
    with((uint32_t)__shfl_xor((int)b, 16, 64));
    return b;
}

__device__ __forceinline__ float block_scale(uint32_t amax)
{
    const float s = __builtin_bit_cast(float, amax) * (1.0f / 448.0f);
    return s < 0x1p-100f ? 0x1p-100f : s;   // a NaN stays
}

// What is rounded to a code: not zero where x is not.
__device__ __forceinline__ float scaled(float x, float inv)
{
    const float u = x * inv;
    return u > 0.0f && u < 0x1p-9f ? 0x1p-9f : u < 0.0f && u > -0x1p-9f ? -0x1p-9f : u;
}

__device__ __forceinline__ void from_codes(float (&x)[8], const uint32_t (&w)[2], float scale)
{
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const f32x2 a = __builtin_amdgcn_cvt_pk_f32_fp8(w[h], false), b = __builtin_amdgcn_cvt_pk_f32_fp8(w[h], true);
        x[h * 4] = a.x * scale, x[h * 4 + 1] = a.y * scale;
        x[h * 4 + 2] = b.x * scale, x[h * 4 + 3] = b.y * scale;
    }
}

__device__ __forceinline__ void to_codes(uint32_t (&w)[2], const float (&x)[8], float inv)
{
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(scaled(x[h * 4], inv), scaled(x[h * 4 + 1], inv), 0, false);
        w[h] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(scaled(x[h * 4 + 2], inv), scaled(x[h * 4 + 3], inv), lo, true);
    }
}

// Moments in 8 bits.  Half a wave takes a block of 256 elements, eight a lane, so a wave's
// two blocks share its reductions; kAt pairs of blocks are loaded before the first is computed.  134 M elements in bf16:
// 262 us, 5.1 TB/s, in a long loop (the first hundred passes, while the clocks settle, 270 to 310).
template <typename P, typename G>
__global__ __launch_bounds__(kThreadsA) void k_adamw8(AdamwBatch batch, AdamwScalars sc)
{
    static_assert(HQML_ADAMW_BLOCK == 256, "32 lanes of eight");
    constexpr int kAt = 2, kPer = kThreadsA * 8;   // elements the workgroup takes at once
    const int ti = tensor_of(batch, blockIdx.x);
    const AdamwTensor t = batch.t[ti];
    const long long base = (long long)(blockIdx.x - batch.first[ti]) * kChunk;
    const Coef<float> k(sc);
    P *p = (P *)t.p + base;
    const G *g = (const G *)t.g + base;
    uint8_t *m = (uint8_t *)t.m + base, *v = (uint8_t *)t.v + base;
    float *ms = t.ms + base / HQML_ADAMW_BLOCK, *vs = t.vs + base / HQML_ADAMW_BLOCK;
    const long long left = t.n - base;
    const int end = left < kChunk ? (int)left : kChunk;
#pragma unroll 1
    for (int i0 = threadIdx.x * 8; (i0 & ~511) < end; i0 += kPer * kAt) {   // whole waves: their halves reduce
        P pe[kAt][8];
        G ge[kAt][8];
        uint32_t mw[kAt][2], vw[kAt][2];
        float sm[kAt], sv[kAt];
#pragma unroll
        for (int a = 0; a < kAt; ++a) {
            const int i = i0 + a * kPer;
            if (i + 8 <= end) {
                get(pe[a], p + i), get(ge[a], g + i);
                get(mw[a], (const uint32_t *)(m + i)), get(vw[a], (const uint32_t *)(v + i));
            } else {
                mw[a][0] = mw[a][1] = vw[a][0] = vw[a][1] = 0;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    pe[a][e] = P{}, ge[a][e] = G{};
                    if (i + e >= end) continue;
                    pe[a][e] = p[i + e], ge[a][e] = g[i + e];
                    mw[a][e / 4] |= (uint32_t)m[i + e] << (e % 4 * 8);
                    vw[a][e / 4] |= (uint32_t)v[i + e] << (e % 4 * 8);
                }
            }
            const bool some = (i & ~255) < end;   // the block holds elements
            sm[a] = some ? ms[i >> 8] : 0.0f;
            sv[a] = some ? vs[i >> 8] : 0.0f;
        }
#pragma unroll
        for (int a = 0; a < kAt; ++a) {
            const int i = i0 + a * kPer;
            float me[8], ro[8];
            from_codes(me, mw[a], sm[a]);
            from_codes(ro, vw[a], sv[a]);
            uint32_t mb = 0, vb = 0;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                float x = widen(pe[a][e]), vn;
                const float r = ro[e];
                element<float>(k, x, widen(ge[a][e]), me[e], r * r, vn, ro[e]);
                narrow(x, pe[a][e]);
                const uint32_t am = __builtin_bit_cast(uint32_t, me[e]) & 0x7FFFFFFF;
                const uint32_t ar = __builtin_bit_cast(uint32_t, ro[e]) & 0x7FFFFFFF;
                mb = am > mb ? am : mb;
                vb = ar > vb ? ar : vb;
            }
            const float nm = block_scale(half_wave_max(mb)), nv = block_scale(half_wave_max(vb));
            to_codes(mw[a], me, 1.0f / nm);
            to_codes(vw[a], ro, 1.0f / nv);
            if (i + 8 <= end) {
                put(p + i, pe[a]);
                put((uint32_t *)(m + i), mw[a]), put((uint32_t *)(v + i), vw[a]);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    if (i + e >= end) continue;
                    p[i + e] = pe[a][e];
                    m[i + e] = (uint8_t)(mw[a][e / 4] >> (e % 4 * 8));
                    v[i + e] = (uint8_t)(vw[a][e / 4] >> (e % 4 * 8));
                }
            }
            if ((threadIdx.x & 31) == 0 && (i & ~255) < end) {
                ms[i >> 8] = nm;
                vs[i >> 8] = nv;
            }
        }
    }
}

template <typename F>
hipError_t each_batch(int n, const hqml_adamw_tensor *t, F launch)
{
    int i = 0;
    while (i < n) {
        AdamwBatch b;
        b.count = 0;
        unsigned long long wgs = 0;
        for (; i < n && b.count < kAdamwTensors; ++i) {
            if (t[i].numel == 0) continue;
            const unsigned long long here = (unsigned long long)((t[i].numel + kChunk - 1) / kChunk);
            if (wgs + here > 0x7FFFFFFFull) break;
            b.first[b.count] = (unsigned)wgs;
            b.t[b.count] = {t[i].param, t[i].grad, t[i].m, t[i].v, t[i].m_scale, t[i].v_scale, t[i].numel};
            ++b.count;
            wgs += here;
        }
        if (!b.count) break;
        launch(b, (unsigned)wgs);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

template <typename P, typename G>
hipError_t launch_as(bool eight, const AdamwScalars &k, int n, const hqml_adamw_tensor *t, hipStream_t s)
{
    return each_batch(n, t, [&](const AdamwBatch &b, unsigned wgs) {
        if (eight) k_adamw8<P, G><<<wgs, kThreadsA, 0, s>>>(b, k);
        else k_adamw<P, G, float><<<wgs, kThreadsA, 0, s>>>(b, k);
    });
}

}  // namespace

hipError_t launch_adamw(const hqml_adamw_config &cfg, const AdamwScalars &k, int n, const hqml_adamw_tensor *t,
                        hipStream_t s)
{
    const bool eight = cfg.moments == HQML_MOMENTS_8;
    if (cfg.param_dtype == HQML_DTYPE_FP64)
        return each_batch(n, t, [&](const AdamwBatch &b, unsigned wgs) {
            k_adamw<double, double, double><<<wgs, kThreadsA, 0, s>>>(b, k);
        });
    const bool pb = cfg.param_dtype == HQML_DTYPE_BF16, gb = cfg.grad_dtype == HQML_DTYPE_BF16;
    if (pb) return gb ? launch_as<bf16, bf16>(eight, k, n, t, s) : launch_as<bf16, float>(eight, k, n, t, s);
    return gb ? launch_as<float, bf16>(eight, k, n, t, s) : launch_as<float, float>(eight, k, n, t, s);
}

}  // namespace hqml
