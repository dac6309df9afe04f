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
    int wide;                        // 1 bit would do: every array of every tensor allows 16-byte access
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
__device__ __forceinline__ void narrow(float x, bf16 &o)
{
    const uint32_t b = __builtin_bit_cast(uint32_t, x);
    o.u = x != x ? (uint16_t)((b >> 16) | 0x40) : (uint16_t)((b + 0x7FFF + ((b >> 16) & 1)) >> 16);
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

// Moments in 32 bits (fp64 for fp64 parameters).
template <typename P, typename G, typename R>
__global__ __launch_bounds__(kThreadsA) void k_adamw(AdamwBatch batch, AdamwScalars sc)
{
    const int ti = tensor_of(batch, blockIdx.x);
    const AdamwTensor t = batch.t[ti];
    const long long base = (long long)(blockIdx.x - batch.first[ti]) * kChunk;
    const Coef<R> k(sc);
    P *p = (P *)t.p;
    const G *g = (const G *)t.g;
    R *m = (R *)t.m, *v = (R *)t.v;
    for (int i = threadIdx.x; i < kChunk; i += kThreadsA) {
        const long long at = base + i;
        if (at >= t.n) break;
        R pe = widen(p[at]), me = m[at], vn, root;
        element<R>(k, pe, (R)widen(g[at]), me, v[at], vn, root);
        narrow(pe, p[at]);
        m[at] = me;
        v[at] = vn;
    }
}

__device__ __forceinline__ float from_e4m3(uint32_t code)
{
    return __builtin_amdgcn_cvt_f32_fp8(code, 0);
}

__device__ __forceinline__ uint32_t to_e4m3(float x)
{
    return __builtin_amdgcn_cvt_pk_fp8_f32(x, 0.0f, 0, false) & 0xFF;
}

// Largest magnitude of a block over the wave, as bits: magnitudes order as integers and a
// NaN is above them all, so it is kept.
__device__ __forceinline__ float wave_max(uint32_t b)
{
    for (int o = 32; o; o >>= 1) {
        const uint32_t other = __shfl_xor(b, o, 64);
        b = b > other ? b : other;
    }
    return __builtin_bit_cast(float, b);
}

__device__ __forceinline__ float block_scale(float amax)
{
    const float s = amax * (1.0f / 448.0f);
    return s < 0x1p-100f ? 0x1p-100f : s;   // a NaN stays
}

__device__ __forceinline__ float scaled(float x, float inv)
{
    const float u = x * inv;
    return u > 0.0f && u < 0x1p-9f ? 0x1p-9f : u < 0.0f && u > -0x1p-9f ? -0x1p-9f : u;
}

// Moments in 8 bits.  A wave takes one block of 256 elements at a time, four a lane.
template <typename P, typename G>
__global__ __launch_bounds__(kThreadsA) void k_adamw8(AdamwBatch batch, AdamwScalars sc)
{
    const int ti = tensor_of(batch, blockIdx.x);
    const AdamwTensor t = batch.t[ti];
    const long long base = (long long)(blockIdx.x - batch.first[ti]) * kChunk;
    const Coef<float> k(sc);
    P *p = (P *)t.p;
    const G *g = (const G *)t.g;
    uint8_t *m = (uint8_t *)t.m, *v = (uint8_t *)t.v;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    for (int b = wave; b < kChunk / HQML_ADAMW_BLOCK; b += kThreadsA / 64) {
        const long long at0 = base + b * HQML_ADAMW_BLOCK;
        if (at0 >= t.n) break;
        const long long blk = at0 / HQML_ADAMW_BLOCK;
        const float ms = t.ms[blk], vs = t.vs[blk];
        float me[4], ro[4];
        uint32_t mb = 0, vb = 0;
        for (int j = 0; j < 4; ++j) {
            const long long at = at0 + lane * 4 + j;
            me[j] = ro[j] = 0.0f;
            if (at < t.n) {
                float pe = widen(p[at]), vn;
                me[j] = from_e4m3(m[at]) * ms;
                const float r = from_e4m3(v[at]) * vs;
                element<float>(k, pe, widen(g[at]), me[j], r * r, vn, ro[j]);
                narrow(pe, p[at]);
                const uint32_t a = __builtin_bit_cast(uint32_t, me[j]) & 0x7FFFFFFF;
                const uint32_t c = __builtin_bit_cast(uint32_t, ro[j]) & 0x7FFFFFFF;
                mb = a > mb ? a : mb;
                vb = c > vb ? c : vb;
            }
        }
        const float sm = block_scale(wave_max(mb)), sv = block_scale(wave_max(vb));
        const float im = 1.0f / sm, iv = 1.0f / sv;
        for (int j = 0; j < 4; ++j) {
            const long long at = at0 + lane * 4 + j;
            if (at < t.n) {
                m[at] = (uint8_t)to_e4m3(scaled(me[j], im));
                v[at] = (uint8_t)to_e4m3(scaled(ro[j], iv));
            }
        }
        if (lane == 0) {
            t.ms[blk] = sm;
            t.vs[blk] = sv;
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
        b.wide = 1;
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
