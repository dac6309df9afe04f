// Dense layer: y = alpha act(x w^T + bias) + residual and its gradients.
//
// All three products of the layer are one tile kernel, C(i, j) = sum_k A(i, k) B(k, j), with
// the operands addressed by two strides each:
//   forward  C = x w^T      dx = dz w      dw = dz^T x
// and an epilogue that finishes the value where the sum ends.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>

#include "hqml_ops.hpp"

namespace hqml {
namespace {

struct bf16 {
    uint16_t u;
};

__device__ __forceinline__ float widen(float x) { return x; }
__device__ __forceinline__ float widen(bf16 x) { return __builtin_bit_cast(float, (uint32_t)x.u << 16); }
__device__ __forceinline__ void narrow(float x, float &o) { o = x; }
// round to nearest even; a NaN stays one
__device__ __forceinline__ void narrow(float x, bf16 &o)
{
    const uint32_t b = __builtin_bit_cast(uint32_t, x);
    o.u = x != x ? (uint16_t)((b >> 16) | 0x40) : (uint16_t)((b + 0x7FFF + ((b >> 16) & 1)) >> 16);
}

// Phi(z), the normal distribution function.
__device__ __forceinline__ float normal_cdf(float z) { return 0.5f * (1.0f + erff(z * 0.70710678f)); }
__device__ __forceinline__ float logistic(float z) { return 1.0f / (1.0f + expf(-z)); }

__device__ __forceinline__ float activate(float z, int act)
{
    switch (act) {
    case HQML_ACT_RELU: return z < 0.0f ? 0.0f : z;
    case HQML_ACT_GELU: return z * normal_cdf(z);
    case HQML_ACT_SILU: return z * logistic(z);
    case HQML_ACT_TANH: return tanhf(z);
    case HQML_ACT_SIGMOID: return logistic(z);
    default: return z;
    }
}

__device__ __forceinline__ float slope(float z, int act)
{
    switch (act) {
    case HQML_ACT_RELU: return z > 0.0f ? 1.0f : 0.0f;
    case HQML_ACT_GELU: return normal_cdf(z) + z * expf(-0.5f * z * z) * 0.39894228f;
    case HQML_ACT_SILU: {
        const float f = logistic(z);
        return f * (1.0f + z * (1.0f - f));
    }
    case HQML_ACT_TANH: {
        const float t = tanhf(z);
        return 1.0f - t * t;
    }
    case HQML_ACT_SIGMOID: {
        const float f = logistic(z);
        return f * (1.0f - f);
    }
    default: return 1.0f;
    }
}

template <typename T>
struct Product {
    const T *a, *b;          // A(i, k) = a[i * ai + k * ak], B(k, j) = b[k * bk + j * bj]
    long long ai, ak, bk, bj;
    int I, J, K;
    T *c;                    // C(i, j) at c[i * ci + j]
    long long ci;
    // epilogue
    const T *bias, *residual;
    long long ri;
    T *z;                    // [I][J]
    int act;
    float alpha;
};

constexpr int kTile = 64, kStep = 16;

// A 64 x 64 tile of C by 256 threads, 4 x 4 sums a thread.
template <typename T>
__global__ __launch_bounds__(256) void k_product(Product<T> P)
{
    __shared__ float as[kStep][kTile + 1], bs[kStep][kTile + 1];
    const int ti = (P.I + kTile - 1) / kTile;
    const int i0 = (int)(blockIdx.x % ti) * kTile, j0 = (int)(blockIdx.x / ti) * kTile;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    float acc[4][4] = {};
    for (int k0 = 0; k0 < P.K; k0 += kStep) {
        for (int e = threadIdx.x; e < kTile * kStep; e += 256) {
            // consecutive threads along whichever index is contiguous
            const int ia = P.ak == 1 ? e / kStep : e % kTile, ka = P.ak == 1 ? e % kStep : e / kTile;
            const int jb = P.bk == 1 ? e / kStep : e % kTile, kb = P.bk == 1 ? e % kStep : e / kTile;
            as[ka][ia] = i0 + ia < P.I && k0 + ka < P.K ? widen(P.a[(i0 + ia) * P.ai + (k0 + ka) * P.ak]) : 0.0f;
            bs[kb][jb] = j0 + jb < P.J && k0 + kb < P.K ? widen(P.b[(k0 + kb) * P.bk + (j0 + jb) * P.bj]) : 0.0f;
        }
        __syncthreads();
        for (int k = 0; k < kStep; ++k)
            for (int r = 0; r < 4; ++r)
                for (int c = 0; c < 4; ++c) acc[r][c] += as[k][ty + 16 * r] * bs[k][tx + 16 * c];
        __syncthreads();
    }
    for (int r = 0; r < 4; ++r)
        for (int c = 0; c < 4; ++c) {
            const int i = i0 + ty + 16 * r, j = j0 + tx + 16 * c;
            if (i >= P.I || j >= P.J) continue;
            float z = acc[r][c];
            if (P.bias) z += widen(P.bias[j]);
            if (P.z) narrow(z, P.z[(long long)i * P.J + j]);
            float y = P.alpha * activate(z, P.act);
            if (P.residual) y += widen(P.residual[i * P.ri + j]);
            narrow(y, P.c[i * P.ci + j]);
        }
}

template <typename T>
hipError_t run_product(const Product<T> &P, hipStream_t s)
{
    const unsigned tiles = (unsigned)((P.I + kTile - 1) / kTile) * (unsigned)((P.J + kTile - 1) / kTile);
    k_product<T><<<tiles, 256, 0, s>>>(P);
    return hipGetLastError();
}

constexpr int kRowChunk = 64;    // rows whose dz one workgroup forms and sums

// dz = alpha act'(z) dy (written if dz is not null) and its sums over kRowChunk rows.
template <typename T>
__global__ __launch_bounds__(256) void k_slope(const T *dy, long long lddy, const T *z, T *dz, float *rows, int M,
                                               int N, int act, float alpha)
{
    const int col = blockIdx.x * 256 + threadIdx.x;
    if (col >= N) return;
    const int r0 = blockIdx.y * kRowChunk, r1 = min(M, r0 + kRowChunk);
    float sum = 0.0f;
    for (int r = r0; r < r1; ++r) {
        float d = alpha * widen(dy[r * lddy + col]);
        if (act != HQML_ACT_NONE) d *= slope(widen(z[(long long)r * N + col]), act);
        if (dz) narrow(d, dz[(long long)r * N + col]);
        sum += d;
    }
    if (rows) rows[(long long)blockIdx.y * N + col] = sum;
}

template <typename T>
__global__ __launch_bounds__(256) void k_row_sum(const float *rows, int chunks, int N, T *db)
{
    const int col = blockIdx.x * 256 + threadIdx.x;
    if (col >= N) return;
    float sum = 0.0f;
    for (int c = 0; c < chunks; ++c) sum += rows[(long long)c * N + col];
    narrow(sum, db[col]);
}

template <typename T>
__global__ void k_zero(T *p, long long n)
{
    const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
    if (i < n) p[i] = T{};
}

template <typename T>
hipError_t zero(void *p, long long n, hipStream_t s)
{
    if (!p) return hipSuccess;
    k_zero<T><<<(unsigned)((n + 255) / 256), 256, 0, s>>>((T *)p, n);
    return hipGetLastError();
}

template <typename T>
hipError_t forward(const DenseForward &a, hipStream_t s)
{
    Product<T> P{};
    P.a = (const T *)a.x, P.ai = a.ldx, P.ak = 1;
    P.b = (const T *)a.w, P.bk = 1, P.bj = a.ldw;
    P.I = a.M, P.J = a.N, P.K = a.K;
    P.c = (T *)a.y, P.ci = a.ldy;
    P.bias = (const T *)a.bias, P.residual = (const T *)a.residual, P.ri = a.ldr;
    P.z = a.act == HQML_ACT_NONE ? nullptr : (T *)a.z;
    P.act = a.act, P.alpha = a.alpha;
    return run_product(P, s);
}

template <typename T>
hipError_t backward(const DenseBackward &a, const DenseWorkspace &ws, hipStream_t s)
{
    hipError_t e = hipSuccess;
    if (a.M == 0) {
        e = zero<T>(a.dw, (long long)a.N * a.K, s);
        return e != hipSuccess ? e : zero<T>(a.db, a.N, s);
    }
    const T *dz = (const T *)a.dy;
    long long lddz = a.lddy;
    float alpha = a.alpha;
    const bool form = a.act != HQML_ACT_NONE && (a.dx || a.dw);
    const int chunks = (a.M + kRowChunk - 1) / kRowChunk;
    if (form || a.db) {
        for (int c0 = 0; c0 < chunks; c0 += 65535) {   // grid limit in y
            const int n = std::min(65535, chunks - c0);
            const long long r0 = (long long)c0 * kRowChunk;
            k_slope<T><<<dim3((unsigned)((a.N + 255) / 256), (unsigned)n), 256, 0, s>>>(
                (const T *)a.dy + r0 * a.lddy, a.lddy, a.z ? (const T *)a.z + r0 * a.N : nullptr,
                form ? (T *)ws.dz + r0 * a.N : nullptr, a.db ? ws.rows + (long long)c0 * a.N : nullptr,
                (int)std::min<long long>(a.M - r0, (long long)n * kRowChunk), a.N, a.act, a.alpha);
            if ((e = hipGetLastError()) != hipSuccess) return e;
        }
        if (a.db) {
            k_row_sum<T><<<(unsigned)((a.N + 255) / 256), 256, 0, s>>>(ws.rows, chunks, a.N, (T *)a.db);
            if ((e = hipGetLastError()) != hipSuccess) return e;
        }
        if (form) dz = (const T *)ws.dz, lddz = a.N, alpha = 1.0f;
    }
    Product<T> P{};
    P.act = HQML_ACT_NONE, P.alpha = alpha;
    if (a.dx) {
        P.a = dz, P.ai = lddz, P.ak = 1;
        P.b = (const T *)a.w, P.bk = a.ldw, P.bj = 1;
        P.I = a.M, P.J = a.K, P.K = a.N;
        P.c = (T *)a.dx, P.ci = a.lddx;
        if ((e = run_product(P, s)) != hipSuccess) return e;
    }
    if (a.dw) {
        P.a = dz, P.ai = 1, P.ak = lddz;
        P.b = (const T *)a.x, P.bk = a.ldx, P.bj = 1;
        P.I = a.N, P.J = a.K, P.K = a.M;
        P.c = (T *)a.dw, P.ci = a.K;
        if ((e = run_product(P, s)) != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace

DenseWorkspace dense_workspace(const hqml_dense_config &cfg)
{
    DenseWorkspace ws;
    const size_t M = (size_t)cfg.max_batch, N = (size_t)cfg.out_features;
    if (cfg.activation != HQML_ACT_NONE) ws.dz_bytes = M * N * (cfg.dtype == HQML_DTYPE_BF16 ? 2 : 4);
    ws.rows_bytes = (M + kRowChunk - 1) / kRowChunk * N * 4;
    return ws;
}

hipError_t launch_dense_forward(const DenseForward &a, int dtype, const DenseWorkspace &, hipStream_t s)
{
    return dtype == HQML_DTYPE_BF16 ? forward<bf16>(a, s) : forward<float>(a, s);
}

hipError_t launch_dense_backward(const DenseBackward &a, int dtype, const DenseWorkspace &ws, hipStream_t s)
{
    return dtype == HQML_DTYPE_BF16 ? backward<bf16>(a, ws, s) : backward<float>(a, ws, s);
}

}  // namespace hqml
