// Dense layer: y = alpha act(x w^T + bias) + residual and its gradients.
//
// All three products of the layer are one kernel family (hqml_gemm.hpp):
//   forward  C = x w^T      dx = dz w      dw = dz^T x
// This file chooses their tiles and splits, and forms dz = alpha act'(z) dy with its row sums.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>

#include "hqml_gemm.hpp"

namespace hqml {
namespace {

using namespace gemm;

// z becomes d act / dz.
template <bool FAST, int n>
__device__ __forceinline__ void slope(float (&z)[n], int act)
{
    switch (act) {
    case HQML_ACT_RELU:
#pragma unroll
        for (int k = 0; k < n; ++k) z[k] = z[k] > 0.0f ? 1.0f : 0.0f;
        break;
    case HQML_ACT_GELU:
#pragma unroll
        for (int k = 0; k < n; ++k) {
            float e;
            const float f = normal_cdf(z[k], e);
            z[k] = f + z[k] * e * 0.39894228f;
        }
        break;
    case HQML_ACT_SILU:
#pragma unroll
        for (int k = 0; k < n; ++k) {
            const float f = logistic<FAST>(z[k]);
            z[k] = f * (1.0f + z[k] * (1.0f - f));
        }
        break;
    case HQML_ACT_TANH:
#pragma unroll
        for (int k = 0; k < n; ++k) {
            const float t = tanh_of<FAST>(z[k]);
            z[k] = 1.0f - t * t;
        }
        break;
    case HQML_ACT_SIGMOID:
#pragma unroll
        for (int k = 0; k < n; ++k) {
            const float f = logistic<FAST>(z[k]);
            z[k] = f * (1.0f - f);
        }
        break;
    default: break;
    }
}

constexpr size_t kPartBytes = 64u << 20;   // most that partial sums take
constexpr int kMostParts = 64;

// How a product is cut up.
struct Cut {
    Shape shape;
    int parts, k_part;
};

int ceil_div(int a, int b) { return (a + b - 1) / b; }

Cut cut(int I, int J, int K, bool direct, size_t part_bytes)
{
    auto tiles = [&](int n) { return (long long)ceil_div(I, n) * ceil_div(J, n); };
    Cut c{TILE_64, 1, (K + 63) / 64 * 64};
    if (direct && tiles(256) >= 192) c.shape = TILE_256;
    else if (tiles(128) >= 256) c.shape = TILE_128;
    if (c.shape == TILE_64 && tiles(64) < 256) {
        long long parts = std::min<long long>(512 / tiles(64), K / 128);
        parts = std::min<long long>(parts, kMostParts);
        parts = std::min<long long>(parts, (long long)(part_bytes / ((size_t)I * J * 4)));
        if (parts > 1) {
            c.k_part = ceil_div(ceil_div(K, (int)parts), 64) * 64;
            c.parts = ceil_div(K, c.k_part);
        }
    }
    return c;
}

bool aligned(const void *p, long long ld, size_t elem)
{
    return (uintptr_t)p % 16 == 0 && ld * (long long)elem % 16 == 0;
}

// Runs one product; P holds everything but its cut.
template <typename T>
hipError_t run_product(Args P, int la, int lb, const DenseWorkspace &ws, hipStream_t s)
{
    const bool direct = sizeof(T) == 2 && aligned(P.a, P.lda, 2) && aligned(P.b, P.ldb, 2) &&
                        ((la == K_COLS && lb == K_COLS) || P.K % 8 == 0);
    P.wide = aligned(P.c, P.ldc, sizeof(T)) && P.J % 8 == 0 && (!P.bias || aligned(P.bias, 0, sizeof(T))) &&
             (!P.residual || aligned(P.residual, P.ldr, sizeof(T))) && (!P.z || aligned(P.z, 0, 4));
    const Cut c = cut(P.I, P.J, P.K, direct, ws.part_bytes);
    const int side = c.shape == TILE_64 ? 64 : c.shape == TILE_128 ? 128 : 256;
    P.tiles_i = ceil_div(P.I, side), P.tiles_j = ceil_div(P.J, side);
    P.k_part = c.k_part;
    P.part = c.parts > 1 ? ws.part : nullptr;
    const hipError_t e = sizeof(T) == 2 ? launch_bf16(P, la, lb, direct, c.shape, c.parts, s)
                                        : launch_fp32(P, la, lb, c.shape, c.parts, s);
    if (e != hipSuccess || c.parts == 1) return e;
    const long long all = (long long)P.I * P.J;
    k_join<T><<<(unsigned)std::min<long long>((all + 255) / 256, 4096), 256, 0, s>>>(P, c.parts);
    return hipGetLastError();
}

constexpr int kRowChunk = 64;    // rows whose dz one workgroup forms and sums
constexpr int kSlopeCols = 256;  // and columns: 32 lanes of eight; eight threads go down the rows

// dz = alpha act'(z) dy (written if dz is not null) and its sums over kRowChunk rows.  Bound by
// memory.  VEC: the rows allow 16-byte access and a lane's eight columns are neighbours; otherwise
// they are 32 apart, so that a row is still read in runs.
template <typename T, bool VEC>
__global__ __launch_bounds__(256) void k_slope(const T *dy, long long lddy, const float *z, T *dz, float *rows, int M,
                                               int N, int act, float alpha)
{
    __shared__ float part[8][kSlopeCols];
    const int lane = threadIdx.x & 31, down = threadIdx.x >> 5;
    const int c0 = blockIdx.x * kSlopeCols;
    const int r0 = blockIdx.y * kRowChunk, r1 = min(M, r0 + kRowChunk);
    float sum[8] = {};
    for (int r = r0 + down; r < r1; r += 8) {
        float d[8], f[8];
        if (VEC) {
            const int c = c0 + lane * 8;
            if (c >= N) break;
            T t[8];
            __builtin_memcpy(t, __builtin_assume_aligned(dy + r * lddy + c, 16), sizeof t);
#pragma unroll
            for (int k = 0; k < 8; ++k) d[k] = alpha * widen(t[k]);
            if (act != HQML_ACT_NONE) __builtin_memcpy(f, __builtin_assume_aligned(z + (long long)r * N + c, 16), sizeof f);
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const int c = c0 + lane + 32 * k;
                d[k] = c < N ? alpha * widen(dy[r * lddy + c]) : 0.0f;
                f[k] = c < N && act != HQML_ACT_NONE ? z[(long long)r * N + c] : 0.0f;
            }
        }
        if (act != HQML_ACT_NONE) {
            slope<sizeof(T) == 2>(f, act);
#pragma unroll
            for (int k = 0; k < 8; ++k) d[k] *= f[k];
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) sum[k] += d[k];
        if (!dz) continue;
        if (VEC) {
            T t[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) narrow(d[k], t[k]);
            __builtin_memcpy(__builtin_assume_aligned(dz + (long long)r * N + c0 + lane * 8, 16), t, sizeof t);
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const int c = c0 + lane + 32 * k;
                if (c < N) narrow(d[k], dz[(long long)r * N + c]);
            }
        }
    }
    if (!rows) return;
#pragma unroll
    for (int k = 0; k < 8; ++k) part[down][VEC ? lane * 8 + k : lane + 32 * k] = sum[k];
    __syncthreads();
    const int c = c0 + threadIdx.x;
    if (c >= N) return;
    float s = 0.0f;
#pragma unroll
    for (int q = 0; q < 8; ++q) s += part[q][threadIdx.x];
    rows[(long long)blockIdx.y * N + c] = s;
}

// db: the sums of all row chunks, 32 columns a workgroup, eight threads down the chunks.
template <typename T>
__global__ __launch_bounds__(256) void k_row_sum(const float *rows, int chunks, int N, T *db)
{
    __shared__ float part[8][32];
    const int lane = threadIdx.x & 31, down = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane;
    float s = 0.0f;
    if (c < N)
#pragma unroll 4
        for (int q = down; q < chunks; q += 8) s += rows[(long long)q * N + c];
    part[down][lane] = s;
    __syncthreads();
    if (down || c >= N) return;
#pragma unroll
    for (int q = 1; q < 8; ++q) s += part[q][lane];
    narrow(s, db[c]);
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
hipError_t forward(const DenseForward &a, const DenseWorkspace &ws, hipStream_t s)
{
    Args P{};
    P.a = a.x, P.lda = a.ldx;
    P.b = a.w, P.ldb = a.ldw;
    P.I = a.M, P.J = a.N, P.K = a.K;
    P.c = a.y, P.ldc = a.ldy;
    P.bias = a.bias, P.residual = a.residual, P.ldr = a.ldr;
    P.z = a.act == HQML_ACT_NONE ? nullptr : (float *)a.z;
    P.act = a.act, P.alpha = a.alpha;
    return run_product<T>(P, K_ROWS, K_ROWS, ws, s);
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
            const dim3 grid((unsigned)ceil_div(a.N, kSlopeCols), (unsigned)n);
            const T *dy = (const T *)a.dy + r0 * a.lddy;
            const float *z = a.act != HQML_ACT_NONE ? a.z + r0 * a.N : nullptr;
            T *to = form ? (T *)ws.dz + r0 * a.N : nullptr;
            float *rows = a.db ? ws.rows + (long long)c0 * a.N : nullptr;
            const int m = (int)std::min<long long>(a.M - r0, (long long)n * kRowChunk);
            if (a.N % 8 == 0 && aligned(a.dy, a.lddy, sizeof(T)) && aligned(a.z, 0, 4))
                k_slope<T, true><<<grid, 256, 0, s>>>(dy, a.lddy, z, to, rows, m, a.N, a.act, a.alpha);
            else k_slope<T, false><<<grid, 256, 0, s>>>(dy, a.lddy, z, to, rows, m, a.N, a.act, a.alpha);
            if ((e = hipGetLastError()) != hipSuccess) return e;
        }
        if (a.db) {
            k_row_sum<T><<<(unsigned)ceil_div(a.N, 32), 256, 0, s>>>(ws.rows, chunks, a.N, (T *)a.db);
            if ((e = hipGetLastError()) != hipSuccess) return e;
        }
        if (form) dz = (const T *)ws.dz, lddz = a.N, alpha = 1.0f;
    }
    Args P{};
    P.a = dz, P.lda = lddz;
    P.act = HQML_ACT_NONE, P.alpha = alpha;
    if (a.dx) {
        P.b = a.w, P.ldb = a.ldw;
        P.I = a.M, P.J = a.K, P.K = a.N;
        P.c = a.dx, P.ldc = a.lddx;
        if ((e = run_product<T>(P, K_ROWS, K_COLS, ws, s)) != hipSuccess) return e;
    }
    if (a.dw) {
        P.b = a.x, P.ldb = a.ldx;
        P.I = a.N, P.J = a.K, P.K = a.M;
        P.c = a.dw, P.ldc = a.K;
        if ((e = run_product<T>(P, K_COLS, K_COLS, ws, s)) != hipSuccess) return e;
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
    // partial sums: up to kMostParts of the largest result
    const size_t K = (size_t)cfg.in_features, most = std::max({M * N, M * K, N * K});
    ws.part_bytes = std::min(kPartBytes, most * 4 * kMostParts);
    return ws;
}

hipError_t launch_dense_forward(const DenseForward &a, int dtype, const DenseWorkspace &ws, hipStream_t s)
{
    return dtype == HQML_DTYPE_BF16 ? forward<bf16>(a, ws, s) : forward<float>(a, ws, s);
}

hipError_t launch_dense_backward(const DenseBackward &a, int dtype, const DenseWorkspace &ws, hipStream_t s)
{
    return dtype == HQML_DTYPE_BF16 ? backward<bf16>(a, ws, s) : backward<float>(a, ws, s);
}

}  // namespace hqml
