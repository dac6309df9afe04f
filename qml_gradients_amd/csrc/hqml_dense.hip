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
#include "hqml_ops.hpp"

namespace hqml {
namespace {

using namespace gemm;

// Work is split over k where a product has fewer tiles than kFewTiles: into parts of kPartK at least, as many
// as make kPartTiles of them.
constexpr int kFewTiles = 256, kPartTiles = 512, kPartK = 128;

int ceil_div(int a, int b) { return (a + b - 1) / b; }

// The most tiles of partial sums that products of up to I rows leave.
size_t part_tiles(size_t I, size_t J, size_t K)
{
    if (K < 2 * kPartK) return 0;
    const size_t tiles = ((I + 63) / 64) * ((J + 63) / 64);
    return std::min<size_t>(kPartTiles, tiles * (K / kPartK));
}

bool aligned(const void *p, long long ld, size_t elem)
{
    return (uintptr_t)p % 16 == 0 && ld * (long long)elem % 16 == 0;
}

// Cuts a product into tiles of `side` and, if they are the 64 x 64 ones and few, its k into parts, whose
// sums go to the workspace.
void cut(Args &P, int side, const DenseWorkspace &ws)
{
    P.tiles_i = ceil_div(P.I, side);
    P.tiles_j = ceil_div(P.J, side);
    P.parts = 1;
    P.k_part = ceil_div(P.K, 32) * 32;
    const long long tiles = (long long)P.tiles_i * P.tiles_j;
    if (side != 64 || tiles >= kFewTiles) return;
    const int parts = std::min((int)(kPartTiles / tiles), P.K / kPartK);
    if (parts < 2) return;
    P.k_part = ceil_div(ceil_div(P.K, parts), 32) * 32;
    P.parts = ceil_div(P.K, P.k_part);
    P.part = ws.part;
    P.ticket = ws.ticket;
}

// Runs one product; P holds everything but its cut.
template <typename T>
hipError_t run_product(Args P, int la, int lb, const DenseWorkspace &ws, hipStream_t s)
{
    const bool direct = sizeof(T) == 2 && aligned(P.a, P.lda, 2) && aligned(P.b, P.ldb, 2) &&
                        ((la == K_COLS && lb == K_COLS) || P.K % 8 == 0);
    P.wide = aligned(P.c, P.ldc, sizeof(T)) && P.J % 8 == 0 &&
             (!P.residual || aligned(P.residual, P.ldr, sizeof(T))) && (!P.z || aligned(P.z, 0, 4));
    auto tiles = [&](int n) { return (long long)ceil_div(P.I, n) * ceil_div(P.J, n); };
    const Shape shape = direct && tiles(256) >= 192 ? TILE_256 : tiles(128) >= 256 ? TILE_128 : TILE_64;
    cut(P, shape == TILE_64 ? 64 : shape == TILE_128 ? 128 : 256, ws);
    return sizeof(T) == 2 ? launch_bf16(P, la, lb, direct, shape, s) : launch_fp32(P, la, lb, shape, s);
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

// Tiles and waves of a small product or two.
void cut_small(Args &P, int fi)
{
    P.tiles_i = ceil_div(P.I, 16 * fi);
    P.tiles_j = ceil_div(P.J + (P.ones ? 1 : 0), 16);
}

long long small_tiles(const Args &P, int fi)
{
    return (long long)ceil_div(P.I, 16 * fi) * ceil_div(P.J + (P.ones ? 1 : 0), 16);
}

int small_waves(int K, long long tiles, int most)
{
    int waves = 1;
    while (waves < most && waves * 2 <= ceil_div(K, 32) && tiles * waves < 4096) waves *= 2;
    return waves;
}

bool small(int M, int N, int K)
{
    return (long long)M * N * K <= 1ll << 27;
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
    if (small(a.M, a.N, a.K)) {
        const int fi = small_tiles(P, 4) >= 512 ? 4 : 1;
        cut_small(P, fi);
        return launch_small_forward(P, sizeof(T) == 2, fi, small_waves(P.K, small_tiles(P, fi), fi == 1 ? 16 : 8), s);
    }
    return run_product<T>(P, K_ROWS, K_ROWS, ws, s);
}

template <typename T>
hipError_t gradients(const DenseBackward &a, hipStream_t s)
{
    Args X{}, W{};
    X.a = W.a = a.dy, X.lda = W.lda = a.lddy;
    X.z = W.z = const_cast<float *>(a.z);
    X.act = W.act = a.act, X.alpha = W.alpha = a.alpha;
    if (a.dx) {
        X.b = a.w, X.ldb = a.ldw;
        X.I = a.M, X.J = a.K, X.K = a.N;
        X.c = a.dx, X.ldc = a.lddx;
    }
    if (a.dw || a.db) {
        W.b = a.x, W.ldb = a.ldx;
        W.I = a.N, W.J = a.dw ? a.K : 0, W.K = a.M;
        W.c = a.dw, W.ldc = a.K;
        W.ones = a.db;
    }
    const int fi = small_tiles(X, 4) + small_tiles(W, 4) >= 512 ? 4 : 1;
    cut_small(X, fi);
    cut_small(W, fi);
    const int waves = small_waves(std::max(X.K, W.K), small_tiles(X, fi) + small_tiles(W, fi), 8);
    return launch_small_gradients(X, W, sizeof(T) == 2, fi, waves, s);
}

template <typename T>
hipError_t backward(const DenseBackward &a, const DenseWorkspace &ws, hipStream_t s)
{
    hipError_t e = hipSuccess;
    if (a.M == 0) {
        e = zero<T>(a.dw, (long long)a.N * a.K, s);
        return e != hipSuccess ? e : zero<T>(a.db, a.N, s);
    }
    if (small(a.M, a.N, a.K)) return gradients<T>(a, s);
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
    const size_t K = (size_t)cfg.in_features;
    const size_t tiles = std::max({part_tiles(M, N, K), part_tiles(M, K, N), part_tiles(N, K, M)});
    ws.part_bytes = tiles * 64 * 64 * 4;
    ws.ticket_bytes = tiles * sizeof(unsigned);
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
