// Dense layer: y = alpha act(x w^T + bias) + residual and its gradients.
//
// All three products of the layer are one kernel family (hqml_gemm.hpp):
//   forward  C = x w^T      dx = dz w      dw = dz^T x
// hqml_dense_cut.hpp chooses their tiles and splits; this file runs them and forms dz = alpha act'(z) dy with its row sums.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>

#include "hqml_dense_cut.hpp"
#include "hqml_gemm.hpp"
#include "hqml_ops.hpp"

namespace hqml {
namespace {

using namespace gemm;

// The most 64 x 64 tiles of partial sums that a product of up to these sizes leaves, 64 MB of them.
size_t part_tiles(size_t I, size_t J, size_t K)
{
    if (K <= 96) return 0;   // three steps: never split
    const size_t tiles = ((I + 255) / 256) * ((J + 255) / 256) * 16;   // whole tiles of any shape
    return std::min<size_t>(kPartTiles, tiles * std::min<size_t>(kMostParts, (K + 31) / 64));
}

bool aligned(const void *p, long long ld, size_t elem)
{
    return (uintptr_t)p % 16 == 0 && ld * (long long)elem % 16 == 0;
}

// Whether a bf16 operand can be loaded straight into LDS: 16-byte rows, and zeros (or nothing) after the last k.
bool straight(const void *p, long long ld, int layout, int K)
{
    return aligned(p, ld, 2) && (layout == K_COLS || K % 8 == 0);
}

// Whether the rows of a bf16 operand begin on whole words.
bool whole_words(const void *p, long long ld)
{
    return (uintptr_t)p % 4 == 0 && ld % 2 == 0;
}

// Whether a product's partial sums and tickets fit the workspace.
bool fits(const Args &P, int tile_values, const DenseWorkspace &ws)
{
    const size_t tiles = (size_t)P.tiles_i * P.tiles_j;
    return P.parts == 1 ||
           (tiles * P.parts * tile_values * 4 <= ws.part_bytes && tiles * sizeof(unsigned) <= ws.ticket_bytes);
}

// Runs one product on tiles; P holds everything but its cut.
template <typename T>
hipError_t run_product(Args P, int la, int lb, const Cut &c, bool direct, const DenseWorkspace &ws, hipStream_t s)
{
    P.tiles_i = ceil_div(P.I, kSides[c.shape][0]);
    P.tiles_j = ceil_div(P.J, kSides[c.shape][1]);
    P.k_part = ceil_div(ceil_div(P.K, c.parts), 32) * 32;
    P.parts = ceil_div(P.K, P.k_part);
    P.part = ws.part;
    P.ticket = ws.ticket;
    if (!fits(P, kSides[c.shape][0] * kSides[c.shape][1], ws)) return hipErrorInvalidValue;
    return sizeof(T) == 2 ? launch_bf16(P, la, lb, direct, c.shape, s) : launch_fp32(P, la, lb, c.shape, s);
}

// ---- bf16 rows that cannot be loaded straight into LDS ----
//
// Their products run at about half the rate (2049 x 2051 x 2047: 57 us; 2048^3: 24).  Where that costs more than a copy
// in rows of a multiple of eight, zeros after the last value, the copy is made first.

int pad8(int n) { return (n + 7) & ~7; }

// Up to two arrays [rows][K] copied into rows of Kp.  Bound by memory: 2049 and 2047 rows of 2051, 34 MB, 7.6 us.
__global__ __launch_bounds__(256) void k_pad(const uint16_t *a, long long lda, int rows_a, const uint16_t *b, long long ldb,
                                             int rows_b, int K, int Kp, uint16_t *to_a, uint16_t *to_b)
{
    const int chunks = Kp / 8;
    const long long all = (long long)(rows_a + rows_b) * chunks;
    for (long long e = (long long)blockIdx.x * 256 + threadIdx.x; e < all; e += (long long)gridDim.x * 256) {
        const long long row = e / chunks;
        const int c = (int)(e % chunks) * 8, n = min(8, K - c);
        const bool second = row >= rows_a;
        const uint16_t *from = second ? b + (row - rows_a) * ldb + c : a + row * lda + c;
        uint16_t *to = (second ? to_b + (row - rows_a) * Kp : to_a + row * Kp) + c;
        u32x4 w;
        if (n == 8) {
            w = *(const u32x4_any *)from;
        } else {
            uint16_t t[8] = {};
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (k < n) t[k] = from[k];
            __builtin_memcpy(&w, t, 16);
        }
        *(u32x4 *)to = w;
    }
}

// Copies of x and w; an array that is not wanted has no rows.
struct Padded {
    const void *x, *w;
    hipError_t e;
};

Padded pad(const void *x, long long ldx, int rows_x, const void *w, long long ldw, int rows_w, int K,
           const DenseWorkspace &ws, hipStream_t s)
{
    const int Kp = pad8(K);
    uint16_t *to_x = (uint16_t *)ws.pad, *to_w = to_x + (size_t)rows_x * Kp;
    const long long chunks = (long long)(rows_x + rows_w) * (Kp / 8);
    k_pad<<<(unsigned)std::min<long long>((chunks + 255) / 256, 8192), 256, 0, s>>>(
        (const uint16_t *)x, ldx, rows_x, (const uint16_t *)w, ldw, rows_w, K, Kp, to_x, to_w);
    return {to_x, to_w, hipGetLastError()};
}

constexpr int kSlopeCols = 256;   // columns of a workgroup: 32 lanes of eight; eight threads go down the rows

// dz = alpha act'(z) dy (written, if dz is not null, in rows of lddz: N, or the next multiple of eight) and its sums
// over `chunk` rows.  Bound by memory (8192 x 4096 bf16: 268 MB in 55 us, 4.9 TB/s); 16 bytes at any alignment, single
// values where a row ends.  The sums take dz before it is rounded to its type and leave as one row a chunk, so that no
// atomic's order changes them.  In bf16 that is the one rounding that a form in 32 bits has not: the matrix cores take
// bf16, and a second plane for the rest of dz would double both products (196 and 184 us at that size).  It makes dx and dw
// 0.0024 off in the norm where the results' own rounding makes them 0.0017.
template <typename T>
__global__ __launch_bounds__(256) void k_slope(const T *dy, long long lddy, const float *z, T *dz, int lddz, float *rows,
                                               int M, int N, int chunk, int act, float alpha)
{
    __shared__ float part[8][kSlopeCols];
    const int lane = threadIdx.x & 31, down = threadIdx.x >> 5;
    const int c0 = blockIdx.x * kSlopeCols, c = c0 + lane * 8, n = min(8, N - c);
    const int r0 = blockIdx.y * chunk, r1 = min(M, r0 + chunk);
    constexpr int kV = (int)sizeof(T) / 2;   // 16-byte words of eight values
    float sum[8] = {};
#pragma unroll 2
    for (int r = r0 + down; r < r1; r += 8) {
        if (n <= 0) break;
        float d[8], f[8] = {};
        T t[8] = {};
        if (n == 8) {
            u32x4 w[kV];
#pragma unroll
            for (int k = 0; k < kV; ++k) w[k] = ((const u32x4_any *)(dy + r * lddy + c))[k];
            __builtin_memcpy(t, w, sizeof t);
            if (act != HQML_ACT_NONE) {
                const f32x4_any *from = (const f32x4_any *)(z + (long long)r * N + c);
                const f32x4 lo = from[0], hi = from[1];
#pragma unroll
                for (int k = 0; k < 4; ++k) f[k] = lo[k], f[4 + k] = hi[k];
            }
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                if (k >= n) continue;
                t[k] = dy[r * lddy + c + k];
                if (act != HQML_ACT_NONE) f[k] = z[(long long)r * N + c + k];
            }
        }
        if (act != HQML_ACT_NONE) {
            slope<sizeof(T) == 2>(f, act);
#pragma unroll
            for (int k = 0; k < 8; ++k) d[k] = alpha * widen(t[k]) * f[k];
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k) d[k] = alpha * widen(t[k]);
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) sum[k] += d[k], narrow(d[k], t[k]);
        if (!dz) continue;
        T *to = dz + (long long)r * lddz + c;
        if (n == 8 || lddz != N) {   // rows of a multiple of eight end with zeros
            u32x4 w[kV];
            __builtin_memcpy(w, t, sizeof t);
#pragma unroll
            for (int k = 0; k < kV; ++k) ((u32x4_any *)to)[k] = w[k];
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (k < n) to[k] = t[k];
        }
    }
    if (!rows) return;
#pragma unroll
    for (int k = 0; k < 8; ++k) part[down][lane * 8 + k] = sum[k];
    __syncthreads();
    const int col = c0 + threadIdx.x;
    if (col >= N) return;
    float s = 0.0f;
#pragma unroll
    for (int q = 0; q < 8; ++q) s += part[q][threadIdx.x];
    rows[(long long)blockIdx.y * N + col] = s;
}

// db: the sums of all row chunks, eight columns a workgroup, 32 threads down the chunks.  Bound by latency: 3 to 5 us.
template <typename T>
__global__ __launch_bounds__(256) void k_row_sum(const float *rows, int chunks, int N, T *db)
{
    __shared__ float part[32][8];
    const int lane = threadIdx.x & 7, down = threadIdx.x >> 3;
    const int c = blockIdx.x * 8 + lane;
    float s = 0.0f;
    if (c < N)
#pragma unroll 4
        for (int q = down; q < chunks; q += 32) s += rows[(long long)q * N + c];
    part[down][lane] = s;
    __syncthreads();
    if (down || c >= N) return;
#pragma unroll
    for (int q = 1; q < 32; ++q) s += part[q][lane];
    narrow(s, db[c]);
}

// Rows that a workgroup of k_slope sums: 16, or 64 where that leaves enough of them.
constexpr int kFewRows = 64 * 1024;

int row_chunk(int M, int N)
{
    return M <= kFewRows && (long long)ceil_div(M, 64) * ceil_div(N, kSlopeCols) < 1024 ? 16 : 64;
}

template <typename T>
__global__ void k_zero(T *p, long long n)
{
    for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < n; i += (long long)gridDim.x * 256) p[i] = T{};
}

template <typename T>
hipError_t zero(void *p, long long n, hipStream_t s)
{
    if (!p) return hipSuccess;
    // a grid has fewer than 2^32 threads
    k_zero<T><<<(unsigned)std::min<long long>((n + 255) / 256, 1 << 16), 256, 0, s>>>((T *)p, n);
    return hipGetLastError();
}

void cut_small(Args &P, int fi)
{
    P.parts = 1;
    P.tiles_i = ceil_div(P.I, 16 * fi);
    P.tiles_j = ceil_div(P.J + (P.ones ? 1 : 0), 16);
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
    const ForwardChoice f = choose_forward(a.M, a.K, a.N, sizeof(T), straight(a.x, a.ldx, K_ROWS, a.K),
                                           straight(a.w, a.ldw, K_ROWS, a.K),
                                           whole_words(a.x, a.ldx) && whole_words(a.w, a.ldw), ws.pad);
    if (f.small) {
        cut_small(P, f.few.fi);
        P.k_part = ceil_div(ceil_div(a.K, f.few.parts), 32) * 32;
        P.parts = ceil_div(a.K, P.k_part);
        P.part = ws.part;
        P.ticket = ws.ticket;
        if (!fits(P, f.few.fi * 16 * 16, ws)) return hipErrorInvalidValue;
        return launch_small_forward(P, sizeof(T) == 2, f.few.fi, f.few.waves, s);
    }
    if (f.copy_x || f.copy_w) {
        const Padded p = pad(a.x, a.ldx, f.copy_x ? a.M : 0, a.w, a.ldw, f.copy_w ? a.N : 0, a.K, ws, s);
        if (p.e != hipSuccess) return p.e;
        if (f.copy_x) P.a = p.x, P.lda = pad8(a.K);
        if (f.copy_w) P.b = p.w, P.ldb = pad8(a.K);
    }
    return run_product<T>(P, K_ROWS, K_ROWS, f.tiles, f.direct, ws, s);
}

// dx, dw and db in one launch.
template <typename T>
hipError_t gradients(const DenseBackward &a, const SmallCut &c, hipStream_t s)
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
    cut_small(X, c.fi);
    cut_small(W, c.fi);
    return launch_small_gradients(X, W, sizeof(T) == 2, c.fi, c.waves, s);
}

template <typename T>
hipError_t backward(const DenseBackward &a, const DenseWorkspace &ws, hipStream_t s)
{
    hipError_t e = hipSuccess;
    if (a.M == 0) {
        e = zero<T>(a.dw, (long long)a.N * a.K, s);
        return e != hipSuccess ? e : zero<T>(a.db, a.N, s);
    }
    const BackwardChoice b =
        choose_backward(a.M, a.K, a.N, sizeof(T), a.act != HQML_ACT_NONE, a.dx, a.dw, straight(a.dy, a.lddy, K_ROWS, a.N),
                        straight(a.x, a.ldx, K_COLS, 0), straight(a.w, a.ldw, K_COLS, 0),
                        whole_words(a.x, a.ldx) && whole_words(a.w, a.ldw) && whole_words(a.dy, a.lddy), ws.dz, ws.pad);
    if (b.small) return gradients<T>(a, b.few, s);
    const T *dz = (const T *)a.dy;
    long long lddz = a.lddy;
    float alpha = a.alpha;
    const bool form = b.form && (a.dx || a.dw);
    const int Np = sizeof(T) == 2 ? pad8(a.N) : a.N;   // a row of dz in the workspace
    if (form || a.db) {
        const int chunk = row_chunk(a.M, a.N), chunks = ceil_div(a.M, chunk);
        for (int c0 = 0; c0 < chunks; c0 += 65535) {   // grid limit in y
            const int n = std::min(65535, chunks - c0);
            const long long r0 = (long long)c0 * chunk;
            const dim3 grid((unsigned)ceil_div(a.N, kSlopeCols), (unsigned)n);
            k_slope<T><<<grid, 256, 0, s>>>((const T *)a.dy + r0 * a.lddy, a.lddy,
                                            a.act != HQML_ACT_NONE ? a.z + r0 * a.N : nullptr,
                                            form ? (T *)ws.dz + r0 * Np : nullptr, Np,
                                            a.db ? ws.rows + (long long)c0 * a.N : nullptr,
                                            (int)std::min<long long>(a.M - r0, (long long)n * chunk), a.N, chunk, a.act,
                                            a.alpha);
            if ((e = hipGetLastError()) != hipSuccess) return e;
        }
        if (a.db) {
            k_row_sum<T><<<(unsigned)ceil_div(a.N, 8), 256, 0, s>>>(ws.rows, chunks, a.N, (T *)a.db);
            if ((e = hipGetLastError()) != hipSuccess) return e;
        }
        if (form) dz = (const T *)ws.dz, lddz = Np, alpha = 1.0f;
    }
    const void *x = a.x, *w = a.w;
    long long ldx = a.ldx, ldw = a.ldw;
    if (b.copy_x || b.copy_w) {
        const Padded p = pad(a.x, a.ldx, b.copy_x ? a.M : 0, a.w, a.ldw, b.copy_w ? a.N : 0, a.K, ws, s);
        if (p.e != hipSuccess) return p.e;
        if (b.copy_x) x = p.x, ldx = pad8(a.K);
        if (b.copy_w) w = p.w, ldw = pad8(a.K);
    }
    Args P{};
    P.a = dz, P.lda = lddz;
    P.act = HQML_ACT_NONE, P.alpha = alpha;
    if (a.dx) {
        P.b = w, P.ldb = ldw;
        P.I = a.M, P.J = a.K, P.K = a.N;
        P.c = a.dx, P.ldc = a.lddx;
        if ((e = run_product<T>(P, K_ROWS, K_COLS, b.dx, b.direct, ws, s)) != hipSuccess) return e;
    }
    if (a.dw) {
        P.b = x, P.ldb = ldx;
        P.I = a.N, P.J = a.K, P.K = a.M;
        P.c = a.dw, P.ldc = a.K;
        if ((e = run_product<T>(P, K_COLS, K_COLS, b.dw, b.direct, ws, s)) != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace

DenseWorkspace dense_workspace(const hqml_dense_config &cfg)
{
    DenseWorkspace ws;
    const size_t M = (size_t)cfg.max_batch, N = (size_t)cfg.out_features;
    const bool two = cfg.dtype == HQML_DTYPE_BF16;
    if (cfg.activation != HQML_ACT_NONE || (two && N % 8)) ws.dz_bytes = M * (two ? pad8(cfg.out_features) * 2 : N * 4);
    if (two && cfg.in_features % 8) ws.pad_bytes = (M + N) * (size_t)pad8(cfg.in_features) * 2;
    // a smaller batch may have more chunks of fewer rows
    const size_t chunk = (size_t)row_chunk(cfg.max_batch, cfg.out_features);
    ws.rows_bytes = std::max((M + chunk - 1) / chunk, (std::min(M, (size_t)kFewRows) + 15) / 16) * N * 4;
    const size_t K = (size_t)cfg.in_features;
    const size_t tiles = std::max({part_tiles(M, N, K), part_tiles(M, K, N), part_tiles(N, K, M)});
    // small products split over k: up to one workgroup a compute unit, of tiles of up to 64 x 16
    ws.part_bytes = tiles ? std::max(tiles * 64 * 64, (size_t)kUnits * 64 * 16) * 4 : 0;
    ws.ticket_bytes = tiles ? std::max(tiles, (size_t)kUnits) * sizeof(unsigned) : 0;
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
