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

int ceil_div(int a, int b) { return (a + b - 1) / b; }

// ---- how a product is run: the estimate that is least ----
//
// Times in us, fitted to sweeps of every cut over 71 products of 64 to 16384 rows, 7 to 8192 columns and k 7 to 16384 and
// 90 smaller ones, of each type and layout: the cut chosen took 2 to 5 % more than the fastest in the mean, 40 % at worst.

constexpr int kUnits = 256;    // compute units
constexpr int kPartTiles = 4096, kMostParts = 64;
constexpr int kParts[] = {1, 2, 3, 4, 6, 8, 12, 16, 24, 32, 48, kMostParts};

// A tile kernel: a workgroup spends `step` on 32 k when alone on its compute unit, n of them n * share; fixed:
// launch, first loads, epilogue; work split over k costs join + parts * join_part and the way of its sums to memory and
// back (9 TB/s: most stay in the caches).  Memory gives `rate` bytes a us where a compute unit's workgroups, up to
// `most` together, have `enough` bytes under way; the result's bytes count `out` times as much again.
struct TileCost {
    Shape shape;
    int most;
    float fixed, step, share, join, join_part;
};
struct MemoryCost {
    float rate, enough, out;
};
constexpr TileCost kFp32Cost[] = {{TILE_64, 4, 4.6f, 0.65f, 0.45f, 0.3f, 0.23f}, {TILE_128, 2, 5.0f, 1.18f, 1.25f, 0.1f, 1.0f},
                                  {TILE_64x32, 6, 4.6f, 0.75f, 0.23f, 0.3f, 0.2f},
                                  {TILE_32x64, 6, 4.6f, 0.75f, 0.23f, 0.3f, 0.2f}};
constexpr TileCost kStagedCost[] = {{TILE_64, 4, 4.5f, 0.27f, 0.184f, 0.6f, 0.4f}, {TILE_128, 2, 4.5f, 0.435f, 0.35f, 0.8f, 1.0f}};
constexpr TileCost kDirectCost[] = {{TILE_64, 4, 2.6f, 0.18f, 0.137f, 0.65f, 0.42f},
                                    {TILE_128, 2, 4.6f, 0.2f, 0.24f, 2.0f, 1.06f},
                                    {TILE_256, 1, 8.6f, 0.45f, 0.525f, 4.6f, 4.0f}};
constexpr MemoryCost kFp32Memory{4.6e6f, 90e3f, 0.0f}, kStagedMemory{5e6f, 29e3f, 2.0f}, kDirectMemory{5e6f, 18e3f, 1.0f};

struct Cut {
    Shape shape;
    int parts;
    float us;
};

Cut best_cut(int I, int J, int K, size_t elem, const TileCost *cost, int n, const MemoryCost &m)
{
    const int steps = ceil_div(K, 32);
    const float out = (float)I * J * elem, bytes = ((float)I * K + (float)J * K) * elem + out;
    Cut best{TILE_64, 0, 0.0f};
    for (int c = 0; c < n; ++c) {
        const int *side = kSides[cost[c].shape];
        // narrow tiles are for operands that a wider one would not fill
        if ((side[0] < side[1] && I > side[0]) || (side[1] < side[0] && J > side[1])) continue;
        const long long tiles = (long long)ceil_div(I, side[0]) * ceil_div(J, side[1]);
        const float step_bytes = 32.0f * elem * (std::min(side[0], I) + std::min(side[1], J));
        for (int parts : kParts) {
            const long long groups = tiles * parts;
            if (parts > 1 && (groups > kPartTiles * 64 * 64 / (side[0] * side[1]) || parts * 2 > steps)) break;
            const float each = (float)((groups + kUnits - 1) / kUnits);
            // three steps of a workgroup are under way
            const float under_way = std::min((float)groups / kUnits, (float)cost[c].most) * 3 * step_bytes;
            const float memory = bytes / (m.rate * std::min(1.0f, under_way / m.enough)) + out * m.out / m.rate;
            float us = cost[c].fixed + std::max(memory, ceil_div(steps, parts) * std::max(cost[c].step, each * cost[c].share)) +
                       0.1f * each;   // starts and ends
            if (parts > 1) us += cost[c].join + parts * cost[c].join_part + (float)groups * (side[0] * side[1] * 8) / 9e6f;
            if (!best.parts || us < best.us) best = {cost[c].shape, parts, us};
        }
    }
    return best;
}

Cut best_cut(int I, int J, int K, size_t elem, bool direct)
{
    if (elem == 4) return best_cut(I, J, K, elem, kFp32Cost, 4, kFp32Memory);
    return direct ? best_cut(I, J, K, elem, kDirectCost, 3, kDirectMemory)
                  : best_cut(I, J, K, elem, kStagedCost, 2, kStagedMemory);
}

// A small forward product: every tile reads its own rows, at `rate` bytes a us and compute unit (bf16 rows whose
// elements straddle words: a sixth of fp32's rate); the fp32 matrix instruction takes 8 x 32 cycles and more for
// 16 x 16 x 32; a wave waits for its loads once in a few steps.
struct SmallCut {
    int fi, waves, parts;
    float us;
};

SmallCut small_cut(int I, int J, int K, size_t elem, bool words)
{
    SmallCut best{0, 1, 1, 0.0f};
    const int steps = ceil_div(K, 32);
    const float bytes = ((float)I * K + (float)J * K + (float)I * J) * elem;
    const float rate = elem == 4 ? 81e3f : words ? 51e3f : 14.3e3f;
    for (int fi : {1, 2, 4}) {
        if (fi > 1 && I <= 8 * fi) break;
        const long long tiles = (long long)ceil_div(I, 16 * fi) * ceil_div(J, 16);
        const int rows = std::min(16 * fi, I) + std::min(16, J), at = fi == 4 ? 2 : 4;   // steps a wave loads together
        for (int parts : {1, 2, 3, 4, 6, 8}) {
            const int own = ceil_div(steps, parts);   // of one workgroup
            if (parts > 1 && (tiles * parts > kUnits || own < 4)) break;
            const float each = (float)((tiles * parts + kUnits - 1) / kUnits);
            for (int waves : {1, 2, 4, 8, 16}) {
                if (waves > 1 && (waves > own || (waves == 16 && fi > 1))) break;
                const float load = each * own * (32 * elem * rows) / rate;
                const float mul = elem == 2 ? 0.0f : each * own * fi * 0.037f, work = load + mul;
                const float wait = ceil_div(own, waves * at) * (elem == 4 ? 0.3f + 0.63f * fi : 0.14f + 0.45f * fi) *
                                   std::max(1.0f, each * waves / 16);
                // memory's rate needs about 40 KB under way on a compute unit
                const float under_way = each * waves * at * (16 * 16 * elem * (fi + 1));
                const float memory = bytes / (4.6e6f * std::min(1.0f, under_way / 40e3f));
                const float us = 2.9f + std::max(std::max(work, wait) + 0.3f * std::min(work, wait), memory) +
                                 each * (0.35f + 0.065f * waves) + (parts > 1 ? 1.65f + 0.07f * parts : 0.0f);
                if (!best.fi || us < best.us) best = {fi, waves, parts, us};
            }
        }
    }
    return best;
}

// Small gradients in one launch.  What counts is forming dz anew in every tile (1,300 to 1,770 cycles of a SIMD for
// 16 rows and 32 k, the matrix instructions with them) and the waits of the longer product's waves.  Over 70 products
// of each type the choice took 1 to 3 % more than the best in the mean.
SmallCut small_gradients_cut(int M, int N, int K, size_t elem, bool words)
{
    SmallCut best{0, 1, 1, 0.0f};
    const int steps_x = ceil_div(N, 32), steps_w = ceil_div(M, 32), steps = std::max(steps_x, steps_w);
    for (int fi : {1, 4}) {
        const float block_us = ((elem == 4 ? 1420.0f : words ? 1300.0f : 1570.0f) + (fi == 4 ? 200.0f : 0.0f)) / 2.15e6f;
        for (int waves : {1, 2, 4, 8}) {
            if (waves > 1 && waves > steps) break;
            const long long tx = (long long)ceil_div(M, 16 * fi) * ceil_div(K, 16);
            const long long tw = (long long)ceil_div(N, 16 * fi) * ceil_div(K + 1, 16);
            const float work = ((float)tx * steps_x * std::min(M, 16 * fi) + (float)tw * steps_w * std::min(N, 16 * fi)) /
                               16 * block_us;
            const int at = fi == 1 ? 2 : 1;   // steps a wave loads together
            const float wait = ceil_div(steps, waves * at) * (fi == 1 ? 1.55f : 2.9f);
            const float ends = (tx + tw) * waves * 4.4f / (kUnits * 32);   // workgroups' starts and epilogues
            const float us = 3.6f + std::max(work, wait) + 0.37f * std::min(work, wait) + ends;
            if (!best.fi || us < best.us) best = {fi, waves, 1, us};
        }
    }
    return best;
}

// dz and its row sums by themselves.
float slope_us(int M, int N, size_t elem)
{
    return 6.0f + (float)M * N * (4 + 2 * elem) / 5e6f;
}

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

float pad_us(int rows, int K)
{
    return rows ? 4.0f + (float)rows * K * 4 / 4.5e6f : 0.0f;
}

constexpr int kSlopeCols = 256;   // columns of a workgroup: 32 lanes of eight; eight threads go down the rows

// dz = alpha act'(z) dy (written, if dz is not null, in rows of lddz: N, or the next multiple of eight) and its sums
// over `chunk` rows.  Bound by memory (8192 x 4096 bf16: 268 MB in 55 us, 4.9 TB/s); 16 bytes at any alignment, single
// values where a row ends.  The sums take dz before it is rounded to its type (bf16: the matrix cores take it so) and
// leave as one row a chunk, so that no atomic's order changes them.
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
    bool direct = false;
    int copy_x = 0, copy_w = 0;   // rows to copy
    Cut c = best_cut(P.I, P.J, P.K, sizeof(T), false);
    if (sizeof(T) == 2) {
        if (!straight(a.x, a.ldx, K_ROWS, a.K)) copy_x = a.M;
        if (!straight(a.w, a.ldw, K_ROWS, a.K)) copy_w = a.N;
        const Cut d = best_cut(P.I, P.J, P.K, 2, true);
        direct = !(copy_x + copy_w) || (ws.pad && d.us + pad_us(copy_x + copy_w, a.K) < c.us);
        if (direct) c = d, c.us += pad_us(copy_x + copy_w, a.K);
    }
    const SmallCut sc = small_cut(P.I, P.J, P.K, sizeof(T), whole_words(a.x, a.ldx) && whole_words(a.w, a.ldw));
    if (sc.us <= c.us) {
        cut_small(P, sc.fi);
        P.k_part = ceil_div(ceil_div(a.K, sc.parts), 32) * 32;
        P.parts = ceil_div(a.K, P.k_part);
        P.part = ws.part;
        P.ticket = ws.ticket;
        if (!fits(P, sc.fi * 16 * 16, ws)) return hipErrorInvalidValue;
        return launch_small_forward(P, sizeof(T) == 2, sc.fi, sc.waves, s);
    }
    if (direct && copy_x + copy_w) {
        const Padded p = pad(a.x, a.ldx, copy_x, a.w, a.ldw, copy_w, a.K, ws, s);
        if (p.e != hipSuccess) return p.e;
        if (copy_x) P.a = p.x, P.lda = pad8(a.K);
        if (copy_w) P.b = p.w, P.ldb = pad8(a.K);
    }
    return run_product<T>(P, K_ROWS, K_ROWS, c, direct, ws, s);
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
    // dx = dz w and dw = dz^T x: the cuts, and for bf16 whether to copy what cannot be loaded straight
    Cut cx = best_cut(a.M, a.K, a.N, sizeof(T), false), cw = best_cut(a.N, a.K, a.M, sizeof(T), false);
    bool form = a.act != HQML_ACT_NONE, direct = false;
    int copy_x = 0, copy_w = 0;   // rows to copy
    if (sizeof(T) == 2) {
        if (!straight(a.x, a.ldx, K_COLS, 0) && a.dw) copy_x = a.M;
        if (!straight(a.w, a.ldw, K_COLS, 0) && a.dx) copy_w = a.N;
        const bool dy_straight = straight(a.dy, a.lddy, K_ROWS, a.N);
        const Cut dx = best_cut(a.M, a.K, a.N, 2, true), dw = best_cut(a.N, a.K, a.M, 2, true);
        const float copies = pad_us(copy_x + copy_w, a.K) + (form || dy_straight ? 0.0f : pad_us(a.M, a.N));
        direct = (form || dy_straight || ws.dz) && (!(copy_x + copy_w) || ws.pad) && dx.us + dw.us + copies < cx.us + cw.us;
        if (direct) {
            cx = dx, cw = dw, cx.us += copies;
            form = form || !dy_straight;   // dz in rows of a multiple of eight
        }
    }
    const bool words = whole_words(a.x, a.ldx) && whole_words(a.w, a.ldw) && whole_words(a.dy, a.lddy);
    const SmallCut c = small_gradients_cut(a.M, a.N, a.K, sizeof(T), words);
    if (c.us <= slope_us(a.M, a.N, sizeof(T)) + cx.us + cw.us) return gradients<T>(a, c, s);
    const T *dz = (const T *)a.dy;
    long long lddz = a.lddy;
    float alpha = a.alpha;
    form = form && (a.dx || a.dw);
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
    if (direct && copy_x + copy_w) {
        const Padded p = pad(a.x, a.ldx, copy_x, a.w, a.ldw, copy_w, a.K, ws, s);
        if (p.e != hipSuccess) return p.e;
        if (copy_x) x = p.x, ldx = pad8(a.K);
        if (copy_w) w = p.w, ldw = pad8(a.K);
    }
    Args P{};
    P.a = dz, P.lda = lddz;
    P.act = HQML_ACT_NONE, P.alpha = alpha;
    if (a.dx) {
        P.b = w, P.ldb = ldw;
        P.I = a.M, P.J = a.K, P.K = a.N;
        P.c = a.dx, P.ldc = a.lddx;
        if ((e = run_product<T>(P, K_ROWS, K_COLS, cx, direct, ws, s)) != hipSuccess) return e;
    }
    if (a.dw) {
        P.b = x, P.ldb = ldx;
        P.I = a.N, P.J = a.K, P.K = a.M;
        P.c = a.dw, P.ldc = a.K;
        if ((e = run_product<T>(P, K_COLS, K_COLS, cw, direct, ws, s)) != hipSuccess) return e;
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
