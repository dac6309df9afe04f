// Dense layer in 8-bit integers, for serving.
//
//   x ~ sx_m cx_mk,  w ~ sw_n cw_nk  (codes of -127..127, a scale for each row)
//   y_mn = alpha act(sx_m sw_n sum_k cx_mk cw_nk + bias_n) + residual_mn
//
// The weights come as codes and scales, laid out once; x is rounded to codes within the call (k_quantise).  The product's
// sums are 32-bit integers, so it is exact up to its one conversion to fp32, and 64 k of codes take the place of 32 of bf16 in every
// tile of hqml_gemm.hpp: rows of codes are padded to 16 bytes with zeros, and a pair of codes counts as one value there.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "hqml_dense_cut.hpp"
#include "hqml_gemm.hpp"
#include "hqml_layers.hpp"

namespace hqml {
namespace {

using namespace gemm;

// ---- rows to codes ----
//
// scale = max(largest magnitude / 127, 2^-100); code = the nearest integer to x / scale (scale before its own rounding),
// ties to even.  A row that is not finite has scale NaN and codes 0.

// What a row's codes are formed with: code = rint(x num / den).
struct RowScale {
    float num, den, inv;   // inv = num / den, rounded
};

__device__ __forceinline__ RowScale row_scale(uint32_t bits, float &scale)
{
    const float size = __builtin_bit_cast(float, bits);
    if (bits >= 0x7F800000u) {
        scale = __builtin_nanf("");
        return {0.0f, 1.0f, 0.0f};
    }
    if (size <= 127 * 0x1p-100f) {
        scale = 0x1p-100f;
        return {0x1p100f, 1.0f, 0x1p100f};
    }
    scale = size / 127.0f;
    return {127.0f, size, 127.0f / size};
}

__device__ __forceinline__ int code_of(float x, const RowScale &s)
{
    if (s.num == 0.0f) return 0;
    const float t = x * s.inv, k = __builtin_rintf(t);
    // t is off by up to 2^-16: a quotient next to the middle of two codes is decided in 64 bits, where x num is exact and
    // a quotient that is not a tie rounds to none (it is at least 2^-26 of itself away)
    if (__builtin_fabsf(t - k) < 0.5f - 0x1p-13f) return (int)k;
    return (int)__builtin_rint((double)x * (double)s.num / (double)s.den);
}

// Largest magnitude as bits: magnitudes order as integers, and a NaN is above them all.
__device__ __forceinline__ uint32_t wave_max(uint32_t b)
{
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) {
        const uint32_t o = (uint32_t)__shfl_xor((int)b, m, 64);
        b = b > o ? b : o;
    }
    return b;
}

// Sixteen values of a row from c on, zeros past its end.
template <typename T>
__device__ __forceinline__ void get16(float (&x)[16], const T *row, int c, int K)
{
    constexpr int kV = (int)sizeof(T);   // 16-byte words of sixteen values
    if (c + 16 <= K) {
        T t[16];
        u32x4 w[kV];
#pragma unroll
        for (int k = 0; k < kV; ++k) w[k] = ((const u32x4_any *)(row + c))[k];
        __builtin_memcpy(t, w, sizeof t);
#pragma unroll
        for (int k = 0; k < 16; ++k) x[k] = widen(t[k]);
    } else {
#pragma unroll
        for (int k = 0; k < 16; ++k) x[k] = c + k < K ? widen(row[c + k]) : 0.0f;
    }
}

__device__ __forceinline__ uint32_t largest16(const float (&x)[16])
{
    uint32_t b = 0;
#pragma unroll
    for (int k = 0; k < 16; ++k) {
        const uint32_t a = __builtin_bit_cast(uint32_t, x[k]) & 0x7FFFFFFFu;
        b = a > b ? a : b;
    }
    return b;
}

__device__ __forceinline__ u32x4 codes16(const float (&x)[16], const RowScale &s)
{
    u32x4 w = {0, 0, 0, 0};
#pragma unroll
    for (int k = 0; k < 16; ++k) w[k / 4] |= (uint32_t)(uint8_t)code_of(x[k], s) << (k % 4 * 8);
    return w;
}

constexpr int kHeld = 2;   // sixteens of a thread that stay in registers between the two passes over a row

// kWaves waves a row, 4 / kWaves rows a workgroup; the codes' rows end with zeros.
template <typename T, int kWaves>
__global__ __launch_bounds__(256) void k_quantise(const T *x, long long ldx, long long rows, int K, int8_t *codes, long long ldc,
                                                  float *scales)
{
    __shared__ uint32_t part[4];
    constexpr int kThreads = 64 * kWaves;
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & (kThreads - 1);
    const int Kp = (K + 15) & ~15;
    const long long step = (long long)gridDim.x * (4 / kWaves);
    for (long long r0 = (long long)blockIdx.x * (4 / kWaves); r0 < rows; r0 += step) {
        const long long r = r0 + (kWaves == 4 ? 0 : wave);
        const bool some = r < rows;   // the same in all threads of a row
        const T *row = x + r * ldx;
        float v[kHeld][16];
        uint32_t b = 0;
        if (some) {
#pragma unroll
            for (int h = 0; h < kHeld; ++h) {
                const int c = (h * kThreads + lane) * 16;
                if (c < Kp) get16(v[h], row, c, K), b = max(b, largest16(v[h]));
            }
            for (int c = (kHeld * kThreads + lane) * 16; c < Kp; c += kThreads * 16) {
                float t[16];
                get16(t, row, c, K);
                b = max(b, largest16(t));
            }
        }
        b = wave_max(b);
        if (kWaves == 4) {
            __syncthreads();   // the row before is done with part
            if ((threadIdx.x & 63) == 0) part[wave] = b;
            __syncthreads();
            b = max(max(part[0], part[1]), max(part[2], part[3]));
        }
        if (!some) continue;
        float scale;
        const RowScale s = row_scale(b, scale);
        int8_t *to = codes + r * ldc;
#pragma unroll
        for (int h = 0; h < kHeld; ++h) {
            const int c = (h * kThreads + lane) * 16;
            if (c < Kp) *(u32x4 *)(to + c) = codes16(v[h], s);
        }
        for (int c = (kHeld * kThreads + lane) * 16; c < Kp; c += kThreads * 16) {
            float t[16];
            get16(t, row, c, K);
            *(u32x4 *)(to + c) = codes16(t, s);
        }
        if (lane == 0) scales[r] = scale;
    }
}

template <typename T>
hipError_t quantise(const void *x, long long ldx, long long rows, int K, int8_t *codes, long long ldc, float *scales, hipStream_t s)
{
    // a wave a row up to two sixteens a lane
    if (K <= 64 * 16 * kHeld) {
        const unsigned grid = (unsigned)std::min<long long>((rows + 3) / 4, 1 << 16);
        k_quantise<T, 1><<<grid, 256, 0, s>>>((const T *)x, ldx, rows, K, codes, ldc, scales);
    } else {
        const unsigned grid = (unsigned)std::min<long long>(rows, 1 << 16);
        k_quantise<T, 4><<<grid, 256, 0, s>>>((const T *)x, ldx, rows, K, codes, ldc, scales);
    }
    return hipGetLastError();
}

// ---- the product ----

// Sums of codes' products as fp32 values: scaled by their row and column.
template <int FI, int FJ>
__device__ __forceinline__ void scaled(f32x4 (&to)[FI][FJ], const i32x4 (&acc)[FI][FJ], const Args &P, const Scales8 &q, int i0, int j0)
{
    const int lane = threadIdx.x & 63;
    float sx[FI];
#pragma unroll
    for (int f = 0; f < FI; ++f) {
        const int i = i0 + f * 16 + (lane & 15);
        sx[f] = i < P.I ? q.x[i] : 0.0f;
    }
#pragma unroll
    for (int g = 0; g < FJ; ++g) {
        const int j = j0 + g * 16 + (lane >> 4) * 4;
        float sw[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) sw[k] = j + k < P.J ? q.w[j + k] : 0.0f;
#pragma unroll
        for (int f = 0; f < FI; ++f)
#pragma unroll
            for (int k = 0; k < 4; ++k) to[f][g][k] = (float)acc[f][g][k] * (sx[f] * sw[k]);
    }
}

template <typename T, int BM, int BN, int WI, int WJ>
__global__ __launch_bounds__(64 * WI *WJ, 2) void k_product8(Args P, Scales8 q)
{
    using D = Direct<K_ROWS, K_ROWS, BM, BN, 32, WI, WJ, MulI8>;
    using TA = typename D::TA;
    using TB = typename D::TB;
    __shared__ __attribute__((aligned(1024))) char a0[TA::kBytes], a1[TA::kBytes], a2[TA::kBytes], a3[TA::kBytes];
    __shared__ __attribute__((aligned(1024))) char b0[TB::kBytes], b1[TB::kBytes], b2[TB::kBytes], b3[TB::kBytes];
    int ti, tj;
    tile_of(blockIdx.x, P.tiles_i, P.tiles_j, ti, tj);
    const int part = blockIdx.y, kb = part * P.k_part;
    const int kn = P.K - kb < P.k_part ? P.K - kb : P.k_part;
    D d;
    d.ta.init(P.a, P.lda, ti * BM, P.I, kn, kb);
    d.tb.init(P.b, P.ldb, tj * BN, P.J, kn, kb);
    d.run((kn + 31) / 32, a0, a1, a2, a3, b0, b1, b2, b3);
    const int i0 = ti * BM + d.wi * D::TI, j0 = tj * BN + d.wj * D::TJ;
    if (P.parts > 1 && !joined<D::FI, D::FJ, 64 * D::kWaves>(P, d.acc, ti * P.tiles_j + tj, part, i0)) return;
    f32x4 sums[D::FI][D::FJ];
    scaled(sums, d.acc, P, q, i0, j0);
    finish<T, D::FI, D::FJ, D::PR, true, false>(P, sums, i0, j0, own_buffer(a0, a1, a2, a3, b0, b1, b2, b3),
                                                [](int, int, const bool (&)[4]) { return f32x4{}; });
}

// Few rows of x: tiles of 16 FI x 16 straight from memory, as k_small_forward's.
template <typename T, int FI>
__global__ __launch_bounds__(FI == 1 ? 1024 : 512) void k_small8(Args P, Scales8 q)
{
    extern __shared__ float small_lds[];
    constexpr int kAt = FI == 4 ? 2 : 4;
    const int i0 = blockIdx.x % P.tiles_i * (16 * FI), j0 = blockIdx.x / P.tiles_i * 16;
    i32x4 acc[FI] = {};
    int first, last;
    const int begin = blockIdx.y * P.k_part;
    small_share(begin, P.K - begin < P.k_part ? P.K : begin + P.k_part, first, last);
    for (int k0 = first; k0 < last; k0 += 32 * kAt) {
        Piece<bf16, K_ROWS> a[kAt][FI], b[kAt];
#pragma unroll
        for (int n = 0; n < kAt; ++n) {   // steps past the share: empty buffers, nothing is read
            const int k = k0 + 32 * n < last ? k0 + 32 * n : P.K;
            b[n].load(P.b, P.ldb, j0, P.J, k, P.K);
#pragma unroll
            for (int f = 0; f < FI; ++f) a[n][f].load(P.a, P.lda, i0 + f * 16, P.I, k, P.K);
        }
#pragma unroll
        for (int n = 0; n < kAt; ++n)
#pragma unroll
            for (int f = 0; f < FI; ++f) {
                bf16x8 va, vb;
                __builtin_memcpy(&va, a[n][f].w, 16);
                __builtin_memcpy(&vb, b[n].w, 16);
                acc[f] = MulI8::mul(vb, va, acc[f]);
            }
    }
    small_finish<T, FI, true>(P, acc, blockIdx.x, i0, j0, small_lds,
                              [&](int sum, int i, int j) { return (float)sum * (q.x[i] * q.w[j]); });
}

template <typename T>
hipError_t product8(const Args &P, const Scales8 &q, Shape shape, hipStream_t s)
{
    const dim3 grid((unsigned)P.tiles_i * (unsigned)P.tiles_j, (unsigned)P.parts);
    if (shape == TILE_64) k_product8<T, 64, 64, 2, 2><<<grid, 256, 0, s>>>(P, q);
    else if (shape == TILE_128) k_product8<T, 128, 128, 2, 2><<<grid, 256, 0, s>>>(P, q);
    else k_product8<T, 256, 256, 4, 2><<<grid, 512, 0, s>>>(P, q);
    return hipGetLastError();
}

template <typename T>
hipError_t small8(const Args &P, const Scales8 &q, int fi, int waves, hipStream_t s)
{
    const dim3 grid((unsigned)P.tiles_i * (unsigned)P.tiles_j, (unsigned)P.parts);
    const unsigned threads = 64u * waves, lds = (unsigned)(waves * fi * 1024);
    if (fi == 1) k_small8<T, 1><<<grid, threads, lds, s>>>(P, q);
    else if (fi == 2) k_small8<T, 2><<<grid, threads, lds, s>>>(P, q);
    else k_small8<T, 4><<<grid, threads, lds, s>>>(P, q);
    return hipGetLastError();
}

template <typename T>
hipError_t forward(const Dense8Forward &a, const Dense8Workspace &ws, hipStream_t s)
{
    const int pairs = (a.K + 15) / 16 * 8;
    const hipError_t e = quantise<T>(a.x, a.ldx, a.M, a.K, ws.codes, 2ll * pairs, ws.scales, s);
    if (e != hipSuccess) return e;
    Args P{};
    P.a = ws.codes, P.lda = pairs;
    P.b = a.codes, P.ldb = a.ldw / 2;
    P.I = a.M, P.J = a.N, P.K = pairs;
    P.c = a.y, P.ldc = a.ldy;
    P.bias = a.bias, P.residual = a.residual, P.ldr = a.ldr;
    P.act = a.act, P.alpha = a.alpha;
    P.part = ws.part, P.ticket = ws.ticket;
    const Scales8 q{ws.scales, a.scales};
    const Cut tiles = best_cut(P.I, P.J, P.K, 2, true);
    const SmallCut few = small_cut(P.I, P.J, P.K, 2, true);
    const bool small = few.us <= tiles.us;
    const int side_i = small ? 16 * few.fi : kSides[tiles.shape][0], side_j = small ? 16 : kSides[tiles.shape][1];
    const int parts = small ? few.parts : tiles.parts;
    P.tiles_i = ceil_div(P.I, side_i), P.tiles_j = ceil_div(P.J, side_j);
    P.k_part = ceil_div(ceil_div(P.K, parts), 32) * 32;
    P.parts = ceil_div(P.K, P.k_part);
    const size_t all = (size_t)P.tiles_i * P.tiles_j;
    if (P.parts > 1 && (all * P.parts * side_i * side_j * 4 > ws.part_bytes || all * sizeof(unsigned) > ws.ticket_bytes))
        return hipErrorInvalidValue;
    return small ? small8<T>(P, q, few.fi, few.waves, s) : product8<T>(P, q, tiles.shape, s);
}

}  // namespace

Dense8Workspace dense8_workspace(const hqml_dense_config &cfg)
{
    Dense8Workspace ws;
    const size_t M = (size_t)cfg.max_batch, N = (size_t)cfg.out_features, Kp = ((size_t)cfg.in_features + 15) / 16 * 16;
    ws.codes_bytes = M * Kp;
    ws.scales_bytes = M * 4;
    if (Kp / 2 > 96) {   // three steps: never split
        const size_t tiles = ((M + 255) / 256) * ((N + 255) / 256) * 16;   // whole tiles of any shape
        const size_t most = std::min<size_t>(kPartTiles, tiles * std::min<size_t>(kMostParts, (Kp / 2 + 31) / 64));
        ws.part_bytes = std::max(most * 64 * 64, (size_t)kUnits * 64 * 16) * 4;
        ws.ticket_bytes = std::max(most, (size_t)kUnits) * sizeof(unsigned);
    }
    return ws;
}

hipError_t launch_dense8_forward(const Dense8Forward &a, int dtype, const Dense8Workspace &ws, hipStream_t s)
{
    return dtype == HQML_DTYPE_BF16 ? forward<bf16>(a, ws, s) : forward<float>(a, ws, s);
}

hipError_t launch_quantise_rows(const void *x, long long ldx, long long rows, int K, int dtype, int8_t *codes, long long ldc,
                                float *scales, hipStream_t s)
{
    return dtype == HQML_DTYPE_BF16 ? quantise<bf16>(x, ldx, rows, K, codes, ldc, scales, s)
                                    : quantise<float>(x, ldx, rows, K, codes, ldc, scales, s);
}

}  // namespace hqml
