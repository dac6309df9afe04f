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
    float num, den, inv;   // inv = num / den, rounded; x num does not overflow
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
    const float less = size > 0x1p100f ? 0x1p-20f : 1.0f;
    return {127.0f * less, size * less, 127.0f / size};
}

// The largest of a wave, in all its lanes; magnitudes as bits order as integers, and a NaN is above them all.
__device__ __forceinline__ uint32_t wave_max(uint32_t b)
{
    auto with = [&](uint32_t other) { b = b > other ? b : other; };
    with((uint32_t)__builtin_amdgcn_update_dpp(0, (int)b, 0xB1, 0xF, 0xF, true));    // lane ^ 1
    with((uint32_t)__builtin_amdgcn_update_dpp(0, (int)b, 0x4E, 0xF, 0xF, true));    // lane ^ 2
    with((uint32_t)__builtin_amdgcn_update_dpp(0, (int)b, 0x141, 0xF, 0xF, true));   // mirrored in eight
    with((uint32_t)__builtin_amdgcn_update_dpp(0, (int)b, 0x140, 0xF, 0xF, true));   // mirrored in sixteen
    with((uint32_t)__shfl_xor((int)b, 16, 64));
    with((uint32_t)__shfl_xor((int)b, 32, 64));
    return b;
}

// Sixteen values of a row from c on, zeros past its end, as they are stored.
template <typename T>
struct Sixteen {
    static constexpr int kV = (int)sizeof(T);   // 16-byte words
    u32x4 w[kV];

    __device__ __forceinline__ void load(const T *row, int c, int K)
    {
        if (c + 16 <= K) {
#pragma unroll
            for (int k = 0; k < kV; ++k) w[k] = ((const u32x4_any *)(row + c))[k];
        } else {
            T t[16];
#pragma unroll
            for (int k = 0; k < 16; ++k) t[k] = c + k < K ? row[c + k] : T{};
            __builtin_memcpy(w, t, sizeof t);
        }
    }
    // The same through a buffer that ends with the row's last whole word.  The last of an odd number of bf16 comes by itself: its
    // word's other half may lie past the array.
    __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t buffer, const T *row, int c, int K)
    {
#pragma unroll
        for (int k = 0; k < kV; ++k) w[k] = __builtin_amdgcn_raw_buffer_load_b128(buffer, c * (int)sizeof(T) + k * 16, 0, 0);
        if (sizeof(T) == 2 && (K & 1) && c < K && c + 16 > K) {
            uint16_t last;
            __builtin_memcpy(&last, row + K - 1, 2);
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (c + 2 * k + 1 == K) w[k / 4][k % 4] = last;
        }
    }
    __device__ __forceinline__ void values(float (&x)[16]) const
    {
        T t[16];
        __builtin_memcpy(t, w, sizeof t);
#pragma unroll
        for (int k = 0; k < 16; ++k) x[k] = widen(t[k]);
    }
    // What was formed of the values is not kept: the words are, which take half the registers in bf16.
    __device__ __forceinline__ void keep()
    {
#pragma unroll
        for (int k = 0; k < kV; ++k) asm volatile("" : "+v"(w[k]));
    }
};

template <typename T>
__device__ __forceinline__ uint32_t largest16(const Sixteen<T> &v)
{
    float x[16];
    v.values(x);
    uint32_t b = 0;
#pragma unroll
    for (int k = 0; k < 16; ++k) {
        const uint32_t a = __builtin_bit_cast(uint32_t, x[k]) & 0x7FFFFFFFu;
        b = a > b ? a : b;
    }
    return b;
}

// The code of x where x num / den lies next to the middle h of two codes: x num and h den are compared exactly, each as the sum
// of two values in 32 bits (they have 32 bits at most, 24 and 8).
__device__ __forceinline__ float next_to_middle(float x, const RowScale &s, float h)
{
#pragma clang fp contract(off)
    const float q = x * s.num, p = h * s.den;
    const float r = (q - p) + (__builtin_fmaf(x, s.num, -q) - __builtin_fmaf(h, s.den, -p));
    return r > 0.0f ? h + 0.5f : r < 0.0f ? h - 0.5f : __builtin_rintf(h);
}

// Adding 3 2^22 rounds to an integer, to nearest even, and leaves it in the low byte.  x num / den as x inv is off by up to
// 2^-16: a quotient that is that near to the middle of two codes (one in 16,000) is looked at again.
template <typename T>
__device__ __forceinline__ u32x4 codes16(const Sixteen<T> &v, const RowScale &s)
{
    float x[16];
    v.values(x);
    if (s.num == 0.0f) return u32x4{0, 0, 0, 0};
    constexpr float kRound = 12582912.0f;
    float u[16], worst = 0.0f;
#pragma unroll
    for (int k = 0; k < 16; ++k) {
        const float t = x[k] * s.inv;
        u[k] = t + kRound;
        worst = fmaxf(worst, __builtin_fabsf(t - (u[k] - kRound)));
    }
    if (worst >= 0.5f - 0x1p-15f) {
#pragma unroll
        for (int k = 0; k < 16; ++k) {
            const float t = x[k] * s.inv, c = u[k] - kRound;
            if (__builtin_fabsf(t - c) >= 0.5f - 0x1p-15f) u[k] = next_to_middle(x[k], s, c + (t > c ? 0.5f : -0.5f)) + kRound;
        }
    }
    u32x4 w;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const uint32_t lo = __builtin_amdgcn_perm(__builtin_bit_cast(uint32_t, u[q * 4 + 1]), __builtin_bit_cast(uint32_t, u[q * 4]), 0x0C0C0400);
        const uint32_t hi = __builtin_amdgcn_perm(__builtin_bit_cast(uint32_t, u[q * 4 + 3]), __builtin_bit_cast(uint32_t, u[q * 4 + 2]), 0x04000C0C);
        w[q] = lo | hi;
    }
    return w;
}

constexpr int kHeld = 4;   // sixteens of a thread that stay in registers between the two passes over a row

// kWaves waves a row, 4 / kWaves rows a workgroup; the codes' rows end with zeros.  A row stays in registers between the pass that
// finds its scale and the one that forms its codes.  Bound by memory: 8192 x 4096 fp32 31 us, 5.5 TB/s; bf16 24 us, 4.2 TB/s, with
// arithmetic nearly as long.
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
        const long long r = r0 + (kWaves == 4 ? 0 : __builtin_amdgcn_readfirstlane(wave));
        const bool some = r < rows;   // the same in all threads of a row
        const T *row = x + (some ? r : 0) * ldx;
        const auto buffer = __builtin_amdgcn_make_buffer_rsrc((void *)row, 0, K * (int)sizeof(T) & ~3, 0x00027000);
        Sixteen<T> v[kHeld];
        uint32_t b = 0;
        if (some) {
#pragma unroll
            for (int h = 0; h < kHeld; ++h) v[h].load(buffer, row, (h * kThreads + lane) * 16, K);   // zeros past its end
#pragma unroll
            for (int h = 0; h < kHeld; ++h) {
                b = max(b, largest16(v[h]));
                __builtin_amdgcn_sched_barrier(0);
            }
            for (int c = (kHeld * kThreads + lane) * 16; c < Kp; c += kThreads * 16) {
                Sixteen<T> t;
                t.load(buffer, row, c, K);
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
            if (c >= Kp) continue;
            v[h].keep();
            *(u32x4 *)(to + c) = codes16(v[h], s);
            __builtin_amdgcn_sched_barrier(0);   // one at a time: registers for more waves
        }
        for (int c = (kHeld * kThreads + lane) * 16; c < Kp; c += kThreads * 16) {
            Sixteen<T> t;
            t.load(buffer, row, c, K);
            *(u32x4 *)(to + c) = codes16(t, s);
        }
        if (lane == 0) scales[r] = scale;
    }
}

template <typename T>
hipError_t quantise(const void *x, long long ldx, long long rows, int K, int8_t *codes, long long ldc, float *scales, hipStream_t s)
{
    // A wave a row where its registers hold it and there are rows for all compute units' waves; a workgroup a row otherwise, whose
    // two barriers cost less than a long row's way through one wave.
    if (K <= 64 * 16 * kHeld && (K <= 64 * 16 || rows >= 2048)) {
        const unsigned grid = (unsigned)std::min<long long>((rows + 3) / 4, 1 << 16);
        k_quantise<T, 1><<<grid, 256, 0, s>>>((const T *)x, ldx, rows, K, codes, ldc, scales);
    } else {
        const unsigned grid = (unsigned)std::min<long long>(rows, 1 << 16);
        k_quantise<T, 4><<<grid, 256, 0, s>>>((const T *)x, ldx, rows, K, codes, ldc, scales);
    }
    return hipGetLastError();
}

// ---- the product ----

// The scale of a row of x, as a value and a power of two.  The product of two scales may leave fp32's range where its product with
// a sum (or a sum of 0) does not.  Scales lie between 2^-100 and 2^121.1, so this one's fraction times 2^-25, from 2^-26 on, with
// one of w's is normal (2^-126 to 2^96.1) and, times a sum below 2^31, finite; the power goes into the result at once: the same bits
// where nothing overflows, one rounding below the normal range.
struct Scale {
    float part;
    int power;
};

__device__ __forceinline__ Scale split(float scale)
{
    return {__builtin_amdgcn_frexp_mantf(scale) * 0x1p-25f, __builtin_amdgcn_frexp_expf(scale) + 25};
}

__device__ __forceinline__ float scaled(int sum, const Scale &x, float w)
{
    return __builtin_amdgcn_ldexpf((float)sum * (x.part * w), x.power);
}

// Sums of codes' products as fp32 values: scaled by their row and column.
template <int FI, int FJ>
__device__ __forceinline__ void scaled(f32x4 (&to)[FI][FJ], const i32x4 (&acc)[FI][FJ], const Args &P, const Scales8 &q, int i0, int j0)
{
    const int lane = threadIdx.x & 63;
    Scale sx[FI];
#pragma unroll
    for (int f = 0; f < FI; ++f) {
        const int i = i0 + f * 16 + (lane & 15);
        sx[f] = split(i < P.I ? q.x[i] : 0.0f);
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
            for (int k = 0; k < 4; ++k) to[f][g][k] = scaled(acc[f][g][k], sx[f], sw[k]);
    }
}

// Larger products: the dense layer's tiles and choice of them (at twice the k of a bf16 tile), split along k where they are few.
// Bound by the matrix instructions, half of the compute units' busy cycles, and the epilogue's memory, in bursts between them:
// 8192 x 4096 x 4096 bf16 with gelu and residual 149 to 162 us, 1,700 to 1,840 TOP/s; a library's bare product takes 131.
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

// Few rows of x: tiles of 16 FI x 16, codes of w straight from memory as k_small_forward's, x's codes from the workspace.  Bound by
// latency: 45 x 1531 -> 803 fp32 5.4 us, behind 3.8 for the codes.
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
                              [&](int sum, int i, int j) { return scaled(sum, split(q.x[i]), q.w[j]); });
}

constexpr int kOwnHeld = 2;   // sixteens of a thread's
constexpr int kOwnLds = 40 * 1024;

// Floats of LDS that a tile's own codes take: up to 16 rows, 16 bytes apart beyond their length, for the banks; their largest
// magnitudes behind them.
__host__ __device__ inline int own_pitch(int pairs) { return pairs * 2 + 16; }
__host__ __device__ inline int own_bytes(int rows, int pairs) { return rows * own_pitch(pairs) + 64; }

// As k_small8<T, 1>, and every workgroup rounds its tile's rows of x by itself, while its first codes of w are under way: one launch
// instead of two.  P.a: x.  784 -> 20 4.2 us, launched by two 12; 4096 -> 4096 8.6 us (16.8 MB of codes), 12.1 by two.
template <typename T>
__global__ __launch_bounds__(1024) void k_small8_own(Args P, Scales8 q, int K)
{
    extern __shared__ float small_lds[];
    constexpr int kAt = 4;
    const int i0 = blockIdx.x % P.tiles_i * 16, j0 = blockIdx.x / P.tiles_i * 16;
    const int rows = P.I - i0 < 16 ? P.I - i0 : 16, pitch = own_pitch(P.K);
    int8_t *codes = (int8_t *)small_lds;
    uint32_t *largest = (uint32_t *)(codes + rows * pitch);
    float *sums = (float *)(largest + 16);
    int first, last;
    const int begin = blockIdx.y * P.k_part;
    small_share(begin, P.K - begin < P.k_part ? P.K : begin + P.k_part, first, last);
    Piece<bf16, K_ROWS> b[kAt];
    auto load = [&](int k0) {
#pragma unroll
        for (int n = 0; n < kAt; ++n) b[n].load(P.b, P.ldb, j0, P.J, k0 + 32 * n < last ? k0 + 32 * n : P.K, P.K);
    };
    const int sixteens = P.K >> 3, all = rows * sixteens;   // of a row, of the tile
    // x is asked for first: loads arrive in order, and it is needed before w
    Sixteen<T> v[kOwnHeld];
    int r_of[kOwnHeld];
#pragma unroll
    for (int h = 0; h < kOwnHeld; ++h) {
        const int at = h * blockDim.x + threadIdx.x;
        r_of[h] = rows == 1 ? 0 : at < all ? at / sixteens : rows - 1;
        if (at < all) v[h].load((const T *)P.a + (i0 + r_of[h]) * P.lda, (at - r_of[h] * sixteens) * 16, K);
    }
    load(first);
    if (threadIdx.x < 16) largest[threadIdx.x] = 0;
    __syncthreads();
#pragma unroll
    for (int h = 0; h < kOwnHeld; ++h) {
        if (h * (int)blockDim.x >= all) continue;   // the same in the whole workgroup
        const bool some = h * (int)blockDim.x + (int)threadIdx.x < all;
        uint32_t most = some ? largest16(v[h]) : 0;
        if (__builtin_amdgcn_readfirstlane(r_of[h]) == __builtin_amdgcn_readlane(r_of[h], 63)) {   // one row's
            most = wave_max(most);
            if ((threadIdx.x & 63) == 0 && some) atomicMax(largest + r_of[h], most);
        } else if (some) {
            atomicMax(largest + r_of[h], most);
        }
    }
    __syncthreads();
#pragma unroll
    for (int h = 0; h < kOwnHeld; ++h) {
        const int at = h * blockDim.x + threadIdx.x;
        if (at >= all) continue;
        float scale;
        *(u32x4 *)(codes + r_of[h] * pitch + (at - r_of[h] * sixteens) * 16) = codes16(v[h], row_scale(largest[r_of[h]], scale));
    }
    __syncthreads();
    const int lane = threadIdx.x & 63, row = (lane & 15) < rows ? lane & 15 : rows - 1;
    const int8_t *mine = codes + row * pitch + (lane >> 4) * 16;
    i32x4 acc[1] = {};
    for (int k0 = first; k0 < last; k0 += 32 * kAt) {
        bf16x8 vb[kAt];
#pragma unroll
        for (int n = 0; n < kAt; ++n) __builtin_memcpy(&vb[n], b[n].w, 16);
        if (k0 + 32 * kAt < last) load(k0 + 32 * kAt);
#pragma unroll
        for (int n = 0; n < kAt; ++n) {
            // past the share, or the row, w's codes are zeros
            const int k = k0 + 32 * n;
            const bool there = k < last && k * 2 + (lane >> 4) * 16 < P.K * 2;
            const u32x4 a = *(const u32x4 *)(there ? mine + k * 2 : codes);
            acc[0] = MulI8::mul(vb[n], __builtin_bit_cast(bf16x8, a), acc[0]);
        }
    }
    small_finish<T, 1, true>(P, acc, blockIdx.x, i0, j0, sums, [&](int sum, int i, int j) {
        float scale;
        (void)row_scale(largest[i - i0], scale);
        return scaled(sum, split(scale), q.w[j]);
    });
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
    Args P{};
    P.a = ws.codes, P.lda = pairs;
    P.b = a.codes, P.ldb = a.ldw / 2;
    P.I = a.M, P.J = a.N, P.K = pairs;
    P.c = a.y, P.ldc = a.ldy;
    P.bias = a.bias, P.residual = a.residual, P.ldr = a.ldr;
    P.act = a.act, P.alpha = a.alpha;
    P.part = ws.part, P.ticket = ws.ticket;
    const Scales8 q{ws.scales, a.scales};
    // Codes of x by the workgroups that use them, or by a launch before: the least of estimates.  The launch takes 4.5 us and
    // memory's time; a workgroup's own codes 1.2, and 0.6 for each sixteen values of a thread.
    const Cut tiles = best_cut(P.I, P.J, P.K, 2, true);
    SmallCut few = small_cut(P.I, P.J, P.K, 2, true);
    const SmallCut few16 = small_cut(P.I, P.J, P.K, 2, true, 1);
    const int rows = std::min(a.M, 16), each = ceil_div(rows * (pairs / 8), 64 * few16.waves);
    const float before = 4.5f + (float)a.M * a.K * (sizeof(T) + 1) / 3.5e6f;
    const bool own = each <= kOwnHeld && own_bytes(rows, pairs) <= kOwnLds &&
                     few16.us + 1.2f + 0.6f * (float)each <= before + std::min(few.us, tiles.us);
    const bool small = own || few.us <= tiles.us;
    if (own) few = few16;
    const int side_i = small ? 16 * few.fi : kSides[tiles.shape][0], side_j = small ? 16 : kSides[tiles.shape][1];
    const int parts = small ? few.parts : tiles.parts;
    P.tiles_i = ceil_div(P.I, side_i), P.tiles_j = ceil_div(P.J, side_j);
    P.k_part = ceil_div(ceil_div(P.K, parts), 32) * 32;
    P.parts = ceil_div(P.K, P.k_part);
    const size_t all = (size_t)P.tiles_i * P.tiles_j;
    if (P.parts > 1 && (all * P.parts * side_i * side_j * 4 > ws.part_bytes || all * sizeof(unsigned) > ws.ticket_bytes))
        return hipErrorInvalidValue;
    if (own) {
        P.a = a.x, P.lda = a.ldx;
        const dim3 grid((unsigned)all, (unsigned)P.parts);
        k_small8_own<T><<<grid, 64 * few.waves, own_bytes(rows, pairs) + few.waves * 1024, s>>>(P, q, a.K);
        return hipGetLastError();
    }
    const hipError_t e = quantise<T>(a.x, a.ldx, a.M, a.K, ws.codes, 2ll * pairs, ws.scales, s);
    if (e != hipSuccess) return e;
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
