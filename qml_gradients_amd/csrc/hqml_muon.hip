// Muon: momentum, and updates orthogonalised by Newton-Schulz products (K. Jordan et al., 2024).
//
//   m = mu m + (1 - mu) g,  u = mu m + (1 - mu) g (Nesterov) or m
//   X = u / max(|u|, eps);  `steps` times:  A = X X^T,  X <- a X + (b A + c A^2) X
//   p = p (1 - lr wd) - lr f X
//
// The polynomial acts on the singular values alone, so a matrix with more rows than columns takes A = X^T X and
// X <- a X + X (b A + c A^2): A is as small as it can be, and no matrix is transposed.  Three products a step, on the matrix
// cores, of operands in fp16 (products exact, sums in fp32):
//   two values for each, x = hi + lo, 22 bits; of their four products the three that count, one after the other along k
//   one value for each, 11 bits, where the caller of bf16 parameters (`precise` 0) takes that: a third of the products
// With two, X is as exact as 32 bits make it: off by 1e-6 to 2e-6 of its size after five steps, and by 2e-5 to 3e-5 where a gradient
// has few directions (8 in 512 x 2048; the steps in fp32 throughout 4e-6 and 3e-5 to 5e-5): roundings fill the others, and each step
// lifts those by a = 3.4.  With one it is off by 1.5e-3 and 4e-2.  A bf16 parameter's own rounding hides such errors in one step, but
// not in the sum of many.
// X's values are at most a little over 1 and often small, so X, A and B = b A + c A^2 are held times 2^10: fp16's normal range then
// goes from 2^-24 to 64 of them.
//
// All larger matrices of a call go through each product in one launch, a workgroup a tile (or a part of one along k).  Bound by the
// matrix instructions (two 4096 x 4096 bf16, a step, of two values: X X^T 452 us, b A + c A^2 453, X 750, 1,100 fp16 TFLOP/s in the
// last; of one: 154, 160 and 243, 1,130; two 1024 x 4096 fp32: 41, 19 and 58, 890 in the last), below some 800 x 800 by the launches
// and the steps' latency (four 803 x 517 fp32: 16, 12 and 20).  Small matrices take one launch for all steps (three 64 x 32 14.2 us
// for 76), thin ones three.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>
#include <type_traits>

#include "hqml_gemm.hpp"
#include "hqml_layers.hpp"

namespace hqml {
namespace {

using namespace gemm;

constexpr float kScale = 1024.0f, kUnscale = 1.0f / kScale;
constexpr int kMatrices = 24;              // of one launch
constexpr long long kChunk = 8192;         // values of a workgroup of the momentum kernel
constexpr size_t kBatchBytes = 1ull << 30; // workspace from which matrices go in several rounds

int pad8(int n) { return (n + 7) & ~7; }

struct Half {   // fp16 by its bits
    uint16_t u;
};

// A matrix of a call.  Planes of X, A and B follow each other.
struct Matrix {
    void *p;
    const void *g;
    float *m;
    Half *x[2], *a, *b;   // thin matrices: x[0] is P, in 64 bits
    double *sums;         // of squares, one a chunk; thin matrices: of products
    int rows, cols;
    float size;           // lr f
};

struct Batch {
    int count;
    unsigned first[kMatrices];   // first workgroup of each
    Matrix t[kMatrices];
};
static_assert(sizeof(Batch) <= 3584, "kernel arguments");

struct Scalars {
    float mu, nu;      // nu = 1 - mu
    int nesterov;
    float eps;
    float decay;       // lr wd
    float a, b, c;
};

__device__ __forceinline__ int matrix_of(const unsigned *first, int count, unsigned wg)
{
    int lo = 0, hi = count - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (first[mid] <= wg) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

__device__ __forceinline__ float update_of(const Scalars &k, float m, float g) { return k.nesterov ? m * k.mu + g * k.nu : m; }

// n neighbouring values, 16 bytes or fewer at a time and at any alignment of the element: the hardware takes them so.
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

// The sum over a wave, in all its lanes.
__device__ __forceinline__ double wave_sum(double v)
{
    auto with = [&](auto move) {
        const unsigned long long b = __builtin_bit_cast(unsigned long long, v);
        const unsigned long long m = (unsigned)move((int)b) | (unsigned long long)(unsigned)move((int)(b >> 32)) << 32;
        v += __builtin_bit_cast(double, m);
    };
    with([](int x) { return __builtin_amdgcn_update_dpp(0, x, 0xB1, 0xF, 0xF, true); });    // lane ^ 1
    with([](int x) { return __builtin_amdgcn_update_dpp(0, x, 0x4E, 0xF, 0xF, true); });    // lane ^ 2
    with([](int x) { return __builtin_amdgcn_update_dpp(0, x, 0x141, 0xF, 0xF, true); });   // mirrored in eight
    with([](int x) { return __builtin_amdgcn_update_dpp(0, x, 0x140, 0xF, 0xF, true); });   // mirrored in sixteen
    with([](int x) { return __shfl_xor(x, 16, 64); });
    with([](int x) { return __shfl_xor(x, 32, 64); });
    return v;
}

// m, and the sums of u^2 of each chunk, in 64 bits: they neither overflow nor lose a small chunk beside a large one.
// The first workgroup clears the tickets of the products that follow.
template <typename G>
__global__ __launch_bounds__(256) void k_momentum(Batch batch, Scalars k, unsigned *tickets, int n_tickets)
{
    __shared__ double part[4];
    if (blockIdx.x == 0)
        for (int i = threadIdx.x; i < n_tickets; i += 256) tickets[i] = 0;
    const int ti = matrix_of(batch.first, batch.count, blockIdx.x);
    const Matrix &t = batch.t[ti];
    const long long chunk = blockIdx.x - batch.first[ti], n = (long long)t.rows * t.cols, base = chunk * kChunk;
    const int end = n - base < kChunk ? (int)(n - base) : (int)kChunk;
    const G *g = (const G *)t.g + base;
    float *m = t.m + base;
    double sum = 0.0;
    constexpr int kV = 4, kAt = 4;   // values of a thread at once, and how often before the first is used
    for (int i0 = threadIdx.x * kV; i0 < end; i0 += 256 * kV * kAt) {
        float mv[kAt][kV];
        G gv[kAt][kV];
#pragma unroll
        for (int a = 0; a < kAt; ++a) {
            const int i = i0 + a * 256 * kV;
            if (i + kV <= end) get(mv[a], m + i), get(gv[a], g + i);
        }
#pragma unroll
        for (int a = 0; a < kAt; ++a) {
            const int i = i0 + a * 256 * kV;
            if (i + kV <= end) {
#pragma unroll
                for (int e = 0; e < kV; ++e) {
                    const float gi = widen(gv[a][e]);
                    mv[a][e] = mv[a][e] * k.mu + gi * k.nu;
                    const double u = update_of(k, mv[a][e], gi);
                    sum += u * u;
                }
                put(m + i, mv[a]);
            } else {
                for (int j = i; j < end; ++j) {
                    const float gi = widen(g[j]), mj = m[j] * k.mu + gi * k.nu;
                    m[j] = mj;
                    const double u = update_of(k, mj, gi);
                    sum += u * u;
                }
            }
        }
    }
    sum = wave_sum(sum);
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = sum;
    __syncthreads();
    if (threadIdx.x == 0) t.sums[chunk] = part[0] + part[1] + part[2] + part[3];
}

__device__ __forceinline__ void to_planes(float v, Half &hi, Half &lo)
{
    const _Float16 h = (_Float16)v;
    hi.u = __builtin_bit_cast(uint16_t, h);
    lo.u = __builtin_bit_cast(uint16_t, (_Float16)(v - (float)h));
}

__device__ __forceinline__ float from_half(Half h) { return (float)__builtin_bit_cast(_Float16, h.u); }

// 1 / max(|u|, eps), in 64 bits: 32 do not hold it for the least eps.  NaN where |u| is.
__device__ __forceinline__ double inverse_norm(const Matrix &t, float eps)
{
    __shared__ double part[4];
    const int chunks = (int)(((long long)t.rows * t.cols + kChunk - 1) / kChunk);
    double sum = 0.0;
    for (int i = threadIdx.x; i < chunks; i += 256) sum += t.sums[i];
    sum = wave_sum(sum);
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = sum;
    __syncthreads();
    const double norm = sqrt(part[0] + part[1] + part[2] + part[3]);
    return 1.0 / (norm <= (double)eps ? (double)eps : norm);
}

// X, normalised, in rows of a multiple of eight that end with zeros.
template <typename G, int PLANES>
__global__ __launch_bounds__(256) void k_begin(Batch batch, Scalars k)
{
    const int ti = matrix_of(batch.first, batch.count, blockIdx.x);
    const Matrix &t = batch.t[ti];
    // as a value and a power of two, which u meets first: it is no more than 2^11 then.  A product in 64 bits takes longer than
    // memory (two 4096 x 4096 bf16 62 us instead of 51)
    const double inv = inverse_norm(t, k.eps) * kScale;
    const float part = (float)__builtin_amdgcn_frexp_mant(inv);
    const int power = __builtin_amdgcn_frexp_exp(inv);
    const int ld = (t.cols + 7) & ~7, eights = ld / 8;
    const long long n = (long long)t.rows * eights, plane = (long long)t.rows * ld;
    const unsigned groups = (ti + 1 < batch.count ? batch.first[ti + 1] : gridDim.x) - batch.first[ti];
    const G *g = (const G *)t.g;
    for (long long i = (long long)(blockIdx.x - batch.first[ti]) * 256 + threadIdx.x; i < n; i += (long long)groups * 256) {
        const int row = (int)(i / eights), c = (int)(i - (long long)row * eights) * 8;
        const long long at = (long long)row * t.cols + c;
        Half hi[8], lo[8];
        float mv[8] = {};
        G gv[8] = {};
        if (c + 8 <= t.cols) {
            get(mv, t.m + at);
            if (k.nesterov) get(gv, g + at);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (c + e < t.cols) mv[e] = t.m[at + e], gv[e] = g[at + e];
        }
#pragma unroll
        for (int e = 0; e < 8; ++e)
            to_planes(c + e < t.cols ? __builtin_amdgcn_ldexpf(update_of(k, mv[e], widen(gv[e])), power) * part : 0.0f, hi[e], lo[e]);
        *(u32x4 *)(t.x[0] + (long long)row * ld + c) = __builtin_bit_cast(u32x4, hi);
        if (PLANES == 2) *(u32x4 *)(t.x[0] + plane + (long long)row * ld + c) = __builtin_bit_cast(u32x4, lo);
    }
}

// ---- the products ----
//
// A product's tiles, for few of them each in several parts along k, are the workgroups.  A and B are symmetric: of their tiles
// those on and below the diagonal are formed, and each is written to its mirrored place too.

enum Stage { GRAM, POLY, APPLY };

// C = sum_k A(i, k) B(j, k), and what becomes of it.
struct Product {
    const Half *a, *b, *with;   // with: what a multiple of is added, laid out as C
    Half *c;
    void *p;                    // the last step's: the parameter
    float *part;                // partial sums
    unsigned *ticket;
    long long plane_a, plane_b, plane_c;   // values from one plane to the next
    int lda, ldb, ldc, I, J, K;
    int tiles_i, tiles_j;
    int tiles, skip;            // of this launch; tiles of twice the side that another one took
    int parts, steps;           // steps of a part
    short cols;                 // A and B across k (GRAM), B across k (APPLY)
    short mirrored;
    float size;
};

template <int MOST>
struct ProductsOf {
    int count;
    unsigned first[MOST];   // multiples of eight: the XCD of a tile follows from its number
    Product t[MOST];
};
using Products = ProductsOf<kMatrices>;

struct Finish {
    float one, two;   // C = one sum + two with
    float decay;
    int last;
};
static_assert(sizeof(Products) + sizeof(Finish) <= 4096, "kernel arguments");

// Operands of two planes: gemm::Direct with both planes of a step's tiles in a buffer, and three matrix instructions for its one:
// lo hi, hi lo and hi hi.  A step has 4/3 of the loads and barriers of three steps of one plane (1024 x 4096, X X^T: 56 us so).
template <int LA, int LB, int BM, int BN, int WI, int WJ>
struct DirectPair {
    static constexpr int BK = 32, kWaves = WI * WJ, TI = BM / WI, TJ = BN / WJ, FI = TI / 16, FJ = TJ / 16;
    using TA = DirectTile<LA, BM, BK, kWaves>;
    using TB = DirectTile<LB, BN, BK, kWaves>;
    static constexpr int kPlaneA = TA::kBytes, kPlaneB = TB::kBytes, kLoads = 2 * (TA::kLoads + TB::kLoads);
    TA ta;
    TB tb;
    long long plane_a, plane_b;   // bytes
    int wi, wj;
    f32x4 acc[FI][FJ];
    static constexpr int kAhead = 1, kMid = FI / 2, kPer = FJ / (FI - kMid);
    bf16x8 fa[FI][2], fb[FJ][2];

    // Queue load n of kLoads.
    __device__ __forceinline__ void load_one(const typename TA::Step &sa, const typename TB::Step &sb, char *A, char *B, int n) const
    {
        const int plane = n & 1;
        n >>= 1;
        if (n < TA::kLoads) {
            auto st = sa;
            st.p += plane * plane_a;
            ta.load(st, (lds_char *)A + plane * kPlaneA, n);
        } else {
            auto st = sb;
            st.p += plane * plane_b;
            tb.load(st, (lds_char *)B + plane * kPlaneB, n - TA::kLoads);
        }
    }
    __device__ __forceinline__ void load(char *A, char *B, int t) const
    {
        const auto sa = ta.begin(t * BK);
        const auto sb = tb.begin(t * BK);
#pragma unroll
        for (int n = 0; n < kLoads; ++n) load_one(sa, sb, A, B, n);
    }
    __device__ __forceinline__ void get_a(bf16x8 (&to)[2], const char *A, int f) const
    {
#pragma unroll
        for (int p = 0; p < 2; ++p) to[p] = ta.fragment((const lds_char *)A + p * kPlaneA, wi * TI + f * 16, 0);
    }
    __device__ __forceinline__ void get_b(bf16x8 (&to)[2], const char *B, int g) const
    {
#pragma unroll
        for (int p = 0; p < 2; ++p) to[p] = tb.fragment((const lds_char *)B + p * kPlaneB, wj * TJ + g * 16, 0);
    }
    __device__ __forceinline__ void step(const char *A, const char *A1, const char *B1, char *A3, char *B3, int t)
    {
        const auto sa = ta.begin((t + 3) * BK);
        const auto sb = tb.begin((t + 3) * BK);
        bf16x8 na[kAhead][2], nb[FJ][2];
        wait_loads<kLoads>();   // step t + 1 is there, and every wave is done with step t - 1
        barrier();
#pragma unroll
        for (int f = 0; f < FI; ++f) {
            if (f + kAhead < FI) get_a(fa[f + kAhead], A, f + kAhead);
            else get_a(na[f + kAhead - FI], A1, f + kAhead - FI);
            if (f >= kMid) {
#pragma unroll
                for (int g = (f - kMid) * kPer; g < (f - kMid + 1) * kPer; ++g) get_b(nb[g], B1, g);
            }
            // a wave's loads among its matrix instructions, a few at a time: more would hold those up behind them
#pragma unroll
            for (int c = 0; c < 3; ++c) {   // small products first
#pragma unroll
                for (int g = 0; g < FJ; ++g) acc[f][g] = MulF16::mul(fb[g][c == 1], fa[f][c == 0], acc[f][g]);
                constexpr int kSlots = FI * 3;
                const int slot = f * 3 + c;
#pragma unroll
                for (int n = slot * kLoads / kSlots; n < (slot + 1) * kLoads / kSlots; ++n) load_one(sa, sb, A3, B3, n);
                __builtin_amdgcn_sched_barrier(0);
            }
        }
#pragma unroll
        for (int p = 0; p < 2; ++p) {
#pragma unroll
            for (int f = 0; f < kAhead; ++f) fa[f][p] = na[f][p];
#pragma unroll
            for (int g = 0; g < FJ; ++g) fb[g][p] = nb[g][p];
        }
    }
    __device__ __forceinline__ void run(int n, char *a0, char *a1, char *a2, char *a3, char *b0, char *b1, char *b2, char *b3)
    {
        const int wave = threadIdx.x >> 6;
        wi = wave / WJ, wj = wave % WJ;
#pragma unroll
        for (int f = 0; f < FI; ++f)
#pragma unroll
            for (int g = 0; g < FJ; ++g) acc[f][g] = f32x4{};
        load(a0, b0, 0);
        load(a1, b1, 1);
        load(a2, b2, 2);
        wait_loads<2 * kLoads>();
        barrier();
#pragma unroll
        for (int f = 0; f < kAhead; ++f) get_a(fa[f], a0, f);
#pragma unroll
        for (int g = 0; g < FJ; ++g) get_b(fb[g], b0, g);
        int t = 0;
        for (; t + 4 <= n; t += 4) {
            step(a0, a1, b1, a3, b3, t);
            step(a1, a2, b2, a0, b0, t + 1);
            step(a2, a3, b3, a1, b1, t + 2);
            step(a3, a0, b0, a2, b2, t + 3);
        }
        if (t < n) {
            step(a0, a1, b1, a3, b3, t);
            if (t + 1 < n) {
                step(a1, a2, b2, a0, b0, t + 1);
                if (t + 2 < n) step(a2, a3, b3, a1, b1, t + 2);
            }
        }
        wait_loads<0>();
        barrier();
    }
    static constexpr int kFit = 2 * (kPlaneA < kPlaneB ? kPlaneA : kPlaneB) / (TJ * 4), PR = kFit >= TI ? TI : kFit;
};

// Tile t of a lower triangle, in rows.
__device__ __forceinline__ void triangle(int t, int &i, int &j)
{
    i = (int)((sqrtf(8.0f * (float)t + 1.0f) - 1.0f) * 0.5f);
    while (i * (i + 1) / 2 > t) --i;
    while ((i + 1) * (i + 2) / 2 <= t) ++i;
    j = t - i * (i + 1) / 2;
}

// Tile t of ti x tj, in bands of eight rows.
__device__ __forceinline__ void banded(int t, int ti, int tj, int &i, int &j)
{
    const int band = t / (8 * tj), first = band * 8, rows = ti - first < 8 ? ti - first : 8, in = t - band * 8 * tj;
    i = first + in % rows;
    j = in / rows;
}

template <int PLANES>
__device__ __forceinline__ void read_planes(float (&x)[8], const Half *from, long long plane)
{
    Half h[8];
    u32x4 w = *(const u32x4 *)from;
    __builtin_memcpy(h, &w, 16);
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = from_half(h[e]);
    if (PLANES == 1) return;
    w = *(const u32x4 *)(from + plane);
    __builtin_memcpy(h, &w, 16);
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] += from_half(h[e]);
}

template <int PLANES>
__device__ __forceinline__ void write_planes(Half *to, long long plane, const float (&v)[8])
{
    Half hi[8], lo[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) to_planes(v[e], hi[e], lo[e]);
    *(u32x4 *)to = __builtin_bit_cast(u32x4, hi);
    if (PLANES == 2) *(u32x4 *)(to + plane) = __builtin_bit_cast(u32x4, lo);
}

// T: the parameter's type.
template <int STAGE, int LA, int LB, int PLANES, typename T, int BM, int BN, int WI, int WJ>
__device__ __forceinline__ void product(const Product &P, const Finish &F, int ti, int tj, int tile, int part, char *a0, char *a1,
                                        char *a2, char *a3, char *b0, char *b1, char *b2, char *b3)
{
    using D = std::conditional_t<PLANES == 2, DirectPair<LA, LB, BM, BN, WI, WJ>, Direct<LA, LB, BM, BN, 32, WI, WJ, MulF16>>;
    D d;
    const int kb = part * P.steps * 32, kn = P.K - kb < P.steps * 32 ? P.K - kb : P.steps * 32;
    d.ta.init(P.a, P.lda, ti * BM, P.I, kn, kb);
    d.tb.init(P.b, P.ldb, tj * BN, P.J, kn, kb);
    if constexpr (PLANES == 2) d.plane_a = P.plane_a * 2, d.plane_b = P.plane_b * 2;
    d.run((kn + 31) / 32, a0, a1, a2, a3, b0, b1, b2, b3);
    constexpr int TJ = D::TJ, FI = D::FI, FJ = D::FJ, PR = D::PR, kRow = TJ * 4, kMask = TJ / 4 - 1;
    const int lane = threadIdx.x & 63, i0 = ti * BM + d.wi * D::TI, j0 = tj * BN + d.wj * TJ;
    if (P.parts > 1) {
        Args at{};
        at.I = P.I, at.parts = P.parts, at.part = P.part, at.ticket = P.ticket;
        if (!joined<FI, FJ, 64 * D::kWaves>(at, d.acc, tile, part, i0)) return;
    }

    // a wave's part is turned around in LDS, so that a lane ends with eight neighbouring j of a row
    constexpr int kGroups = TJ / 8, kRows = 64 / kGroups, kRounds = PR / kRows;
    const int c = lane % kGroups * 8, j = j0 + c;
    const bool mirror = STAGE != APPLY && ti != tj;
    lds_char *const buf = own_buffer(a0, a1, a2, a3, b0, b1, b2, b3);
#pragma unroll
    for (int f0 = 0; f0 < FI; f0 += PR / 16) {
#pragma unroll
        for (int f = 0; f < PR / 16; ++f)
#pragma unroll
            for (int g = 0; g < FJ; ++g)
                *(__attribute__((address_space(3))) f32x4 *)(buf + (f * 16 + (lane & 15)) * kRow +
                                                             (((g * 4 + (lane >> 4)) ^ (lane & kMask & 15)) << 4)) =
                    d.acc[f0 + f][g];
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");   // the wave's own writes, read by its other lanes
        for (int round = 0; round < kRounds; ++round) {
            const int r = round * kRows + lane / kGroups, i = i0 + f0 * 16 + r, key = r & kMask & 15;
            const auto *src = (const __attribute__((address_space(3))) f32x4 *)(buf + r * kRow);
            const f32x4 lo4 = src[(c >> 2) ^ key], hi4 = src[((c >> 2) + 1) ^ key];
            if (i >= P.I || j >= P.J) continue;
            float v[8], x[8];
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = lo4[e] * F.one, v[4 + e] = hi4[e] * F.one;
            const long long at = (long long)i * P.ldc + j;
            if (STAGE != GRAM) {   // rows end with zeros, and so do sums over them
                read_planes<PLANES>(x, P.with + at, P.plane_c);
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] = __builtin_fmaf(x[e], F.two, v[e]);
            }
            if (STAGE != APPLY || !F.last) {
                write_planes<PLANES>(P.c + at, P.plane_c, v);
                if (mirror) {   // finished, for the mirrored place
                    auto *back = (__attribute__((address_space(3))) f32x4 *)(buf + r * kRow);
                    back[(c >> 2) ^ key] = f32x4{v[0], v[1], v[2], v[3]};
                    back[((c >> 2) + 1) ^ key] = f32x4{v[4], v[5], v[6], v[7]};
                }
                continue;
            }
            T *p = (T *)P.p + (long long)i * P.J + j, t[8];
            const float size = P.size * kUnscale;
            if (j + 8 <= P.J) {
                get(t, p);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float y = widen(t[e]);
                    // one rounding for the decayed parameter: 1 - lr wd, held in 32 bits, would add its own
                    narrow(__builtin_fmaf(y, -F.decay, y) - size * v[e], t[e]);
                }
                put(p, t);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    if (j + e >= P.J) continue;
                    const float y = widen(p[e]);
                    narrow(__builtin_fmaf(y, -F.decay, y) - size * v[e], p[e]);
                }
            }
        }
        if (mirror) {   // eight rows of a column are eight neighbours of a row there; lanes beside each other take its next ones
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
            constexpr int kDown = PR / 8, kAcross = 64 / kDown;
            const int r0 = lane % kDown * 8, i = i0 + f0 * 16 + r0;
#pragma unroll 2
            for (int cj = lane / kDown; cj < TJ; cj += kAcross) {
                const int jj = j0 + cj;
                float v[8];
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    v[e] = *(const __attribute__((address_space(3))) float *)(buf + (r0 + e) * kRow +
                                                                              (((cj >> 2) ^ ((r0 + e) & kMask & 15)) << 4) + (cj & 3) * 4);
                if (jj < P.J && i < P.I) write_planes<PLANES>(P.c + (long long)jj * P.ldc + i, P.plane_c, v);
            }
        }
        asm volatile("" ::: "memory");
    }
}

template <int STAGE, int PLANES, typename T, int SIDE, int WAVES, int MOST>
__global__ __launch_bounds__(64 * WAVES, PLANES == 2 && SIDE == 128 && WAVES == 4 ? 1 : 2) void k_product(ProductsOf<MOST> G, Finish F)
{
    constexpr int kBytes = SIDE * 64 * PLANES;
    static_assert(PLANES == 1 || SIDE <= 128, "room for two planes");
    __shared__ __attribute__((aligned(1024))) char a0[kBytes], a1[kBytes], a2[kBytes], a3[kBytes];
    __shared__ __attribute__((aligned(1024))) char b0[kBytes], b1[kBytes], b2[kBytes], b3[kBytes];
    const int m = matrix_of(G.first, G.count, blockIdx.x);
    const Product &P = G.t[m];
    // Workgroups go round the eight XCDs in turn; each XCD takes a run of the product's tiles, part by part, so that what it
    // works on together shares rows and k in its L2.
    const int id = blockIdx.x - G.first[m], units = P.tiles * P.parts, xcd = id & 7, q = units >> 3, r = units & 7;
    if ((id >> 3) >= q + (xcd < r ? 1 : 0)) return;
    const int unit = xcd * q + (xcd < r ? xcd : r) + (id >> 3), part = unit / P.tiles, tile = unit - part * P.tiles;
    int ti, tj;
    if (P.skip < 0) {
        if (STAGE != APPLY) triangle(tile, ti, tj);
        else banded(tile, P.tiles_i, P.tiles_j, ti, tj);
    } else {   // quarters of larger tiles
        const int large = P.skip + (tile >> 2);
        if (STAGE != APPLY) triangle(large, ti, tj);
        else banded(large, (P.tiles_i + 1) >> 1, (P.tiles_j + 1) >> 1, ti, tj);
        ti = ti * 2 + ((tile >> 1) & 1), tj = tj * 2 + (tile & 1);
        if (ti >= P.tiles_i || tj >= P.tiles_j || (STAGE != APPLY && tj > ti)) return;
    }
    // 256 x 256: waves of 64 x 128 where both operands lie along k, of 128 x 64 elsewhere, as the dense layer's
    constexpr int WI = 2, WJ = WAVES / 2, WIR = WAVES / 2, WJR = 2;
    if (STAGE == POLY || !P.cols)
        product<STAGE, K_ROWS, K_ROWS, PLANES, T, SIDE, SIDE, WIR, WJR>(P, F, ti, tj, tile, part, a0, a1, a2, a3, b0, b1, b2, b3);
    else if (STAGE == GRAM)
        product<STAGE, K_COLS, K_COLS, PLANES, T, SIDE, SIDE, WI, WJ>(P, F, ti, tj, tile, part, a0, a1, a2, a3, b0, b1, b2, b3);
    else
        product<STAGE, K_ROWS, K_COLS, PLANES, T, SIDE, SIDE, WI, WJ>(P, F, ti, tj, tile, part, a0, a1, a2, a3, b0, b1, b2, b3);
}

// ---- small matrices ----
//
// A workgroup takes a whole matrix through the whole step: X (the smaller side as rows), A and B in fp32 in LDS, products by the
// fp32 matrix instruction, nothing rounded to fewer bits.  What counts is latency: three products and as many barriers a
// step, one launch instead of 2 + 3 for each step.

constexpr int kSmallSide = 64, kSmallWaves = 16, kTinyWaves = 4;
constexpr int kSmallLds = 160 * 1024 - 1024;
// Up to where: in values, where the rest may be thin (16 x 1000 31 us, as thin ones 28; 48 x 128 27 and 45, 48 x 400 62 and 50;
// 64 x 200 58 and 72, 64 x 350 84 and 72), in multiply-adds of X X^T otherwise (64 x 350 84 us, by tiles 89; 64 x 420 99 and 92).
constexpr int kSmallValues = 14 << 10;
constexpr long long kSmallWork = 3 << 19;

// Four waves a matrix where all of a launch have up to so many padded values, sixteen otherwise: barriers and joins of four cost less,
// products of sixteen (us by four and sixteen: 16 x 16 7.8 and 8.5, 16 x 64 9.2 and 11.6, 32 x 32 10.8 and 13.3, 16 x 128 12.0 and 12.5,
// 32 x 64 14.2 and 14.3, 32 x 128 22.3 and 17.7).  Matrices run beside each other, so the largest decides.
constexpr int kTinyValues = 2048;
static_assert(48 * 48 > kTinyValues, "matrices of three tiles of sixteen rows take sixteen waves");

__host__ __device__ inline int pad16(int n) { return (n + 15) & ~15; }

struct SmallSize {
    int n, m, ldx, lda;   // sides, padded; floats from a row to the next, four more than they hold: other banks
    __host__ __device__ SmallSize(int rows, int cols)
        : n(pad16(rows < cols ? rows : cols)), m(pad16(rows < cols ? cols : rows)), ldx(m + 4), lda(n + 4)
    {
    }
    __host__ __device__ size_t bytes() const { return ((size_t)n * ldx + 2 * (size_t)n * lda + kSmallWaves * 256) * 4; }
};

bool is_small(int rows, int cols, bool thin)
{
    const SmallSize z(rows, cols);
    return z.n <= kSmallSide && z.bytes() <= (size_t)kSmallLds &&
           (thin ? z.n * z.m <= kSmallValues : (long long)z.n * z.n * z.m <= kSmallWork);
}

// Four k of a 16 x 16 block: lane % 16 is the row of either operand, lane / 16 its k.
__device__ __forceinline__ f32x4 multiply(float b, float a, f32x4 c) { return __builtin_amdgcn_mfma_f32_16x16x4f32(b, a, c, 0, 0, 0); }

// The steps of a matrix of NT tiles of sixteen rows.  What counts is the way from LDS to the matrix instructions, so each loop
// reads all its operands, or many, before it uses the first.
template <int NT, int WAVES>
__device__ __forceinline__ void small_steps(const SmallSize &z, const Scalars &k, int steps, float *X, float *A, float *B, float *P)
{
    constexpr int kThreads = 64 * WAVES, kTiles = NT * (NT + 1) / 2;
    constexpr int kParts = kTiles < WAVES ? WAVES / kTiles : 1;   // of k, for A: a wave each
    constexpr int kAt = 8;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, row = lane & 15, quad = lane >> 4;
    const int kp = wave / kTiles, fours = z.m / 4, share = (fours + kParts - 1) / kParts;
    const int from = kp * share, to = from + share < fours ? from + share : fours;
    auto tile_at = [](int tile, int &i, int &j) {   // of a lower triangle, in rows
        i = 0, j = tile;
        while (j > i) j -= ++i;
    };
    int wi, wj;
    tile_at(wave % kTiles, wi, wj);
    auto mirrored = [&](float *to, int i, int j, float v) {
        to[i * z.lda + j] = v;
        if (i >> 4 != j >> 4) to[j * z.lda + i] = v;
    };
    for (int step = 0; step < steps; ++step) {
        if (kp < kParts) {   // A = X X^T
            const float *a = X + (wi * 16 + row) * z.ldx + quad, *b = X + (wj * 16 + row) * z.ldx + quad;
            f32x4 s[2] = {};
            for (int f = from; f < to; f += kAt) {
                float av[kAt], bv[kAt];
#pragma unroll
                for (int e = 0; e < kAt; ++e) {
                    const int at = f + e < to ? f + e : from;
                    av[e] = f + e < to ? a[at * 4] : 0.0f;
                    bv[e] = b[at * 4];
                }
#pragma unroll
                for (int e = 0; e < kAt; ++e) s[e & 1] = multiply(bv[e], av[e], s[e & 1]);
            }
            s[0] += s[1];
            if (kParts > 1) {
                *(f32x4 *)(P + wave * 256 + row * 16 + quad * 4) = s[0];
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e) mirrored(A, wi * 16 + row, wj * 16 + quad * 4 + e, s[0][e]);
            }
        }
        __syncthreads();
        if (kParts > 1) {
            for (int i = threadIdx.x; i < kTiles * 256; i += kThreads) {
                int bi, bj;
                tile_at(i >> 8, bi, bj);
                float s = 0.0f;
#pragma unroll
                for (int q = 0; q < kParts; ++q) s += P[q * kTiles * 256 + i];
                mirrored(A, bi * 16 + ((i >> 4) & 15), bj * 16 + (i & 15), s);
            }
            __syncthreads();
        }
        for (int tile = wave; tile < kTiles; tile += WAVES) {   // B = b A + c A^2
            int ti, tj;
            tile_at(tile, ti, tj);
            const float *a = A + (ti * 16 + row) * z.lda + quad, *b = A + (tj * 16 + row) * z.lda + quad;
            float av[NT * 4], bv[NT * 4];
#pragma unroll
            for (int f = 0; f < NT * 4; ++f) av[f] = a[f * 4], bv[f] = b[f * 4];
            const f32x4 own = *(const f32x4 *)(A + (ti * 16 + row) * z.lda + tj * 16 + quad * 4);
            f32x4 s[2] = {};
#pragma unroll
            for (int f = 0; f < NT * 4; ++f) s[f & 1] = multiply(bv[f], av[f], s[f & 1]);
#pragma unroll
            for (int e = 0; e < 4; ++e)
                mirrored(B, ti * 16 + row, tj * 16 + quad * 4 + e, __builtin_fmaf(k.b, own[e], k.c * (s[0][e] + s[1][e])));
        }
        __syncthreads();
        for (int cb = wave; cb < z.m / 16; cb += WAVES) {   // X = a X + B X, sixteen columns a wave: no other reads them
            float x[NT * 4];
            f32x4 own[NT], s[NT] = {};
#pragma unroll
            for (int f = 0; f < NT * 4; ++f) x[f] = X[(f * 4 + quad) * z.ldx + cb * 16 + row];
#pragma unroll
            for (int it = 0; it < NT; ++it) own[it] = *(const f32x4 *)(X + (it * 16 + row) * z.ldx + cb * 16 + quad * 4);
#pragma unroll
            for (int f0 = 0; f0 < NT * 4; f0 += 4) {
                float b[4][NT];
#pragma unroll
                for (int f = 0; f < 4; ++f)
#pragma unroll
                    for (int it = 0; it < NT; ++it) b[f][it] = B[(it * 16 + row) * z.lda + (f0 + f) * 4 + quad];
#pragma unroll
                for (int f = 0; f < 4; ++f)
#pragma unroll
                    for (int it = 0; it < NT; ++it) s[it] = multiply(x[f0 + f], b[f][it], s[it]);
            }
#pragma unroll
            for (int it = 0; it < NT; ++it) {
#pragma unroll
                for (int e = 0; e < 4; ++e) s[it][e] = __builtin_fmaf(k.a, own[it][e], s[it][e]);
                *(f32x4 *)(X + (it * 16 + row) * z.ldx + cb * 16 + quad * 4) = s[it];
            }
        }
        __syncthreads();
    }
}

template <typename T, typename G, int WAVES>
__global__ __launch_bounds__(64 * WAVES) void k_small(Batch batch, Scalars k, int steps)
{
    extern __shared__ float small_lds[];
    constexpr int kThreads = 64 * WAVES;
    __shared__ double part[WAVES];
    const Matrix &t = batch.t[blockIdx.x];
    const SmallSize z(t.rows, t.cols);
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const bool tall = t.rows > t.cols;
    float *X = small_lds, *A = X + z.n * z.ldx, *B = A + z.n * z.lda, *P = B + z.n * z.lda;
    const G *g = (const G *)t.g;
    T *p = (T *)t.p;
    const int all = t.rows * t.cols;
    // a thread's elements are kThreads apart: row and column go on by as much, without a division
    const int dr = kThreads / t.cols, dc = kThreads - dr * t.cols;
    const int r0 = (int)threadIdx.x / t.cols, c0 = (int)threadIdx.x - r0 * t.cols;
    auto each = [&](auto f) {
        int r = r0, c = c0;
        for (int i = threadIdx.x; i < all; i += kThreads) {
            f(i, X + (tall ? c * z.ldx + r : r * z.ldx + c));
            r += dr, c += dc;
            if (c >= t.cols) c -= t.cols, ++r;
        }
    };
    for (int i = threadIdx.x; i < z.n * z.ldx; i += kThreads) X[i] = 0.0f;
    __syncthreads();
    double sum = 0.0;
    constexpr int kAt = 4;   // elements loaded before the first is used
    {
        int r = r0, c = c0;
        for (int i0 = threadIdx.x; i0 < all; i0 += kThreads * kAt) {
            float gv[kAt], mv[kAt];
#pragma unroll
            for (int a = 0; a < kAt; ++a) {
                const int i = i0 + a * kThreads;
                gv[a] = i < all ? widen(g[i]) : 0.0f;
                mv[a] = i < all ? t.m[i] : 0.0f;
            }
#pragma unroll
            for (int a = 0; a < kAt; ++a) {
                const int i = i0 + a * kThreads;
                if (i < all) {
                    const float m = mv[a] * k.mu + gv[a] * k.nu, u = update_of(k, m, gv[a]);
                    t.m[i] = m;
                    X[tall ? c * z.ldx + r : r * z.ldx + c] = u;
                    sum += (double)u * u;
                }
                r += dr, c += dc;
                if (c >= t.cols) c -= t.cols, ++r;
            }
        }
    }
    sum = wave_sum(sum);
    if (lane == 0) part[wave] = sum;
    __syncthreads();
    sum = 0.0;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) sum += part[w];
    const double norm = sqrt(sum);
    const double inv = 1.0 / (norm <= (double)k.eps ? (double)k.eps : norm);   // beyond 32 bits for the least eps
    for (int i = threadIdx.x; i < z.n * z.ldx; i += kThreads) X[i] = (float)(X[i] * inv);
    __syncthreads();
    switch (z.n / 16) {
    case 1: small_steps<1, WAVES>(z, k, steps, X, A, B, P); break;
    case 2: small_steps<2, WAVES>(z, k, steps, X, A, B, P); break;
    default:
        if constexpr (WAVES == kSmallWaves) {   // those of three tiles have more than kTinyValues
            if (z.n == 48) small_steps<3, WAVES>(z, k, steps, X, A, B, P);
            else small_steps<4, WAVES>(z, k, steps, X, A, B, P);
        }
    }
    each([&](int i, const float *x) {
        const float y = widen(p[i]);
        narrow(__builtin_fmaf(y, -k.decay, y) - t.size * *x, p[i]);
    });
}

// ---- thin matrices ----
//
// All steps together multiply X by a polynomial P of A = X X^T: with Q = a + b A + c A^2, a step makes Q P of P and Q A Q of A, all
// of the smaller side alone.  So X is read twice, for A and for P X, in three launches, where each step of k_product takes three
// and reads it twice.  The price: an error of A grows by up to a^2 = 12 a step, and P's values reach a^5 = 485 and cancel in P X,
// so everything is held in 64 bits (those of 32 would leave errors of 1e-3), and only few steps go this way (thin_steps).
// 4 x 3664 fp32 23 us, by k_product 101; 48 x 2000 49 and 103; 64 x 5000 73 and 123: 13 for the chunks, 48 for the chain (five
// times four products of 64^3, by one workgroup at 7 us), 11 for P X.

constexpr int kThinSide = 64, kThinWaves = 4, kChainWaves = 16;
constexpr int kThinChunks = 64;     // of a matrix: what its workgroup of k_chain adds up
constexpr float kThinGrowth = 1 << 22;

// Positions of a workgroup along the longer side at once: for A, and for P X.
__host__ __device__ constexpr int thin_gram_width(int nt) { return nt == 1 ? 512 : nt == 2 ? 256 : 128; }
__host__ __device__ constexpr int thin_apply_width(int nt) { return nt == 1 ? 256 : nt == 2 ? 128 : 64; }
// Parts of a chunk: waves beside each other along k, where there is one tile.
__host__ __device__ constexpr int thin_parts(int nt) { return nt == 1 ? kThinWaves : 1; }
__host__ __device__ constexpr int thin_tiles(int nt) { return nt * (nt + 1) / 2; }
// Floats of u that a workgroup holds, of any size.
template <class F>
constexpr int most_floats(F width)
{
    int most = 0;
    for (int nt = 1; nt <= kThinSide / 16; ++nt) most = std::max(most, 16 * nt * (width(nt) + 4));
    return most;
}

struct ThinSize {
    int n, nt, m, chunks;   // smaller side, its tiles, larger side
    __host__ __device__ ThinSize(int rows, int cols)
        : n(rows < cols ? rows : cols), nt((n + 15) / 16), m(rows < cols ? cols : rows),
          chunks((m + thin_gram_width(nt) - 1) / thin_gram_width(nt))
    {
        if (chunks > kThinChunks) chunks = kThinChunks;
    }
    __host__ __device__ int parts() const { return chunks * thin_parts(nt); }
};

using f64x4 = __attribute__((ext_vector_type(4))) double;

// Four k of a 16 x 16 block: lane % 16 is the row of either operand, lane / 16 its k; of the result lane % 16 is b's row, and
// 4 e + lane / 16 a's.
__device__ __forceinline__ f64x4 multiply(double a, double b, f64x4 c)
{
    return __builtin_amdgcn_mfma_f64_16x16x4f64(a, b, c, 0, 0, 0);
}

// Positions p0 .. p0 + width of the longer side: u = f(place in the matrix) to U[smaller side][width + 4].
template <int WIDTH, class F>
__device__ __forceinline__ void thin_load(const Matrix &t, const ThinSize &z, int p0, float *U, F f)
{
    constexpr int kThreads = 64 * kThinWaves, kAt = F::kAt, kPitch = WIDTH + 4;
    const int here = z.m - p0 < WIDTH ? z.m - p0 : WIDTH;
    if (t.rows > t.cols) {   // neighbours lie along the smaller side
        const long long base = (long long)p0 * z.n;
        const int all = here * z.n, dp = kThreads / z.n, dc = kThreads - dp * z.n;
        int p = (int)threadIdx.x / z.n, c = (int)threadIdx.x - p * z.n;
        for (int i0 = threadIdx.x; i0 < all; i0 += kThreads * kAt) {
            float u[kAt];
            f.template many<kAt>(u, base + i0, kThreads, (all - i0 + kThreads - 1) / kThreads);
#pragma unroll
            for (int a = 0; a < kAt; ++a) {
                if (i0 + a * kThreads < all) U[c * kPitch + p] = u[a];
                p += dp, c += dc;
                if (c >= z.n) c -= z.n, ++p;
            }
        }
    } else {
        constexpr int kDown = kThreads > WIDTH ? kThreads / WIDTH : 1, kAcross = kThreads < WIDTH ? WIDTH / kThreads : 1;
#pragma unroll
        for (int q = 0; q < kAcross; ++q) {
            const int c = q * kThreads + (int)threadIdx.x % WIDTH, r0 = kDown > 1 ? (int)threadIdx.x / WIDTH : 0;
            if (c >= here) continue;
            for (int r = r0; r < z.n; r += kDown * kAt) {
                float u[kAt];
                f.template many<kAt>(u, (long long)r * t.cols + p0 + c, (long long)kDown * t.cols, (z.n - r + kDown - 1) / kDown);
#pragma unroll
                for (int a = 0; a < kAt; ++a)
                    if (r + a * kDown < z.n) U[(r + a * kDown) * kPitch + c] = u[a];
            }
        }
    }
}

// u at `count` places, `step` apart; updating m, or of an m that has been updated.
template <typename G, bool UPDATE>
struct ThinUpdate {
    static constexpr int kAt = UPDATE ? 8 : 16;   // places before the first is used
    const G *g;
    float *m;
    const Scalars &k;
    template <int N>
    __device__ __forceinline__ void many(float (&u)[N], long long at, long long step, int count) const
    {
        float gv[N], mv[N];
#pragma unroll
        for (int a = 0; a < N; ++a) {
            gv[a] = a < count && (UPDATE || k.nesterov) ? widen(g[at + a * step]) : 0.0f;
            mv[a] = a < count ? m[at + a * step] : 0.0f;
        }
#pragma unroll
        for (int a = 0; a < N; ++a) {
            if (UPDATE) {
                mv[a] = mv[a] * k.mu + gv[a] * k.nu;
                if (a < count) m[at + a * step] = mv[a];
            }
            u[a] = update_of(k, mv[a], gv[a]);
        }
    }
};

__device__ __forceinline__ void clear(float *U, int floats)
{
    for (int i = threadIdx.x; i < floats; i += blockDim.x) U[i] = 0.0f;
    __syncthreads();
}

// Tile t of a lower triangle, in rows, of few.
__device__ __forceinline__ void small_triangle(int t, int &i, int &j)
{
    i = 0, j = t;
    while (j > i) j -= ++i;
}

// m, and the products of u with itself over a chunk: lower tiles, as the lanes hold them.
template <typename G, int NT>
__device__ __forceinline__ void thin_gram(const Matrix &t, const Scalars &k, int chunk, float *U)
{
    constexpr int kWidth = thin_gram_width(NT), kPitch = kWidth + 4, kParts = thin_parts(NT), kTiles = thin_tiles(NT);
    constexpr int kOwn = (kTiles * kParts + kThinWaves - 1) / kThinWaves;   // tiles of a wave
    const ThinSize z(t.rows, t.cols);
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, row = lane & 15, quad = lane >> 4;
    const ThinUpdate<G, true> update{(const G *)t.g, t.m, k};
    f64x4 s[kOwn] = {};
    clear(U, 16 * NT * kPitch);
    for (int p0 = chunk * kWidth; p0 < z.m; p0 += z.chunks * kWidth) {
        if (z.m - p0 < kWidth) clear(U, 16 * NT * kPitch);   // the last one: what was there before goes
        thin_load<kWidth>(t, z, p0, U, update);
        __syncthreads();
#pragma unroll
        for (int o = 0; o < kOwn; ++o) {
            const int tile = kParts > 1 ? 0 : o * kThinWaves + wave, part = kParts > 1 ? wave : 0;
            if (tile >= kTiles) continue;
            int ti, tj;
            small_triangle(tile, ti, tj);
            constexpr int kSteps = kWidth / 4 / kParts, kAt = 8;
            const float *from = U + row * kPitch + part * kSteps * 4 + quad, *a = from + ti * 16 * kPitch, *b = from + tj * 16 * kPitch;
            for (int f = 0; f < kSteps; f += kAt) {
                float av[kAt], bv[kAt];
#pragma unroll
                for (int e = 0; e < kAt; ++e) av[e] = a[(f + e) * 4], bv[e] = b[(f + e) * 4];
#pragma unroll
                for (int e = 0; e < kAt; ++e) s[o] = multiply((double)av[e], (double)bv[e], s[o]);
            }
        }
        __syncthreads();
    }
#pragma unroll
    for (int o = 0; o < kOwn; ++o) {
        const int tile = kParts > 1 ? 0 : o * kThinWaves + wave, part = kParts > 1 ? wave : 0;
        if (tile < kTiles) *(f64x4 *)(t.sums + ((long long)(chunk * kParts + part) * kTiles + tile) * 256 + lane * 4) = s[o];
    }
}

template <typename G>
__global__ __launch_bounds__(64 * kThinWaves) void k_thin_gram(Batch batch, Scalars k)
{
    __shared__ float U[most_floats(thin_gram_width)];
    const int ti = matrix_of(batch.first, batch.count, blockIdx.x), chunk = blockIdx.x - batch.first[ti];
    const Matrix &t = batch.t[ti];
    switch (ThinSize(t.rows, t.cols).nt) {
    case 1: thin_gram<G, 1>(t, k, chunk, U); break;
    case 2: thin_gram<G, 2>(t, k, chunk, U); break;
    case 3: thin_gram<G, 3>(t, k, chunk, U); break;
    default: thin_gram<G, 4>(t, k, chunk, U); break;
    }
}

__host__ __device__ constexpr int chain_pitch(int nt) { return 16 * nt + 2; }
// Sums of the chunks' values by so many threads each.
__host__ __device__ constexpr int chain_down(int nt)
{
    const int down = 64 * kChainWaves / (thin_tiles(nt) * 128);
    return down > 1 ? down : 1;
}
constexpr size_t chain_bytes(int nt)
{
    return (4 * (size_t)(16 * nt) * chain_pitch(nt) + (chain_down(nt) > 1 ? chain_down(nt) * thin_tiles(nt) * 256 : 0)) * 8;
}

// A matrix's P / max(|u|, eps), from the chunks' products: one workgroup, in LDS.
template <int NT>
__device__ __forceinline__ void chain(const Matrix &t, const Scalars &k, int steps, double *lds)
{
    constexpr int kThreads = 64 * kChainWaves, kTiles = thin_tiles(NT), kValues = kTiles * 256;
    constexpr int kPitch = chain_pitch(NT), kN = 16 * NT;
    const ThinSize z(t.rows, t.cols);
    double *A = lds, *Q = A + kN * kPitch, *R = Q + kN * kPitch, *P = R + kN * kPitch, *held = P + kN * kPitch;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, row = lane & 15, quad = lane >> 4;
    // chunks' products, threads across the values and down the chunks
    constexpr int kPairs = kValues / 2, kDown = chain_down(NT), kAt = 16;
    using f64x2 = __attribute__((ext_vector_type(2))) double;
    const int down = kDown > 1 ? (int)threadIdx.x / kPairs : 0, parts = z.parts();
    auto put_at = [&](double *to, int tile, int l, int e, double v) {   // value e of lane l, to both places
        int ti, tj;
        small_triangle(tile, ti, tj);
        const int i = ti * 16 + 4 * e + (l >> 4), j = tj * 16 + (l & 15);
        to[i * kPitch + j] = v;
        if (ti != tj) to[j * kPitch + i] = v;
    };
    for (int i = kDown > 1 ? (int)threadIdx.x % kPairs : (int)threadIdx.x; i < kPairs && down < kDown; i += kThreads) {
        f64x2 s = {};
        for (int c0 = down; c0 < parts; c0 += kDown * kAt) {
            f64x2 v[kAt];
#pragma unroll
            for (int a = 0; a < kAt; ++a)
                v[a] = c0 + a * kDown < parts ? *(const f64x2 *)(t.sums + (long long)(c0 + a * kDown) * kValues + 2 * i) : f64x2{};
#pragma unroll
            for (int a = 0; a < kAt; ++a) s += v[a];
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int at = 2 * i + e;
            if (kDown > 1) held[down * kValues + at] = s[e];
            else put_at(A, at >> 8, (at & 255) >> 2, at & 3, s[e]);
        }
    }
    __syncthreads();
    if (kDown > 1) {
        for (int i = threadIdx.x; i < kValues; i += kThreads) {
            double s = 0.0;
#pragma unroll
            for (int d = 0; d < kDown; ++d) s += held[d * kValues + i];
            put_at(A, i >> 8, (i & 255) >> 2, i & 3, s);
        }
        __syncthreads();
    }
    double square = 0.0;   // |u|^2, the trace; the same in every wave
    if (lane < kN) square = A[lane * kPitch + lane];
    square = wave_sum(square);
    const double norm = sqrt(square), inv = 1.0 / (norm <= (double)k.eps ? (double)k.eps : norm);
    __syncthreads();
    for (int i = threadIdx.x; i < kN * kN; i += kThreads) A[i / kN * kPitch + i % kN] *= inv * inv;
    __syncthreads();
    auto tile_product = [&](const double *a, const double *b, int ti, int tj) {
        a += (ti * 16 + row) * kPitch + quad, b += (tj * 16 + row) * kPitch + quad;
        double av[NT * 4], bv[NT * 4];
#pragma unroll
        for (int f = 0; f < NT * 4; ++f) av[f] = a[f * 4], bv[f] = b[f * 4];
        f64x4 s = {};
#pragma unroll
        for (int f = 0; f < NT * 4; ++f) s = multiply(av[f], bv[f], s);
        return s;
    };
    auto put_tile = [&](double *to, int tile, f64x4 v) {
#pragma unroll
        for (int e = 0; e < 4; ++e) put_at(to, tile, lane, e, v[e]);
    };
    for (int step = 0; step < steps; ++step) {
        const bool last = step + 1 == steps;
        for (int tile = wave; tile < kTiles; tile += kChainWaves) {   // Q = a + b A + c A^2
            int ti, tj;
            small_triangle(tile, ti, tj);
            f64x4 s = tile_product(A, A, ti, tj);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int i = ti * 16 + 4 * e + quad, j = tj * 16 + row;
                s[e] = (double)k.c * s[e] + (double)k.b * A[i * kPitch + j] + (i == j ? (double)k.a : 0.0);
            }
            put_tile(Q, tile, s);
            if (step == 0) put_tile(P, tile, s);
        }
        __syncthreads();
        // R = Q A, and Q P; P is read by all before any of it is replaced
        constexpr int kOwn = (2 * kTiles + kChainWaves - 1) / kChainWaves;
        f64x4 s[kOwn];
#pragma unroll
        for (int o = 0; o < kOwn; ++o) {
            const int at = o * kChainWaves + wave, tile = at % kTiles;
            if (at >= 2 * kTiles || (at < kTiles ? last : step == 0)) continue;
            int ti, tj;
            small_triangle(tile, ti, tj);
            s[o] = tile_product(Q, at < kTiles ? A : P, ti, tj);
        }
        __syncthreads();
#pragma unroll
        for (int o = 0; o < kOwn; ++o) {
            const int at = o * kChainWaves + wave, tile = at % kTiles;
            if (at >= 2 * kTiles || (at < kTiles ? last : step == 0)) continue;
            put_tile(at < kTiles ? R : P, tile, s[o]);
        }
        __syncthreads();
        if (last) break;
        for (int tile = wave; tile < kTiles; tile += kChainWaves) {   // A = Q (Q A)
            int ti, tj;
            small_triangle(tile, ti, tj);
            put_tile(A, tile, tile_product(Q, R, ti, tj));
        }
        __syncthreads();
    }
    double *to = (double *)t.x[0];
    for (int i = threadIdx.x; i < kN * kN; i += kThreads) to[i] = P[i / kN * kPitch + i % kN] * inv;
}

__global__ __launch_bounds__(64 * kChainWaves) void k_chain(Batch batch, Scalars k, int steps)
{
    extern __shared__ double chain_lds[];
    const Matrix &t = batch.t[blockIdx.x];
    switch (ThinSize(t.rows, t.cols).nt) {
    case 1: chain<1>(t, k, steps, chain_lds); break;
    case 2: chain<2>(t, k, steps, chain_lds); break;
    case 3: chain<3>(t, k, steps, chain_lds); break;
    default: chain<4>(t, k, steps, chain_lds); break;
    }
}

// P X, and the parameter.
template <typename T, typename G, int NT>
__device__ __forceinline__ void thin_apply(const Matrix &t, const Scalars &k, int wg, float *U, double *P)
{
    constexpr int kWidth = thin_apply_width(NT), kPitch = kWidth + 4, kN = 16 * NT, kPitchP = chain_pitch(NT);
    const ThinSize z(t.rows, t.cols);
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, row = lane & 15, quad = lane >> 4, p0 = wg * kWidth;
    const bool tall = t.rows > t.cols;
    const double *from = (const double *)t.x[0];
    double q[NT * NT];   // on its way while u is loaded
#pragma unroll
    for (int i = 0; i < NT * NT; ++i) q[i] = from[i * 64 * kThinWaves + threadIdx.x];
    clear(U, kN * kPitch);
    thin_load<kWidth>(t, z, p0, U, ThinUpdate<G, false>{(const G *)t.g, t.m, k});
#pragma unroll
    for (int i = 0; i < NT * NT; ++i) {
        const int at = i * 64 * kThinWaves + (int)threadIdx.x;
        P[at / kN * kPitchP + at % kN] = q[i];
    }
    __syncthreads();
    T *p = (T *)t.p;
    for (int c = wave; c < kWidth / 16; c += kThinWaves) {
        if (p0 + c * 16 >= z.m) break;
        double u[NT * 4];
        float y[NT][4];
        auto at = [&](int it, int e, long long &place) {
            const int own = it * 16 + (tall ? row : 4 * e + quad), along = p0 + c * 16 + (tall ? 4 * e + quad : row);
            place = tall ? (long long)along * t.cols + own : (long long)own * t.cols + along;
            return own < z.n && along < z.m;
        };
#pragma unroll
        for (int it = 0; it < NT; ++it)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                long long place;
                y[it][e] = at(it, e, place) ? widen(p[place]) : 0.0f;
            }
#pragma unroll
        for (int f = 0; f < NT * 4; ++f) u[f] = (double)U[(f * 4 + quad) * kPitch + c * 16 + row];
#pragma unroll
        for (int it = 0; it < NT; ++it) {
            f64x4 s = {};
#pragma unroll
            for (int f = 0; f < NT * 4; ++f) {
                const double v = P[(it * 16 + row) * kPitchP + f * 4 + quad];
                s = tall ? multiply(u[f], v, s) : multiply(v, u[f], s);   // neighbours of the matrix in neighbouring lanes
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                long long place;
                if (at(it, e, place)) narrow(__builtin_fmaf(y[it][e], -k.decay, y[it][e]) - t.size * (float)s[e], p[place]);
            }
        }
    }
}

template <typename T, typename G>
__global__ __launch_bounds__(64 * kThinWaves) void k_thin_apply(Batch batch, Scalars k)
{
    __shared__ float U[most_floats(thin_apply_width)];
    __shared__ double P[kThinSide * chain_pitch(kThinSide / 16)];
    const int ti = matrix_of(batch.first, batch.count, blockIdx.x), wg = blockIdx.x - batch.first[ti];
    const Matrix &t = batch.t[ti];
    switch (ThinSize(t.rows, t.cols).nt) {
    case 1: thin_apply<T, G, 1>(t, k, wg, U, P); break;
    case 2: thin_apply<T, G, 2>(t, k, wg, U, P); break;
    case 3: thin_apply<T, G, 3>(t, k, wg, U, P); break;
    default: thin_apply<T, G, 4>(t, k, wg, U, P); break;
    }
}

// Whether errors of A stay small over the steps: how much one grows, for any singular value.
bool thin_steps(const hqml_muon_config &c)
{
    for (int i = 0; i <= 64; ++i) {
        double x = i ? exp2(-(i - 1) * 0.5) : 0.0, grown = 1.0;   // an eigenvalue of A
        for (int step = 0; step < c.steps; ++step) {
            const double q = c.a + c.b * x + c.c * x * x, slope = q * (q + 2 * x * (c.b + 2 * c.c * x));
            grown *= std::max({1.0, q * q, fabs(slope)});
            x *= q * q;
            if (!(grown <= kThinGrowth)) return false;
        }
    }
    return true;
}

// ---- a call ----

struct Bytes {
    size_t x, gram, sums;   // one X, one A, the chunks' sums
    size_t all() const { return 2 * x + 2 * gram + sums; }
};

size_t up256(size_t b) { return (b + 255) & ~(size_t)255; }

Bytes bytes_of(const hqml_muon_tensor &t, int planes)
{
    const size_t n = (size_t)std::min(t.rows, t.cols);
    Bytes b;
    b.x = up256((size_t)planes * t.rows * pad8(t.cols) * 2);
    b.gram = up256((size_t)planes * n * pad8((int)n) * 2);
    b.sums = up256((((size_t)t.rows * t.cols + kChunk - 1) / kChunk) * 8);
    return b;
}

struct ThinBytes {
    size_t p, sums;   // P, the chunks' products
    size_t all() const { return p + sums; }
};

ThinBytes thin_bytes(const hqml_muon_tensor &t)
{
    const ThinSize z(t.rows, t.cols);
    return {up256((size_t)256 * z.nt * z.nt * 8), up256((size_t)z.parts() * thin_tiles(z.nt) * 256 * 8)};
}

// Partial sums of a launch: at most this much, in tiles that at most so many tickets count.
constexpr size_t kPartBytes = 64ull << 20;
constexpr int kTickets = 4096;
constexpr size_t kJoinBytes = kPartBytes + kTickets * sizeof(unsigned);

int planes_of(const hqml_muon_config &cfg) { return cfg.param_dtype == HQML_DTYPE_FP32 || cfg.precise ? 2 : 1; }

enum Kind { SMALL, THIN, LARGE };

// Which way a call's matrices go.
class KindOf {
public:
    explicit KindOf(const hqml_muon_config &cfg) : cfg_(cfg) {}
    Kind operator()(const hqml_muon_tensor &t)
    {
        if (std::min(t.rows, t.cols) > kThinSide) return LARGE;
        if (is_small(t.rows, t.cols, true)) return SMALL;
        if (few_ < 0) few_ = thin_steps(cfg_);
        return few_ ? THIN : is_small(t.rows, t.cols, false) ? SMALL : LARGE;
    }

private:
    const hqml_muon_config &cfg_;
    int few_ = -1;
};

// Calls f(first, last, bytes) for each round of matrices that go together.
template <typename F>
void rounds(const hqml_muon_config &cfg, int n, const hqml_muon_tensor *t, F f)
{
    KindOf kind_of(cfg);
    for (int i = 0; i < n;) {
        size_t bytes = 0;
        int last = i, count[3] = {};
        for (; last < n && *std::max_element(count, count + 3) < kMatrices; ++last) {
            if (!t[last].rows || !t[last].cols) continue;
            const Kind kind = kind_of(t[last]);
            const size_t here = kind == LARGE  ? bytes_of(t[last], planes_of(cfg)).all()
                                : kind == THIN ? thin_bytes(t[last]).all()
                                               : 0;
            if (bytes && bytes + here > kBatchBytes) break;
            bytes += here;
            ++count[kind];
        }
        if (count[SMALL] || count[THIN] || count[LARGE]) f(i, last, count[LARGE] ? bytes + kJoinBytes : bytes);
        i = last;
    }
}

// All tiles of a product.
int tiles_of(const Product &P, int side)
{
    const int i = ceil_div(P.I, side), j = ceil_div(P.J, side);
    return P.mirrored ? i * (i + 1) / 2 : i * j;
}

int steps_of(const Product &P) { return ceil_div(P.K, 32); }

// A kernel's times in us, as the dense layer's TileCost: a step of a workgroup alone on its compute unit, and of n of them
// n share; launch and epilogue; joining parts.  Fitted to sweeps of sides and parts over the three products of matrices of 300 x
// 200 to 4096 x 4096.
constexpr TileCost kOneCost[] = {{TILE_64, 4, 3.0f, 0.2f, 0.165f, 0.65f, 0.42f},
                                 {TILE_128, 2, 5.0f, 0.32f, 0.36f, 2.0f, 1.06f},
                                 {TILE_256, 1, 10.0f, 0.66f, 0.88f, 4.6f, 4.0f}};
constexpr TileCost kPairCost[] = {{TILE_64, 2, 4.5f, 0.33f, 0.43f, 0.65f, 0.42f}, {TILE_128, 1, 10.0f, 0.52f, 0.7f, 2.0f, 1.06f}};

struct Pieces {
    int side, steps;   // tile side, steps of a part
    float us;
};

// How tiles[i] tiles of side `side` of the products are cut best, with kernels of up to that side.  A tile makes four of half
// its side.
Pieces cut_of(const Products &G, const int *tiles, int side, int planes, bool smaller)
{
    Pieces best{0, 1 << 30, 0.0f};
    int most = 0;
    for (int i = 0; i < G.count; ++i)
        if (tiles[i]) most = std::max(most, steps_of(G.t[i]));
    const TileCost *cost = planes == 2 ? kPairCost : kOneCost;
    for (int n_cost = planes == 2 ? 2 : 3; n_cost > 0; --n_cost, ++cost) {
        const TileCost &c = *cost;
        const int own = kSides[c.shape][0];
        if (own != (smaller ? side / 2 : side)) continue;
        int last = 0;
        for (int parts : kParts) {
            const int u = ceil_div(most, parts);
            if (u == last || (parts > 1 && u < 4)) continue;
            last = u;
            long long groups = 0, split = 0, joins = 0;
            float work = 0.0f;
            for (int i = 0; i < G.count; ++i) {
                const int steps = steps_of(G.t[i]), n = ceil_div(steps, u);
                const long long t = smaller ? tiles[i] * 4 : tiles[i];
                groups += t * n;
                work += (float)t * (float)steps;
                if (n > 1) split += t * n, joins += t;
            }
            if (split * own * own * 4 > (long long)kPartBytes || joins > kTickets) continue;
            // a compute unit's workgroups share it, or, of the largest tiles, come one after the other; shorter ones than the
            // longest fill in
            const float each = (float)groups / kUnits, even = std::min(each, work / kUnits / (float)u + 1.0f);
            const float whole = floorf(even), last_round = even - whole;
            const float busy = c.most > 1 ? std::max(c.step, even * c.share)
                                          : whole * c.share + (last_round > 0.0f ? std::max(c.step, last_round * c.share) : 0.0f);
            float us = c.fixed + (float)u * busy + (float)own / 160 * each;
            if (split) us += c.join + (float)parts * c.join_part + (float)split * (own * own * 8) / 9e6f;
            if (!best.side || us < best.us) best = {own, u, us};
        }
    }
    return best;
}

// How a stage runs: `first` tiles of a side, the rest, if any, as quarters of them in a second launch.
struct Plan {
    Pieces main, rest;
    int first;
};

// A compute unit holds one workgroup of the largest tiles, so those that go beyond whole rounds of all compute units would take
// a round of their own: quarters of them, split along k, take less.  Two 4096 x 4096, X X^T of one plane: 272 tiles of 256 in two
// rounds 206 us, 256 and quarters of 16 150.
Plan plan_of(const Products &G, int planes)
{
    Plan best{{0, 0, 0.0f}, {0, 0, 0.0f}, 0};
    int tiles[kMatrices], rest[kMatrices];
    for (int side : {64, 128, 256}) {
        long long all = 0;
        for (int i = 0; i < G.count; ++i) all += tiles[i] = tiles_of(G.t[i], side);
        if (all > 1 << 28) continue;   // tiles in 32 bits, quarters among them
        const Pieces whole = cut_of(G, tiles, side, planes, false);
        if (whole.side && (!best.main.side || whole.us < best.main.us + best.rest.us)) best = {whole, {0, 0, 0.0f}, (int)all};
        const int first = (int)(all / kUnits) * kUnits;
        if (side < (planes == 2 ? 128 : 256) || !first || first == all) continue;
        int left = first;
        for (int i = 0; i < G.count; ++i) {
            const int here = std::min(left, tiles[i]);
            left -= here;
            rest[i] = tiles[i] - here, tiles[i] = here;
        }
        const Pieces rounds = cut_of(G, tiles, side, planes, false), quarters = cut_of(G, rest, side, planes, true);
        if (rounds.side && quarters.side && rounds.us + quarters.us < best.main.us + best.rest.us) best = {rounds, quarters, first};
    }
    return best;
}

// The arguments of few products are few: three 100 x 120, 17 launches, take 95 us a step so, 100 with room for 24 in each.
constexpr int kFew = 4;

template <int STAGE, int PLANES, typename T, int MOST>
void launch(const ProductsOf<MOST> &G, const Finish &F, int side, unsigned groups, hipStream_t s)
{
    if (side == 64) {
        k_product<STAGE, PLANES, T, 64, 4, MOST><<<groups, 256, 0, s>>>(G, F);
    } else if constexpr (PLANES == 2) {
        k_product<STAGE, 2, T, 128, 8, MOST><<<groups, 512, 0, s>>>(G, F);
    } else {
        if (side == 128) k_product<STAGE, 1, T, 128, 4, MOST><<<groups, 256, 0, s>>>(G, F);
        else k_product<STAGE, 1, T, 256, 8, MOST><<<groups, 512, 0, s>>>(G, F);
    }
}

template <int STAGE, int PLANES, typename T>
hipError_t run_cut(Products &G, const Finish &F, const Pieces &cut, const int *tiles, const int *skip, float *part, unsigned *ticket,
                   hipStream_t s)
{
    unsigned at = 0;
    float *part_end = part + kPartBytes / 4;
    unsigned *ticket_end = ticket + kTickets;
    for (int i = 0; i < G.count; ++i) {
        Product &P = G.t[i];
        P.tiles_i = ceil_div(P.I, cut.side), P.tiles_j = ceil_div(P.J, cut.side);
        P.skip = skip ? skip[i] : -1;
        P.tiles = skip ? tiles[i] * 4 : tiles[i];
        P.steps = std::min(cut.steps, steps_of(P));
        P.parts = ceil_div(steps_of(P), P.steps);
        if (P.parts > 1 && P.tiles) {
            P.part = part, P.ticket = ticket;
            if ((long long)P.tiles * P.parts * cut.side * cut.side > part_end - part || P.tiles > ticket_end - ticket)
                return hipErrorInvalidValue;
            part += (size_t)P.tiles * P.parts * cut.side * cut.side;
            ticket += P.tiles;
        }
        G.first[i] = at;
        at += ((unsigned)P.tiles * (unsigned)P.parts + 7) & ~7u;
    }
    if (G.count > kFew) {
        launch<STAGE, PLANES, T>(G, F, cut.side, at, s);
    } else {
        ProductsOf<kFew> few;
        few.count = G.count;
        std::copy_n(G.first, kFew, few.first);
        std::copy_n(G.t, kFew, few.t);
        launch<STAGE, PLANES, T>(few, F, cut.side, at, s);
    }
    return hipGetLastError();
}

template <int STAGE, int PLANES, typename T>
hipError_t run_stage(Products &G, const Finish &F, const Plan &plan, float *part, unsigned *ticket, hipStream_t s)
{
    if (!plan.main.side) return hipErrorInvalidValue;
    int tiles[kMatrices], skip[kMatrices], left = plan.first;
    for (int i = 0; i < G.count; ++i) {
        const int all = tiles_of(G.t[i], plan.main.side);
        tiles[i] = std::min(left, all);
        left -= tiles[i];
        skip[i] = tiles[i];
    }
    hipError_t e = run_cut<STAGE, PLANES, T>(G, F, plan.main, tiles, nullptr, part, ticket, s);
    if (e != hipSuccess || !plan.rest.side) return e;
    for (int i = 0; i < G.count; ++i) tiles[i] = tiles_of(G.t[i], plan.main.side) - skip[i];
    return run_cut<STAGE, PLANES, T>(G, F, plan.rest, tiles, skip, part, ticket, s);
}

template <typename T, typename G, int PLANES>
hipError_t run(const hqml_muon_config &cfg, int n, const hqml_muon_tensor *t, char *work, hipStream_t s)
{
    Scalars k;
    k.mu = (float)cfg.momentum, k.nu = (float)(1.0 - cfg.momentum);
    k.nesterov = cfg.nesterov;
    k.eps = (float)cfg.eps;
    k.decay = (float)(cfg.lr * cfg.weight_decay);
    k.a = (float)cfg.a, k.b = (float)cfg.b, k.c = (float)cfg.c;
    Batch b{}, thin{}, few{};   // large matrices, thin ones, small ones
    KindOf kind_of(cfg);
    unsigned groups = 0;
    auto each = [&](Batch &b, auto count_of) {   // first workgroups
        groups = 0;
        for (int i = 0; i < b.count; ++i) {
            b.first[i] = groups;
            groups += count_of(b.t[i]);
        }
    };
    for (int i = 0; i < n; ++i) {
        if (!t[i].rows || !t[i].cols) continue;
        const Kind kind = kind_of(t[i]);
        Batch &to = kind == SMALL ? few : kind == THIN ? thin : b;
        Matrix &m = to.t[to.count++];
        m.p = t[i].param, m.g = t[i].grad, m.m = t[i].momentum;
        m.rows = t[i].rows, m.cols = t[i].cols;
        m.size = (float)(cfg.lr * t[i].scale);
        if (kind == SMALL) continue;
        auto take = [&](size_t bytes) {
            char *here = work;
            work += bytes;
            return here;
        };
        if (kind == THIN) {
            const ThinBytes z = thin_bytes(t[i]);
            m.x[0] = (Half *)take(z.p);
            m.sums = (double *)take(z.sums);
            continue;
        }
        const Bytes z = bytes_of(t[i], PLANES);
        m.x[0] = (Half *)take(z.x), m.x[1] = (Half *)take(z.x);
        m.a = (Half *)take(z.gram), m.b = (Half *)take(z.gram);
        m.sums = (double *)take(z.sums);
    }
    hipError_t e = hipSuccess;
    if (few.count) {
        size_t lds = 0;
        bool tiny = true;
        for (int i = 0; i < few.count; ++i) {
            const SmallSize z(few.t[i].rows, few.t[i].cols);
            lds = std::max(lds, z.bytes());
            tiny = tiny && z.n * z.m <= kTinyValues;
        }
        if (lds > 32 * 1024) {   // with what the kernel holds besides, more than a launch may take unasked
            e = hipFuncSetAttribute((const void *)k_small<T, G, kSmallWaves>, hipFuncAttributeMaxDynamicSharedMemorySize, kSmallLds);
            if (e != hipSuccess) return e;
        }
        if (tiny) k_small<T, G, kTinyWaves><<<few.count, 64 * kTinyWaves, lds, s>>>(few, k, cfg.steps);
        else k_small<T, G, kSmallWaves><<<few.count, 64 * kSmallWaves, lds, s>>>(few, k, cfg.steps);
        if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    if (thin.count) {
        int nt = 0;
        for (int i = 0; i < thin.count; ++i) nt = std::max(nt, ThinSize(thin.t[i].rows, thin.t[i].cols).nt);
        if (chain_bytes(nt) > 64 * 1024) {
            e = hipFuncSetAttribute((const void *)k_chain, hipFuncAttributeMaxDynamicSharedMemorySize,
                                    (int)chain_bytes(kThinSide / 16));
            if (e != hipSuccess) return e;
        }
        each(thin, [](const Matrix &m) { return (unsigned)ThinSize(m.rows, m.cols).chunks; });
        k_thin_gram<G><<<groups, 64 * kThinWaves, 0, s>>>(thin, k);
        if ((e = hipGetLastError()) != hipSuccess) return e;
        k_chain<<<thin.count, 64 * kChainWaves, chain_bytes(nt), s>>>(thin, k, cfg.steps);
        if ((e = hipGetLastError()) != hipSuccess) return e;
        each(thin, [](const Matrix &m) {
            const ThinSize z(m.rows, m.cols);
            return (unsigned)ceil_div(z.m, thin_apply_width(z.nt));
        });
        k_thin_apply<T, G><<<groups, 64 * kThinWaves, 0, s>>>(thin, k);
        if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    if (!b.count) return hipSuccess;
    float *const part = (float *)work;
    unsigned *const ticket = (unsigned *)(work + kPartBytes);
    each(b, [](const Matrix &m) { return (unsigned)(((long long)m.rows * m.cols + kChunk - 1) / kChunk); });
    k_momentum<G><<<groups, 256, 0, s>>>(b, k, ticket, kTickets);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    each(b, [](const Matrix &m) { return (unsigned)std::min<long long>(((long long)m.rows * pad8(m.cols) / 8 + 255) / 256, 4096); });
    k_begin<G, PLANES><<<groups, 256, 0, s>>>(b, k);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    Products gram{}, poly{}, apply{};
    gram.count = poly.count = apply.count = b.count;
    for (int i = 0; i < b.count; ++i) {
        const Matrix &m = b.t[i];
        const bool tall = m.rows > m.cols;
        const int small = std::min(m.rows, m.cols), ldx = pad8(m.cols), lda = pad8(small);
        const long long plane_x = (long long)m.rows * ldx, plane_a = (long long)small * lda;
        Product &A = gram.t[i];
        A.c = m.a;
        A.lda = A.ldb = ldx, A.ldc = lda;
        A.plane_a = A.plane_b = plane_x, A.plane_c = plane_a;
        A.I = A.J = small, A.K = tall ? m.rows : m.cols, A.cols = tall, A.mirrored = true;
        Product &B = poly.t[i];
        B.a = B.b = B.with = m.a, B.c = m.b;
        B.lda = B.ldb = B.ldc = lda;
        B.plane_a = B.plane_b = B.plane_c = plane_a;
        B.I = B.J = B.K = small, B.mirrored = true;
        Product &X = apply.t[i];
        X.lda = tall ? ldx : lda, X.ldb = tall ? lda : ldx, X.ldc = ldx;
        X.plane_a = tall ? plane_x : plane_a, X.plane_b = tall ? plane_a : plane_x, X.plane_c = plane_x;
        X.I = m.rows, X.J = m.cols, X.K = small, X.cols = !tall;
        X.p = m.p, X.size = m.size;
    }
    const Plan plan_gram = plan_of(gram, PLANES), plan_poly = plan_of(poly, PLANES), plan_apply = plan_of(apply, PLANES);
    for (int step = 0; step < cfg.steps; ++step) {
        const bool last = step + 1 == cfg.steps;
        for (int i = 0; i < b.count; ++i) {   // X goes from one array to the other
            const Matrix &m = b.t[i];
            const bool tall = m.rows > m.cols;
            const Half *x = m.x[step & 1];
            Product &A = gram.t[i], &X = apply.t[i];
            A.a = A.b = x;
            X.a = tall ? x : m.b, X.b = tall ? m.b : x, X.with = x, X.c = m.x[1 - (step & 1)];
        }
        if ((e = run_stage<GRAM, PLANES, float>(gram, {kUnscale, 0.0f, 0.0f, 0}, plan_gram, part, ticket, s)) != hipSuccess) return e;
        if ((e = run_stage<POLY, PLANES, float>(poly, {k.c * kUnscale, k.b, 0.0f, 0}, plan_poly, part, ticket, s)) != hipSuccess) return e;
        if ((e = run_stage<APPLY, PLANES, T>(apply, {kUnscale, k.a, k.decay, last}, plan_apply, part, ticket, s)) != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace

size_t muon_workspace(const hqml_muon_config &cfg, int n, const hqml_muon_tensor *t)
{
    size_t most = 0;
    rounds(cfg, n, t, [&](int, int, size_t bytes) { most = std::max(most, bytes); });
    return most;
}

hipError_t launch_muon(const hqml_muon_config &cfg, int n, const hqml_muon_tensor *t, void *workspace, hipStream_t s)
{
    hipError_t e = hipSuccess;
    rounds(cfg, n, t, [&](int first, int last, size_t) {
        if (e != hipSuccess) return;
        auto run_all = [&](auto of_param, auto of_grad) {
            using T = decltype(of_param);
            using G = decltype(of_grad);
            char *work = (char *)workspace;
            if constexpr (sizeof(T) == 2)
                if (planes_of(cfg) == 1) return run<T, G, 1>(cfg, last - first, t + first, work, s);
            return run<T, G, 2>(cfg, last - first, t + first, work, s);
        };
        const bool gb = cfg.grad_dtype == HQML_DTYPE_BF16;
        if (cfg.param_dtype == HQML_DTYPE_BF16) e = gb ? run_all(bf16{}, bf16{}) : run_all(bf16{}, 0.0f);
        else e = gb ? run_all(0.0f, bf16{}) : run_all(0.0f, 0.0f);
    });
    return e;
}

}  // namespace hqml
