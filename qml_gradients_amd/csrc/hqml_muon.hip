// Muon: momentum, and updates orthogonalised by Newton-Schulz products (K. Jordan et al., 2024).
//
//   m = mu m + (1 - mu) g,  u = mu m + (1 - mu) g (Nesterov) or m
//   X = u / max(|u|, eps);  `steps` times:  A = X X^T,  X <- a X + (b A + c A^2) X
//   p = p (1 - lr wd) - lr f X
//
// The polynomial acts on the singular values alone, so a matrix with more rows than columns takes A = X^T X and
// X <- a X + X (b A + c A^2): A is as small as it can be, and no matrix is transposed.  Three products a step, on the matrix
// cores, of operands in fp16 (products exact, sums in fp32):
//   bf16 parameters  one fp16 value for each: 11 bits, where the parameter keeps 8
//   fp32 parameters  two, x = hi + lo, 22 bits; of their four products the three that count, one after the other along k
// X's values are at most a little over 1 and often small, so X, A and B = b A + c A^2 are held times 2^10: fp16's normal range then
// goes from 2^-24 to 64 of them.
//
// All matrices of a call go through each product in one launch, a workgroup a tile.
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
constexpr int kMatrices = 32;              // of one launch
constexpr long long kChunk = 16384;        // values of a workgroup of the momentum kernel
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
    Half *x[2], *a, *b;
    double *sums;         // of squares, one a chunk
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

// m, and the sums of u^2 of each chunk, in 64 bits: they neither overflow nor lose a small chunk beside a large one.
template <typename G>
__global__ __launch_bounds__(256) void k_momentum(Batch batch, Scalars k)
{
    __shared__ double part[4];
    const int ti = matrix_of(batch.first, batch.count, blockIdx.x);
    const Matrix &t = batch.t[ti];
    const long long chunk = blockIdx.x - batch.first[ti], n = (long long)t.rows * t.cols, base = chunk * kChunk;
    const long long end = n - base < kChunk ? n : base + kChunk;
    const G *g = (const G *)t.g;
    double sum = 0.0;
    for (long long i = base + threadIdx.x; i < end; i += 256) {
        const float gi = widen(g[i]), m = t.m[i] * k.mu + gi * k.nu;
        t.m[i] = m;
        const double u = update_of(k, m, gi);
        sum += u * u;
    }
#pragma unroll
    for (int h = 1; h < 64; h <<= 1) sum += __shfl_xor(sum, h, 64);
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

// 1 / max(|u|, eps); NaN where |u| is.
__device__ __forceinline__ float inverse_norm(const Matrix &t, float eps)
{
    __shared__ double part[4];
    const int chunks = (int)(((long long)t.rows * t.cols + kChunk - 1) / kChunk);
    double sum = 0.0;
    for (int i = threadIdx.x; i < chunks; i += 256) sum += t.sums[i];
#pragma unroll
    for (int h = 1; h < 64; h <<= 1) sum += __shfl_xor(sum, h, 64);
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = sum;
    __syncthreads();
    const double norm = sqrt(part[0] + part[1] + part[2] + part[3]);
    return (float)(1.0 / (norm <= (double)eps ? (double)eps : norm));
}

// X, normalised, in rows of a multiple of eight that end with zeros.
template <typename G, int PLANES>
__global__ __launch_bounds__(256) void k_begin(Batch batch, Scalars k)
{
    const int ti = matrix_of(batch.first, batch.count, blockIdx.x);
    const Matrix &t = batch.t[ti];
    const float inv = inverse_norm(t, k.eps) * kScale;
    const int ld = (t.cols + 7) & ~7, eights = ld / 8;
    const long long n = (long long)t.rows * eights, plane = (long long)t.rows * ld;
    const unsigned groups = (ti + 1 < batch.count ? batch.first[ti + 1] : gridDim.x) - batch.first[ti];
    const G *g = (const G *)t.g;
    for (long long i = (long long)(blockIdx.x - batch.first[ti]) * 256 + threadIdx.x; i < n; i += (long long)groups * 256) {
        const int row = (int)(i / eights), c = (int)(i - (long long)row * eights) * 8;
        const long long at = (long long)row * t.cols + c;
        Half hi[8], lo[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float u = c + e < t.cols ? update_of(k, t.m[at + e], widen(g[at + e])) : 0.0f;
            to_planes(c + e < t.cols ? u * inv : 0.0f, hi[e], lo[e]);
        }
        *(u32x4 *)(t.x[0] + (long long)row * ld + c) = __builtin_bit_cast(u32x4, hi);
        if (PLANES == 2) *(u32x4 *)(t.x[0] + plane + (long long)row * ld + c) = __builtin_bit_cast(u32x4, lo);
    }
}

// ---- the products ----

enum Stage { GRAM, POLY, APPLY };

// C = sum_k A(i, k) B(j, k), and what becomes of it.
struct Product {
    const Half *a, *b, *with;   // with: what a multiple of is added, laid out as C
    Half *c;
    void *p;                    // the last step's: the parameter
    long long plane_a, plane_b, plane_c;   // values from one plane to the next
    int lda, ldb, ldc, I, J, K;
    int cols;                   // A and B across k (GRAM), B across k (APPLY)
    int tiles_i, tiles_j;
    float size;
};

struct Products {
    int count;
    unsigned first[kMatrices];   // multiples of eight: the XCD of a tile follows from its number
    Product t[kMatrices];
};

struct Finish {
    float one, two;   // C = one sum + two with
    float decay;
    int last;
};
static_assert(sizeof(Products) + sizeof(Finish) <= 4096, "kernel arguments");

// The operands' tiles along k: with two planes, the small products first: lo hi, hi lo, hi hi.
template <int PLANES>
struct Planes {
    int per;                     // steps of a plane
    long long plane_a, plane_b;  // bytes
    template <bool kSecond, class Tile>
    __device__ __forceinline__ typename Tile::Step begin(const Tile &tile, int t, int bk) const
    {
        if (PLANES == 1) return tile.begin(t * bk);
        const int turn = t >= 2 * per ? 2 : t >= per ? 1 : 0;
        auto st = tile.begin((t - turn * per) * bk);
        if (turn == (kSecond ? 1 : 0)) st.p += kSecond ? plane_b : plane_a;
        return st;
    }
};

template <int LA, int LB, int PLANES, int BM, int BN, int WI, int WJ>
__device__ __forceinline__ void product(const Product &P, const Finish &F, int id, char *a0, char *a1, char *a2, char *a3, char *b0,
                                        char *b1, char *b2, char *b3)
{
    using D = Direct<LA, LB, BM, BN, 32, WI, WJ, MulF16, Planes<PLANES>>;
    int ti, tj;
    tile_of(id, P.tiles_i, P.tiles_j, ti, tj);
    D d;
    d.ta.init(P.a, P.lda, ti * BM, P.I, P.K, 0);
    d.tb.init(P.b, P.ldb, tj * BN, P.J, P.K, 0);
    d.steps.per = (P.K + 31) / 32;
    d.steps.plane_a = P.plane_a * 2;
    d.steps.plane_b = P.plane_b * 2;
    d.run(d.steps.per * (PLANES == 2 ? 3 : 1), a0, a1, a2, a3, b0, b1, b2, b3);

    // a wave's part is turned around in LDS, so that a lane ends with eight neighbouring j of a row
    constexpr int TJ = D::TJ, FI = D::FI, FJ = D::FJ, PR = D::PR, kRow = TJ * 4, kMask = TJ / 4 - 1;
    constexpr int kGroups = TJ / 8, kRows = 64 / kGroups, kRounds = PR / kRows;
    const int lane = threadIdx.x & 63, i0 = ti * BM + d.wi * D::TI, j0 = tj * BN + d.wj * TJ;
    const int c = lane % kGroups * 8, j = j0 + c;
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
            float v[8];
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = lo4[e] * F.one, v[4 + e] = hi4[e] * F.one;
            const long long at = (long long)i * P.ldc + j;
            if (P.with) {   // rows end with zeros, and so do sums over them
                Half h[8];
                u32x4 w = *(const u32x4 *)(P.with + at);
                __builtin_memcpy(h, &w, 16);
                float x[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] = from_half(h[e]);
                if (PLANES == 2) {
                    w = *(const u32x4 *)(P.with + P.plane_c + at);
                    __builtin_memcpy(h, &w, 16);
#pragma unroll
                    for (int e = 0; e < 8; ++e) x[e] += from_half(h[e]);
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] = __builtin_fmaf(x[e], F.two, v[e]);
            }
            if (!F.last) {
                Half hi[8], lo[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) to_planes(v[e], hi[e], lo[e]);
                *(u32x4 *)(P.c + at) = __builtin_bit_cast(u32x4, hi);
                if (PLANES == 2) *(u32x4 *)(P.c + P.plane_c + at) = __builtin_bit_cast(u32x4, lo);
                continue;
            }
            using T = std::conditional_t<PLANES == 2, float, bf16>;
            T *p = (T *)P.p + (long long)i * P.J + j;
            const float size = P.size * kUnscale;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                if (j + e >= P.J) continue;
                const float x = widen(p[e]);
                // one rounding for the decayed parameter: 1 - lr wd, held in 32 bits, would add its own
                narrow(__builtin_fmaf(x, -F.decay, x) - size * v[e], p[e]);
            }
        }
        asm volatile("" ::: "memory");
    }
}

template <int STAGE, int PLANES, int SIDE>
__global__ __launch_bounds__(SIDE == 256 ? 512 : 256, 2) void k_product(Products G, Finish F)
{
    constexpr int kBytes = SIDE * 64;
    __shared__ __attribute__((aligned(1024))) char a0[kBytes], a1[kBytes], a2[kBytes], a3[kBytes];
    __shared__ __attribute__((aligned(1024))) char b0[kBytes], b1[kBytes], b2[kBytes], b3[kBytes];
    const int ti = matrix_of(G.first, G.count, blockIdx.x), id = blockIdx.x - G.first[ti];
    const Product &P = G.t[ti];
    if (id >= P.tiles_i * P.tiles_j) return;
    // 256 x 256: waves of 64 x 128 where both operands lie along k, of 128 x 64 elsewhere, as the dense layer's
    constexpr int WI = 2, WJ = SIDE == 256 ? 4 : 2, WIR = SIDE == 256 ? 4 : 2, WJR = 2;
    if (STAGE == POLY || (STAGE == GRAM && !P.cols) || (STAGE == APPLY && !P.cols))
        product<K_ROWS, K_ROWS, PLANES, SIDE, SIDE, WIR, WJR>(P, F, id, a0, a1, a2, a3, b0, b1, b2, b3);
    else if (STAGE == GRAM) product<K_COLS, K_COLS, PLANES, SIDE, SIDE, WI, WJ>(P, F, id, a0, a1, a2, a3, b0, b1, b2, b3);
    else product<K_ROWS, K_COLS, PLANES, SIDE, SIDE, WI, WJ>(P, F, id, a0, a1, a2, a3, b0, b1, b2, b3);
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

int planes_of(const hqml_muon_config &cfg) { return cfg.param_dtype == HQML_DTYPE_FP32 ? 2 : 1; }

// Calls f(first, last, bytes) for each round of matrices that go together.
template <typename F>
void rounds(const hqml_muon_config &cfg, int n, const hqml_muon_tensor *t, F f)
{
    for (int i = 0; i < n;) {
        size_t bytes = 0;
        int last = i, count = 0;
        for (; last < n && count < kMatrices; ++last) {
            if (!t[last].rows || !t[last].cols) continue;
            const size_t here = bytes_of(t[last], planes_of(cfg)).all();
            if (count && bytes + here > kBatchBytes) break;
            bytes += here;
            ++count;
        }
        if (count) f(i, last, bytes);
        i = last;
    }
}

// Tile side of a launch: times in us as the dense layer's estimate has them.
int side_of(const Products &G, int planes)
{
    static constexpr struct {
        int side, most;
        float fixed, step, share;
    } kCost[] = {{64, 4, 2.6f, 0.18f, 0.137f}, {128, 2, 4.6f, 0.2f, 0.24f}, {256, 1, 8.6f, 0.45f, 0.525f}};
    int best = 64;
    float least = 0.0f;
    for (const auto &c : kCost) {
        float steps = 0.0f, longest = 0.0f;
        for (int i = 0; i < G.count; ++i) {
            const Product &P = G.t[i];
            const float own = (float)(ceil_div(P.K, 32) * (planes == 2 ? 3 : 1));
            steps += own * (float)ceil_div(P.I, c.side) * (float)ceil_div(P.J, c.side);
            longest = std::max(longest, own);
        }
        const float us = c.fixed + std::max(longest * c.step, steps * c.share / kUnits);
        if (c.side == 64 || us < least) least = us, best = c.side;
    }
    return best;
}

template <int STAGE, int PLANES>
hipError_t run_stage(Products &G, const Finish &F, hipStream_t s)
{
    const int side = side_of(G, PLANES);
    unsigned at = 0;
    for (int i = 0; i < G.count; ++i) {
        Product &P = G.t[i];
        P.tiles_i = ceil_div(P.I, side), P.tiles_j = ceil_div(P.J, side);
        G.first[i] = at;
        at += ((unsigned)P.tiles_i * (unsigned)P.tiles_j + 7) & ~7u;
    }
    if (side == 64) k_product<STAGE, PLANES, 64><<<at, 256, 0, s>>>(G, F);
    else if (side == 128) k_product<STAGE, PLANES, 128><<<at, 256, 0, s>>>(G, F);
    else k_product<STAGE, PLANES, 256><<<at, 512, 0, s>>>(G, F);
    return hipGetLastError();
}

template <typename G, int PLANES>
hipError_t run(const hqml_muon_config &cfg, int n, const hqml_muon_tensor *t, char *work, hipStream_t s)
{
    Scalars k;
    k.mu = (float)cfg.momentum, k.nu = (float)(1.0 - cfg.momentum);
    k.nesterov = cfg.nesterov;
    k.eps = (float)cfg.eps;
    k.decay = (float)(cfg.lr * cfg.weight_decay);
    k.a = (float)cfg.a, k.b = (float)cfg.b, k.c = (float)cfg.c;
    Batch b{};
    unsigned groups = 0;
    auto each = [&](auto count_of) {   // first workgroups
        groups = 0;
        for (int i = 0; i < b.count; ++i) {
            b.first[i] = groups;
            groups += count_of(b.t[i]);
        }
    };
    for (int i = 0; i < n; ++i) {
        if (!t[i].rows || !t[i].cols) continue;
        const Bytes z = bytes_of(t[i], PLANES);
        Matrix &m = b.t[b.count++];
        m.p = t[i].param, m.g = t[i].grad, m.m = t[i].momentum;
        m.rows = t[i].rows, m.cols = t[i].cols;
        m.size = (float)(cfg.lr * t[i].scale);
        auto take = [&](size_t bytes) {
            char *here = work;
            work += bytes;
            return here;
        };
        m.x[0] = (Half *)take(z.x), m.x[1] = (Half *)take(z.x);
        m.a = (Half *)take(z.gram), m.b = (Half *)take(z.gram);
        m.sums = (double *)take(z.sums);
    }
    each([](const Matrix &m) { return (unsigned)(((long long)m.rows * m.cols + kChunk - 1) / kChunk); });
    k_momentum<G><<<groups, 256, 0, s>>>(b, k);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    each([](const Matrix &m) { return (unsigned)std::min<long long>(((long long)m.rows * pad8(m.cols) / 8 + 255) / 256, 4096); });
    k_begin<G, PLANES><<<groups, 256, 0, s>>>(b, k);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    for (int step = 0; step < cfg.steps; ++step) {
        const bool last = step + 1 == cfg.steps;
        Products gram{}, poly{}, apply{};
        gram.count = poly.count = apply.count = b.count;
        for (int i = 0; i < b.count; ++i) {
            const Matrix &m = b.t[i];
            const bool tall = m.rows > m.cols;
            const int small = std::min(m.rows, m.cols), ldx = pad8(m.cols), lda = pad8(small);
            const long long plane_x = (long long)m.rows * ldx, plane_a = (long long)small * lda;
            const Half *x = m.x[step & 1];
            Product &A = gram.t[i];
            A.a = A.b = x, A.c = m.a;
            A.lda = A.ldb = ldx, A.ldc = lda;
            A.plane_a = A.plane_b = plane_x, A.plane_c = plane_a;
            A.I = A.J = small, A.K = tall ? m.rows : m.cols, A.cols = tall;
            Product &B = poly.t[i];
            B.a = B.b = B.with = m.a, B.c = m.b;
            B.lda = B.ldb = B.ldc = lda;
            B.plane_a = B.plane_b = B.plane_c = plane_a;
            B.I = B.J = B.K = small;
            Product &X = apply.t[i];
            X.a = tall ? x : m.b, X.b = tall ? m.b : x, X.with = x, X.c = m.x[1 - (step & 1)];
            X.lda = tall ? ldx : lda, X.ldb = tall ? lda : ldx, X.ldc = ldx;
            X.plane_a = tall ? plane_x : plane_a, X.plane_b = tall ? plane_a : plane_x, X.plane_c = plane_x;
            X.I = m.rows, X.J = m.cols, X.K = small, X.cols = !tall;
            X.p = m.p, X.size = m.size;
        }
        if ((e = run_stage<GRAM, PLANES>(gram, {kUnscale, 0.0f, 0.0f, 0}, s)) != hipSuccess) return e;
        if ((e = run_stage<POLY, PLANES>(poly, {k.c * kUnscale, k.b, 0.0f, 0}, s)) != hipSuccess) return e;
        if ((e = run_stage<APPLY, PLANES>(apply, {kUnscale, k.a, k.decay, last}, s)) != hipSuccess) return e;
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
        const bool gb = cfg.grad_dtype == HQML_DTYPE_BF16;
        char *work = (char *)workspace;
        if (cfg.param_dtype == HQML_DTYPE_BF16)
            e = gb ? run<bf16, 1>(cfg, last - first, t + first, work, s) : run<float, 1>(cfg, last - first, t + first, work, s);
        else
            e = gb ? run<bf16, 2>(cfg, last - first, t + first, work, s) : run<float, 2>(cfg, last - first, t + first, work, s);
    });
    return e;
}

}  // namespace hqml
