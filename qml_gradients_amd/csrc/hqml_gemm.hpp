// The matrix product under the dense layer, on the matrix cores.
//
//   C(i, j) = sum_k A(i, k) B(j, k)
//
// An operand is stored with k along its rows (K_ROWS: x and w of the forward product) or with
// k across them (K_COLS: w of dx = dz w, both operands of dw = dz^T x).  A workgroup forms a
// BM x BN tile of C; each of its waves a TI x TJ part of it as 16 x 16 blocks
// (v_mfma_f32_16x16x32_bf16, sums in fp32 registers).  Tiles of the operands go through LDS:
//   K_ROWS  [row][BK], 16-byte chunks permuted by the row so that eight lanes reading one
//           chunk of eight rows meet eight different banks; a fragment is one 16-byte read
//   K_COLS  [k][rows], a fragment is two transposing reads (ds_read_b64_tr_b16), each of which
//           hands a lane four k of its own column; 32-byte units permuted by k for the banks
// The block of C is handed to the matrix core transposed (B's rows as its rows), so a lane
// ends with four neighbouring j of one row i.  The epilogue turns a wave's part around in
// LDS and works on eight neighbouring values of a row: one 16-byte access in bf16.
#pragma once
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "hqml_ops.hpp"

namespace hqml {
namespace gemm {

struct bf16 {
    uint16_t u;
};

__device__ __forceinline__ float widen(float x) { return x; }
__device__ __forceinline__ float widen(bf16 x) { return __builtin_bit_cast(float, (uint32_t)x.u << 16); }
__device__ __forceinline__ void narrow(float x, float &o) { o = x; }
// round to nearest even; a NaN stays one
__device__ __forceinline__ void narrow(float x, bf16 &o) { o.u = __builtin_bit_cast(uint16_t, (__bf16)x); }

// Phi(z), the normal distribution function, and e = exp(-z^2 / 2).  With t = 1 / (1 + 0.3 |z|),
// Phi(-|z|) exp(z^2 / 2) / t is smooth in t on (0, 1]; the polynomial is its least largest relative
// error there, 1.5e-7 (weighted least squares, reweighted to the largest error), and 2e-7 is what fp32
// adds.  So the tail keeps its relative precision.  An eighth of erff and expf's instructions.
__device__ __forceinline__ float normal_cdf(float z, float &e)
{
    const float a = __builtin_fabsf(z);
    const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(0.3f, a, 1.0f));
    e = __builtin_amdgcn_exp2f(a * a * -0.72134752f);
    float p = 0.0356756443f;
    p = __builtin_fmaf(p, t, -0.157206790f);
    p = __builtin_fmaf(p, t, 0.206360008f);
    p = __builtin_fmaf(p, t, -0.0536897052f);
    p = __builtin_fmaf(p, t, 0.128564859f);
    p = __builtin_fmaf(p, t, 0.0999125095f);
    p = __builtin_fmaf(p, t, 0.120754113f);
    p = __builtin_fmaf(p, t, 0.119629289f);
    const float q = p * t * e;
    return z < 0.0f ? q : 1.0f - q;
}

// 1 / (1 + exp(-z)) and tanh.  FAST, for results held in bf16: the hardware's exp2 and reciprocal, good to
// (1 + |z|) 2^-23 or so against bf16's 2^-9.
template <bool FAST>
__device__ __forceinline__ float logistic(float z)
{
    if (FAST) return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(z * -1.44269504f));
    return 1.0f / (1.0f + expf(-z));
}

template <bool FAST>
__device__ __forceinline__ float tanh_of(float z)
{
    if (!FAST) return tanhf(z);
    // near 0 the quotient would cancel: two more terms of the series, off by z^6 17/315 below 0.1
    const float s = z * z, near = z * __builtin_fmaf(s, __builtin_fmaf(s, 2.0f / 15.0f, -1.0f / 3.0f), 1.0f);
    const float far = 1.0f - 2.0f * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(z * 2.88539008f));
    return s < 0.01f ? near : far;
}

// n values through one activation.
template <bool FAST, int n>
__device__ __forceinline__ void activate(float (&z)[n], int act)
{
    switch (act) {
    case HQML_ACT_RELU:
#pragma unroll
        for (int k = 0; k < n; ++k) z[k] = z[k] < 0.0f ? 0.0f : z[k];
        break;
    case HQML_ACT_GELU:
#pragma unroll
        for (int k = 0; k < n; ++k) {
            float e;
            z[k] *= normal_cdf(z[k], e);
        }
        break;
    case HQML_ACT_SILU:
#pragma unroll
        for (int k = 0; k < n; ++k) z[k] *= logistic<FAST>(z[k]);
        break;
    case HQML_ACT_TANH:
#pragma unroll
        for (int k = 0; k < n; ++k) z[k] = tanh_of<FAST>(z[k]);
        break;
    case HQML_ACT_SIGMOID:
#pragma unroll
        for (int k = 0; k < n; ++k) z[k] = logistic<FAST>(z[k]);
        break;
    default: break;
    }
}

using bf16x8 = __attribute__((ext_vector_type(8))) __bf16;
using s16x4 = __attribute__((ext_vector_type(4))) short;
using f32x4 = __attribute__((ext_vector_type(4))) float;
using u32x4 = __attribute__((ext_vector_type(4))) uint32_t;
using lds_char = __attribute__((address_space(3))) char;

enum Layout { K_ROWS = 0, K_COLS = 1 };

struct Args {
    const void *a, *b;
    long long lda, ldb;      // elements from one stored row to the next
    int I, J, K;
    int tiles_i, tiles_j;
    // epilogue: y = alpha act(sum + bias) + residual
    void *c;
    long long ldc;
    const void *bias, *residual;
    long long ldr;
    float *z;                // [I][J], sum + bias
    int act;
    float alpha;
    int wide;                // every row of c, residual and z, and bias, allows 16-byte access
    // work split over k
    int k_part;              // k of one part, a multiple of BK
    float *part;             // [parts][I][J]: sums of one part, no epilogue; null: whole sums
};

// Tile of a workgroup.  Workgroups go round the eight XCDs in turn; each XCD takes a run of
// neighbouring tiles, and the run walks bands of eight tile rows, so that the tiles an XCD
// works on together share operand rows in its L2.
__device__ __forceinline__ void tile_of(int id, int ti, int tj, int &i, int &j)
{
    const int all = ti * tj, xcd = id & 7, q = all >> 3, r = all & 7;
    const int t = xcd * q + (xcd < r ? xcd : r) + (id >> 3);
    const int band = t / (8 * tj), first = band * 8;
    const int rows = ti - first < 8 ? ti - first : 8;
    const int in = t - band * 8 * tj;
    i = first + in % rows;
    j = in / rows;
}

// vmcnt(n): at most n of this wave's loads are still under way.
template <int n>
__device__ __forceinline__ void wait_loads()
{
    __builtin_amdgcn_s_waitcnt((n & 15) | ((n >> 4) << 14) | (7 << 4) | (15 << 8));
}

__device__ __forceinline__ void barrier()
{
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// One bf16 operand tile of R rows (i or j) and BK k, loaded straight into LDS.
// Loads go through a buffer resource that ends with the operand's last element: rows past
// the end read as zero by themselves; k past the end of a row is sent past the end of the buffer.
template <int L, int R, int BK, int WAVES>
struct DirectTile {
    static constexpr int kBytes = R * BK * 2;
    static constexpr int kLoads = kBytes / (WAVES * 1024);   // 16-byte loads of a lane
    static_assert(kBytes % (WAVES * 1024) == 0, "whole loads");
    static constexpr int kRow = (L == K_ROWS ? BK : R) * 2;   // bytes of an LDS row
    static constexpr int kChunks = kRow / 16;

    const char *base;
    long long ld;      // bytes
    int rows, K;
    int off[kLoads];   // byte offset of a lane's chunk in the tile; K_COLS: past the end if its rows are
    int at;            // K_ROWS: first k of a lane's chunk (the same in all its rows: they are 8 n apart)
    int frag;          // byte of a lane's part of the fragment at row 0, k 0

    static __device__ __forceinline__ int key(int r)
    {
        if (L == K_ROWS) return kChunks == 4 ? (r >> 1) & 3 : r & 7;
        return (((r & 3) | ((r >> 1) & 12)) << 1) & (kChunks - 1);
    }

    __device__ __forceinline__ void init(const void *p, long long ld_elems, int row0, int n_rows, int n_k, int k0)
    {
        ld = ld_elems * 2;
        rows = n_rows - row0;
        K = n_k;
        base = (const char *)p + (L == K_ROWS ? row0 * ld + k0 * 2ll : k0 * ld + row0 * 2ll);
        const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
        for (int n = 0; n < kLoads; ++n) {
            const int slot = (n * WAVES + wave) * 64 + lane;
            const int r = slot / kChunks, c = (slot % kChunks) ^ key(r);
            if (L == K_ROWS) {
                off[n] = (int)(r * ld) + c * 16;
                at = c * 8;
            } else {
                off[n] = c * 8 < rows ? (int)(r * ld) + c * 16 : 0x7FFFFFF0;
            }
        }
        init_fragment();
    }

    __device__ __forceinline__ void init_fragment()
    {
        const int lane = threadIdx.x & 63;
        if (L == K_ROWS) {
            frag = (lane & 15) * kRow + (((lane >> 4) ^ key(lane & 15)) << 4);
        } else {
            const int k = (lane >> 4) * 8 + ((lane >> 2) & 3);
            frag = k * kRow + (key(k) << 4) + (lane & 3) * 8;
        }
    }

    // What the loads of one step share.
    struct Step {
        const char *p;
        int end, left;
    };

    // The tile at k (relative to init's k0, which left n_k); past the end: an empty buffer, nothing is read.
    __device__ __forceinline__ Step begin(int k) const
    {
        const int left = K - k;
        long long bytes;
        const char *p;
        if (L == K_ROWS) {
            p = base + 2ll * k;
            bytes = (long long)(rows - 1) * ld + 2ll * left;
        } else {
            p = base + k * ld;
            bytes = (long long)(left - 1) * ld + 2ll * rows;
        }
        const int end = left <= 0 ? 0 : bytes > 0x7FFFFFE0 ? 0x7FFFFFE0 : (int)bytes;
        return {p, end, left};
    }

    // Queue load n of kLoads.
    __device__ __forceinline__ void load(const Step &st, lds_char *to, int n) const
    {
        const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        const auto rsrc = __builtin_amdgcn_make_buffer_rsrc((void *)st.p, 0, st.end, 0x00027000);
        int o = off[n];
        if (L == K_ROWS) o = at < st.left ? o : 0x7FFFFFF0;
        __builtin_amdgcn_raw_ptr_buffer_load_lds(
            rsrc, (__attribute__((address_space(3))) void *)(to + (n * WAVES + wave) * 1024), 16, o, 0, 0, 0);
    }

    // Fragment of 16 rows from row r0 (a multiple of 16), 32 k from k0 (of 32).  Neither changes a
    // row's or k's key, so both enter the lane's byte as a sum or one exclusive or.
    __device__ __forceinline__ bf16x8 fragment(const lds_char *t, int r0, int k0) const
    {
        if (L == K_ROWS)
            return *(const __attribute__((address_space(3))) bf16x8 *)(t + (frag ^ (k0 << 1)) + r0 * kRow);
        union {
            s16x4 s[2];
            bf16x8 v;
        } u;
        // sixteen lanes read four k rows of sixteen values and receive them transposed
        const lds_char *p = t + (frag ^ (r0 << 1)) + k0 * kRow;
#pragma unroll
        for (int h = 0; h < 2; ++h)
            u.s[h] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4 *)(p + h * 4 * kRow));
        return u.v;
    }
};

// Epilogue of a wave's TI x TJ part (16 x 16 blocks acc[FI][FJ], four j of row lane % 16 a lane)
// that begins at (i0, j0) of C; buf: this wave's own LDS, PR rows of TJ floats, whose 16-byte
// chunks are permuted by the row (a lane writes one chunk of its row).
// Only a forward product has more to finish than alpha.  again(i, j): the sum at (i, j) formed anew where it is not finite (kAgain).
template <typename TC, int FI, int FJ, int PR, bool kForward, bool kAgain, typename F>
__device__ __forceinline__ void finish(const Args &P, f32x4 (&acc)[FI][FJ], int i0, int j0, int part, lds_char *buf,
                                       F again)
{
    constexpr int TJ = FJ * 16, kRow = TJ * 4, kMask = TJ / 4 - 1;
    static_assert((TJ & (TJ - 1)) == 0, "chunk permutation");
    constexpr int kGroups = TJ / 8, kRows = 64 / kGroups;   // a wave takes kRows rows of kGroups values of eight at once
    constexpr int kRounds = PR / kRows, kU = kRounds % 4 == 0 ? 4 : kRounds % 2 == 0 ? 2 : 1;
    constexpr int kV = (int)sizeof(TC) / 2;                 // 16-byte words of eight values
    static_assert(PR % kRows == 0 && FI * 16 % PR == 0, "whole turns");
    constexpr bool kFast = sizeof(TC) == 2;
    const int lane = threadIdx.x & 63;
    const int c = lane % kGroups * 8, j = j0 + c, n = P.J - j < 8 ? P.J - j : 8;
    float *out = P.part ? P.part + (long long)part * P.I * P.J : nullptr;
    float bias[8] = {};
    if (kForward && P.bias && !out)
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (k < n) bias[k] = widen(((const TC *)P.bias)[j + k]);
#pragma unroll
    for (int f0 = 0; f0 < FI; f0 += PR / 16) {
#pragma unroll
        for (int f = 0; f < PR / 16; ++f)
#pragma unroll
            for (int g = 0; g < FJ; ++g)
                *(__attribute__((address_space(3))) f32x4 *)(buf + (f * 16 + (lane & 15)) * kRow +
                                                             (((g * 4 + (lane >> 4)) ^ (lane & kMask & 15)) << 4)) =
                    acc[f0 + f][g];
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");   // the wave's own writes, read by its other lanes
        for (int round = 0; round < kRounds; round += kU) {
            const int r0 = round * kRows + lane / kGroups, i_of = i0 + f0 * 16 + r0;
            const bool wide = P.wide && j < P.J;   // J is a multiple of 8 then
            u32x4 res[kU][kV];
            if (kForward && wide && P.residual && !out)
#pragma unroll
                for (int u = 0; u < kU; ++u)
#pragma unroll
                    for (int k = 0; k < kV; ++k)
                        if (i_of + u * kRows < P.I)
                            res[u][k] = ((const u32x4 *)((const TC *)P.residual + (i_of + u * kRows) * P.ldr + j))[k];
            float v[kU * 8];
#pragma unroll
            for (int u = 0; u < kU; ++u) {
                const int r = r0 + u * kRows, key = r & kMask & 15;
                const auto *src = (const __attribute__((address_space(3))) f32x4 *)(buf + r * kRow);
                const f32x4 lo = src[(c >> 2) ^ key], hi = src[((c >> 2) + 1) ^ key];
#pragma unroll
                for (int k = 0; k < 4; ++k) v[u * 8 + k] = lo[k], v[u * 8 + 4 + k] = hi[k];
                if (kAgain && i_of + u * kRows < P.I) {
                    float worst = 0.0f;
#pragma unroll
                    for (int k = 0; k < 8; ++k) worst += k < n ? v[u * 8 + k] * 0.0f : 0.0f;
                    if (worst != worst)
                        for (int k = 0; k < n; ++k) {
                            const float s = again(i_of + u * kRows, j + k);
#pragma unroll
                            for (int q = 0; q < 8; ++q) v[u * 8 + q] = q == k ? s : v[u * 8 + q];
                        }
                }
            }
            if (out) {
#pragma unroll
                for (int u = 0; u < kU; ++u) {
                    const int i = i_of + u * kRows;
                    if (i >= P.I) continue;
                    float *o = out + (long long)i * P.J + j;
                    if (wide) {
                        ((f32x4 *)o)[0] = f32x4{v[u * 8], v[u * 8 + 1], v[u * 8 + 2], v[u * 8 + 3]};
                        ((f32x4 *)o)[1] = f32x4{v[u * 8 + 4], v[u * 8 + 5], v[u * 8 + 6], v[u * 8 + 7]};
                    } else {
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            if (k < n) o[k] = v[u * 8 + k];
                    }
                }
                continue;
            }
            if (kForward) {
#pragma unroll
                for (int u = 0; u < kU; ++u)
#pragma unroll
                    for (int k = 0; k < 8; ++k) v[u * 8 + k] += bias[k];
                if (P.z)
#pragma unroll
                    for (int u = 0; u < kU; ++u) {
                        const int i = i_of + u * kRows;
                        if (i >= P.I) continue;
                        float *o = P.z + (long long)i * P.J + j;
                        if (wide) {
                            ((f32x4 *)o)[0] = f32x4{v[u * 8], v[u * 8 + 1], v[u * 8 + 2], v[u * 8 + 3]};
                            ((f32x4 *)o)[1] = f32x4{v[u * 8 + 4], v[u * 8 + 5], v[u * 8 + 6], v[u * 8 + 7]};
                        } else {
#pragma unroll
                            for (int k = 0; k < 8; ++k)
                                if (k < n) o[k] = v[u * 8 + k];
                        }
                    }
                activate<kFast>(v, P.act);
            }
#pragma unroll
            for (int u = 0; u < kU; ++u) {
                const int i = i_of + u * kRows;
                if (i >= P.I) continue;
                TC *o = (TC *)P.c + i * P.ldc + j;
                if (wide) {
                    TC t[8];
                    if (kForward && P.residual) {
                        __builtin_memcpy(t, res[u], sizeof t);
#pragma unroll
                        for (int k = 0; k < 8; ++k) narrow(v[u * 8 + k] * P.alpha + widen(t[k]), t[k]);
                    } else {
#pragma unroll
                        for (int k = 0; k < 8; ++k) narrow(v[u * 8 + k] * P.alpha, t[k]);
                    }
                    u32x4 w[kV];
                    __builtin_memcpy(w, t, sizeof t);
#pragma unroll
                    for (int k = 0; k < kV; ++k) ((u32x4 *)o)[k] = w[k];
                } else {
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        if (k >= n) continue;
                        float y = v[u * 8 + k] * P.alpha;
                        if (kForward && P.residual) y += widen(((const TC *)P.residual)[i * P.ldr + j + k]);
                        narrow(y, o[k]);
                    }
                }
            }
        }
        asm volatile("" ::: "memory");
    }
}

// bf16 operands whose rows allow 16-byte access, loaded straight into LDS.  Four LDS buffers of
// a step (32 k) each: the loads of two to three steps are under way while one is computed.  A
// wave reads fragments ahead of the matrix instructions that take them: row blocks of A by
// kAhead, the next step's column blocks of B during the second half of a step.  So the one
// barrier of a step stands in its middle: it makes step t + 1 readable and frees the
// buffer of step t - 1, into which the loads of step t + 3 go out one after each row block (all
// at once, they would hold up the wave's matrix instructions behind them).
// 8192 x 4096 x 4096 at 256 x 256 tiles, by layout pair: 218, 206 and 200 us (1264, 1332 and
// 1377 TFLOP/s), with two buffers of 64 k 228-257; the matrix instructions alone take 135.

// What a wave of k_product_direct holds.
template <int LA, int LB, int BM, int BN, int BK, int WI, int WJ>
struct Direct {
    static constexpr int kWaves = WI * WJ, TI = BM / WI, TJ = BN / WJ, FI = TI / 16, FJ = TJ / 16;
    using TA = DirectTile<LA, BM, BK, kWaves>;
    using TB = DirectTile<LB, BN, BK, kWaves>;
    static constexpr int kLoads = TA::kLoads + TB::kLoads;
    TA ta;
    TB tb;
    int wi, wj;
    f32x4 acc[FI][FJ];
    static constexpr int kAhead = FI >= 4 ? 2 : 1, kMid = FI / 2, kPer = FJ / (FI - kMid);
    bf16x8 fa[FI], fb[FJ];

    // Queue all loads of step t.
    __device__ __forceinline__ void load(char *A, char *B, int t) const
    {
        const auto sa = ta.begin(t * BK);
        const auto sb = tb.begin(t * BK);
#pragma unroll
        for (int n = 0; n < TA::kLoads; ++n) ta.load(sa, (lds_char *)A, n);
#pragma unroll
        for (int n = 0; n < TB::kLoads; ++n) tb.load(sb, (lds_char *)B, n);
    }

    __device__ __forceinline__ void first(const char *A, const char *B)
    {
#pragma unroll
        for (int f = 0; f < kAhead; ++f) fa[f] = ta.fragment((const lds_char *)A, wi * TI + f * 16, 0);
#pragma unroll
        for (int g = 0; g < FJ; ++g) fb[g] = tb.fragment((const lds_char *)B, wj * TJ + g * 16, 0);
    }
    __device__ __forceinline__ void step(const char *A, const char *A1, const char *B1, char *A3, char *B3, int t)
    {
        const auto sa = ta.begin((t + 3) * BK);
        const auto sb = tb.begin((t + 3) * BK);
        bf16x8 na[kAhead], nb[FJ];
#pragma unroll
        for (int f = 0; f < FI; ++f) {
            if (f == kMid) {
                wait_loads<kLoads>();
                barrier();
            }
            if (f + kAhead < FI) fa[f + kAhead] = ta.fragment((const lds_char *)A, wi * TI + (f + kAhead) * 16, 0);
            else na[f + kAhead - FI] = ta.fragment((const lds_char *)A1, wi * TI + (f + kAhead - FI) * 16, 0);
            if (f >= kMid) {
#pragma unroll
                for (int g = (f - kMid) * kPer; g < (f - kMid + 1) * kPer; ++g)
                    nb[g] = tb.fragment((const lds_char *)B1, wj * TJ + g * 16, 0);
            }
#pragma unroll
            for (int g = 0; g < FJ; ++g)
                acc[f][g] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fb[g], fa[f], acc[f][g], 0, 0, 0);
            if (f >= kMid) {
                constexpr int kH = FI - kMid;
#pragma unroll
                for (int n = (f - kMid) * kLoads / kH; n < (f - kMid + 1) * kLoads / kH; ++n) {
                    if (n < TA::kLoads) ta.load(sa, (lds_char *)A3, n);
                    else tb.load(sb, (lds_char *)B3, n - TA::kLoads);
                }
            }
            __builtin_amdgcn_sched_barrier(0);
        }
#pragma unroll
        for (int f = 0; f < kAhead; ++f) fa[f] = na[f];
#pragma unroll
        for (int g = 0; g < FJ; ++g) fb[g] = nb[g];
    }

    // Step t is in LDS for every wave, and every wave is done with the buffer of step t - 1.
    __device__ __forceinline__ void ready() const
    {
        wait_loads<2 * kLoads>();
        barrier();
    }
};

template <int LA, int LB, int BM, int BN, int BK, int WI, int WJ>
__global__ __launch_bounds__(64 * WI *WJ, 2) void k_product_direct(Args P)
{
    using D = Direct<LA, LB, BM, BN, BK, WI, WJ>;
    using TA = typename D::TA;
    using TB = typename D::TB;
    constexpr int kWaves = D::kWaves, TI = D::TI, TJ = D::TJ, FI = D::FI, FJ = D::FJ;
    __shared__ __attribute__((aligned(1024))) char a0[TA::kBytes], a1[TA::kBytes], a2[TA::kBytes], a3[TA::kBytes];
    __shared__ __attribute__((aligned(1024))) char b0[TB::kBytes], b1[TB::kBytes], b2[TB::kBytes], b3[TB::kBytes];

    int ti, tj;
    tile_of(blockIdx.x, P.tiles_i, P.tiles_j, ti, tj);
    const int kb = blockIdx.y * P.k_part;
    const int kn = P.K - kb < P.k_part ? P.K - kb : P.k_part;
    const int wave = threadIdx.x >> 6;
    D d;
    d.ta.init(P.a, P.lda, ti * BM, P.I, kn, kb);
    d.tb.init(P.b, P.ldb, tj * BN, P.J, kn, kb);
    d.wi = wave / WJ, d.wj = wave % WJ;
#pragma unroll
    for (int f = 0; f < FI; ++f)
#pragma unroll
        for (int g = 0; g < FJ; ++g) d.acc[f][g] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

    const int steps = (kn + BK - 1) / BK;
    d.load(a0, b0, 0);
    d.load(a1, b1, 1);
    d.load(a2, b2, 2);
    d.ready();
    d.first(a0, b0);
    int t = 0;
    for (; t + 4 <= steps; t += 4) {
        d.step(a0, a1, b1, a3, b3, t);
        d.step(a1, a2, b2, a0, b0, t + 1);
        d.step(a2, a3, b3, a1, b1, t + 2);
        d.step(a3, a0, b0, a2, b2, t + 3);
    }
    if (t < steps) {
        d.step(a0, a1, b1, a3, b3, t);
        if (t + 1 < steps) {
            d.step(a1, a2, b2, a0, b0, t + 1);
            if (t + 2 < steps) d.step(a2, a3, b3, a1, b1, t + 2);
        }
    }
    wait_loads<0>();
    barrier();
    // each buffer serves a quarter of the waves
    constexpr int kOwn = (TA::kBytes < TB::kBytes ? TA::kBytes : TB::kBytes);
    constexpr int kFit = kOwn / (TJ * 4);
    static_assert(kWaves % 4 == 0 && kWaves <= 8 && kFit >= 16, "room for one block row");
    constexpr int PR = kFit >= TI ? TI : kFit;
    lds_char *const own = wave == 0 ? (lds_char *)a0 : wave == 1 ? (lds_char *)a1 : wave == 2 ? (lds_char *)a2 : wave==3 ? (lds_char *)a3 : wave==4 ? (lds_char*)b0 : wave==5?(lds_char*)b1:wave==6?(lds_char*)b2:(lds_char*)b3;
    finish<bf16, FI, FJ, PR, LA == K_ROWS && LB == K_ROWS, false>(P, d.acc, ti * BM + d.wi * TI, tj * BN + d.wj * TJ, blockIdx.y, own,
                                    [](int, int) { return 0.0f; });
}

// One operand tile that goes through registers on its way to LDS: 32-bit operands, which are
// split there, and bf16 rows that do not allow 16-byte access to LDS.  The LDS layout is
// DirectTile's, PLANES times.  Loads into registers take 16 bytes at any alignment of the element;
// where a chunk may pass the end of its row, its values are loaded one by one.  A 32-bit value is the sum of PLANES bf16 values to 8 PLANES + 1 bits or so
// (exactly, with three, where none underflows): x = h + m + l, each the rounding of what the
// ones before leave.
template <typename T, int PLANES, int L, int R, int BK, int THREADS>
struct StagedTile {
    using Tile = DirectTile<L, R, BK, THREADS / 64>;
    static constexpr int kPlane = R * BK * 2, kBytes = kPlane * PLANES;
    static constexpr int kN = R * BK / 8 / THREADS;   // 8-value chunks of a lane
    static_assert(kN >= 1 && R * BK / 8 % THREADS == 0, "whole chunks");
    static constexpr int kSize = (int)sizeof(T), kWords = kSize * 2;   // registers of a chunk

    const char *base;
    long long ld;   // bytes
    int rows, K;
    int off[kN];
    int at[kN];     // first k (K_COLS: first row) of a lane's chunk in the tile
    int put;        // its LDS byte; chunk n lies n * THREADS * 16 further
    uint32_t reg[kN][kWords];

    __device__ __forceinline__ void init(const void *p, long long ld_elems, int row0, int n_rows, int n_k, int k0)
    {
        ld = ld_elems * kSize;
        rows = n_rows - row0;
        K = n_k;
        base = (const char *)p + (L == K_ROWS ? row0 * ld + (long long)k0 * kSize : k0 * ld + (long long)row0 * kSize);
#pragma unroll
        for (int n = 0; n < kN; ++n) {
            const int slot = n * THREADS + threadIdx.x;
            const int r = slot / Tile::kChunks, c = (slot % Tile::kChunks) ^ Tile::key(r);
            off[n] = (int)(r * ld) + c * 8 * kSize;
            at[n] = c * 8;
        }
        put = threadIdx.x * 16;
    }

    // Load the tile at k into registers.
    __device__ __forceinline__ void load(int k)
    {
        const int left = K - k;
        long long bytes;
        const char *p;
        if (L == K_ROWS) {
            p = base + (long long)k * kSize;
            bytes = (long long)(rows - 1) * ld + (long long)left * kSize;
        } else {
            p = base + k * ld;
            bytes = (long long)(left - 1) * ld + (long long)rows * kSize;
        }
        const int end = left <= 0 ? 0 : bytes > 0x7FFFFFE0 ? 0x7FFFFFE0 : (int)bytes;
        const auto rsrc = __builtin_amdgcn_make_buffer_rsrc((void *)p, 0, end, 0x00027000);
        const int stop = L == K_ROWS ? left : rows;   // values of the chunk's direction that exist
        const bool tail = L == K_ROWS ? left < BK : rows < R;
#pragma unroll
        for (int n = 0; n < kN; ++n) {
            if (!tail) {
#pragma unroll
                for (int h = 0; h < kWords / 4; ++h) {
                    const u32x4 w = __builtin_amdgcn_raw_buffer_load_b128(rsrc, off[n] + h * 16, 0, 0);
#pragma unroll
                    for (int q = 0; q < 4; ++q) reg[n][h * 4 + q] = w[q];
                }
                continue;
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int o = at[n] + e < stop ? off[n] + e * kSize : 0x7FFFFFF0;
                if (kSize == 4) {
                    reg[n][e % kWords] = __builtin_amdgcn_raw_buffer_load_b32(rsrc, o, 0, 0);
                } else {
                    const uint32_t v = (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(rsrc, o, 0, 0);
                    if (e & 1) reg[n][e / 2] |= v << 16;
                    else reg[n][e / 2] = v;
                }
            }
        }
    }

    // Split what load() brought and write it to LDS.
    __device__ __forceinline__ void store(lds_char *to) const
    {
#pragma unroll
        for (int n = 0; n < kN; ++n) {
            lds_char *dst = to + put + n * THREADS * 16;
            if (kSize == 2) {
                *(__attribute__((address_space(3))) u32x4 *)dst = u32x4{reg[n][0], reg[n][1], reg[n][2], reg[n][3]};
            } else {
                float x[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] = __builtin_bit_cast(float, reg[n][e % kWords]);
#pragma unroll
                for (int p = 0; p < PLANES; ++p) {
                    bf16x8 h;
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        h[e] = (__bf16)x[e];
                        if (p + 1 < PLANES) x[e] -= (float)h[e];
                    }
                    *(__attribute__((address_space(3))) bf16x8 *)(dst + p * kPlane) = h;
                }
            }
        }
    }
};

// The sum at (i, j) by itself, in fp32: for values whose split does not hold (infinities, and
// magnitudes that round up to one).
template <typename T, typename U, int LA, int LB>
__device__ __attribute__((noinline)) float plain_sum(const T *a, const U *b, long long lda, long long ldb, int i, int j, int k0, int n)
{
    float s = 0.0f;
    for (int k = k0; k < k0 + n; ++k)
        s += widen(LA == K_ROWS ? a[i * lda + k] : a[k * lda + i]) * widen(LB == K_ROWS ? b[j * ldb + k] : b[k * ldb + j]);
    return s;
}

// Operands of type T and U held as PA and PB bf16 planes; of the products of planes those are
// formed that reach the sum's 24 bits: 6 for 3 x 3 planes, whose left-out ones are below 2^-24 of the
// product of magnitudes.  Step t + 1 is loaded into registers while step t is computed.  With
// BUF = 2 its split and its way to LDS fall between step t's matrix instructions, at one barrier
// a step; with BUF = 1 they come after, and two workgroups share a compute unit, so that one
// computes while the other stores.  2048^3 in fp32 (256 tiles, one a compute unit): 91 us with
// two buffers, 102 with one; 4096^3 (1024 tiles): 693 and 640.
template <typename T, int PA, int LA, typename U, int PB, int LB, typename TC, int BM, int BN, int WI, int WJ, int BUF>
__global__ __launch_bounds__(64 * WI *WJ, 2) void k_product_staged(Args P)
{
    constexpr int BK = 32, kWaves = WI * WJ, kThreads = 64 * kWaves, TI = BM / WI, TJ = BN / WJ, FI = TI / 16,
                  FJ = TJ / 16;
    using TA = StagedTile<T, PA, LA, BM, BK, kThreads>;
    using TB = StagedTile<U, PB, LB, BN, BK, kThreads>;
    constexpr int kTurn = TI < 32 ? TI : 32;   // rows of a wave's part turned at once
    constexpr int kTurnBytes = kTurn * TJ * 4;
    constexpr int kTiles = TA::kBytes + TB::kBytes;
    constexpr int kLds = kTiles * BUF > kWaves * kTurnBytes ? kTiles * BUF : kWaves * kTurnBytes;
    __shared__ __attribute__((aligned(1024))) char lds[kLds];
    lds_char *here = (lds_char *)lds, *next = here + (BUF - 1) * kTiles;

    int ti, tj;
    tile_of(blockIdx.x, P.tiles_i, P.tiles_j, ti, tj);
    const int kb = blockIdx.y * P.k_part;
    const int kn = P.K - kb < P.k_part ? P.K - kb : P.k_part;
    TA ta;
    TB tb;
    ta.init(P.a, P.lda, ti * BM, P.I, kn, kb);
    tb.init(P.b, P.ldb, tj * BN, P.J, kn, kb);
    typename TA::Tile fa_of;   // where a lane's fragments begin
    typename TB::Tile fb_of;
    fa_of.init_fragment();
    fb_of.init_fragment();
    const int wave = threadIdx.x >> 6, wi = wave / WJ, wj = wave % WJ;
    f32x4 acc[FI][FJ] = {};
    ta.load(0);
    tb.load(0);
    ta.store(here);
    tb.store(here + TA::kBytes);
    ta.load(BK);   // past the last step: an empty buffer, nothing is read
    tb.load(BK);
    __builtin_amdgcn_s_waitcnt(0xC07F);   // lgkmcnt(0): the stores are done
    barrier();
    for (int k0 = 0; k0 < kn; k0 += BK) {
        bf16x8 fb[PB][FJ];
#pragma unroll
        for (int p = 0; p < PB; ++p)
#pragma unroll
            for (int g = 0; g < FJ; ++g)
                fb[p][g] = fb_of.fragment(here + TA::kBytes + p * TB::kPlane, wj * TJ + g * 16, 0);
#pragma unroll
        for (int f = 0; f < FI; ++f) {
#pragma unroll
            for (int p = PA - 1; p >= 0; --p) {
                const bf16x8 fa = fa_of.fragment(here + p * TA::kPlane, wi * TI + f * 16, 0);
#pragma unroll
                for (int q = PB - 1; q >= 0; --q) {
                    if (p + q >= (PA > PB ? PA : PB)) continue;
#pragma unroll
                    for (int g = 0; g < FJ; ++g)
                        acc[f][g] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fb[q][g], fa, acc[f][g], 0, 0, 0);
                }
            }
            if (BUF == 2 && f == FI / 2 - 1) {
                ta.store(next);
                ta.load(k0 + 2 * BK);
            }
            if (BUF == 2 && f == FI - 1) {
                tb.store(next + TA::kBytes);
                tb.load(k0 + 2 * BK);
            }
        }
        if (BUF == 1) {
            barrier();
            ta.store(here);
            tb.store(here + TA::kBytes);
            ta.load(k0 + 2 * BK);
            tb.load(k0 + 2 * BK);
        }
        __builtin_amdgcn_s_waitcnt(0xC07F);
        barrier();
        lds_char *const swap = here;
        here = next;
        next = swap;
    }
    finish<TC, FI, FJ, kTurn, LA == K_ROWS && LB == K_ROWS, (PA > 1 || PB > 1)>(
        P, acc, ti * BM + wi * TI, tj * BN + wj * TJ, blockIdx.y, (lds_char *)lds + wave * kTurnBytes,
        [&](int i, int j) {
            return plain_sum<T, U, LA, LB>((const T *)P.a, (const U *)P.b, P.lda, P.ldb, i, j, kb, kn);
        });
}

// y of summed parts: the join after work split over k.
template <typename TC>
__global__ __launch_bounds__(256) void k_join(Args P, int parts)
{
    const long long all = (long long)P.I * P.J;
    for (long long e = (long long)blockIdx.x * 256 + threadIdx.x; e < all; e += (long long)gridDim.x * 256) {
        const int i = (int)(e / P.J), j = (int)(e % P.J);
        float v[1] = {0.0f};
        for (int p = 0; p < parts; ++p) v[0] += P.part[p * all + e];
        if (P.bias) v[0] += widen(((const TC *)P.bias)[j]);
        if (P.z) P.z[e] = v[0];
        activate<sizeof(TC) == 2>(v, P.act);
        float y = v[0] * P.alpha;
        if (P.residual) y += widen(((const TC *)P.residual)[i * P.ldr + j]);
        narrow(y, ((TC *)P.c)[i * P.ldc + j]);
    }
}

// Tile shapes a product can be run with.
enum Shape { TILE_64 = 0, TILE_128 = 1, TILE_256 = 2 };

// The kernels of one operand type, for a layout pair (K_ROWS, K_ROWS), (K_ROWS, K_COLS) or
// (K_COLS, K_COLS).  direct: both bf16 operands' rows allow 16-byte access to LDS; TILE_256 needs it.
hipError_t launch_bf16(const Args &a, int la, int lb, bool direct, Shape shape, int parts, hipStream_t s);
hipError_t launch_fp32(const Args &a, int la, int lb, Shape shape, int parts, hipStream_t s);

}  // namespace gemm
}  // namespace hqml
