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
#include <stdint.h>

#include "hqml_act.hpp"
#include "hqml_dense_cut.hpp"

namespace hqml {
namespace gemm {

using bf16x8 = __attribute__((ext_vector_type(8))) __bf16;
using s16x4 = __attribute__((ext_vector_type(4))) short;
using f32x2 = __attribute__((ext_vector_type(2))) float;
using f32x4 = __attribute__((ext_vector_type(4))) float;
using u32x4 = __attribute__((ext_vector_type(4))) uint32_t;
// 16 bytes at any alignment of an element: the hardware takes them so
using u32x4_any = __attribute__((ext_vector_type(4), aligned(2))) uint32_t;
using f32x4_any = __attribute__((ext_vector_type(4), aligned(4))) float;
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
    void *ones;              // [I]: the sums of A's rows, as a column J of B that is all ones; or null
    // work split over k: every part leaves its sums, the last one of a tile to finish adds them up
    int parts, k_part;       // k of one part, a multiple of 32
    float *part;             // [tiles][parts][BM * BN]
    unsigned *ticket;        // [tiles], 0 between calls
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

// vmcnt(n): at most n of this wave's loads and stores are still under way.  The builtin alone says nothing of memory: the
// compiler might move one past it.
template <int n>
__device__ __forceinline__ void wait_loads()
{
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt((n & 15) | ((n >> 4) << 14) | (7 << 4) | (15 << 8));
}

// This wave's LDS reads and writes are done.
__device__ __forceinline__ void wait_lds()
{
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0xC07F);   // lgkmcnt(0)
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
    int span;          // bytes of the buffer: of the rows before the tile's last one (K_ROWS), of one k (K_COLS)
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
        // an odd number of rows (K_COLS) ends in the middle of a word, which would read as zero: the whole
        // aligned word is let in, and its other half reaches only sums that are not stored
        span = L == K_ROWS ? ((rows < R ? rows : R) - 1) * (int)ld : (2 * rows + 3) & ~3;
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
        const char *p = L == K_ROWS ? base + 2ll * k : base + k * ld;
        // K_ROWS: rows end with zeros up to a multiple of eight
        const int end = L == K_ROWS ? span + ((2 * left + 15) & ~15) : (left < BK ? left - 1 : BK - 1) * (int)ld + span;
        return {p, left <= 0 ? 0 : end, left};
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

// Work split over k.  A workgroup leaves its sums in the workspace and takes a ticket; the one that
// takes a tile's last adds all parts in their order (the result does not depend on who came
// last) and finishes the tile.  Says whether this workgroup is the one.  The sums are written
// and read as device-scope atomics, past the caches that the XCDs do not share, and have
// arrived when the ticket is taken: a fence would write back a whole L2 for each of them (serve
// 4096 -> 4096: 32 us with fences).
// MORE: twice the parts' loads under way, for kernels whose LDS leaves room in the registers.
template <int FI, int FJ, int THREADS, bool MORE = false>
__device__ __forceinline__ bool joined(const Args &P, f32x4 (&acc)[FI][FJ], int tile, int part, int i0)
{
    __shared__ unsigned taken;
    constexpr int kWords = FI * FJ * 2;   // pairs of sums of a lane
    unsigned long long *all = (unsigned long long *)P.part + (long long)tile * P.parts * (kWords * THREADS) + threadIdx.x;
    unsigned long long *own = all + (long long)part * (kWords * THREADS);
    const int rows = P.I - i0 - (threadIdx.x & 15);   // a lane's row of block f exists if 16 f < rows
#pragma unroll
    for (int f = 0; f < FI; ++f) {
        if (f * 16 >= rows) continue;
#pragma unroll
        for (int g = 0; g < FJ; ++g)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const f32x2 pair = {acc[f][g][2 * h], acc[f][g][2 * h + 1]};
                __hip_atomic_store(own + ((f * FJ + g) * 2 + h) * THREADS, __builtin_bit_cast(unsigned long long, pair),
                                   __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            }
    }
    wait_loads<0>();   // and stores: this wave's have arrived
    __syncthreads();   // every wave's have
    if (threadIdx.x == 0)
        taken = __hip_atomic_fetch_add(P.ticket + tile, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    __syncthreads();
    if (taken != (unsigned)P.parts - 1) return false;
    constexpr int kAtOnce = kWords <= 8 ? (MORE ? 8 : 4) : kWords <= 16 ? 2 : 1;   // parts whose loads are under way together
#pragma unroll
    for (int f = 0; f < FI; ++f)
#pragma unroll
        for (int g = 0; g < FJ; ++g) acc[f][g] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    for (int p0 = 0; p0 < P.parts; p0 += kAtOnce) {
        unsigned long long w[kAtOnce][kWords];
#pragma unroll
        for (int p = 0; p < kAtOnce; ++p)
#pragma unroll
            for (int e = 0; e < kWords; ++e)
                w[p][e] = p0 + p < P.parts && e / (FJ * 2) * 16 < rows
                              ? __hip_atomic_load(all + ((long long)(p0 + p) * kWords + e) * THREADS, __ATOMIC_RELAXED,
                                                  __HIP_MEMORY_SCOPE_AGENT)
                              : 0;
#pragma unroll
        for (int p = 0; p < kAtOnce; ++p)
#pragma unroll
            for (int e = 0; e < kWords; ++e) {
                acc[e / (FJ * 2)][e / 2 % FJ][e % 2 * 2] += __builtin_bit_cast(float, (uint32_t)w[p][e]);
                acc[e / (FJ * 2)][e / 2 % FJ][e % 2 * 2 + 1] += __builtin_bit_cast(float, (uint32_t)(w[p][e] >> 32));
            }
    }
    if (threadIdx.x == 0) __hip_atomic_store(P.ticket + tile, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    return true;
}

// Epilogue of a wave's TI x TJ part (16 x 16 blocks acc[FI][FJ], four j of row lane % 16 a lane)
// that begins at (i0, j0) of C; buf: this wave's own LDS, PR rows of TJ floats, whose 16-byte
// chunks are permuted by the row (a lane writes one chunk of its row).
// Only a forward product has more to finish than alpha.  again(i, j, of): the sums of the block at (i, j) formed anew, for
// those that are not finite (kAgain).
template <typename TC, int FI, int FJ, int PR, bool kForward, bool kAgain, typename F>
__device__ __forceinline__ void finish(const Args &P, f32x4 (&acc)[FI][FJ], int i0, int j0, lds_char *buf, F again)
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
    bool bad = false;   // a sum of this wave is not finite
    if (kAgain) {
        float worst = 0.0f;
#pragma unroll
        for (int f = 0; f < FI; ++f)
#pragma unroll
            for (int g = 0; g < FJ; ++g)
#pragma unroll
                for (int k = 0; k < 4; ++k) worst = __builtin_fmaf(acc[f][g][k], 0.0f, worst);
        bad = __any(worst != 0.0f);
    }
    float bias[8] = {};
    if (kForward && P.bias)
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
        if (kAgain && bad) {   // by blocks; a lane's four sums stand where it wrote them
#pragma unroll 1
            for (int b = 0; b < PR / 16 * FJ; ++b) {
                const int bi = i0 + (f0 + b / FJ) * 16, bj = j0 + b % FJ * 16;
                auto *at = (__attribute__((address_space(3))) f32x4 *)(buf + (b / FJ * 16 + (lane & 15)) * kRow +
                                                                       (((b % FJ * 4 + (lane >> 4)) ^ (lane & kMask & 15)) << 4));
                f32x4 v = *at;
                bool again_of[4], some = false;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    again_of[k] = bi + (lane & 15) < P.I && bj + (lane >> 4) * 4 + k < P.J && v[k] * 0.0f != 0.0f;
                    some = some || again_of[k];
                }
                if (!__any(some)) continue;
                const f32x4 s = again(bi, bj, again_of);
#pragma unroll
                for (int k = 0; k < 4; ++k) v[k] = again_of[k] ? s[k] : v[k];
                *at = v;
            }
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        }
        for (int round = 0; round < kRounds; round += kU) {
            const int r0 = round * kRows + lane / kGroups, i_of = i0 + f0 * 16 + r0;
            const bool wide = n == 8;
            u32x4 res[kU][kV];
            if (kForward && wide && P.residual)
#pragma unroll
                for (int u = 0; u < kU; ++u)
#pragma unroll
                    for (int k = 0; k < kV; ++k)
                        if (i_of + u * kRows < P.I)
                            res[u][k] = ((const u32x4_any *)((const TC *)P.residual + (i_of + u * kRows) * P.ldr + j))[k];
            float v[kU * 8];
#pragma unroll
            for (int u = 0; u < kU; ++u) {
                const int r = r0 + u * kRows, key = r & kMask & 15;
                const auto *src = (const __attribute__((address_space(3))) f32x4 *)(buf + r * kRow);
                const f32x4 lo = src[(c >> 2) ^ key], hi = src[((c >> 2) + 1) ^ key];
#pragma unroll
                for (int k = 0; k < 4; ++k) v[u * 8 + k] = lo[k], v[u * 8 + 4 + k] = hi[k];
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
                            ((f32x4_any *)o)[0] = f32x4{v[u * 8], v[u * 8 + 1], v[u * 8 + 2], v[u * 8 + 3]};
                            ((f32x4_any *)o)[1] = f32x4{v[u * 8 + 4], v[u * 8 + 5], v[u * 8 + 6], v[u * 8 + 7]};
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
                    for (int k = 0; k < kV; ++k) ((u32x4_any *)o)[k] = w[k];
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
// 8192 x 4096 x 4096 at 256 x 256 tiles, by layout pair: 201-218, 196-206 and 182-200 us, card to
// card (1264-1370, 1332-1403 and 1377-1510 TFLOP/s), with two buffers of 64 k 228-257; the matrix
// instructions alone take 135.

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
    const int part = blockIdx.y, kb = part * P.k_part;
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
    if (P.parts > 1 && !joined<FI, FJ, 64 * kWaves>(P, d.acc, ti * P.tiles_j + tj, part, ti * BM + d.wi * TI)) return;
    // each wave has a buffer of its own
    constexpr int kOwn = TA::kBytes < TB::kBytes ? TA::kBytes : TB::kBytes, kFit = kOwn / (TJ * 4);
    static_assert(kWaves <= 8 && kFit >= 16, "room for one block row");
    constexpr int PR = kFit >= TI ? TI : kFit;
    lds_char *const own = wave == 0   ? (lds_char *)a0
                          : wave == 1 ? (lds_char *)a1
                          : wave == 2 ? (lds_char *)a2
                          : wave == 3 ? (lds_char *)a3
                          : wave == 4 ? (lds_char *)b0
                          : wave == 5 ? (lds_char *)b1
                          : wave == 6 ? (lds_char *)b2
                                      : (lds_char *)b3;
    finish<bf16, FI, FJ, PR, LA == K_ROWS && LB == K_ROWS, false>(P, d.acc, ti * BM + d.wi * TI, tj * BN + d.wj * TJ,
                                                                  own, [](int, int, const bool (&)[4]) { return f32x4{}; });
}

// One operand tile on its way through registers: 8-value chunks, loaded 16 bytes at a time at any
// alignment of the element.  Where a chunk may pass the end of its row (K_ROWS:
// the last k; K_COLS: the last row of the operand), bf16 values are loaded one at a time where the buffer ends too, as a
// word that is half in it would read as zero; of 32-bit values those past the last k are
// masked afterwards, and those past the last row reach only sums that are not stored.
template <typename T, int L, int R, int BK, int THREADS>
struct Chunks {
    using Tile = DirectTile<L, R, BK, THREADS / 64>;   // whose LDS layout the chunks follow
    static constexpr int kN = R * BK / 8 / THREADS;    // chunks of a lane
    static_assert(kN >= 1 && R * BK / 8 % THREADS == 0, "whole chunks");
    static constexpr int kSize = (int)sizeof(T), kWords = kSize * 2;   // registers of a chunk

    const char *base;
    long long ld;   // bytes
    int rows, K;
    int span;       // bytes of the buffer: of the rows before the tile's last one (K_ROWS), of one k (K_COLS)
    int off[kN];
    int at[kN];     // first k (K_COLS: first row) of a lane's chunk in the tile
    uint32_t reg[kN][kWords];

    __device__ __forceinline__ void init(const void *p, long long ld_elems, int row0, int n_rows, int n_k, int k0)
    {
        ld = ld_elems * kSize;
        rows = n_rows - row0;
        K = n_k;
        span = L == K_ROWS ? ((rows < R ? rows : R) - 1) * (int)ld : rows * kSize;
        base = (const char *)p + (L == K_ROWS ? row0 * ld + (long long)k0 * kSize : k0 * ld + (long long)row0 * kSize);
#pragma unroll
        for (int n = 0; n < kN; ++n) {
            const int slot = n * THREADS + threadIdx.x;
            const int r = slot / Tile::kChunks, c = (slot % Tile::kChunks) ^ Tile::key(r);
            at[n] = c * 8;
            off[n] = L == K_ROWS || at[n] < rows ? (int)(r * ld) + c * 8 * kSize : 0x7FFFFFF0;
        }
    }

    // Load the tile at k; past the end: an empty buffer, nothing is read.
    __device__ __forceinline__ void load(int k)
    {
        const int left = K - k;
        const char *p = L == K_ROWS ? base + (long long)k * kSize : base + k * ld;
        const int bytes = L == K_ROWS ? span + left * kSize : (left <= BK ? left - 1 : BK) * (int)ld + span;
        const int end = left <= 0 ? 0 : bytes;
        const auto rsrc = __builtin_amdgcn_make_buffer_rsrc((void *)p, 0, end, 0x00027000);
        const int stop = L == K_ROWS ? left : rows;   // values of the chunk's direction that exist
        // a K_COLS chunk that passes its row's end reads into the next k's row, until there is none
        const bool tail = kSize == 2 && (L == K_ROWS ? left < BK : rows < R && left <= BK);
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
                const uint32_t v = (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(rsrc, o, 0, 0);
                if (e & 1) reg[n][e / 2] |= v << 16;
                else reg[n][e / 2] = v;
            }
        }
    }

    // What a 32-bit chunk of the tile at k read past its row's last k becomes 0.
    __device__ __forceinline__ void mask(int k)
    {
        if (kSize == 2 || L == K_COLS || K - k >= BK) return;
#pragma unroll
        for (int n = 0; n < kN; ++n)
#pragma unroll
            for (int e = 0; e < 8; ++e) reg[n][e % kWords] = at[n] + e < K - k ? reg[n][e % kWords] : 0;
    }

    __device__ __forceinline__ void values(float (&x)[8], int n) const
    {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            if (kSize == 4) x[e] = __builtin_bit_cast(float, reg[n][e % kWords]);
            else x[e] = __builtin_bit_cast(float, e & 1 ? reg[n][e / 2] & 0xFFFF0000u : reg[n][e / 2] << 16);
        }
    }
};

// x as PLANES bf16 values each, chunk by chunk into LDS planes kPlane bytes apart.  A 32-bit value is the
// sum of its planes to 8 bits and a rounding a plane: x = h + m + l, each the rounding of what the
// ones before leave; exactly, with three, from 2^-109 (1.5e-33) up.  Below, the last planes fall under bf16's
// smallest magnitude, 2^-133, and x is off by up to 2^-134.
template <int PLANES, int kPlane>
__device__ __forceinline__ void split(lds_char *dst, float (&x)[8])
{
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

// A stored operand as planes.
template <typename T, int PLANES_, int L_, int R, int THREADS>
struct Stored {
    static constexpr int PLANES = PLANES_, L = L_, BK = 32, kPlane = R * BK * 2, kBytes = kPlane * PLANES;
    using C = Chunks<T, L, R, BK, THREADS>;
    using Tile = typename C::Tile;
    C c;

    __device__ __forceinline__ void init(const Args &P, bool second, int row0, int n_k, int k0)
    {
        if (second) c.init(P.b, P.ldb, row0, P.J, n_k, k0);
        else c.init(P.a, P.lda, row0, P.I, n_k, k0);
    }
    __device__ __forceinline__ void load(int k)
    {
        c.load(k);
    }
    __device__ __forceinline__ void mask(int k)
    {
        c.mask(k);
    }
    __device__ __forceinline__ void store(lds_char *to) const
    {
#pragma unroll
        for (int n = 0; n < C::kN; ++n) {
            lds_char *dst = to + (n * THREADS + threadIdx.x) * 16;
            if (C::kSize == 2) {
                *(__attribute__((address_space(3))) u32x4 *)dst =
                    u32x4{c.reg[n][0], c.reg[n][1], c.reg[n][2], c.reg[n][3]};
            } else {
                float x[8];
                c.values(x, n);
                split<PLANES, kPlane>(dst, x);
            }
        }
    }
};

// Eight k of one row: k0 + 8 (lane / 16) + 0..7 of row0 + lane % 16.
template <typename T, int L>
struct Piece {
    static constexpr int kSize = (int)sizeof(T), kWords = kSize * 2;
    uint32_t w[kWords];

    // rows and K: those of the operand.
    __device__ __forceinline__ void load(const void *p, long long ld_elems, int row0, int rows, int k0, int K)
    {
        const int lane = threadIdx.x & 63, r = lane & 15, q = (lane >> 4) * 8;
        const long long ld = ld_elems * kSize;
        const int left = K - k0, more = rows - row0;
        const char *base = (const char *)p + (L == K_ROWS ? row0 * ld + (long long)k0 * kSize : k0 * ld + (long long)row0 * kSize);
        const long long bytes = L == K_ROWS ? (more - 1) * ld + (long long)left * kSize : (left - 1) * ld + (long long)more * kSize;
        const int end = left <= 0 || more <= 0 ? 0 : bytes > 0x7FFFFFE0 ? 0x7FFFFFE0 : (int)bytes;
        const auto rsrc = __builtin_amdgcn_make_buffer_rsrc((void *)base, 0, end, 0x00027000);
        if (L == K_ROWS && left >= 32) {
            const int off = (int)(r * ld) + q * kSize;
#pragma unroll
            for (int h = 0; h < kWords / 4; ++h) {
                const u32x4 v = __builtin_amdgcn_raw_buffer_load_b128(rsrc, off + h * 16, 0, 0);
#pragma unroll
                for (int e = 0; e < 4; ++e) w[h * 4 + e] = v[e];
            }
            return;
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int off = L == K_ROWS ? (q + e < left ? (int)(r * ld) + (q + e) * kSize : 0x7FFFFFF0)
                                        : (r < more ? (int)((q + e) * ld) + r * kSize : 0x7FFFFFF0);
            if (kSize == 4) {
                w[e % kWords] = __builtin_amdgcn_raw_buffer_load_b32(rsrc, off, 0, 0);
            } else {
                const uint32_t v = (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(rsrc, off, 0, 0);
                if (e & 1) w[e / 2] |= v << 16;
                else w[e / 2] = v;
            }
        }
    }
    __device__ __forceinline__ float value(int e) const
    {
        if (kSize == 4) return __builtin_bit_cast(float, w[e % kWords]);
        return __builtin_bit_cast(float, e & 1 ? w[e / 2] & 0xFFFF0000u : w[e / 2] << 16);
    }
};

// The sums of the 16 x 16 block at (i, j) by themselves, by the fp32 matrix instruction from fp32 operands: for values
// whose split does not hold (infinities, and magnitudes that round up to one).  Of a NaN nothing more can come: the
// sums end where all that are wanted are.  Two steps are loaded before the first is used (four would take the registers
// of one wave in four).  2048^3: gradients with one sample of NaN 0.78 ms (finite 0.22), the forward with one NaN weight
// 0.28 (0.11), a layer that is all NaN 0.11 and 0.22.
template <class A, class B>
__device__ __forceinline__ f32x4 plain_block(const Args &P, int i, int j, const bool (&of)[4])
{
    constexpr int kAt = 2;
    f32x4 s = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 1
    for (int k0 = 0; k0 < P.K; k0 += 32 * kAt) {
        Piece<float, A::L> a[kAt];
        Piece<float, B::L> b[kAt];
#pragma unroll
        for (int n = 0; n < kAt; ++n) {   // steps past the end: empty buffers
            const int k = k0 + 32 * n < P.K ? k0 + 32 * n : P.K;
            a[n].load(P.a, P.lda, i, P.I, k, P.K);
            b[n].load(P.b, P.ldb, j, P.J, k, P.K);
        }
#pragma unroll
        for (int n = 0; n < kAt; ++n)
#pragma unroll
            for (int e = 0; e < 8; ++e) s = __builtin_amdgcn_mfma_f32_16x16x4f32(b[n].value(e), a[n].value(e), s, 0, 0, 0);
        bool open = false;
#pragma unroll
        for (int k = 0; k < 4; ++k) open = open || (of[k] && s[k] == s[k]);
        if (!__any(open)) break;
    }
    return s;
}

// A product whose operands A and B go through registers and are held in LDS as bf16 planes; of the
// products of planes those are formed that reach the sum's 24 bits: 6 for 3 x 3 planes, whose
// left-out ones are below 2^-24 of the product of magnitudes.  With BUF = 2 the split of step t + 1 and
// its way to LDS fall between step t's matrix instructions, at one barrier a step, and step t + 2 is
// on its way into registers; with BUF = 1 they come after, and two workgroups share a compute
// unit, so that one computes while the other stores.  (Two steps in registers instead of one
// gave nothing: 90 us for 2048^3 either way.)
template <class A, class B, typename TC, int BM, int BN, int WI, int WJ, int BUF, bool kForward>
struct Staged {
    static constexpr int BK = 32, kWaves = WI * WJ, kThreads = 64 * kWaves, TI = BM / WI, TJ = BN / WJ, FI = TI / 16,
                         FJ = TJ / 16, PA = A::PLANES, PB = B::PLANES, kMost = PA > PB ? PA : PB;
    static constexpr int kTurn = TI < 32 ? TI : 32;   // rows of a wave's part turned at once
    static constexpr int kTurnBytes = kTurn * TJ * 4, kTiles = A::kBytes + B::kBytes;
    static constexpr int kLds = kTiles * BUF > kWaves * kTurnBytes ? kTiles * BUF : kWaves * kTurnBytes;

    A ta;
    B tb;
    typename A::Tile fa_of;   // where a lane's fragments begin
    typename B::Tile fb_of;
    int wi, wj;
    f32x4 acc[FI][FJ];

    // Compute step t from here; step t + 1 is in the registers.
    __device__ __forceinline__ void step(lds_char *here, lds_char *next, int t)
    {
        ta.mask((t + 1) * BK);
        tb.mask((t + 1) * BK);
        bf16x8 fb[PB][FJ];
#pragma unroll
        for (int p = 0; p < PB; ++p)
#pragma unroll
            for (int g = 0; g < FJ; ++g)
                fb[p][g] = fb_of.fragment(here + A::kBytes + p * B::kPlane, wj * TJ + g * 16, 0);
#pragma unroll
        for (int f = 0; f < FI; ++f) {
#pragma unroll
            for (int p = PA - 1; p >= 0; --p) {   // small products first
                const bf16x8 fa = fa_of.fragment(here + p * A::kPlane, wi * TI + f * 16, 0);
#pragma unroll
                for (int q = PB - 1; q >= 0; --q) {
                    if (p + q >= kMost) continue;
#pragma unroll
                    for (int g = 0; g < FJ; ++g)
                        acc[f][g] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fb[q][g], fa, acc[f][g], 0, 0, 0);
                }
            }
            if (BUF == 2 && f == FI / 2 - 1) {
                ta.store(next);
                ta.load((t + 2) * BK);
            }
            if (BUF == 2 && f == FI - 1) {
                tb.store(next + A::kBytes);
                tb.load((t + 2) * BK);
            }
        }
        if (BUF == 1) {
            wait_lds();   // the fragments have arrived: the matrix instructions that take them may come after the barrier
            barrier();
            ta.store(here);
            tb.store(here + A::kBytes);
            ta.load((t + 2) * BK);
            tb.load((t + 2) * BK);
        }
        wait_lds();
        barrier();
    }

    __device__ __forceinline__ void run(const Args &P, int id, int part, lds_char *lds)
    {
        int ti, tj;
        tile_of(id, P.tiles_i, P.tiles_j, ti, tj);
        const int kb = part * P.k_part, kn = P.K - kb < P.k_part ? P.K - kb : P.k_part;
        ta.init(P, false, ti * BM, kn, kb);
        tb.init(P, true, tj * BN, kn, kb);
        fa_of.init_fragment();
        fb_of.init_fragment();
        const int wave = threadIdx.x >> 6;
        wi = wave / WJ, wj = wave % WJ;
#pragma unroll
        for (int f = 0; f < FI; ++f)
#pragma unroll
            for (int g = 0; g < FJ; ++g) acc[f][g] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        lds_char *const other = lds + (BUF - 1) * kTiles;
        ta.load(0);
        tb.load(0);
        ta.mask(0);
        tb.mask(0);
        ta.store(lds);
        tb.store(lds + A::kBytes);
        ta.load(BK);
        tb.load(BK);
        wait_lds();
        barrier();
        const int steps = (kn + BK - 1) / BK;
        for (int t = 0; t < steps; ++t) step(t & 1 ? other : lds, t & 1 ? lds : other, t);
        if (P.parts > 1 && !joined<FI, FJ, kThreads, (PA > 1 || PB > 1)>(P, acc, ti * P.tiles_j + tj, part, ti * BM + wi * TI)) return;
        finish<TC, FI, FJ, kTurn, kForward, (PA > 1 || PB > 1)>(P, acc, ti * BM + wi * TI, tj * BN + wj * TJ,
                                                                lds + wave * kTurnBytes,
                                                                [&](int i, int j, const bool (&of)[4]) { return plain_block<A, B>(P, i, j, of); });
    }
};

// Bound by LDS, the matrix cores and the split's arithmetic about equally (a step of two workgroups on a compute unit:
// 2.5 us; its LDS traffic alone 1.4, its matrix instructions 1.4, its split 0.9).  2048^3 in fp32, each product alone in
// a loop: forward 95 to 100 us, dx and dw 88 to 90 (171 to 193 TFLOP/s); one after another in a training step's kernel
// trace, with bias, residual and z: 109 to 111, 98 to 100 and 101 to 103.  4096^3: 640 to 655 us, 210 TFLOP/s.
template <typename T, int PLANES, int LA, int LB, int BM, int BN, int WI, int WJ, int BUF>
__global__ __launch_bounds__(64 * WI *WJ, 2) void k_product_staged(Args P)
{
    using S = Staged<Stored<T, PLANES, LA, BM, 64 * WI * WJ>, Stored<T, PLANES, LB, BN, 64 * WI * WJ>, T, BM, BN, WI, WJ,
                     BUF, LA == K_ROWS && LB == K_ROWS>;
    __shared__ __attribute__((aligned(1024))) char lds[S::kLds];
    S s;
    s.run(P, blockIdx.x, blockIdx.y, (lds_char *)lds);
}

// ---- small products ----
//
// Where latency counts, or one operand has few rows: tiles of 16 FI x 16, whose k the waves of
// a workgroup share out.  Fragments come straight from memory (each value is used by one or FI
// matrix instructions only, so LDS would add a trip and save nothing), kAt steps of 32 k
// before the first is used; the waves' sums meet in LDS and are added in their order.
// fp32, and dz formed in fp32, use the fp32 matrix instruction: nothing is rounded or split.
// Bound by the waits for memory: fp32 1 x 64 -> 4 takes 3.5 us, 1000 x 784 -> 20 6.2, bf16 1 x 4096 -> 4096 in a loop
// of calls 8.0 with its 32 MB of weights in the last-level cache (4.2 TB/s) and 10.1 from HBM (3.3; 24 such weights in turn);
// all gradients of 64 x 12 -> 64 6.3.

// dz of a piece: dy, scaled by act'(z) (alpha is the epilogue's); without an activation, dy alone.
template <typename T, int L>
struct SlopePiece {
    Piece<T, L> d;
    Piece<float, L> z;
    float x[8];

    __device__ __forceinline__ void load(const Args &P, int row0, int k0)
    {
        d.load(P.a, P.lda, row0, P.I, k0, P.K);
        if (P.act != HQML_ACT_NONE) z.load(P.z, L == K_ROWS ? P.K : P.I, row0, P.I, k0, P.K);
    }
    __device__ __forceinline__ void form(int act)
    {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = z.value(e);
        if (act != HQML_ACT_NONE) {
            slope<sizeof(T) == 2>(x, act);
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] *= d.value(e);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = d.value(e);
        }
    }
    __device__ __forceinline__ float value(int e) const { return x[e]; }
};

// One value of a small product, finished.
template <typename T, bool kForward>
__device__ __forceinline__ void small_value(const Args &P, float sum, int i, int j)
{
    if (i >= P.I) return;
    if (!kForward) {
        if (j < P.J) narrow(sum * P.alpha, ((T *)P.c)[i * P.ldc + j]);
        else if (j == P.J && P.ones) narrow(sum * P.alpha, ((T *)P.ones)[i]);
        return;
    }
    if (j >= P.J) return;
    float v[1] = {sum};
    if (P.bias) v[0] += widen(((const T *)P.bias)[j]);
    if (P.z) P.z[(long long)i * P.J + j] = v[0];
    activate<sizeof(T) == 2>(v, P.act);
    float y = v[0] * P.alpha;
    if (P.residual) y += widen(((const T *)P.residual)[i * P.ldr + j]);
    narrow(y, ((T *)P.c)[i * P.ldc + j]);
}

// The waves' sums of a 16 FI x 16 tile, added and finished; split over k, parts meet as joined()'s do.
template <typename T, int FI, bool kForward>
__device__ __forceinline__ void small_finish(const Args &P, f32x4 (&acc)[FI], int tile, int i0, int j0, float *lds)
{
    __shared__ unsigned taken;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
#pragma unroll
    for (int f = 0; f < FI; ++f)   // [wave][row][16 columns]
        *(f32x4 *)(lds + (wave * FI * 16 + f * 16 + (lane & 15)) * 16 + (lane >> 4) * 4) = acc[f];
    __syncthreads();
    float *all = P.part + (long long)tile * P.parts * (FI * 256);
    for (int e = threadIdx.x; e < FI * 256; e += blockDim.x) {
        float sum = 0.0f;
        for (int q = 0; q < waves; ++q) sum += lds[q * FI * 256 + e];
        if (P.parts == 1) small_value<T, kForward>(P, sum, i0 + (e >> 4), j0 + (e & 15));
        else if (i0 + (e >> 4) < P.I)
            __hip_atomic_store(all + blockIdx.y * (FI * 256) + e, sum, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    if (P.parts == 1) return;
    wait_loads<0>();   // and stores: this wave's have arrived
    __syncthreads();   // every wave's have
    if (threadIdx.x == 0)
        taken = __hip_atomic_fetch_add(P.ticket + tile, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    __syncthreads();
    if (taken != (unsigned)P.parts - 1) return;
    for (int e = threadIdx.x; e < FI * 256; e += blockDim.x) {
        if (i0 + (e >> 4) >= P.I) break;
        float sum = 0.0f;
#pragma unroll 4
        for (int p = 0; p < P.parts; ++p)
            sum += __hip_atomic_load(all + p * (FI * 256) + e, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        small_value<T, kForward>(P, sum, i0 + (e >> 4), j0 + (e & 15));
    }
    if (threadIdx.x == 0) __hip_atomic_store(P.ticket + tile, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// k of this wave in [begin, end): [first, last), a multiple of 32 long unless it ends with the range.
__device__ __forceinline__ void small_share(int begin, int end, int &first, int &last)
{
    const int waves = blockDim.x >> 6, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int steps = (end - begin + 31) >> 5, q = steps / waves, r = steps % waves;
    first = begin + (wave * q + (wave < r ? wave : r)) * 32;
    last = first + (q + (wave < r ? 1 : 0)) * 32;
    if (last > end) last = end;
}

// Forward: C = A B^T, both with k along their rows.
template <typename T, int FI>
__global__ __launch_bounds__(FI == 1 ? 1024 : 512) void k_small_forward(Args P)
{
    extern __shared__ float small_lds[];
    constexpr int kAt = FI == 4 ? 2 : 4;
    const int i0 = blockIdx.x % P.tiles_i * (16 * FI), j0 = blockIdx.x / P.tiles_i * 16;
    f32x4 acc[FI] = {};
    int first, last;
    const int begin = blockIdx.y * P.k_part;
    small_share(begin, P.K - begin < P.k_part ? P.K : begin + P.k_part, first, last);
    for (int k0 = first; k0 < last; k0 += 32 * kAt) {
        Piece<T, K_ROWS> a[kAt][FI], b[kAt];
#pragma unroll
        for (int n = 0; n < kAt; ++n) {   // steps past the share: empty buffers, nothing is read
            const int k = k0 + 32 * n < last ? k0 + 32 * n : P.K;
            b[n].load(P.b, P.ldb, j0, P.J, k, P.K);
#pragma unroll
            for (int f = 0; f < FI; ++f) a[n][f].load(P.a, P.lda, i0 + f * 16, P.I, k, P.K);
        }
#pragma unroll
        for (int n = 0; n < kAt; ++n) {
            if (sizeof(T) == 2) {
#pragma unroll
                for (int f = 0; f < FI; ++f) {
                    bf16x8 va, vb;
                    __builtin_memcpy(&va, a[n][f].w, 16);
                    __builtin_memcpy(&vb, b[n].w, 16);
                    acc[f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(vb, va, acc[f], 0, 0, 0);
                }
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e)
#pragma unroll
                    for (int f = 0; f < FI; ++f)
                        acc[f] = __builtin_amdgcn_mfma_f32_16x16x4f32(b[n].value(e), a[n][f].value(e), acc[f], 0, 0, 0);
            }
        }
    }
    small_finish<T, FI, true>(P, acc, blockIdx.x, i0, j0, small_lds);
}

// One gradient product: C = dz B with B's k across its rows; dz's layout L.  A column of ones after B's
// last gives dz's row sums.
template <typename T, int FI, int L>
__device__ __forceinline__ void small_gradient(const Args &P, int id, float *lds)
{
    constexpr int kAt = FI == 1 ? 2 : 1;
    const int i0 = id % P.tiles_i * (16 * FI), j0 = id / P.tiles_i * 16;
    const bool one = P.ones && j0 + (int)(threadIdx.x & 15) == P.J;
    f32x4 acc[FI] = {};
    int first, last;
    small_share(0, P.K, first, last);
    for (int k0 = first; k0 < last; k0 += 32 * kAt) {
        SlopePiece<T, L> a[kAt][FI];
        Piece<T, K_COLS> b[kAt];
#pragma unroll
        for (int n = 0; n < kAt; ++n) {
            const int k = k0 + 32 * n < last ? k0 + 32 * n : P.K;
            b[n].load(P.b, P.ldb, j0, P.J, k, P.K);
#pragma unroll
            for (int f = 0; f < FI; ++f) a[n][f].load(P, i0 + f * 16, k);
        }
#pragma unroll
        for (int n = 0; n < kAt; ++n)
#pragma unroll
            for (int f = 0; f < FI; ++f) {
                a[n][f].form(P.act);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    acc[f] = __builtin_amdgcn_mfma_f32_16x16x4f32(one ? 1.0f : b[n].value(e), a[n][f].value(e), acc[f], 0, 0, 0);
            }
    }
    small_finish<T, FI, false>(P, acc, id, i0, j0, lds);
}

// Small gradients in one launch: dx = dz w from the first workgroups, dw = dz^T x with db as a column
// of ones from the others.  dz is formed anew by every tile that takes it, and never rounded.
template <typename T, int FI>
__global__ __launch_bounds__(512) void k_small_gradients(Args dx, Args dw)
{
    extern __shared__ float small_lds[];
    const int tx = dx.tiles_i * dx.tiles_j, id = blockIdx.x;
    if (id < tx) small_gradient<T, FI, K_ROWS>(dx, id, small_lds);
    else small_gradient<T, FI, K_COLS>(dw, id - tx, small_lds);
}

// The kernels of one operand type, for a layout pair (K_ROWS, K_ROWS), (K_ROWS, K_COLS) or
// (K_COLS, K_COLS).  direct: both bf16 operands' rows allow 16-byte access to LDS; TILE_256 needs it.
hipError_t launch_bf16(const Args &a, int la, int lb, bool direct, Shape shape, hipStream_t s);
hipError_t launch_fp32(const Args &a, int la, int lb, Shape shape, hipStream_t s);
// Small products, in tiles of 16 fi x 16 by `waves` waves (fi = 1 or 4; forward also 2); either gradient may have
// no tiles.
hipError_t launch_small_forward(const Args &a, bool is_bf16, int fi, int waves, hipStream_t s);
hipError_t launch_small_gradients(const Args &dx, const Args &dw, bool is_bf16, int fi, int waves, hipStream_t s);

}  // namespace gemm
}  // namespace hqml
