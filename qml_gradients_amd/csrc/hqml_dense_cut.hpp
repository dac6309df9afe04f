// Which kernel runs a product of the dense layer, and how it is cut.  Host code without a device call: a test compiles it
// by itself.
#pragma once
#include <stddef.h>

#include <algorithm>

namespace hqml {
namespace gemm {

// Tile shapes a product can be run with.
enum Shape { TILE_64, TILE_128, TILE_256, TILE_64x32, TILE_32x64 };
constexpr int kSides[][2] = {{64, 64}, {128, 128}, {256, 256}, {64, 32}, {32, 64}};   // rows, columns

inline int ceil_div(int a, int b) { return (a + b - 1) / b; }

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

inline Cut best_cut(int I, int J, int K, size_t elem, const TileCost *cost, int n, const MemoryCost &m)
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

inline Cut best_cut(int I, int J, int K, size_t elem, bool direct)
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

inline SmallCut small_cut(int I, int J, int K, size_t elem, bool words)
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
inline SmallCut small_gradients_cut(int M, int N, int K, size_t elem, bool words)
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
inline float slope_us(int M, int N, size_t elem)
{
    return 6.0f + (float)M * N * (4 + 2 * elem) / 5e6f;
}

inline float pad_us(int rows, int K)
{
    return rows ? 4.0f + (float)rows * K * 4 / 4.5e6f : 0.0f;
}

// A forward call.  What is known of its operands: whether their rows can be loaded straight into LDS (bf16), and whether
// they begin on whole words; pad: there is room for copies in aligned rows.
struct ForwardChoice {
    bool small;         // k_small_forward, cut as `few`; else tiles, cut as `tiles`
    SmallCut few;
    Cut tiles;
    bool direct;        // bf16 tiles loaded straight into LDS
    bool copy_x, copy_w;   // copied first (direct only)
};

inline ForwardChoice choose_forward(int M, int K, int N, size_t elem, bool x_straight, bool w_straight, bool words, bool pad)
{
    ForwardChoice f{};
    f.tiles = best_cut(M, N, K, elem, false);
    if (elem == 2) {
        const int copies = (x_straight ? 0 : M) + (w_straight ? 0 : N);   // rows
        Cut d = best_cut(M, N, K, 2, true);
        d.us += pad_us(copies, K);
        if (!copies || (pad && d.us < f.tiles.us)) f.direct = true, f.tiles = d, f.copy_x = !x_straight, f.copy_w = !w_straight;
    }
    f.few = small_cut(M, N, K, elem, words);
    f.small = f.few.us <= f.tiles.us;
    return f;
}

// The gradients of a call: dx = dz w and dw = dz^T x.  act: whether dz has a slope in it; room: there is an array for dz.
struct BackwardChoice {
    bool small;         // k_small_gradients, cut as `few`; else tiles
    SmallCut few;
    Cut dx, dw;
    bool direct;
    bool copy_x, copy_w;
    bool form;          // dz is formed in memory
};

inline BackwardChoice choose_backward(int M, int K, int N, size_t elem, bool act, bool want_dx, bool want_dw, bool dy_straight,
                                      bool x_straight, bool w_straight, bool words, bool room, bool pad)
{
    BackwardChoice b{};
    b.dx = best_cut(M, K, N, elem, false), b.dw = best_cut(N, K, M, elem, false);
    b.form = act;
    if (elem == 2) {
        const bool x_copy = !x_straight && want_dw, w_copy = !w_straight && want_dx;
        const int copies = (x_copy ? M : 0) + (w_copy ? N : 0);   // rows
        const Cut dx = best_cut(M, K, N, 2, true), dw = best_cut(N, K, M, 2, true);
        const float us = pad_us(copies, K) + (act || dy_straight ? 0.0f : pad_us(M, N));
        if ((act || dy_straight || room) && (!copies || pad) && dx.us + dw.us + us < b.dx.us + b.dw.us) {
            b.direct = true, b.copy_x = x_copy, b.copy_w = w_copy;
            b.dx = dx, b.dw = dw, b.dx.us += us;
            b.form = act || !dy_straight;   // dz in rows of a multiple of eight
        }
    }
    b.few = small_gradients_cut(M, N, K, elem, words);
    b.small = b.few.us <= slope_us(M, N, elem) + b.dx.us + b.dw.us;
    return b;
}

}  // namespace gemm
}  // namespace hqml
