// Products of fp32 operands, each held as three bf16 planes: the matrix cores multiply bf16 at
// sixteen times their fp32 rate, so six products of planes cost three eighths of one fp32 product.
#include "hqml_gemm.hpp"

namespace hqml {
namespace gemm {
namespace {

template <int LA, int LB, bool WIDE>
void run(const Args &a, Shape shape, dim3 grid, hipStream_t s)
{
    if (shape == TILE_64) k_product_staged<float, 3, LA, float, 3, LB, float, 64, 64, 32, 2, 2, WIDE><<<grid, 256, 0, s>>>(a);
    else k_product_staged<float, 3, LA, float, 3, LB, float, 128, 128, 32, 2, 2, WIDE><<<grid, 256, 0, s>>>(a);
}

template <bool WIDE>
void run(const Args &a, int la, int lb, Shape shape, dim3 grid, hipStream_t s)
{
    if (la == K_ROWS && lb == K_ROWS) run<K_ROWS, K_ROWS, WIDE>(a, shape, grid, s);
    else if (la == K_ROWS) run<K_ROWS, K_COLS, WIDE>(a, shape, grid, s);
    else run<K_COLS, K_COLS, WIDE>(a, shape, grid, s);
}

}  // namespace

hipError_t launch_fp32(const Args &a, int la, int lb, bool wide, Shape shape, int parts, hipStream_t s)
{
    const dim3 grid((unsigned)a.tiles_i * (unsigned)a.tiles_j, (unsigned)parts);
    if (wide) run<true>(a, la, lb, shape, grid, s);
    else run<false>(a, la, lb, shape, grid, s);
    return hipGetLastError();
}

}  // namespace gemm
}  // namespace hqml
