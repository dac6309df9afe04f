// Products of fp32 operands, each held as three bf16 planes: the matrix cores multiply bf16 at
// sixteen times their fp32 rate, so six products of planes cost three eighths of one fp32 product.
#include "hqml_gemm.hpp"

namespace hqml {
namespace gemm {
namespace {

// 128 x 128 tiles: two LDS buffers where every workgroup has a compute unit to itself (2048^3, 256 of them: 94 us against
// 102), one where two share it (432 of 1500 x 1500 x 3000 in three parts: 91 against 99; 4096 x 4096 x 1024: 180 against 191).
// Up to 32 rows or columns: half the matrix instructions of a 64 x 64 tile (8544 x 24 x 7504: 56 us, 4.6 TB/s, against 72;
// 24 x 7504 x 8544, both across k: 51 against 69).
template <int LA, int LB>
void run(const Args &a, Shape shape, dim3 grid, hipStream_t s)
{
    if (shape == TILE_64) k_product_staged<float, 3, LA, LB, 64, 64, 2, 2, 2><<<grid, 256, 0, s>>>(a);
    else if (shape == TILE_64x32) k_product_staged<float, 3, LA, LB, 64, 32, 2, 1, 1><<<grid, 128, 0, s>>>(a);
    else if (shape == TILE_32x64) k_product_staged<float, 3, LA, LB, 32, 64, 1, 2, 1><<<grid, 128, 0, s>>>(a);
    else if (grid.x * grid.y <= 256) k_product_staged<float, 3, LA, LB, 128, 128, 2, 4, 2><<<grid, 512, 0, s>>>(a);
    else k_product_staged<float, 3, LA, LB, 128, 128, 2, 4, 1><<<grid, 512, 0, s>>>(a);
}

}  // namespace

hipError_t launch_fp32(const Args &a, int la, int lb, Shape shape, hipStream_t s)
{
    const dim3 grid((unsigned)a.tiles_i * (unsigned)a.tiles_j, (unsigned)a.parts);
    if (la == K_ROWS && lb == K_ROWS) run<K_ROWS, K_ROWS>(a, shape, grid, s);
    else if (la == K_ROWS) run<K_ROWS, K_COLS>(a, shape, grid, s);
    else run<K_COLS, K_COLS>(a, shape, grid, s);
    return hipGetLastError();
}

}  // namespace gemm
}  // namespace hqml
