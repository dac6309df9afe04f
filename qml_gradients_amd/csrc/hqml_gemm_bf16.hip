// Products of bf16 operands.
#include "hqml_gemm.hpp"

namespace hqml {
namespace gemm {
namespace {

template <int LA, int LB>
void run(const Args &a, bool wide, Shape shape, dim3 grid, hipStream_t s)
{
    if (!wide) {
        if (shape == TILE_64) k_product_staged<bf16, 1, LA, bf16, 1, LB, bf16, 64, 64, 32, 2, 2, false><<<grid, 256, 0, s>>>(a);
        else k_product_staged<bf16, 1, LA, bf16, 1, LB, bf16, 128, 128, 32, 2, 2, false><<<grid, 256, 0, s>>>(a);
        return;
    }
    if (shape == TILE_64) k_product_direct<LA, LB, 64, 64, 64, 2, 2><<<grid, 256, 0, s>>>(a);
    else if (shape == TILE_128) k_product_direct<LA, LB, 128, 128, 64, 2, 2><<<grid, 256, 0, s>>>(a);
    else k_product_direct<LA, LB, 256, 256, 64, 2, 4><<<grid, 512, 0, s>>>(a);
}

}  // namespace

hipError_t launch_bf16(const Args &a, int la, int lb, bool wide, Shape shape, int parts, hipStream_t s)
{
    const dim3 grid((unsigned)a.tiles_i * (unsigned)a.tiles_j, (unsigned)parts);
    if (la == K_ROWS && lb == K_ROWS) run<K_ROWS, K_ROWS>(a, wide, shape, grid, s);
    else if (la == K_ROWS) run<K_ROWS, K_COLS>(a, wide, shape, grid, s);
    else run<K_COLS, K_COLS>(a, wide, shape, grid, s);
    return hipGetLastError();
}

}  // namespace gemm
}  // namespace hqml
