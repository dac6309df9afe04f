// Products of bf16 operands.
#include "hqml_gemm.hpp"

namespace hqml {
namespace gemm {
namespace {

template <int LA, int LB>
void run(const Args &a, bool direct, Shape shape, dim3 grid, hipStream_t s)
{
    if (!direct) {
        if (shape == TILE_64) k_product_staged<bf16, 1, LA, LB, 64, 64, 2, 2, 2><<<grid, 256, 0, s>>>(a);
        else k_product_staged<bf16, 1, LA, LB, 128, 128, 2, 4, 2><<<grid, 512, 0, s>>>(a);
        return;
    }
    // 256 x 256: waves of 64 x 128 where both operands lie along k (218 us against 231 for
    // 8192 x 4096 x 4096), of 128 x 64 elsewhere (206 and 200 against 216 and 212)
    constexpr int WI = LA == K_ROWS && LB == K_ROWS ? 4 : 2;
    if (shape == TILE_64) k_product_direct<LA, LB, 64, 64, 32, 2, 2><<<grid, 256, 0, s>>>(a);
    else if (shape == TILE_128) k_product_direct<LA, LB, 128, 128, 32, 2, 2><<<grid, 256, 0, s>>>(a);
    else k_product_direct<LA, LB, 256, 256, 32, WI, 8 / WI><<<grid, 512, 0, s>>>(a);
}

}  // namespace

hipError_t launch_bf16(const Args &a, int la, int lb, bool direct, Shape shape, hipStream_t s)
{
    const dim3 grid((unsigned)a.tiles_i * (unsigned)a.tiles_j, (unsigned)a.parts);
    if (la == K_ROWS && lb == K_ROWS) run<K_ROWS, K_ROWS>(a, direct, shape, grid, s);
    else if (la == K_ROWS) run<K_ROWS, K_COLS>(a, direct, shape, grid, s);
    else run<K_COLS, K_COLS>(a, direct, shape, grid, s);
    return hipGetLastError();
}

}  // namespace gemm
}  // namespace hqml
