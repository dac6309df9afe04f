// Small products, both types.
#include "hqml_gemm.hpp"

namespace hqml {
namespace gemm {

hipError_t launch_small_forward(const Args &a, bool is_bf16, int fi, int waves, hipStream_t s)
{
    const unsigned grid = (unsigned)a.tiles_i * (unsigned)a.tiles_j, threads = 64 * (unsigned)waves;
    const size_t lds = (size_t)waves * fi * 1024;
    if (is_bf16) {
        if (fi == 1) k_small_forward<bf16, 1><<<grid, threads, lds, s>>>(a);
        else k_small_forward<bf16, 4><<<grid, threads, lds, s>>>(a);
    } else {
        if (fi == 1) k_small_forward<float, 1><<<grid, threads, lds, s>>>(a);
        else k_small_forward<float, 4><<<grid, threads, lds, s>>>(a);
    }
    return hipGetLastError();
}

hipError_t launch_small_gradients(const Args &dx, const Args &dw, bool is_bf16, int fi, int waves, hipStream_t s)
{
    const unsigned grid = (unsigned)(dx.tiles_i * dx.tiles_j + dw.tiles_i * dw.tiles_j), threads = 64 * (unsigned)waves;
    const size_t lds = (size_t)waves * fi * 1024;
    if (is_bf16) {
        if (fi == 1) k_small_gradients<bf16, 1><<<grid, threads, lds, s>>>(dx, dw);
        else k_small_gradients<bf16, 4><<<grid, threads, lds, s>>>(dx, dw);
    } else {
        if (fi == 1) k_small_gradients<float, 1><<<grid, threads, lds, s>>>(dx, dw);
        else k_small_gradients<float, 4><<<grid, threads, lds, s>>>(dx, dw);
    }
    return hipGetLastError();
}

}  // namespace gemm
}  // namespace hqml
