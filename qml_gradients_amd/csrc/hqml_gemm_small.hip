// Small products, both types.
#include "hqml_gemm.hpp"

namespace hqml {
namespace gemm {

template <typename T>
void run_forward(const Args &a, int fi, dim3 grid, unsigned threads, size_t lds, hipStream_t s)
{
    if (fi == 1) k_small_forward<T, 1><<<grid, threads, lds, s>>>(a);
    else if (fi == 2) k_small_forward<T, 2><<<grid, threads, lds, s>>>(a);
    else k_small_forward<T, 4><<<grid, threads, lds, s>>>(a);
}

hipError_t launch_small_forward(const Args &a, bool is_bf16, int fi, int waves, hipStream_t s)
{
    const dim3 grid((unsigned)a.tiles_i * (unsigned)a.tiles_j, (unsigned)a.parts);
    const size_t lds = (size_t)waves * fi * 1024;
    if (is_bf16) run_forward<bf16>(a, fi, grid, 64 * (unsigned)waves, lds, s);
    else run_forward<float>(a, fi, grid, 64 * (unsigned)waves, lds, s);
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
