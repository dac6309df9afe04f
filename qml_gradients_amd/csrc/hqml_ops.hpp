// Internal interface between the entry points of the dense layer and AdamW (hqml_ops.cpp)
// and their kernels (hqml_dense.hip, hqml_adamw.hip).  Not part of the public ABI.
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>

#include "../../include/hqml.h"

namespace hqml {

struct DenseForward {
    int M, K, N;
    const void *x, *w, *bias, *residual;
    long long ldx, ldw, ldr, ldy;
    void *y;
    float *z;
    int act;
    float alpha;
};

struct DenseBackward {
    int M, K, N;
    const void *dy, *x, *w;
    const float *z;
    long long lddy, ldx, ldw, lddx;
    void *dx, *dw, *db;
    int act;
    float alpha;
};

// Parts of a handle's workspace (byte counts and, once reserved, addresses).
struct DenseWorkspace {
    size_t dz_bytes = 0;     // gradient at z in dtype, rows of N (bf16: the next multiple of eight)
    size_t rows_bytes = 0;   // partial row sums of dz, fp32
    size_t part_bytes = 0;   // partial sums of products split over k, fp32
    size_t ticket_bytes = 0; // one counter a tile of them, 0 between calls
    size_t pad_bytes = 0;    // bf16 copies of x and w in aligned rows, where in_features does not allow 16-byte ones
    void *dz = nullptr, *pad = nullptr;
    float *rows = nullptr;
    float *part = nullptr;
    unsigned *ticket = nullptr;
};

DenseWorkspace dense_workspace(const hqml_dense_config &cfg);
hipError_t launch_dense_forward(const DenseForward &a, int dtype, const DenseWorkspace &ws, hipStream_t s);
hipError_t launch_dense_backward(const DenseBackward &a, int dtype, const DenseWorkspace &ws, hipStream_t s);

// One AdamW launch takes this many tensors in its kernel arguments.
constexpr int kAdamwTensors = 48;

struct AdamwScalars {
    double decay;     // lr weight_decay
    double b1, c1;    // beta1, 1 - beta1
    double b2, c2;
    double inv_root;  // 1 / sqrt(1 - beta2^step)
    double eps;
    double size;      // lr / (1 - beta1^step)
};

hipError_t launch_adamw(const hqml_adamw_config &cfg, const AdamwScalars &k, int n, const hqml_adamw_tensor *t,
                        hipStream_t s);

}  // namespace hqml
