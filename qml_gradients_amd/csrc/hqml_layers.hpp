// Internal interface between the entry points of the 8-bit dense layer, group norm and Muon (hqml_layers.cpp) and their
// kernels (hqml_dense8.hip, hqml_norm.hip, hqml_muon.hip).  Not part of the public ABI.
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/hqml.h"

namespace hqml {

// ---- dense layer in 8-bit integers ----

struct Dense8Forward {
    int M, K, N;
    const void *x;
    const int8_t *codes;   // [N][ldw], rows of a multiple of sixteen
    const float *scales;   // [N]
    const void *bias, *residual;
    long long ldx, ldw, ldr, ldy;
    void *y;
    int act;
    float alpha;
};

struct Scales8 {
    const float *x, *w;
};

struct Dense8Workspace {
    size_t codes_bytes = 0;    // x's codes, rows of the next multiple of sixteen
    size_t scales_bytes = 0;   // and their scales
    size_t part_bytes = 0;     // partial sums of products split over k, fp32
    size_t ticket_bytes = 0;   // one counter a tile of them, 0 between calls
    int8_t *codes = nullptr;
    float *scales = nullptr;
    float *part = nullptr;
    unsigned *ticket = nullptr;
};

Dense8Workspace dense8_workspace(const hqml_dense_config &cfg);
hipError_t launch_dense8_forward(const Dense8Forward &a, int dtype, const Dense8Workspace &ws, hipStream_t s);
hipError_t launch_quantise_rows(const void *x, long long ldx, long long rows, int K, int dtype, int8_t *codes, long long ldc,
                                float *scales, hipStream_t s);

// ---- group norm ----

struct NormCall {
    int B, S, C, G;
    const void *x, *gamma, *beta;
    long long ldx, ldy;          // elements from one position to the next
    void *y;                     // forward
    float *mean, *rstd;          // [B][G]; forward: written, or null
    const void *dy;              // backward
    long long lddy, lddx;
    void *dx, *dgamma, *dbeta;
    int act;
    float eps;
};

struct NormWorkspace {
    size_t part_bytes = 0;     // partial statistics or sums
    size_t group_bytes = 0;    // statistics or means of each sample's groups
    size_t ticket_bytes = 0;   // one counter a sample, 0 between calls
    float *part = nullptr, *group = nullptr;
    unsigned *ticket = nullptr;
};

NormWorkspace norm_workspace(const hqml_norm_config &cfg);
// Allows the kernels the LDS they take, on the current device.
hipError_t configure_norm(int dtype);
hipError_t launch_norm_forward(const NormCall &a, int dtype, const NormWorkspace &ws, hipStream_t s);
hipError_t launch_norm_backward(const NormCall &a, int dtype, const NormWorkspace &ws, hipStream_t s);

// ---- Muon ----

size_t muon_workspace(const hqml_muon_config &cfg, int n, const hqml_muon_tensor *t);
hipError_t launch_muon(const hqml_muon_config &cfg, int n, const hqml_muon_tensor *t, void *workspace, hipStream_t s);

}  // namespace hqml
