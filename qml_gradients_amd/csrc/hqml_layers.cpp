// Entry points of the 8-bit dense layer, group norm and Muon: argument checks, the handles' workspaces, and the launches.
// Nothing is queued before every argument has passed, and no exception leaves an entry point.
#include <hip/hip_runtime.h>
#include <math.h>

#include <algorithm>
#include <cstdio>
#include <new>
#include <string>
#include <vector>

#include "../../include/hqml.h"
#include "hqml_entry.hpp"
#include "hqml_layers.hpp"

using namespace hqml;

struct hqml_dense8 {
    hqml_dense_config cfg{};
    Dense8Workspace ws;
    hipStream_t stream = nullptr;
    void *reserved = nullptr;
    std::string err;
};

struct hqml_norm {
    hqml_norm_config cfg{};
    NormWorkspace ws;
    hipStream_t stream = nullptr;
    void *reserved = nullptr;
    std::string err;
};

namespace {

size_t total_bytes(const Dense8Workspace &ws)
{
    return up256(ws.codes_bytes) + up256(ws.scales_bytes) + up256(ws.part_bytes) + up256(ws.ticket_bytes);
}

size_t total_bytes(const NormWorkspace &ws)
{
    return up256(ws.part_bytes) + up256(ws.group_bytes) + up256(ws.ticket_bytes);
}

// Hands out a reservation.
class Taker {
public:
    explicit Taker(void *p) : at_(static_cast<char *>(p)) {}
    template <typename T>
    T *take(size_t bytes)
    {
        char *here = at_;
        at_ += up256(bytes);
        return bytes ? reinterpret_cast<T *>(here) : nullptr;
    }

private:
    char *at_;
};

void place(Dense8Workspace &ws, void *p)
{
    Taker t(p);
    ws.codes = t.take<int8_t>(ws.codes_bytes);
    ws.scales = t.take<float>(ws.scales_bytes);
    ws.part = t.take<float>(ws.part_bytes);
    ws.ticket = t.take<unsigned>(ws.ticket_bytes);
}

void place(NormWorkspace &ws, void *p)
{
    Taker t(p);
    ws.part = t.take<float>(ws.part_bytes);
    ws.group = t.take<float>(ws.group_bytes);
    ws.ticket = t.take<unsigned>(ws.ticket_bytes);
}

// A handle of cfg with its workspace ws reserved on the current device.
template <class H, class C, class W>
int make(const C &cfg, W ws, H **out)
{
    size_t free_b = 0, all_b = 0;
    hipError_t e = hipMemGetInfo(&free_b, &all_b);
    if (e != hipSuccess) return thread_error(HQML_ERR_HIP, hip_text("hipMemGetInfo", e));
    const size_t need = total_bytes(ws);
    if (need > free_b) {
        char msg[160];
        std::snprintf(msg, sizeof msg, "workspace needs %zu bytes, device has %zu free", need, free_b);
        return thread_error(HQML_ERR_OOM, msg);
    }
    void *p = nullptr;
    if (hipMalloc(&p, need) != hipSuccess) {
        (void)hipGetLastError();
        return thread_error(HQML_ERR_OOM, "hipMalloc failed while reserving the workspace");
    }
    H *h = new (std::nothrow) H;
    if (!h) {
        (void)hipFree(p);
        return thread_error(HQML_ERR_OOM, "host allocation failed");
    }
    h->cfg = cfg;
    h->stream = reinterpret_cast<hipStream_t>(cfg.stream);
    h->reserved = p;
    place(ws, p);
    if (ws.ticket_bytes) {
        e = hipMemsetAsync(ws.ticket, 0, ws.ticket_bytes, h->stream);
        if (e == hipSuccess) e = hipStreamSynchronize(h->stream);
        if (e != hipSuccess) {
            (void)hipFree(p);
            delete h;
            return thread_error(HQML_ERR_HIP, hip_text("workspace set-up", e));
        }
    }
    h->ws = ws;
    *out = h;
    return HQML_OK;
}

template <class H>
int destroy(H *h)
{
    if (!h) return HQML_OK;
    const OnDevice on(h->cfg.device);
    (void)hipStreamSynchronize(h->stream);
    (void)hipFree(h->reserved);
    delete h;
    return HQML_OK;
}

template <class H>
int handle_error(H *h, int code, const std::string &msg)
{
    h->err = msg;
    return code;
}

template <class H>
const char *last_error(const H *h)
{
    return h ? h->err.c_str() : "handle is NULL";
}

bool layer_dtype(int dtype) { return dtype == HQML_DTYPE_FP32 || dtype == HQML_DTYPE_BF16; }

bool known_activation(int act) { return act >= HQML_ACT_NONE && act <= HQML_ACT_SIGMOID; }

int refused(const char *why, std::string *err)
{
    if (!why) return HQML_OK;
    *err = why;
    return HQML_ERR_ARG;
}

// ---- dense layer in 8-bit integers ----

int check_config(const hqml_dense_config *c, std::string *err)
{
    const char *why = nullptr;
    if (!c) why = "cfg is NULL";
    else if (c->in_features < 1 || c->in_features > HQML_DENSE8_MAX_IN) why = "in_features must be 1..2^17";
    else if (c->out_features < 1 || c->out_features > HQML_DENSE_MAX_FEATURES) why = "out_features must be 1..2^20";
    else if (c->max_batch < 1 || c->max_batch > HQML_DENSE_MAX_BATCH) why = "max_batch must be 1..2^24";
    else if (!layer_dtype(c->dtype)) why = "dtype must be HQML_DTYPE_FP32 or HQML_DTYPE_BF16";
    else if (!known_activation(c->activation)) why = "unknown activation";
    else if (!isfinite(c->alpha)) why = "alpha must be finite";
    else if (c->device < 0) why = "device must be >= 0";
    return refused(why, err);
}

long long pad16(long long k) { return (k + 15) & ~15ll; }

// Rows of codes are loaded sixteen at a time.
int check_codes(const void *codes, long long rows, long long K, long long ld, std::string *err)
{
    if ((size_t)codes % 16) return refused("codes must be 16-byte aligned", err);
    if (rows > 1 && (ld % 16 || ld < pad16(K))) return refused("row stride of codes must be a multiple of 16, at least K", err);
    return HQML_OK;
}

int quantise_rows(int device, void *stream, int dtype, long long rows, int K, const void *x, long long ldx, signed char *codes,
                  long long ldc, float *scales)
{
    std::string err;
    const char *why = nullptr;
    if (device < 0) why = "device must be >= 0";
    else if (!layer_dtype(dtype)) why = "dtype must be HQML_DTYPE_FP32 or HQML_DTYPE_BF16";
    else if (rows < 0 || rows > (1ll << 31)) why = "rows must be 0..2^31";
    else if (K < 1 || K > HQML_DENSE_MAX_FEATURES) why = "K must be 1..2^20";
    int rc = refused(why, &err);
    if (rc == HQML_OK && rows > 0) rc = check_codes(codes, rows, K, ldc, &err);
    if (rc != HQML_OK) return thread_error(rc, err);
    if (rows == 0) return HQML_OK;
    const OnDevice on(device);
    if (on.error() != hipSuccess) return thread_error(HQML_ERR_HIP, hip_text("device", on.error()));
    const long long Kp = pad16(K);
    const Arg args[] = {{"x", x, rows, K, ldx, false},
                        {"codes", codes, rows, Kp, rows > 1 ? ldc : Kp, false, 1, true},
                        {"scales", scales, 1, rows, rows, false, 4, true}};
    rc = check_args(device, dtype_bytes(dtype), args, 3, &err);
    if (rc != HQML_OK) return thread_error(rc, err);
    const hipError_t e = launch_quantise_rows(x, stride(rows, K, ldx), rows, K, dtype, codes, stride(rows, Kp, ldc), scales,
                                              reinterpret_cast<hipStream_t>(stream));
    return e == hipSuccess ? HQML_OK : thread_error(HQML_ERR_HIP, hip_text("quantise", e));
}

int dense8_create(const hqml_dense_config *cfg, hqml_dense8 **out)
{
    std::string err;
    const int rc = check_config(cfg, &err);
    if (rc != HQML_OK) return thread_error(rc, err);
    const OnDevice on(cfg->device);
    if (on.error() != hipSuccess) return thread_error(HQML_ERR_HIP, hip_text("device", on.error()));
    return make(*cfg, dense8_workspace(*cfg), out);
}

int dense8_forward(hqml_dense8 *h, int M, const void *x, long long ldx, const signed char *codes, long long ldw, const float *scales,
                   const void *bias, const void *residual, long long ldr, void *y, long long ldy)
{
    const hqml_dense_config &c = h->cfg;
    if (M < 0 || M > c.max_batch) return handle_error(h, HQML_ERR_ARG, "M must be 0..max_batch");
    if (M == 0) return HQML_OK;
    const long long K = c.in_features, N = c.out_features, Kp = pad16(K);
    const OnDevice on(c.device);
    if (on.error() != hipSuccess) return handle_error(h, HQML_ERR_HIP, hip_text("device", on.error()));
    std::string err;
    int rc = check_codes(codes, N, K, ldw, &err);
    if (rc != HQML_OK) return handle_error(h, rc, err);
    const Arg args[] = {{"x", x, M, K, ldx, false},
                        {"codes", codes, N, Kp, N > 1 ? ldw : Kp, false, 1},
                        {"scales", scales, 1, N, N, false, 4},
                        {"bias", bias, 1, N, N, true},
                        {"residual", residual, M, N, ldr, true},
                        {"y", y, M, N, ldy, false, 0, true, 4}};
    rc = check_args(c.device, dtype_bytes(c.dtype), args, 6, &err);
    if (rc != HQML_OK) return handle_error(h, rc, err);
    const Dense8Forward a{M,    (int)K,   (int)N, x,
                          codes, scales, bias, residual, stride(M, K, ldx), stride(N, Kp, ldw), stride(M, N, ldr), stride(M, N, ldy),
                          y,    c.activation, c.alpha};
    const hipError_t e = launch_dense8_forward(a, c.dtype, h->ws, h->stream);
    return e == hipSuccess ? HQML_OK : handle_error(h, HQML_ERR_HIP, hip_text("8-bit dense forward", e));
}

// ---- group norm ----

int check_config(const hqml_norm_config *c, std::string *err)
{
    const char *why = nullptr;
    if (!c) why = "cfg is NULL";
    else if (c->channels < 1 || c->channels > HQML_NORM_MAX_CHANNELS) why = "channels must be 1..4096";
    else if (c->groups < 1 || c->channels % c->groups) why = "groups must divide channels";
    else if (c->max_rows < 1 || c->max_rows > HQML_NORM_MAX_ROWS) why = "max_rows must be 1..2^30";
    else if (!layer_dtype(c->dtype)) why = "dtype must be HQML_DTYPE_FP32 or HQML_DTYPE_BF16";
    else if (!known_activation(c->activation)) why = "unknown activation";
    else if (!isfinite(c->eps) || !(c->eps > 0.0f)) why = "eps must be finite and > 0";
    else if (c->device < 0) why = "device must be >= 0";
    return refused(why, err);
}

int norm_create(const hqml_norm_config *cfg, hqml_norm **out)
{
    std::string err;
    const int rc = check_config(cfg, &err);
    if (rc != HQML_OK) return thread_error(rc, err);
    const OnDevice on(cfg->device);
    if (on.error() != hipSuccess) return thread_error(HQML_ERR_HIP, hip_text("device", on.error()));
    const hipError_t e = configure_norm(cfg->dtype);
    if (e != hipSuccess) return thread_error(HQML_ERR_HIP, hip_text("kernel attributes", e));
    return make(*cfg, norm_workspace(*cfg), out);
}

int check_rows(hqml_norm *h, int B, int S)
{
    if (B < 0 || S < 0 || (long long)B * S > h->cfg.max_rows)
        return handle_error(h, HQML_ERR_ARG, "B and S must be >= 0, and B S at most max_rows");
    return HQML_OK;
}

NormCall norm_call(const hqml_norm_config &c, int B, int S)
{
    NormCall a{};
    a.B = B, a.S = S, a.C = c.channels, a.G = c.groups;
    a.act = c.activation, a.eps = c.eps;
    return a;
}

int norm_forward(hqml_norm *h, int B, int S, const void *x, long long ldx, const void *gamma, const void *beta, void *y, long long ldy,
                 float *mean, float *rstd)
{
    const hqml_norm_config &c = h->cfg;
    int rc = check_rows(h, B, S);
    const long long rows = (long long)B * S, C = c.channels, sets = (long long)B * c.groups;
    if (rc != HQML_OK || rows == 0) return rc;
    if (!mean != !rstd) return handle_error(h, HQML_ERR_ARG, "mean and rstd are given together");
    const OnDevice on(c.device);
    if (on.error() != hipSuccess) return handle_error(h, HQML_ERR_HIP, hip_text("device", on.error()));
    const Arg args[] = {{"x", x, rows, C, ldx, false},  {"gamma", gamma, 1, C, C, true},
                        {"beta", beta, 1, C, C, true},  {"y", y, rows, C, ldy, false, 0, true, 0},
                        {"mean", mean, 1, sets, sets, true, 4, true}, {"rstd", rstd, 1, sets, sets, true, 4, true}};
    std::string err;
    rc = check_args(c.device, dtype_bytes(c.dtype), args, 6, &err);
    if (rc != HQML_OK) return handle_error(h, rc, err);
    NormCall a = norm_call(c, B, S);
    a.x = x, a.gamma = gamma, a.beta = beta, a.y = y;
    a.ldx = stride(rows, C, ldx), a.ldy = stride(rows, C, ldy);
    a.mean = mean, a.rstd = rstd;
    const hipError_t e = launch_norm_forward(a, c.dtype, h->ws, h->stream);
    return e == hipSuccess ? HQML_OK : handle_error(h, HQML_ERR_HIP, hip_text("norm forward", e));
}

int norm_backward(hqml_norm *h, int B, int S, const void *dy, long long lddy, const void *x, long long ldx, const void *gamma,
                  const void *beta, const float *mean, const float *rstd, void *dx, long long lddx, void *dgamma, void *dbeta)
{
    const hqml_norm_config &c = h->cfg;
    int rc = check_rows(h, B, S);
    if (rc != HQML_OK) return rc;
    const long long rows = (long long)B * S, C = c.channels, sets = (long long)B * c.groups;
    const OnDevice on(c.device);
    if (on.error() != hipSuccess) return handle_error(h, HQML_ERR_HIP, hip_text("device", on.error()));
    std::string err;
    if (rows) {
        const Arg args[] = {{"dy", dy, rows, C, lddy, false},       {"x", x, rows, C, ldx, false},
                            {"gamma", gamma, 1, C, C, true},        {"beta", beta, 1, C, C, true},
                            {"mean", mean, 1, sets, sets, false, 4}, {"rstd", rstd, 1, sets, sets, false, 4},
                            {"dx", dx, rows, C, lddx, true, 0, true}, {"dgamma", dgamma, 1, C, C, true, 0, true},
                            {"dbeta", dbeta, 1, C, C, true, 0, true}};
        rc = check_args(c.device, dtype_bytes(c.dtype), args, 9, &err);
    } else {
        const Arg args[] = {{"dgamma", dgamma, 1, C, C, true, 0, true}, {"dbeta", dbeta, 1, C, C, true, 0, true}};
        rc = check_args(c.device, dtype_bytes(c.dtype), args, 2, &err);
    }
    if (rc != HQML_OK) return handle_error(h, rc, err);
    if (!dgamma && !dbeta && (!dx || !rows)) return HQML_OK;
    NormCall a = norm_call(c, B, S);
    a.x = x, a.gamma = gamma, a.beta = beta, a.dy = dy;
    a.ldx = stride(rows, C, ldx), a.lddy = stride(rows, C, lddy), a.lddx = stride(rows, C, lddx);
    a.mean = const_cast<float *>(mean), a.rstd = const_cast<float *>(rstd);   // only read
    a.dx = dx, a.dgamma = dgamma, a.dbeta = dbeta;
    const hipError_t e = launch_norm_backward(a, c.dtype, h->ws, h->stream);
    return e == hipSuccess ? HQML_OK : handle_error(h, HQML_ERR_HIP, hip_text("norm backward", e));
}

// ---- Muon ----

int check_muon(const hqml_muon_config *c, int n, const hqml_muon_tensor *t, std::string *err)
{
    const char *why = nullptr;
    auto small = [](double v) { return v >= -16.0 && v <= 16.0; };
    if (!c) why = "cfg is NULL";
    else if (n < 0 || (n > 0 && !t)) why = "tensors is NULL or n_tensors negative";
    else if (!layer_dtype(c->param_dtype) || !layer_dtype(c->grad_dtype)) why = "parameters and gradients must be fp32 or bf16";
    else if (c->steps < 1 || c->steps > HQML_MUON_MAX_STEPS) why = "steps must be 1..100";
    else if (!(c->lr >= 0) || !isfinite(c->lr) || !(c->weight_decay >= 0) || !isfinite(c->weight_decay))
        why = "lr and weight_decay must be finite and >= 0";
    else if (!(c->momentum >= 0 && c->momentum < 1)) why = "momentum must be in [0, 1)";
    else if (!((float)c->eps > 0) || !isfinite((float)c->eps)) why = "eps must be finite and > 0 in fp32";
    else if (!small(c->a) || !small(c->b) || !small(c->c)) why = "coefficients must be -16..16";
    else if (c->device < 0) why = "device must be >= 0";
    for (int i = 0; !why && i < n; ++i) {
        if (t[i].rows < 0 || t[i].rows > HQML_MUON_MAX_SIDE || t[i].cols < 0 || t[i].cols > HQML_MUON_MAX_SIDE)
            why = "rows and cols must be 0..2^16";
        else if (!(t[i].scale >= 0) || !isfinite(t[i].scale)) why = "scale must be finite and >= 0";
    }
    return refused(why, err);
}

// Workgroups update matrices while others still read theirs.
int check_apart(const hqml_muon_config &c, int n, const hqml_muon_tensor *t, const void *workspace, size_t bytes, std::string *err)
{
    struct Span {
        size_t from, to;
        bool output;
    };
    std::vector<Span> all;
    all.reserve(3 * (size_t)n + 1);
    auto add = [&](const void *p, size_t size, bool output) {
        if (p && size) all.push_back({(size_t)p, (size_t)p + size, output});
    };
    add(workspace, bytes, true);
    for (int i = 0; i < n; ++i) {
        const size_t k = (size_t)t[i].rows * t[i].cols;
        add(t[i].param, k * dtype_bytes(c.param_dtype), true);
        add(t[i].grad, k * dtype_bytes(c.grad_dtype), false);
        add(t[i].momentum, k * 4, true);
    }
    std::sort(all.begin(), all.end(), [](const Span &a, const Span &b) { return a.from < b.from; });
    size_t end = 0, outputs_end = 0;   // of those so far
    for (const Span &s : all) {
        if (s.from < outputs_end || (s.output && s.from < end)) return refused("matrices and workspace must not overlap", err);
        end = std::max(end, s.to);
        if (s.output) outputs_end = std::max(outputs_end, s.to);
    }
    return HQML_OK;
}

int muon_step(const hqml_muon_config *c, int n, const hqml_muon_tensor *t, void *workspace, size_t bytes)
{
    std::string err;
    int rc = check_muon(c, n, t, &err);
    if (rc != HQML_OK) return thread_error(rc, err);
    bool some = false;
    for (int i = 0; i < n; ++i) some = some || (t[i].rows && t[i].cols);
    if (!some) return HQML_OK;
    const size_t need = muon_workspace(*c, n, t);
    rc = check_apart(*c, n, t, workspace, need, &err);
    if (rc != HQML_OK) return thread_error(rc, err);
    const OnDevice on(c->device);
    if (on.error() != hipSuccess) return thread_error(HQML_ERR_HIP, hip_text("device", on.error()));
    if (need) {
        if (bytes < need || (size_t)workspace % 256)
            return thread_error(HQML_ERR_ARG, "workspace is too small or not 256-byte aligned");
        rc = check_device_array(c->device, workspace, need, "workspace", &err);
    }
    for (int i = 0; rc == HQML_OK && i < n; ++i) {
        const size_t k = (size_t)t[i].rows * t[i].cols;
        if (!k) continue;
        const struct {
            const char *name;
            const void *p;
            size_t elem;
        } a[] = {{"param", t[i].param, dtype_bytes(c->param_dtype)},
                 {"grad", t[i].grad, dtype_bytes(c->grad_dtype)},
                 {"momentum", t[i].momentum, 4}};
        for (const auto &v : a) {
            if ((size_t)v.p % v.elem) return thread_error(HQML_ERR_ARG, std::string(v.name) + " is not aligned to its element");
            rc = check_device_array(c->device, v.p, v.elem * k, v.name, &err);
            if (rc != HQML_OK) break;
        }
    }
    if (rc != HQML_OK) return thread_error(rc, err);
    const hipError_t e = launch_muon(*c, n, t, workspace, reinterpret_cast<hipStream_t>(c->stream));
    return e == hipSuccess ? HQML_OK : thread_error(HQML_ERR_HIP, hip_text("muon", e));
}

}  // namespace

extern "C" {

int hqml_quantise_rows(int device, void *stream, int dtype, long long rows, int K, const void *x, long long ldx, signed char *codes,
                       long long ldc, float *scales)
{
    return guarded([&] { return quantise_rows(device, stream, dtype, rows, K, x, ldx, codes, ldc, scales); });
}

size_t hqml_dense8_workspace_bytes(const hqml_dense_config *cfg)
{
    size_t bytes = 0;
    (void)guarded([&] {
        std::string err;
        if (check_config(cfg, &err) == HQML_OK) bytes = total_bytes(dense8_workspace(*cfg));
        return (int)HQML_OK;
    });
    return bytes;
}

int hqml_dense8_create(const hqml_dense_config *cfg, hqml_dense8 **out)
{
    return guarded([&] {
        if (!out) return thread_error(HQML_ERR_ARG, "out is NULL");
        *out = nullptr;
        return dense8_create(cfg, out);
    });
}

int hqml_dense8_destroy(hqml_dense8 *h) { return destroy(h); }

const char *hqml_dense8_last_error(const hqml_dense8 *h) { return last_error(h); }

int hqml_dense8_forward(hqml_dense8 *h, int M, const void *x, long long ldx, const signed char *codes, long long ldw,
                        const float *scales, const void *bias, const void *residual, long long ldr, void *y, long long ldy)
{
    if (!h) return HQML_ERR_ARG;
    return guarded([&] { return dense8_forward(h, M, x, ldx, codes, ldw, scales, bias, residual, ldr, y, ldy); });
}

size_t hqml_norm_workspace_bytes(const hqml_norm_config *cfg)
{
    size_t bytes = 0;
    (void)guarded([&] {
        std::string err;
        if (check_config(cfg, &err) == HQML_OK) bytes = total_bytes(norm_workspace(*cfg));
        return (int)HQML_OK;
    });
    return bytes;
}

int hqml_norm_create(const hqml_norm_config *cfg, hqml_norm **out)
{
    return guarded([&] {
        if (!out) return thread_error(HQML_ERR_ARG, "out is NULL");
        *out = nullptr;
        return norm_create(cfg, out);
    });
}

int hqml_norm_destroy(hqml_norm *h) { return destroy(h); }

const char *hqml_norm_last_error(const hqml_norm *h) { return last_error(h); }

int hqml_norm_forward(hqml_norm *h, int B, int S, const void *x, long long ldx, const void *gamma, const void *beta, void *y,
                      long long ldy, float *mean, float *rstd)
{
    if (!h) return HQML_ERR_ARG;
    return guarded([&] { return norm_forward(h, B, S, x, ldx, gamma, beta, y, ldy, mean, rstd); });
}

int hqml_norm_backward(hqml_norm *h, int B, int S, const void *dy, long long lddy, const void *x, long long ldx, const void *gamma,
                       const void *beta, const float *mean, const float *rstd, void *dx, long long lddx, void *dgamma, void *dbeta)
{
    if (!h) return HQML_ERR_ARG;
    return guarded([&] { return norm_backward(h, B, S, dy, lddy, x, ldx, gamma, beta, mean, rstd, dx, lddx, dgamma, dbeta); });
}

size_t hqml_muon_workspace_bytes(const hqml_muon_config *cfg, int n_tensors, const hqml_muon_tensor *tensors)
{
    size_t bytes = 0;
    (void)guarded([&] {
        std::string err;
        if (check_muon(cfg, n_tensors, tensors, &err) == HQML_OK) bytes = muon_workspace(*cfg, n_tensors, tensors);
        return (int)HQML_OK;
    });
    return bytes;
}

int hqml_muon_step(const hqml_muon_config *cfg, int n_tensors, const hqml_muon_tensor *tensors, void *workspace,
                   size_t workspace_bytes)
{
    return guarded([&] { return muon_step(cfg, n_tensors, tensors, workspace, workspace_bytes); });
}

}  // extern "C"
