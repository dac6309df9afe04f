// Entry points of the dense layer and of AdamW: argument checks, the dense handle's
// workspace, and the launches.  Nothing is queued before every argument has passed, and no
// exception leaves an entry point.
#include <hip/hip_runtime.h>
#include <math.h>

#include <cstdio>
#include <new>
#include <string>

#include "../../include/hqml.h"
#include "hqml_host.hpp"
#include "hqml_ops.hpp"

using namespace hqml;

struct hqml_dense {
    hqml_dense_config cfg{};
    DenseWorkspace ws;
    hipStream_t stream = nullptr;
    void *reserved = nullptr;
    std::string err;
};

namespace {

// The calling thread's device, put back at the end of an entry point.
class OnDevice {
public:
    explicit OnDevice(int device)
    {
        e_ = hipGetDevice(&before_);
        if (e_ == hipSuccess && before_ != device) {
            e_ = hipSetDevice(device);
            switched_ = e_ == hipSuccess;
        }
    }
    ~OnDevice()
    {
        if (switched_) (void)hipSetDevice(before_);
    }
    hipError_t error() const { return e_; }

private:
    int before_ = 0;
    bool switched_ = false;
    hipError_t e_;
};

std::string hip_text(const char *what, hipError_t e)
{
    return std::string(what) + ": " + hipGetErrorString(e);
}

size_t dtype_bytes(int dtype)
{
    return dtype == HQML_DTYPE_BF16 ? 2 : dtype == HQML_DTYPE_FP64 ? 8 : 4;
}

size_t up256(size_t b)
{
    return (b + 255) & ~(size_t)255;
}

size_t total_bytes(const DenseWorkspace &ws)
{
    return up256(ws.dz_bytes) + up256(ws.rows_bytes) + up256(ws.part_bytes) +
           up256(ws.ticket_bytes) + up256(ws.pad_bytes);
}

int check_dense_config(const hqml_dense_config *c, std::string *err)
{
    const char *why = nullptr;
    if (!c) why = "cfg is NULL";
    else if (c->in_features < 1 || c->in_features > HQML_DENSE_MAX_FEATURES) why = "in_features must be 1..2^20";
    else if (c->out_features < 1 || c->out_features > HQML_DENSE_MAX_FEATURES) why = "out_features must be 1..2^20";
    else if (c->max_batch < 1 || c->max_batch > HQML_DENSE_MAX_BATCH) why = "max_batch must be 1..2^24";
    else if (c->dtype != HQML_DTYPE_FP32 && c->dtype != HQML_DTYPE_BF16)
        why = "dtype must be HQML_DTYPE_FP32 or HQML_DTYPE_BF16";
    else if (c->activation < HQML_ACT_NONE || c->activation > HQML_ACT_SIGMOID) why = "unknown activation";
    else if (!isfinite(c->alpha)) why = "alpha must be finite";
    else if (c->device < 0) why = "device must be >= 0";
    if (!why) return HQML_OK;
    *err = why;
    return HQML_ERR_ARG;
}

// One caller array of a call: rows rows of len elements, ld elements apart.
struct Arg {
    const char *name;
    const void *p;
    long long rows, len, ld;
    bool optional;
    size_t elem = 0;   // bytes of an element; 0: the handle's
    bool output = false;
    int itself = -1;   // the argument that an output may be
};

// Whether two arrays share bytes.  Where neither lies before the other they may still be columns of one array: rows the
// same distance apart, and the columns apart within it.  Rows at other distances count as shared.
bool overlap(const Arg &a, size_t ea, const Arg &b, size_t eb)
{
    struct Bytes {
        size_t at, rows, len, step;
    };
    auto bytes = [](const Arg &g, size_t e) {
        Bytes r{(size_t)g.p, (size_t)g.rows, e * (size_t)g.len, e * (size_t)g.ld};
        if (r.rows > 1 && r.step == r.len) r.len *= r.rows, r.rows = 1;   // no gaps
        return r;
    };
    const Bytes p = bytes(a, ea), q = bytes(b, eb);
    if (p.at + (p.rows - 1) * p.step + p.len <= q.at || q.at + (q.rows - 1) * q.step + q.len <= p.at) return false;
    if (p.rows == 1 && q.rows == 1) return true;
    if (p.rows > 1 && q.rows > 1 && p.step != q.step) return true;
    const size_t step = p.rows > 1 ? p.step : q.step;
    const size_t from = q.at >= p.at ? (q.at - p.at) % step : (step - (p.at - q.at) % step) % step;
    return p.len > from || from + q.len > step;
}

int check_args(int device, size_t dtype, const Arg *a, int n, std::string *err)
{
    for (int i = 0; i < n; ++i) {
        const size_t elem = a[i].elem ? a[i].elem : dtype;
        if (!a[i].p && a[i].optional) continue;
        if (a[i].ld < a[i].len || (a[i].rows > 1 && a[i].ld > HQML_DENSE_MAX_FEATURES)) {
            *err = std::string("row stride of ") + a[i].name + " must be at least its row's length and at most 2^20";
            return HQML_ERR_ARG;
        }
        if ((size_t)a[i].p % elem) {
            *err = std::string(a[i].name) + " is not aligned to its element";
            return HQML_ERR_ARG;
        }
        if (a[i].rows == 0) continue;
        const size_t bytes = elem * (size_t)((a[i].rows - 1) * a[i].ld + a[i].len);
        const int rc = check_device_array(device, a[i].p, bytes, a[i].name, err);
        if (rc != HQML_OK) return rc;
    }
    // workgroups write rows of an output while others still read their operands
    for (int i = 0; i < n; ++i)
        for (int j = 0; j < n; ++j) {
            if (!a[i].output || i == j || (a[j].output && j > i) || !a[i].p || !a[j].p) continue;
            if (j == a[i].itself && a[i].p == a[j].p && (a[i].ld == a[j].ld || a[i].rows == 1)) continue;
            if (!overlap(a[i], a[i].elem ? a[i].elem : dtype, a[j], a[j].elem ? a[j].elem : dtype)) continue;
            *err = std::string(a[i].name) + " must not overlap " + a[j].name;
            return HQML_ERR_ARG;
        }
    return HQML_OK;
}

// The stride that the kernels take.  They form it for rows past the last one too, and hold it in 32 bits of bytes: that of
// a single row, which may be anything, would bring those back onto the row itself.
long long stride(long long rows, long long len, long long ld)
{
    return rows > 1 ? ld : len;
}

int dense_error(hqml_dense *h, int code, const std::string &msg)
{
    h->err = msg;
    return code;
}

int check_batch(hqml_dense *h, int M)
{
    if (M >= 0 && M <= h->cfg.max_batch) return HQML_OK;
    return dense_error(h, HQML_ERR_ARG, "M must be 0..max_batch");
}

int thread_error(int code, const std::string &msg)
{
    set_thread_error(msg);
    return code;
}

int dense_forward(hqml_dense *h, int M, const void *x, long long ldx, const void *w, long long ldw, const void *bias,
                  const void *residual, long long ldr, void *y, long long ldy, float *z)
{
    const hqml_dense_config &c = h->cfg;
    int rc = check_batch(h, M);
    if (rc != HQML_OK || M == 0) return rc;
    const long long K = c.in_features, N = c.out_features;
    const OnDevice on(c.device);
    if (on.error() != hipSuccess) return dense_error(h, HQML_ERR_HIP, hip_text("device", on.error()));
    if (c.activation == HQML_ACT_NONE) z = nullptr;
    const Arg args[] = {{"x", x, M, K, ldx, false},         {"w", w, N, K, ldw, false},
                        {"bias", bias, 1, N, N, true},      {"residual", residual, M, N, ldr, true},
                        {"y", y, M, N, ldy, false, 0, true, 3}, {"z", z, M, N, N, true, 4, true}};
    std::string err;
    rc = check_args(c.device, dtype_bytes(c.dtype), args, 6, &err);
    if (rc != HQML_OK) return dense_error(h, rc, err);
    DenseForward a{M, (int)K, (int)N, x, w, bias, residual, stride(M, K, ldx), stride(N, K, ldw), stride(M, N, ldr),
                   stride(M, N, ldy), y, z, c.activation, c.alpha};
    const hipError_t e = launch_dense_forward(a, c.dtype, h->ws, h->stream);
    return e == hipSuccess ? HQML_OK : dense_error(h, HQML_ERR_HIP, hip_text("dense forward", e));
}

int dense_backward(hqml_dense *h, int M, const void *dy, long long lddy, const void *x, long long ldx, const void *w,
                   long long ldw, const float *z, void *dx, long long lddx, void *dw, void *db)
{
    const hqml_dense_config &c = h->cfg;
    int rc = check_batch(h, M);
    if (rc != HQML_OK) return rc;
    const long long K = c.in_features, N = c.out_features;
    const OnDevice on(c.device);
    if (on.error() != hipSuccess) return dense_error(h, HQML_ERR_HIP, hip_text("device", on.error()));
    std::string err;
    if (M > 0) {
        if (c.activation == HQML_ACT_NONE) z = nullptr;
        const Arg args[] = {{"dy", dy, M, N, lddy, false},           {"x", x, M, K, ldx, !dw},
                            {"w", w, N, K, ldw, !dx},                {"z", z, M, N, N, c.activation == HQML_ACT_NONE, 4},
                            {"dx", dx, M, K, lddx, true, 0, true},   {"dw", dw, N, K, K, true, 0, true},
                            {"db", db, 1, N, N, true, 0, true}};
        rc = check_args(c.device, dtype_bytes(c.dtype), args, 7, &err);
    } else {
        const Arg args[] = {{"dw", dw, N, K, K, true, 0, true}, {"db", db, 1, N, N, true, 0, true}};
        rc = check_args(c.device, dtype_bytes(c.dtype), args, 2, &err);
    }
    if (rc != HQML_OK) return dense_error(h, rc, err);
    if (!dx && !dw && !db) return HQML_OK;
    DenseBackward a{M, (int)K, (int)N, dy, x, w, z, stride(M, N, lddy), stride(M, K, ldx), stride(N, K, ldw),
                    stride(M, K, lddx), dx, dw, db, c.activation, c.alpha};
    const hipError_t e = launch_dense_backward(a, c.dtype, h->ws, h->stream);
    return e == hipSuccess ? HQML_OK : dense_error(h, HQML_ERR_HIP, hip_text("dense backward", e));
}

int dense_create(const hqml_dense_config *cfg, hqml_dense **out)
{
    std::string err;
    const int rc = check_dense_config(cfg, &err);
    if (rc != HQML_OK) return thread_error(rc, err);
    const OnDevice on(cfg->device);
    if (on.error() != hipSuccess) return thread_error(HQML_ERR_HIP, hip_text("device", on.error()));
    DenseWorkspace ws = dense_workspace(*cfg);
    size_t free_b = 0, all_b = 0;
    hipError_t e = hipMemGetInfo(&free_b, &all_b);
    if (e != hipSuccess) return thread_error(HQML_ERR_HIP, hip_text("hipMemGetInfo", e));
    const size_t need = total_bytes(ws);
    if (need > free_b) {
        char msg[160];
        std::snprintf(msg, sizeof msg, "workspace needs %zu bytes, device has %zu free", need, free_b);
        return thread_error(HQML_ERR_OOM, msg);
    }
    char *p = nullptr;
    if (hipMalloc(reinterpret_cast<void **>(&p), need) != hipSuccess) {
        (void)hipGetLastError();
        return thread_error(HQML_ERR_OOM, "hipMalloc failed while reserving the workspace");
    }
    hqml_dense *h = new (std::nothrow) hqml_dense;
    if (!h) {
        (void)hipFree(p);
        return thread_error(HQML_ERR_OOM, "host allocation failed");
    }
    h->cfg = *cfg;
    h->stream = reinterpret_cast<hipStream_t>(cfg->stream);
    h->reserved = p;
    char *at = p;
    auto take = [&](size_t bytes) -> void * {
        char *here = at;
        at += up256(bytes);
        return bytes ? here : nullptr;
    };
    ws.dz = take(ws.dz_bytes);
    ws.rows = static_cast<float *>(take(ws.rows_bytes));
    ws.part = static_cast<float *>(take(ws.part_bytes));
    ws.ticket = static_cast<unsigned *>(take(ws.ticket_bytes));
    ws.pad = take(ws.pad_bytes);
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

int check_adamw(const hqml_adamw_config *c, int n, const hqml_adamw_tensor *t, std::string *err)
{
    auto bad = [&](const std::string &m) {
        *err = m;
        return (int)HQML_ERR_ARG;
    };
    if (!c) return bad("cfg is NULL");
    if (n < 0 || (n > 0 && !t)) return bad("tensors is NULL or n_tensors negative");
    for (int d : {c->param_dtype, c->grad_dtype})
        if (d != HQML_DTYPE_FP32 && d != HQML_DTYPE_BF16 && d != HQML_DTYPE_FP64) return bad("unknown dtype");
    if ((c->param_dtype == HQML_DTYPE_FP64) != (c->grad_dtype == HQML_DTYPE_FP64))
        return bad("fp64 parameters take fp64 gradients, and no others do");
    if (c->moments != HQML_MOMENTS_32 && c->moments != HQML_MOMENTS_8) return bad("unknown moments");
    if (c->moments == HQML_MOMENTS_8 && c->param_dtype == HQML_DTYPE_FP64) {
        *err = "8-bit moments are for fp32 and bf16 parameters";
        return HQML_ERR_UNSUPPORTED;
    }
    if (c->step < 1) return bad("step counts from 1");
    if (!(c->lr >= 0) || !(c->eps >= 0) || !(c->weight_decay >= 0) || !isfinite(c->lr) || !isfinite(c->eps) ||
        !isfinite(c->weight_decay))
        return bad("lr, eps and weight_decay must be finite and >= 0");
    if (!(c->beta1 >= 0 && c->beta1 < 1) || !(c->beta2 >= 0 && c->beta2 < 1)) return bad("betas must be in [0, 1)");
    if (c->device < 0) return bad("device must be >= 0");
    const size_t pb = dtype_bytes(c->param_dtype), gb = dtype_bytes(c->grad_dtype);
    const bool eight = c->moments == HQML_MOMENTS_8;
    const size_t mb = eight ? 1 : pb == 8 ? 8 : 4;
    for (int i = 0; i < n; ++i) {
        const long long numel = t[i].numel;
        if (numel == 0) continue;
        if (numel < 0 || numel > (1ll << 40)) return bad("numel must be 0..2^40");
        const size_t k = (size_t)numel, scales = (k + HQML_ADAMW_BLOCK - 1) / HQML_ADAMW_BLOCK;
        const struct {
            const char *name;
            const void *p;
            size_t elem, count;
        } a[] = {{"param", t[i].param, pb, k},  {"grad", t[i].grad, gb, k},
                 {"m", t[i].m, mb, k},          {"v", t[i].v, mb, k},
                 {"m_scale", t[i].m_scale, 4, scales}, {"v_scale", t[i].v_scale, 4, scales}};
        for (int j = 0; j < (eight ? 6 : 4); ++j) {
            if ((size_t)a[j].p % a[j].elem) return bad(std::string(a[j].name) + " is not aligned to its element");
            const int rc = check_device_array(c->device, a[j].p, a[j].elem * a[j].count, a[j].name, err);
            if (rc != HQML_OK) return rc;
        }
    }
    return HQML_OK;
}

int adamw_step(const hqml_adamw_config *c, int n, const hqml_adamw_tensor *t)
{
    std::string err;
    if (c && c->device >= 0) {
        const OnDevice on(c->device);
        if (on.error() != hipSuccess) return thread_error(HQML_ERR_HIP, hip_text("device", on.error()));
        const int rc = check_adamw(c, n, t, &err);
        if (rc != HQML_OK) return thread_error(rc, err);
        const hipStream_t s = reinterpret_cast<hipStream_t>(c->stream);
        hipStreamCaptureStatus cap = hipStreamCaptureStatusNone;
        hipError_t e = hipStreamIsCapturing(s, &cap);
        if (e != hipSuccess) return thread_error(HQML_ERR_HIP, hip_text("stream", e));
        if (cap != hipStreamCaptureStatusNone)
            return thread_error(HQML_ERR_UNSUPPORTED,
                                "the step number is a host value: a captured step would repeat this one");
        AdamwScalars k;
        k.decay = c->lr * c->weight_decay;
        k.b1 = c->beta1, k.c1 = 1.0 - c->beta1;
        k.b2 = c->beta2, k.c2 = 1.0 - c->beta2;
        k.inv_root = 1.0 / sqrt(1.0 - pow(c->beta2, (double)c->step));
        k.eps = c->eps;
        k.size = c->lr / (1.0 - pow(c->beta1, (double)c->step));
        e = launch_adamw(*c, k, n, t, s);
        return e == hipSuccess ? HQML_OK : thread_error(HQML_ERR_HIP, hip_text("adamw", e));
    }
    return thread_error(check_adamw(c, n, t, &err), err);
}

// Runs an entry point's body; what the standard library throws becomes a status.
template <typename F>
int guarded(F f) noexcept
{
    try {
        return f();
    } catch (...) {
        return HQML_ERR_OOM;
    }
}

}  // namespace

extern "C" {

size_t hqml_dense_workspace_bytes(const hqml_dense_config *cfg)
{
    size_t bytes = 0;
    (void)guarded([&] {
        std::string err;
        if (check_dense_config(cfg, &err) == HQML_OK) bytes = total_bytes(dense_workspace(*cfg));
        return (int)HQML_OK;
    });
    return bytes;
}

int hqml_dense_create(const hqml_dense_config *cfg, hqml_dense **out)
{
    return guarded([&] {
        if (!out) return thread_error(HQML_ERR_ARG, "out is NULL");
        *out = nullptr;
        return dense_create(cfg, out);
    });
}

int hqml_dense_destroy(hqml_dense *h)
{
    if (!h) return HQML_OK;
    const OnDevice on(h->cfg.device);
    (void)hipStreamSynchronize(h->stream);
    (void)hipFree(h->reserved);
    delete h;
    return HQML_OK;
}

const char *hqml_dense_last_error(const hqml_dense *h)
{
    return h ? h->err.c_str() : "handle is NULL";
}

int hqml_dense_forward(hqml_dense *h, int M, const void *x, long long ldx, const void *w, long long ldw,
                       const void *bias, const void *residual, long long ldr, void *y, long long ldy, float *z)
{
    if (!h) return HQML_ERR_ARG;
    return guarded([&] { return dense_forward(h, M, x, ldx, w, ldw, bias, residual, ldr, y, ldy, z); });
}

int hqml_dense_backward(hqml_dense *h, int M, const void *dy, long long lddy, const void *x, long long ldx,
                        const void *w, long long ldw, const float *z, void *dx, long long lddx, void *dw, void *db)
{
    if (!h) return HQML_ERR_ARG;
    return guarded([&] { return dense_backward(h, M, dy, lddy, x, ldx, w, ldw, z, dx, lddx, dw, db); });
}

int hqml_adamw_step(const hqml_adamw_config *cfg, int n_tensors, const hqml_adamw_tensor *tensors)
{
    return guarded([&] { return adamw_step(cfg, n_tensors, tensors); });
}

}  // extern "C"
