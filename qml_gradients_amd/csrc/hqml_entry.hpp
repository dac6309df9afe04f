// What the entry points of the layers and optimisers share: the calling thread's device, checks of caller arrays,
// messages, and the guard that keeps exceptions inside.
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>

#include <string>

#include "../../include/hqml.h"
#include "hqml_host.hpp"

namespace hqml {

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

inline std::string hip_text(const char *what, hipError_t e)
{
    return std::string(what) + ": " + hipGetErrorString(e);
}

inline size_t dtype_bytes(int dtype)
{
    return dtype == HQML_DTYPE_BF16 ? 2 : dtype == HQML_DTYPE_FP64 ? 8 : 4;
}

inline size_t up256(size_t b)
{
    return (b + 255) & ~(size_t)255;
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
inline bool overlap(const Arg &a, size_t ea, const Arg &b, size_t eb)
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

inline int check_args(int device, size_t dtype, const Arg *a, int n, std::string *err)
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
inline long long stride(long long rows, long long len, long long ld)
{
    return rows > 1 ? ld : len;
}

inline int thread_error(int code, const std::string &msg)
{
    set_thread_error(msg);
    return code;
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

}  // namespace hqml
