// Group norm with an activation, channels last: x [B][S][C], groups of C / G neighbouring channels over all positions of a
// sample.
//
//   xhat = (x - mean) rstd,  rstd = 1 / sqrt(var + eps),  z = gamma xhat + beta,  y = act(z)
//   dz = dy act'(z),  dgamma = sum dz xhat,  dbeta = sum dz  (over samples and positions)
//   dx = rstd (gamma dz - mean(gamma dz) - xhat mean(gamma dz xhat))  (means over the group)
//
// Bound by memory.  A thread keeps V neighbouring channels (16 bytes) and goes down the positions, so that what it sums
// stays by channel, and groups of any size are put together from channels in LDS.
//   k_resident_*  a workgroup holds all positions of a sample and some whole groups in registers: x is read once, and the
//                 variance is formed of what is left after the mean.  Small samples share a workgroup.
//   k_stats, k_sums with k_apply_*  larger samples: workgroups take chunks of positions; the last one of a sample to finish puts
//                 the chunks' statistics together (in their order, so no result depends on timing), and a second kernel reads
//                 x again, in the opposite order, to find its end still in the last-level cache.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "hqml_act.hpp"
#include "hqml_layers.hpp"

namespace hqml {
namespace {

using u32x4 = __attribute__((ext_vector_type(4))) uint32_t;
// 16 bytes at any alignment of an element: the hardware takes them so
using u32x4_any = __attribute__((ext_vector_type(4), aligned(2))) uint32_t;

template <typename T>
constexpr int kVec = 16 / (int)sizeof(T);   // channels of a thread

// How a workgroup's threads share `width` channels (a span of whole groups, or all) and the positions of `subs` samples.
struct Map {
    int width, vecs;    // channels, threads across them
    int lanes;          // threads down the positions of a sample
    int subs;
    int per;            // channels of a group
    int groups;         // of the span
};

struct Norm {
    int B, S, C, G;
    const void *x, *gamma, *beta, *dy;
    long long ldx, ldy, lddy, lddx;
    void *y, *dx;
    float *mean, *rstd;
    int act;
    float eps;
    float *part;        // backward: [workgroups of a span][2][C], dgamma and dbeta
    void *dgamma, *dbeta;   // written by the one workgroup of a span there is, or null
    Map map;
    // split
    int chunk, chunks;      // positions of a chunk, chunks of a sample
    float *stat;            // [B][chunks][G][2]
    float *group;           // [B][G][2]
    unsigned *ticket;       // [B], 0 between calls
};

// A thread's channels and positions.
struct Place {
    int c, n;          // first channel in the span, channels that exist (0: none)
    int row, sub;      // first position, sample of the workgroup's
    bool on;
};

template <int V>
__device__ __forceinline__ Place place(const Map &m, int width)
{
    Place p;
    const int rl = (int)threadIdx.x / m.vecs, cv = (int)threadIdx.x - rl * m.vecs;
    p.c = cv * V;
    p.sub = rl / m.lanes;
    p.row = rl - p.sub * m.lanes;
    p.on = p.sub < m.subs;
    p.n = !p.on || p.c >= width ? 0 : width - p.c < V ? width - p.c : V;
    return p;
}

template <typename T, int V>
__device__ __forceinline__ u32x4 get(const T *from, int n)
{
    if (n == V) return *(const u32x4_any *)from;
    T t[V] = {};
#pragma unroll
    for (int e = 0; e < V; ++e)
        if (e < n) t[e] = from[e];
    return __builtin_bit_cast(u32x4, t);
}

template <typename T, int V>
__device__ __forceinline__ void put(T *to, const float (&v)[V], int n)
{
    T t[V];
#pragma unroll
    for (int e = 0; e < V; ++e) narrow(v[e], t[e]);
    if (n == V) {
        *(u32x4_any *)to = __builtin_bit_cast(u32x4, t);
        return;
    }
#pragma unroll
    for (int e = 0; e < V; ++e)
        if (e < n) to[e] = t[e];
}

template <typename T, int V>
__device__ __forceinline__ void widened(float (&v)[V], const u32x4 &w)
{
    T t[V];
    __builtin_memcpy(t, &w, 16);
#pragma unroll
    for (int e = 0; e < V; ++e) v[e] = widen(t[e]);
}

template <typename T, int V>
__device__ __forceinline__ void parameters(float (&v)[V], const void *from, int c, int n, float without)
{
#pragma unroll
    for (int e = 0; e < V; ++e) v[e] = e < n && from ? widen(((const T *)from)[c + e]) : without;
}

// Sums over a group of Q values that every thread has for each of its channels: to LDS by channel and thread, summed down the
// positions, then over the group's channels.  all: reduce_floats() of work.  Each quantity's sums end in
// groups[q][sub][group].
template <int V, int Q>
__device__ __forceinline__ void group_sums(const Map &m, const Place &p, const float (&s)[Q][V], float *all, float *groups)
{
    const int T = blockDim.x, pitch = m.vecs * V, items = m.subs * pitch;
    float *red = all, *col = all + Q * T * V;
    if (p.on)
#pragma unroll
        for (int q = 0; q < Q; ++q)
#pragma unroll
            for (int e = 0; e < V; ++e) red[(q * T + (int)threadIdx.x) * V + e] = e < p.n ? s[q][e] : 0.0f;
    __syncthreads();
    // `parts` threads a channel where there are that many
    int parts = T / items;
    parts = parts < 1 ? 1 : parts > m.lanes ? m.lanes : parts;
    for (int i = threadIdx.x; i < items * parts; i += T) {
        const int part = i / items, at = i - part * items, sub = at / pitch, c = at - sub * pitch;
#pragma unroll
        for (int q = 0; q < Q; ++q) {
            float sum = 0.0f;
            for (int l = part; l < m.lanes; l += parts) sum += red[q * T * V + (sub * m.lanes + l) * pitch + c];
            col[q * T * V + i] = sum;
        }
    }
    __syncthreads();
    const int sets = m.subs * m.groups, each = m.per * parts;
    if (each <= 32) {
        for (int i = threadIdx.x; i < sets * Q; i += T) {
            const int q = i / sets, at = i - q * sets, sub = at / m.groups, g = at - sub * m.groups;
            float sum = 0.0f;
            for (int part = 0; part < parts; ++part)
                for (int k = 0; k < m.per; ++k) sum += col[q * T * V + part * items + sub * pitch + g * m.per + k];
            groups[q * sets + at] = sum;
        }
    } else {   // a wave a group
        const int lane = threadIdx.x & 63;
        for (int i = threadIdx.x >> 6; i < sets * Q; i += T >> 6) {
            const int q = i / sets, at = i - q * sets, sub = at / m.groups, g = at - sub * m.groups;
            float sum = 0.0f;
            for (int part = 0; part < parts; ++part)
                for (int k = lane; k < m.per; k += 64) sum += col[q * T * V + part * items + sub * pitch + g * m.per + k];
#pragma unroll
            for (int h = 1; h < 64; h <<= 1) sum += __shfl_xor(sum, h, 64);
            if (lane == 0) groups[q * sets + at] = sum;
        }
    }
    __syncthreads();
}

// Floats of LDS that group_sums takes for its work.
__host__ __device__ constexpr int reduce_floats(int threads, int V, int Q) { return 2 * Q * threads * V; }
// At most: 512 threads of eight channels and two quantities, or 1024 of four, and two sums of each of 4096 groups.
constexpr int kMostLds = (reduce_floats(512, 8, 2) + 2 * 4096) * 4;
static_assert(reduce_floats(1024, 4, 2) <= reduce_floats(512, 8, 2), "either type");

// A thread's group of each of its channels.
template <int V>
__device__ __forceinline__ void groups_of(int (&g)[V], const Map &m, const Place &p)
{
#pragma unroll
    for (int e = 0; e < V; ++e) g[e] = e < p.n ? p.sub * m.groups + (p.c + e) / m.per : 0;
}

// ---- all positions of a sample in registers ----

template <typename T, int ROWS, int MOST>
__global__ __launch_bounds__(MOST) void k_resident_forward(Norm P)
{
    extern __shared__ float norm_lds[];
    constexpr int V = kVec<T>;
    const Map &m = P.map;
    const int c0 = blockIdx.y * m.width, width = P.C - c0 < m.width ? P.C - c0 : m.width, g0 = c0 / m.per;
    const int groups = width / m.per, sets = m.subs * m.groups;
    const Place p = place<V>(m, width);
    float *first = norm_lds + reduce_floats(blockDim.x, V, 1), *second = first + sets;
    float gamma[V], beta[V];
    int of[V];
    parameters<T, V>(gamma, P.gamma, c0 + p.c, p.n, 1.0f);
    parameters<T, V>(beta, P.beta, c0 + p.c, p.n, 0.0f);
    groups_of(of, m, p);
    const float inv = 1.0f / ((float)P.S * (float)m.per);
    for (long long b0 = (long long)blockIdx.x * m.subs; b0 < P.B; b0 += (long long)gridDim.x * m.subs) {
        const long long b = b0 + p.sub;
        const int S = b < P.B && p.n ? P.S : 0;   // positions of this thread's
        const T *x = (const T *)P.x + b * P.S * P.ldx + c0 + p.c;
        u32x4 w[ROWS];
        float s[1][V] = {};
#pragma unroll
        for (int k = 0; k < ROWS; ++k) {
            const int row = p.row + k * m.lanes;
            w[k] = u32x4{0, 0, 0, 0};
            if (row < S) w[k] = get<T, V>(x + row * P.ldx, p.n);
        }
#pragma unroll
        for (int k = 0; k < ROWS; ++k) {
            float v[V];
            widened<T, V>(v, w[k]);
#pragma unroll
            for (int e = 0; e < V; ++e) s[0][e] += v[e];
        }
        group_sums<V, 1>(m, p, s, norm_lds, first);
        float mean[V];
#pragma unroll
        for (int e = 0; e < V; ++e) mean[e] = first[of[e]] * inv, s[0][e] = 0.0f;
#pragma unroll
        for (int k = 0; k < ROWS; ++k) {
            if (p.row + k * m.lanes >= S) continue;
            float v[V];
            widened<T, V>(v, w[k]);
#pragma unroll
            for (int e = 0; e < V; ++e) s[0][e] = __builtin_fmaf(v[e] - mean[e], v[e] - mean[e], s[0][e]);
        }
        group_sums<V, 1>(m, p, s, norm_lds, second);
        if (P.mean)
            for (int i = threadIdx.x; i < sets; i += blockDim.x) {
                const int sub = i / m.groups, g = i - sub * m.groups;
                if (b0 + sub >= P.B || g >= groups) continue;
                P.mean[(b0 + sub) * P.G + g0 + g] = first[i] * inv;
                P.rstd[(b0 + sub) * P.G + g0 + g] = 1.0f / sqrtf(second[i] * inv + P.eps);
            }
        float a[V];
#pragma unroll
        for (int e = 0; e < V; ++e) a[e] = gamma[e] / sqrtf(second[of[e]] * inv + P.eps);
        T *y = (T *)P.y + b * P.S * P.ldy + c0 + p.c;
#pragma unroll
        for (int k = 0; k < ROWS; ++k) {
            const int row = p.row + k * m.lanes;
            if (row >= S) continue;
            float v[V];
            widened<T, V>(v, w[k]);
#pragma unroll
            for (int e = 0; e < V; ++e) v[e] = __builtin_fmaf(v[e] - mean[e], a[e], beta[e]);
            activate<sizeof(T) == 2>(v, P.act);
            put<T, V>(y + row * P.ldy, v, p.n);
        }
        __syncthreads();   // the sums have been read
    }
}

// dz of a thread's channels at one position, and xhat.
template <typename T, int V>
__device__ __forceinline__ void gradient_at(float (&dz)[V], float (&hat)[V], const u32x4 &x, const u32x4 &dy, const float (&mean)[V],
                                            const float (&rstd)[V], const float (&gamma)[V], const float (&beta)[V], int act)
{
    widened<T, V>(hat, x);
    widened<T, V>(dz, dy);
#pragma unroll
    for (int e = 0; e < V; ++e) hat[e] = (hat[e] - mean[e]) * rstd[e];
    if (act == HQML_ACT_NONE) return;
    float z[V];
#pragma unroll
    for (int e = 0; e < V; ++e) z[e] = __builtin_fmaf(hat[e], gamma[e], beta[e]);
    slope<sizeof(T) == 2>(z, act);
#pragma unroll
    for (int e = 0; e < V; ++e) dz[e] *= z[e];
}

// The workgroup's sums by channel of dz and dz xhat: added over its threads, to the workgroup's row of `part`, or, if it is
// the only one of its channels, to the results.
template <typename T, int V>
__device__ __forceinline__ void parameter_sums(const Norm &P, const Place &p, const float (&s)[2][V], int c0, int width, long long row,
                                               float *lds)
{
    const Map &m = P.map;
    const int T_ = blockDim.x, pitch = m.vecs * V, down = m.lanes * m.subs;
    __syncthreads();
    if (p.on)
#pragma unroll
        for (int q = 0; q < 2; ++q)
#pragma unroll
            for (int e = 0; e < V; ++e) lds[(q * T_ + (int)threadIdx.x) * V + e] = s[q][e];
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * width; i += T_) {
        const int q = i >= width, c = i - q * width;
        float sum = 0.0f;
        for (int l = 0; l < down; ++l) sum += lds[q * T_ * V + l * pitch + c];
        if (P.part) P.part[(row * 2 + q) * P.C + c0 + c] = sum;
        else if (q && P.dgamma) narrow(sum, ((T *)P.dgamma)[c0 + c]);
        else if (!q && P.dbeta) narrow(sum, ((T *)P.dbeta)[c0 + c]);
    }
}

template <typename T, int ROWS, int MOST>
__global__ __launch_bounds__(MOST) void k_resident_backward(Norm P)
{
    extern __shared__ float norm_lds[];
    constexpr int V = kVec<T>;
    const Map &m = P.map;
    const int c0 = blockIdx.y * m.width, width = P.C - c0 < m.width ? P.C - c0 : m.width, g0 = c0 / m.per;
    const int sets = m.subs * m.groups;
    const Place p = place<V>(m, width);
    float *groups = norm_lds + reduce_floats(blockDim.x, V, 2);
    float gamma[V], beta[V], all[2][V] = {};
    int of[V];
    parameters<T, V>(gamma, P.gamma, c0 + p.c, p.n, 1.0f);
    parameters<T, V>(beta, P.beta, c0 + p.c, p.n, 0.0f);
    groups_of(of, m, p);
    const float inv = 1.0f / ((float)P.S * (float)m.per);
    for (long long b0 = (long long)blockIdx.x * m.subs; b0 < P.B; b0 += (long long)gridDim.x * m.subs) {
        const long long b = b0 + p.sub;
        const int S = b < P.B && p.n ? P.S : 0;
        const T *x = (const T *)P.x + b * P.S * P.ldx + c0 + p.c;
        const T *dy = (const T *)P.dy + b * P.S * P.lddy + c0 + p.c;
        u32x4 w[ROWS];
        float dz[ROWS][V], mean[V], rstd[V];
        u32x4 d[ROWS];
#pragma unroll
        for (int k = 0; k < ROWS; ++k) {
            const int row = p.row + k * m.lanes;
            w[k] = d[k] = u32x4{0, 0, 0, 0};
            if (row < S) w[k] = get<T, V>(x + row * P.ldx, p.n), d[k] = get<T, V>(dy + row * P.lddy, p.n);
        }
#pragma unroll
        for (int e = 0; e < V; ++e) {
            const bool some = S > 0 && e < p.n;
            const long long g = b * P.G + g0 + (p.c + e) / m.per;
            mean[e] = some ? P.mean[g] : 0.0f;
            rstd[e] = some ? P.rstd[g] : 0.0f;
        }
        float s[2][V] = {};
#pragma unroll
        for (int k = 0; k < ROWS; ++k) {
            float hat[V];
            gradient_at<T, V>(dz[k], hat, w[k], d[k], mean, rstd, gamma, beta, P.act);
            const bool some = p.row + k * m.lanes < S;
#pragma unroll
            for (int e = 0; e < V; ++e) {
                s[0][e] += some ? dz[k][e] : 0.0f;
                s[1][e] += some ? dz[k][e] * hat[e] : 0.0f;
            }
        }
#pragma unroll
        for (int e = 0; e < V; ++e) {
            all[0][e] += s[0][e], all[1][e] += s[1][e];
            s[0][e] *= gamma[e], s[1][e] *= gamma[e];
        }
        if (P.dx) {
            group_sums<V, 2>(m, p, s, norm_lds, groups);
            T *dx = (T *)P.dx + b * P.S * P.lddx + c0 + p.c;
#pragma unroll
            for (int k = 0; k < ROWS; ++k) {
                const int row = p.row + k * m.lanes;
                if (row >= S) continue;
                float v[V];
                widened<T, V>(v, w[k]);
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    const float hat = (v[e] - mean[e]) * rstd[e];
                    v[e] = rstd[e] * (gamma[e] * dz[k][e] - (groups[of[e]] + hat * groups[sets + of[e]]) * inv);
                }
                put<T, V>(dx + row * P.lddx, v, p.n);
            }
            __syncthreads();   // the sums have been read
        }
    }
    if (P.part || P.dgamma || P.dbeta) parameter_sums<T, V>(P, p, all, c0, width, blockIdx.x, norm_lds);
}

// ---- chunks of positions ----

// Takes a ticket of sample b; whether this workgroup is the sample's last.  What it left before, as device-scope atomics, has
// arrived.
__device__ __forceinline__ bool last_of(const Norm &P, int b)
{
    __shared__ unsigned taken;
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // this wave's stores have arrived
    __syncthreads();                                   // every wave's have
    if (threadIdx.x == 0) taken = __hip_atomic_fetch_add(P.ticket + b, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    __syncthreads();
    if (taken != (unsigned)P.chunks - 1) return false;
    if (threadIdx.x == 0) __hip_atomic_store(P.ticket + b, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    return true;
}

__device__ __forceinline__ void leave(float *to, float v)
{
    __hip_atomic_store(to, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

__device__ __forceinline__ float fetch(const float *from)
{
    return __hip_atomic_load(from, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// Sums over the chunks of a sample of f(chunk, group), for groups g0 .. g0 + n - 1: threads across the groups and down the
// chunks, which meet in lds (a float a thread).  A thread below n receives its group's.
template <typename F>
__device__ __forceinline__ float over_chunks(const Norm &P, int n, float *lds, F f)
{
    const int parts = blockDim.x / n, part = threadIdx.x / n, g = threadIdx.x - part * n;
    float sum = 0.0f;
    if (part < parts)
#pragma unroll 4
        for (int i = part; i < P.chunks; i += parts) sum += f(i, g);
    __syncthreads();   // lds is free
    lds[threadIdx.x] = sum;
    int h = 1;
    while (h < parts) h <<= 1;
    for (h >>= 1; h; h >>= 1) {
        __syncthreads();
        if (part < h && part + h < parts) lds[threadIdx.x] += lds[threadIdx.x + h * n];
    }
    __syncthreads();
    return lds[(int)threadIdx.x < n ? threadIdx.x : 0];
}

constexpr int kStep = 8;   // positions of a thread under way together

// Mean and squared distance from it, of a chunk's groups; the sample's last workgroup joins them.
template <typename T>
__global__ __launch_bounds__(1024) void k_stats(Norm P)
{
    extern __shared__ float norm_lds[];
    constexpr int V = kVec<T>;
    const Map &m = P.map;
    const Place p = place<V>(m, P.C);
    const int b = blockIdx.x / P.chunks, chunk = blockIdx.x - b * P.chunks;
    const int s0 = chunk * P.chunk, s1 = P.S - s0 < P.chunk ? P.S : s0 + P.chunk;
    const T *x = (const T *)P.x + (long long)b * P.S * P.ldx + p.c;
    float *first = norm_lds + reduce_floats(blockDim.x, V, 1), *second = first + m.groups;
    int of[V];
    groups_of(of, m, p);
    // by channel: mean and squared distance of the positions so far, joined eight at a time
    float mean[V] = {}, far[V] = {};
    float count = 0.0f;
    for (int r0 = s0 + p.row; r0 < s1 && p.n; r0 += kStep * m.lanes) {
        u32x4 w[kStep];
        int k_n = 0;
#pragma unroll
        for (int k = 0; k < kStep; ++k) {
            const int row = r0 + k * m.lanes;
            w[k] = u32x4{0, 0, 0, 0};
            if (row < s1) w[k] = get<T, V>(x + (long long)row * P.ldx, p.n), ++k_n;
        }
        const float n = (float)k_n, inv = 1.0f / n, all = count + n, share = n / all;
        float sum[V] = {}, sq[V] = {};
#pragma unroll
        for (int k = 0; k < kStep; ++k) {
            float v[V];
            widened<T, V>(v, w[k]);
#pragma unroll
            for (int e = 0; e < V; ++e) sum[e] += v[e];
        }
#pragma unroll
        for (int e = 0; e < V; ++e) sum[e] *= inv;
#pragma unroll
        for (int k = 0; k < kStep; ++k) {
            if (k >= k_n) continue;
            float v[V];
            widened<T, V>(v, w[k]);
#pragma unroll
            for (int e = 0; e < V; ++e) sq[e] = __builtin_fmaf(v[e] - sum[e], v[e] - sum[e], sq[e]);
        }
#pragma unroll
        for (int e = 0; e < V; ++e) {
            const float d = sum[e] - mean[e];
            far[e] += __builtin_fmaf(d * d, count * share, sq[e]);
            mean[e] = __builtin_fmaf(d, share, mean[e]);
        }
        count = all;
    }
    float s[1][V];
#pragma unroll
    for (int e = 0; e < V; ++e) s[0][e] = mean[e] * count;
    group_sums<V, 1>(m, p, s, norm_lds, first);
    const float values = (float)(s1 - s0) * (float)m.per;
#pragma unroll
    for (int e = 0; e < V; ++e) {
        const float d = mean[e] - first[of[e]] / values;
        s[0][e] = count > 0.0f ? __builtin_fmaf(d * d, count, far[e]) : 0.0f;
    }
    group_sums<V, 1>(m, p, s, norm_lds, second);
    float *mine = P.stat + ((long long)b * P.chunks + chunk) * P.G * 2;
    for (int g = threadIdx.x; g < P.G; g += blockDim.x) {
        leave(mine + g * 2, first[g] / values);
        leave(mine + g * 2 + 1, second[g]);
    }
    if (!last_of(P, b)) return;
    const float *stat = P.stat + (long long)b * P.chunks * P.G * 2;
    auto size = [&](int i) { return (float)((i + 1 == P.chunks ? P.S - i * P.chunk : P.chunk)); };   // positions of a chunk
    const float inv = 1.0f / (float)P.S;
    for (int g0 = 0; g0 < P.G; g0 += blockDim.x) {
        const int n = P.G - g0 < (int)blockDim.x ? P.G - g0 : (int)blockDim.x;
        float *held = norm_lds + blockDim.x;
        const float sum = over_chunks(P, n, norm_lds, [&](int i, int g) {
            return fetch(stat + ((long long)i * P.G + g0 + g) * 2) * (size(i) * inv);
        });
        if ((int)threadIdx.x < n) held[threadIdx.x] = sum;
        __syncthreads();
        const float sq = over_chunks(P, n, norm_lds, [&](int i, int g) {
            const float *at = stat + ((long long)i * P.G + g0 + g) * 2;
            const float d = fetch(at) - held[g];
            return __builtin_fmaf(d * d, size(i) * (float)m.per, fetch(at + 1));
        });
        if ((int)threadIdx.x < n) {
            const long long at = (long long)b * P.G + g0 + threadIdx.x;
            P.mean[at] = held[threadIdx.x];
            P.rstd[at] = 1.0f / sqrtf(sq / ((float)P.S * (float)m.per) + P.eps);
        }
        __syncthreads();
    }
}

template <typename T>
__global__ __launch_bounds__(1024) void k_apply_forward(Norm P)
{
    constexpr int V = kVec<T>;
    const Map &m = P.map;
    const Place p = place<V>(m, P.C);
    const int id = gridDim.x - 1 - blockIdx.x, b = id / P.chunks, chunk = id - b * P.chunks;
    const int s0 = chunk * P.chunk, s1 = P.S - s0 < P.chunk ? P.S : s0 + P.chunk;
    if (!p.n) return;
    const T *x = (const T *)P.x + (long long)b * P.S * P.ldx + p.c;
    T *y = (T *)P.y + (long long)b * P.S * P.ldy + p.c;
    float a[V], beta[V], mean[V];
    parameters<T, V>(a, P.gamma, p.c, p.n, 1.0f);
    parameters<T, V>(beta, P.beta, p.c, p.n, 0.0f);
#pragma unroll
    for (int e = 0; e < V; ++e) {
        const long long g = (long long)b * P.G + (p.c + (e < p.n ? e : 0)) / m.per;
        mean[e] = P.mean[g];
        a[e] *= P.rstd[g];
    }
    for (int r0 = s0 + p.row; r0 < s1; r0 += kStep * m.lanes) {
        u32x4 w[kStep];
#pragma unroll
        for (int k = 0; k < kStep; ++k) {
            const int row = r0 + k * m.lanes;
            w[k] = u32x4{0, 0, 0, 0};
            if (row < s1) w[k] = get<T, V>(x + (long long)row * P.ldx, p.n);
        }
#pragma unroll
        for (int k = 0; k < kStep; ++k) {
            const int row = r0 + k * m.lanes;
            if (row >= s1) continue;
            float v[V];
            widened<T, V>(v, w[k]);
#pragma unroll
            for (int e = 0; e < V; ++e) v[e] = __builtin_fmaf(v[e] - mean[e], a[e], beta[e]);
            activate<sizeof(T) == 2>(v, P.act);
            put<T, V>(y + (long long)row * P.ldy, v, p.n);
        }
    }
}

constexpr int kStepBack = 4;

// The sums behind a chunk's gradients: by channel to `part`, by group, with gamma, joined by the sample's last workgroup.
template <typename T>
__global__ __launch_bounds__(1024) void k_sums(Norm P)
{
    extern __shared__ float norm_lds[];
    constexpr int V = kVec<T>;
    const Map &m = P.map;
    const Place p = place<V>(m, P.C);
    const int b = blockIdx.x / P.chunks, chunk = blockIdx.x - b * P.chunks;
    const int s0 = chunk * P.chunk, s1 = P.S - s0 < P.chunk ? P.S : s0 + P.chunk;
    const T *x = (const T *)P.x + (long long)b * P.S * P.ldx + p.c;
    const T *dy = (const T *)P.dy + (long long)b * P.S * P.lddy + p.c;
    float *groups = norm_lds + reduce_floats(blockDim.x, V, 2);
    float gamma[V], beta[V], mean[V], rstd[V], s[2][V] = {};
    parameters<T, V>(gamma, P.gamma, p.c, p.n, 1.0f);
    parameters<T, V>(beta, P.beta, p.c, p.n, 0.0f);
#pragma unroll
    for (int e = 0; e < V; ++e) {
        const long long g = (long long)b * P.G + (p.c + e) / m.per;
        mean[e] = e < p.n ? P.mean[g] : 0.0f;
        rstd[e] = e < p.n ? P.rstd[g] : 0.0f;
    }
    for (int r0 = s0 + p.row; r0 < s1 && p.n; r0 += kStepBack * m.lanes) {
        u32x4 w[kStepBack], d[kStepBack];
#pragma unroll
        for (int k = 0; k < kStepBack; ++k) {
            const int row = r0 + k * m.lanes;
            w[k] = d[k] = u32x4{0, 0, 0, 0};
            if (row < s1) {
                w[k] = get<T, V>(x + (long long)row * P.ldx, p.n);
                d[k] = get<T, V>(dy + (long long)row * P.lddy, p.n);
            }
        }
#pragma unroll
        for (int k = 0; k < kStepBack; ++k) {
            if (r0 + k * m.lanes >= s1) continue;
            float dz[V], hat[V];
            gradient_at<T, V>(dz, hat, w[k], d[k], mean, rstd, gamma, beta, P.act);
#pragma unroll
            for (int e = 0; e < V; ++e) s[0][e] += dz[e], s[1][e] = __builtin_fmaf(dz[e], hat[e], s[1][e]);
        }
    }
    if (P.part) parameter_sums<T, V>(P, p, s, 0, P.C, (long long)b * P.chunks + chunk, norm_lds);
    if (!P.dx) return;
#pragma unroll
    for (int e = 0; e < V; ++e) s[0][e] *= gamma[e], s[1][e] *= gamma[e];
    __syncthreads();
    group_sums<V, 2>(m, p, s, norm_lds, groups);
    float *mine = P.stat + ((long long)b * P.chunks + chunk) * P.G * 2;
    for (int g = threadIdx.x; g < P.G; g += blockDim.x) {
        leave(mine + g * 2, groups[g]);
        leave(mine + g * 2 + 1, groups[m.groups + g]);
    }
    if (!last_of(P, b)) return;
    const float *stat = P.stat + (long long)b * P.chunks * P.G * 2;
    const float inv = 1.0f / ((float)P.S * (float)m.per);
    const int all = P.G * 2;   // both sums of a group
    for (int g0 = 0; g0 < all; g0 += blockDim.x) {
        const int n = all - g0 < (int)blockDim.x ? all - g0 : (int)blockDim.x;
        const float sum = over_chunks(P, n, norm_lds, [&](int i, int g) { return fetch(stat + (long long)i * all + g0 + g); });
        if ((int)threadIdx.x < n) P.group[(long long)b * all + g0 + threadIdx.x] = sum * inv;
    }
}

template <typename T>
__global__ __launch_bounds__(1024) void k_apply_backward(Norm P)
{
    constexpr int V = kVec<T>;
    const Map &m = P.map;
    const Place p = place<V>(m, P.C);
    const int id = gridDim.x - 1 - blockIdx.x, b = id / P.chunks, chunk = id - b * P.chunks;
    const int s0 = chunk * P.chunk, s1 = P.S - s0 < P.chunk ? P.S : s0 + P.chunk;
    if (!p.n) return;
    const T *x = (const T *)P.x + (long long)b * P.S * P.ldx + p.c;
    const T *dy = (const T *)P.dy + (long long)b * P.S * P.lddy + p.c;
    T *dx = (T *)P.dx + (long long)b * P.S * P.lddx + p.c;
    float gamma[V], beta[V], mean[V], rstd[V], one[V], two[V];
    parameters<T, V>(gamma, P.gamma, p.c, p.n, 1.0f);
    parameters<T, V>(beta, P.beta, p.c, p.n, 0.0f);
#pragma unroll
    for (int e = 0; e < V; ++e) {
        const long long g = (long long)b * P.G + (p.c + (e < p.n ? e : 0)) / m.per;
        mean[e] = P.mean[g], rstd[e] = P.rstd[g];
        one[e] = P.group[g * 2], two[e] = P.group[g * 2 + 1];
    }
    for (int r0 = s0 + p.row; r0 < s1; r0 += kStepBack * m.lanes) {
        u32x4 w[kStepBack], d[kStepBack];
#pragma unroll
        for (int k = 0; k < kStepBack; ++k) {
            const int row = r0 + k * m.lanes;
            w[k] = d[k] = u32x4{0, 0, 0, 0};
            if (row < s1) {
                w[k] = get<T, V>(x + (long long)row * P.ldx, p.n);
                d[k] = get<T, V>(dy + (long long)row * P.lddy, p.n);
            }
        }
#pragma unroll
        for (int k = 0; k < kStepBack; ++k) {
            const int row = r0 + k * m.lanes;
            if (row >= s1) continue;
            float dz[V], hat[V];
            gradient_at<T, V>(dz, hat, w[k], d[k], mean, rstd, gamma, beta, P.act);
#pragma unroll
            for (int e = 0; e < V; ++e) dz[e] = rstd[e] * (gamma[e] * dz[e] - (one[e] + hat[e] * two[e]));
            put<T, V>(dx + (long long)row * P.lddx, dz, p.n);
        }
    }
}

// dgamma and dbeta: the sums over `rows` partial ones, eight channels a workgroup, 32 threads down the rows.
template <typename T>
__global__ __launch_bounds__(256) void k_parameters(const float *part, int rows, int C, T *dgamma, T *dbeta)
{
    __shared__ float held[32][8];
    const int lane = threadIdx.x & 7, down = threadIdx.x >> 3, c = blockIdx.x * 8 + lane, q = blockIdx.y;
    float s = 0.0f;
    if (c < C)
#pragma unroll 4
        for (int r = down; r < rows; r += 32) s += part[((long long)r * 2 + q) * C + c];
    held[down][lane] = s;
    __syncthreads();
    if (down || c >= C) return;
#pragma unroll
    for (int k = 1; k < 32; ++k) s += held[k][lane];
    T *to = q ? dgamma : dbeta;
    if (to) narrow(s, to[c]);
}

template <typename T>
__global__ void k_zero(T *a, T *b, int n)
{
    const int i = blockIdx.x * 256 + threadIdx.x;
    if (i < n && a) a[i] = T{};
    if (i < n && b) b[i] = T{};
}

// ---- which runs, and how it is cut ----

constexpr int kUnits = 256;          // compute units
constexpr int kSplitGroups = 2048;   // workgroups that a split call aims at
constexpr int kResidentMost = 1024;  // workgroups of a span in a resident backward pass
constexpr int kMinSegment = 64;      // bytes of a row that a span has at least, unless the array is small
constexpr long long kSmallArray = 1 << 20;

int ceil_div(long long a, long long b) { return (int)((a + b - 1) / b); }

// Threads of a split kernel, and those down the positions, for C channels.
template <typename T>
int split_threads(int C)
{
    const int vecs = ceil_div(C, kVec<T>);
    return vecs <= 256 ? 256 : vecs <= 512 ? 512 : 1024;
}
template <typename T>
int split_lanes(int C)
{
    return split_threads<T>(C) / ceil_div(C, kVec<T>);
}

// The most positions of a thread: what its registers hold (backward: x, and dz in 32 bits), by the size of the workgroup.
constexpr int kMostForward = 16, kMostBackward = 8, kMostOf1024 = 4;

struct Resident {
    bool fits;
    int threads, rows, spans;
    Map map;
};

template <typename T>
Resident resident(int B, int S, int C, int G, int most)
{
    constexpr int V = kVec<T>;
    const int per = C / G;
    Resident r{};
    Map &m = r.map;
    // spans of whole groups: as many as give every compute unit one workgroup, of at least kMinSegment bytes of a row
    const bool small = (long long)B * S * C * (int)sizeof(T) <= kSmallArray;
    const int least = small ? per : std::max(1, ceil_div(kMinSegment / (int)sizeof(T), per)) * per;
    int all = 0;   // threads down the positions that there can be
    for (int spans = std::min(ceil_div(kUnits, B), std::max(1, C / least));; ++spans) {
        const int each = ceil_div(G, std::min(spans, G));   // groups of a span
        r.spans = ceil_div(G, each);
        m.width = each * per;
        m.groups = each;
        m.vecs = ceil_div(m.width, V);
        const int threads = m.vecs <= 512 ? 512 : 1024;
        all = threads / m.vecs;
        const long long room = (long long)all * (threads == 512 ? most : kMostOf1024);
        if (room >= S) break;
        if (m.width <= least || spans >= G) return r;   // does not fit
    }
    r.fits = true;
    m.per = per;
    r.rows = ceil_div(S, all);
    m.lanes = ceil_div(S, r.rows);
    // small samples share a workgroup of four waves
    m.subs = std::max(1, std::min({all / m.lanes, 256 / (m.vecs * m.lanes), B}));
    r.threads = ceil_div(m.vecs * m.lanes * m.subs, 64) * 64;
    return r;
}

Norm common(const NormCall &a)
{
    Norm P{};
    P.B = a.B, P.S = a.S, P.C = a.C, P.G = a.G;
    P.x = a.x, P.gamma = a.gamma, P.beta = a.beta, P.dy = a.dy;
    P.ldx = a.ldx, P.ldy = a.ldy, P.lddy = a.lddy, P.lddx = a.lddx;
    P.y = a.y, P.dx = a.dx;
    P.mean = a.mean, P.rstd = a.rstd;
    P.act = a.act, P.eps = a.eps;
    return P;
}

// Cuts a split call; the threads of its workgroups.
template <typename T>
int cut(Norm &P, const NormWorkspace &ws)
{
    Map &m = P.map;
    m.width = P.C;
    m.vecs = ceil_div(P.C, kVec<T>);
    m.lanes = split_lanes<T>(P.C);
    m.subs = 1;
    m.per = P.C / P.G;
    m.groups = P.G;
    const long long rows = (long long)P.B * P.S;
    P.chunk = (int)std::min<long long>(P.S, std::max<long long>(m.lanes * kStep, (rows + kSplitGroups - 1) / kSplitGroups));
    P.chunks = ceil_div(P.S, P.chunk);
    P.stat = ws.part;
    P.group = ws.group;
    P.ticket = ws.ticket;
    return split_threads<T>(P.C);
}

// What a split call of up to `rows` positions in all takes at most: samples, and chunks of all of them.  A sample that is
// split has more positions than any resident workgroup holds across all channels.
template <typename T>
void split_most(long long rows, int C, long long &samples, long long &chunks)
{
    samples = rows / (split_lanes<T>(C) * kMostOf1024 + 1);
    chunks = samples ? kSplitGroups + samples : 0;
}

bool fits(const Norm &P, const NormWorkspace &ws, bool parameters)
{
    const size_t chunks = (size_t)P.B * P.chunks;
    return chunks * (2 * P.G + (parameters ? 2 * P.C : 0)) * 4 <= ws.part_bytes && (size_t)P.B * P.G * 8 <= ws.group_bytes &&
           (size_t)P.B * sizeof(unsigned) <= ws.ticket_bytes;
}

size_t lds_bytes(int threads, int V, int Q, int sets) { return (size_t)(reduce_floats(threads, V, Q) + 2 * sets) * 4; }

template <typename T>
hipError_t forward(const NormCall &a, const NormWorkspace &ws, hipStream_t s)
{
    Norm P = common(a);
    const Resident r = resident<T>(a.B, a.S, a.C, a.G, kMostForward);
    if (r.fits) {
        P.map = r.map;
        const dim3 grid((unsigned)std::min(ceil_div(a.B, r.map.subs), 1 << 20), (unsigned)r.spans);
        const size_t lds = lds_bytes(r.threads, kVec<T>, 1, r.map.subs * r.map.groups);
        if (r.threads > 512) k_resident_forward<T, kMostOf1024, 1024><<<grid, r.threads, lds, s>>>(P);
        else if (r.rows <= 1) k_resident_forward<T, 1, 512><<<grid, r.threads, lds, s>>>(P);
        else if (r.rows <= 4) k_resident_forward<T, 4, 512><<<grid, r.threads, lds, s>>>(P);
        else k_resident_forward<T, kMostForward, 512><<<grid, r.threads, lds, s>>>(P);
        return hipGetLastError();
    }
    const int threads = cut<T>(P, ws);
    if (!fits(P, ws, false)) return hipErrorInvalidValue;
    if (!P.mean) P.mean = ws.group, P.rstd = ws.group + (size_t)a.B * a.G;
    const unsigned grid = (unsigned)a.B * (unsigned)P.chunks;
    k_stats<T><<<grid, threads, lds_bytes(threads, kVec<T>, 1, a.G), s>>>(P);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    k_apply_forward<T><<<grid, threads, 0, s>>>(P);
    return hipGetLastError();
}

template <typename T>
hipError_t backward(const NormCall &a, const NormWorkspace &ws, hipStream_t s)
{
    Norm P = common(a);
    const bool parameters = a.dgamma || a.dbeta;
    int rows = 0;   // of partial sums
    const Resident r = resident<T>(a.B, a.S, a.C, a.G, kMostBackward);
    if (r.fits) {
        P.map = r.map;
        const dim3 grid((unsigned)std::min(ceil_div(a.B, r.map.subs), kResidentMost), (unsigned)r.spans);
        if (parameters && grid.x > 1) {
            rows = (int)grid.x;
            P.part = ws.part;
            if ((size_t)rows * 2 * a.C * 4 > ws.part_bytes) return hipErrorInvalidValue;
        } else {
            P.dgamma = a.dgamma, P.dbeta = a.dbeta;
        }
        const size_t lds = lds_bytes(r.threads, kVec<T>, 2, r.map.subs * r.map.groups);
        if (r.threads > 512) k_resident_backward<T, kMostOf1024, 1024><<<grid, r.threads, lds, s>>>(P);
        else if (r.rows <= 1) k_resident_backward<T, 1, 512><<<grid, r.threads, lds, s>>>(P);
        else if (r.rows <= 4) k_resident_backward<T, 4, 512><<<grid, r.threads, lds, s>>>(P);
        else k_resident_backward<T, kMostBackward, 512><<<grid, r.threads, lds, s>>>(P);
    } else {
        const int threads = cut<T>(P, ws);
        if (!fits(P, ws, parameters)) return hipErrorInvalidValue;
        const unsigned grid = (unsigned)a.B * (unsigned)P.chunks;
        if (parameters) rows = (int)grid, P.part = ws.part + (size_t)grid * 2 * a.G;
        k_sums<T><<<grid, threads, lds_bytes(threads, kVec<T>, 2, a.G), s>>>(P);
        hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        if (a.dx) k_apply_backward<T><<<grid, threads, 0, s>>>(P);
    }
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || !rows) return e;
    k_parameters<T><<<dim3((unsigned)ceil_div(a.C, 8), 2), 256, 0, s>>>(P.part, rows, a.C, (T *)a.dgamma, (T *)a.dbeta);
    return hipGetLastError();
}

// More dynamic LDS than 64 KB has to be allowed.
template <typename T>
hipError_t configure()
{
    const void *kernels[] = {(const void *)k_resident_forward<T, 1, 512>,          (const void *)k_resident_forward<T, 4, 512>,
                             (const void *)k_resident_forward<T, kMostForward, 512>, (const void *)k_resident_forward<T, kMostOf1024, 1024>,
                             (const void *)k_resident_backward<T, 1, 512>,         (const void *)k_resident_backward<T, 4, 512>,
                             (const void *)k_resident_backward<T, kMostBackward, 512>,
                             (const void *)k_resident_backward<T, kMostOf1024, 1024>, (const void *)k_stats<T>, (const void *)k_sums<T>};
    for (const void *k : kernels) {
        const hipError_t e = hipFuncSetAttribute(k, hipFuncAttributeMaxDynamicSharedMemorySize, kMostLds);
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

template <typename T>
NormWorkspace workspace(const hqml_norm_config &c)
{
    NormWorkspace ws;
    long long samples, chunks;
    split_most<T>(c.max_rows, c.channels, samples, chunks);
    const size_t C = (size_t)c.channels, G = (size_t)c.groups;
    ws.part_bytes = std::max((size_t)chunks * (2 * G + 2 * C), std::min<size_t>(kResidentMost, (size_t)c.max_rows) * 2 * C) * 4;
    ws.group_bytes = (size_t)samples * G * 8;
    ws.ticket_bytes = (size_t)samples * sizeof(unsigned);
    return ws;
}

}  // namespace

NormWorkspace norm_workspace(const hqml_norm_config &cfg)
{
    return cfg.dtype == HQML_DTYPE_BF16 ? workspace<bf16>(cfg) : workspace<float>(cfg);
}

hipError_t configure_norm(int dtype)
{
    return dtype == HQML_DTYPE_BF16 ? configure<bf16>() : configure<float>();
}

hipError_t launch_norm_forward(const NormCall &a, int dtype, const NormWorkspace &ws, hipStream_t s)
{
    return dtype == HQML_DTYPE_BF16 ? forward<bf16>(a, ws, s) : forward<float>(a, ws, s);
}

hipError_t launch_norm_backward(const NormCall &a, int dtype, const NormWorkspace &ws, hipStream_t s)
{
    if ((long long)a.B * a.S == 0) {
        const unsigned grid = (unsigned)ceil_div(a.C, 256);
        if (dtype == HQML_DTYPE_BF16) k_zero<bf16><<<grid, 256, 0, s>>>((bf16 *)a.dgamma, (bf16 *)a.dbeta, a.C);
        else k_zero<float><<<grid, 256, 0, s>>>((float *)a.dgamma, (float *)a.dbeta, a.C);
        return hipGetLastError();
    }
    return dtype == HQML_DTYPE_BF16 ? backward<bf16>(a, ws, s) : backward<float>(a, ws, s);
}

}  // namespace hqml
