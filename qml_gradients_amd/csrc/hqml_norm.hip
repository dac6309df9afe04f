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
//                 variance is formed of what is left after the mean.  Small samples share a workgroup.  Bound by latency
//                 (a load, two reductions with barriers, a store): 784 x 32 fp32 7.7 us (6.6 at least), 1000 x 784 fp32 9.5
//                 forward and 10.2 + 3.9 backward.
//   k_stats, k_sums with k_apply_*  larger samples: workgroups take chunks of positions; the last one of a sample to finish puts
//                 the chunks' statistics together (in their order, so no result depends on timing), and a second kernel reads
//                 x again, in the opposite order, to find its end still in the last-level cache.  32 x 4096 x 512 bf16,
//                 silu: statistics 30 us (4.5 TB/s), forward 47 (5.7), sums 64 (4.2; arithmetic takes 59 % of their
//                 busy cycles), backward 70 (5.7).
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

// Division of numbers below 2^16 by one of those, by the high half of a product (an integer division takes forty
// instructions): with magic = ceil(2^32 / by), magic by is less than `by` above 2^32, and n times that less than 2^32.
struct Div {
    unsigned by, magic;
    Div() = default;
    explicit Div(int d) : by((unsigned)d), magic((unsigned)(((1ull << 32) + d - 1) / d)) {}   // 0 for 1
    __device__ __forceinline__ int operator()(int n) const { return magic ? (int)__umulhi((unsigned)n, magic) : n; }
};

// How a workgroup's threads share `width` channels (a span of whole groups, or all) and the positions of `subs` samples.  Every
// thread leaves one value for its groups' sums where all its channels are of one group, one for each of them otherwise; `each`
// lanes (a power of two, up to a wave) put a group's together.
struct Map {
    int width, vecs;    // channels, threads across them
    int lanes;          // threads down the positions of a sample
    int subs;
    int per;            // channels of a group
    int groups;         // of the span
    int wide, pitch, mine;   // values of a thread, of a position; of a group in it
    int sets, each;          // groups of all samples
    float channels;          // that a value stands for
    Div by_vecs, by_lanes, by_per, by_groups, by_mine;
};

struct Norm {
    int B, S, C, G;
    const void *x, *gamma, *beta, *dy;
    long long ldx, ldy, lddy, lddx;
    void *y, *dx;
    float *mean, *rstd;
    int act;
    float eps;
    float *part;        // backward: partial sums [rows][2][C] of dbeta and dgamma; null: the only workgroup of a span writes those
    void *dgamma, *dbeta;
    int add;            // whether they are added to what an earlier launch left there
    int rows, extra;
    int ahead;          // rows that hold a thread's channels at least
    Map map;
    // split
    int chunk, chunks;      // positions of a chunk, chunks of a sample
    float *stat;            // [B][chunks][G][2]
    float *group;           // [B][G][2]
    unsigned *ticket;       // [B], kTicketStep apart, 0 between calls
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
    const int rl = m.by_vecs((int)threadIdx.x), cv = (int)threadIdx.x - rl * m.vecs;
    p.c = cv * V;
    p.sub = m.by_lanes(rl);
    p.row = rl - p.sub * m.lanes;
    p.on = p.sub < m.subs;
    p.n = !p.on || p.c >= width ? 0 : width - p.c < V ? width - p.c : V;
    return p;
}

// Positions of sample b from which V channels may be read from channel c on, though they pass the row's end: all but the last
// ones of the array.
template <int V>
__device__ __forceinline__ int rows_before_the_end(const Norm &P, long long b, int c)
{
    if (c + V <= P.C) return P.S;
    const long long left = (P.B - b) * (long long)P.S - P.ahead;
    return left < P.S ? (int)left : P.S;
}

// A thread's channels at one position, of which n exist.  beyond: those that follow in memory may be read in their stead (they
// are the row's next ones, or the next row's), which costs one load where n take one each.
template <typename T, int V>
__device__ __forceinline__ u32x4 get(const T *from, int n, bool beyond)
{
    if (n == V || beyond) return *(const u32x4_any *)from;
    T t[V] = {};
#pragma unroll
    for (int e = 0; e < V; ++e)
        if (e < n) t[e] = from[e];
    return __builtin_bit_cast(u32x4, t);
}

template <typename T, int V>
__device__ __forceinline__ void put(T *to, const float (&v)[V], int n)
{
    using u32x2_any = __attribute__((ext_vector_type(2), aligned(2))) uint32_t;
    using u32_any = __attribute__((aligned(2))) uint32_t;
    T t[V];
#pragma unroll
    for (int e = 0; e < V; ++e) narrow(v[e], t[e]);
    const u32x4 w = __builtin_bit_cast(u32x4, t);
    if (n == V) {
        *(u32x4_any *)to = w;
        return;
    }
    const int bytes = n * (int)sizeof(T);   // halves of what is left
    char *at = (char *)to;
    if (bytes & 8) *(u32x2_any *)at = u32x2_any{w[0], w[1]};
    if (bytes & 4) *(u32_any *)(at + (bytes & 8)) = bytes & 8 ? w[2] : w[0];
    if (bytes & 2) *(uint16_t *)(at + (bytes & 12)) = (uint16_t)(bytes & 8 ? bytes & 4 ? w[3] : w[2] : bytes & 4 ? w[1] : w[0]);
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

// The sum of n lanes beside each other (a power of two, the same in the whole wave), in all of them.
__device__ __forceinline__ float lanes_sum(float v, int n)
{
    auto with = [&](int moved) { v += __builtin_bit_cast(float, moved); };
    auto bits = [&] { return __builtin_bit_cast(int, v); };
    if (n >= 2) with(__builtin_amdgcn_update_dpp(0, bits(), 0xB1, 0xF, 0xF, true));    // lane ^ 1
    if (n >= 4) with(__builtin_amdgcn_update_dpp(0, bits(), 0x4E, 0xF, 0xF, true));    // lane ^ 2
    if (n >= 8) with(__builtin_amdgcn_update_dpp(0, bits(), 0x141, 0xF, 0xF, true));   // mirrored in eight
    if (n >= 16) with(__builtin_amdgcn_update_dpp(0, bits(), 0x140, 0xF, 0xF, true));  // mirrored in sixteen
    if (n >= 32) v += __shfl_xor(v, 16, 64);
    if (n >= 64) v += __shfl_xor(v, 32, 64);
    return v;
}

// A thread's Q values for each of its channels, left for its workgroup.
template <int V, int Q>
__device__ __forceinline__ void leave_sums(const Map &m, const Place &p, const float (&s)[Q][V], float *all)
{
    const int T = blockDim.x;
    if (!p.on) return;
#pragma unroll
    for (int q = 0; q < Q; ++q) {
        float sum = 0.0f;
#pragma unroll
        for (int e = 0; e < V; ++e) {
            if (m.wide == 1) sum += e < p.n ? s[q][e] : 0.0f;
            else all[(q * T + (int)threadIdx.x) * V + e] = e < p.n ? s[q][e] : 0.0f;
        }
        if (m.wide == 1) all[q * T + (int)threadIdx.x] = sum;
    }
}

// Calls f(at, l) for the values of a set that are this lane's: at is the value's place, l the thread down the positions.
template <typename F>
__device__ __forceinline__ void each_value(const Map &m, int set, int lane, F take)
{
    const int sub = m.by_groups(set), g = set - sub * m.groups;
    const int from = sub * m.lanes * m.pitch + g * m.mine;
    int l = m.by_mine(lane), k = lane - l * m.mine;
    const int dl = m.by_mine(m.each), dk = m.each - dl * m.mine, n = (m.mine * m.lanes - lane + m.each - 1) >> __builtin_ctz(m.each);
#pragma unroll 4
    for (int i = 0; i < n; ++i) {
        take(from + l * m.pitch + k, l);
        l += dl, k += dk;
        if (k >= m.mine) k -= m.mine, ++l;
    }
}

// Sums over a group of Q values that every thread has for each of its channels; each quantity's end in groups[q][set].
template <int V, int Q>
__device__ __forceinline__ void group_sums(const Map &m, const Place &p, const float (&s)[Q][V], float *all, float *groups)
{
    const int T = blockDim.x;
    leave_sums<V, Q>(m, p, s, all);
    __syncthreads();
    const int lane = threadIdx.x & (m.each - 1), stride = m.wide == 1 ? T : T * V;
    for (int set = (int)(threadIdx.x >> __builtin_ctz(m.each)); set < m.sets; set += T >> __builtin_ctz(m.each)) {
        float sum[Q] = {};
        each_value(m, set, lane, [&](int at, int) {
#pragma unroll
            for (int q = 0; q < Q; ++q) sum[q] += all[q * stride + at];
        });
#pragma unroll
        for (int q = 0; q < Q; ++q) {
            sum[q] = lanes_sum(sum[q], m.each);
            if (lane == 0) groups[q * m.sets + set] = sum[q];
        }
    }
    __syncthreads();
}

// Mean of a group, and the sum of squared distances from it, of what the threads have: the sum of each channel over the
// thread's positions (count: positions), and the squared distances from its own mean.  Values that stand for several channels
// (wide == 1) are joined in the thread first.  positions: of the sample or chunk.  The results end in groups[0][set],
// groups[1][set].
template <int V>
__device__ __forceinline__ void group_moments(const Map &m, const Place &p, float (&sum)[V], float (&far)[V], float count,
                                              int positions, float *all, float *groups)
{
    const int T = blockDim.x;
    float s[2][V];
    if (m.wide == 1) {
        float total = 0.0f, squares = 0.0f;
#pragma unroll
        for (int e = 0; e < V; ++e) total += sum[e];
        const float one = count > 0.0f ? 1.0f / count : 0.0f, mean = total * one * (1.0f / V);
#pragma unroll
        for (int e = 0; e < V; ++e) {
            const float d = __builtin_fmaf(sum[e], one, -mean);
            squares += __builtin_fmaf(d * d, count, far[e]);
        }
#pragma unroll
        for (int e = 0; e < V; ++e) s[0][e] = e ? 0.0f : total, s[1][e] = e ? 0.0f : squares;
    } else {
#pragma unroll
        for (int e = 0; e < V; ++e) s[0][e] = sum[e], s[1][e] = far[e];
    }
    leave_sums<V, 2>(m, p, s, all);
    __syncthreads();
    const int lane = threadIdx.x & (m.each - 1), stride = m.wide == 1 ? T : T * V;
    const int some = positions / m.lanes, more = positions - some * m.lanes;   // positions of a thread: one more for the first ones
    const float inv = 1.0f / ((float)positions * (float)m.per);
    const float n0 = (float)some * m.channels, n1 = (float)(some + 1) * m.channels, i0 = some ? 1.0f / n0 : 0.0f, i1 = 1.0f / n1;
    for (int set = (int)(threadIdx.x >> __builtin_ctz(m.each)); set < m.sets; set += T >> __builtin_ctz(m.each)) {
        float total = 0.0f, squares = 0.0f;
        each_value(m, set, lane, [&](int at, int) { total += all[at]; });
        const float mean = lanes_sum(total, m.each) * inv;
        each_value(m, set, lane, [&](int at, int l) {
            const float d = __builtin_fmaf(all[at], l < more ? i1 : i0, -mean);
            squares += l < more || some ? __builtin_fmaf(d * d, l < more ? n1 : n0, all[stride + at]) : 0.0f;
        });
        squares = lanes_sum(squares, m.each);
        if (lane == 0) groups[set] = mean, groups[m.sets + set] = squares;
    }
    __syncthreads();
}

// Floats of LDS that these take for their work.
__host__ __device__ constexpr int reduce_floats(int threads, int V) { return 2 * threads * V; }
// At most: 1024 threads of eight channels, and two sums of each of their channels' groups.
constexpr int kMostLds = 160 * 1024 - 4096;

// A thread's group of each of its channels.
template <int V>
__device__ __forceinline__ void groups_of(int (&g)[V], const Map &m, const Place &p)
{
#pragma unroll
    for (int e = 0; e < V; ++e) g[e] = e < p.n ? p.sub * m.groups + m.by_per(p.c + e) : 0;
}

// ---- all positions of a sample in registers ----

template <typename T, int ROWS, int MOST>
__global__ __launch_bounds__(MOST) void k_resident_forward(Norm P)
{
    extern __shared__ float norm_lds[];
    constexpr int V = kVec<T>;
    const Map &m = P.map;
    const int c0 = blockIdx.y * m.width, width = P.C - c0 < m.width ? P.C - c0 : m.width, g0 = m.by_per(c0);
    const int groups = m.by_per(width), sets = m.sets;
    const Place p = place<V>(m, width);
    float *first = norm_lds + reduce_floats(blockDim.x, V), *second = first + sets;
    float gamma[V], beta[V];
    int of[V];
    parameters<T, V>(gamma, P.gamma, c0 + p.c, p.n, 1.0f);
    parameters<T, V>(beta, P.beta, c0 + p.c, p.n, 0.0f);
    groups_of(of, m, p);
    const float inv = 1.0f / ((float)P.S * (float)m.per);
    for (long long b0 = (long long)blockIdx.x * m.subs; b0 < P.B; b0 += (long long)gridDim.x * m.subs) {
        const long long b = b0 + p.sub;
        const int S = b < P.B && p.n ? P.S : 0;   // positions of this thread's
        const int beyond = rows_before_the_end<V>(P, b, c0 + p.c);
        const T *x = (const T *)P.x + b * P.S * P.ldx + c0 + p.c;
        u32x4 w[ROWS];
        float sum[V] = {}, far[V] = {}, count = 0.0f;
#pragma unroll
        for (int k = 0; k < ROWS; ++k) {
            const int row = p.row + k * m.lanes;
            w[k] = u32x4{0, 0, 0, 0};
            if (row < S) w[k] = get<T, V>(x + row * P.ldx, p.n, row < beyond), count += 1.0f;
        }
#pragma unroll
        for (int k = 0; k < ROWS; ++k) {
            float v[V];
            widened<T, V>(v, w[k]);
#pragma unroll
            for (int e = 0; e < V; ++e) sum[e] += v[e];
        }
        if (ROWS > 1) {
            const float one = 1.0f / count;
#pragma unroll
            for (int k = 0; k < ROWS; ++k) {
                if (p.row + k * m.lanes >= S) continue;
                float v[V];
                widened<T, V>(v, w[k]);
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    const float d = __builtin_fmaf(sum[e], -one, v[e]);
                    far[e] = __builtin_fmaf(d, d, far[e]);
                }
            }
        }
        group_moments<V>(m, p, sum, far, count, P.S, norm_lds, first);
        float mean[V];
#pragma unroll
        for (int e = 0; e < V; ++e) mean[e] = first[of[e]];
        if (P.mean)
            for (int i = threadIdx.x; i < sets; i += blockDim.x) {
                const int sub = m.by_groups(i), g = i - sub * m.groups;
                if (b0 + sub >= P.B || g >= groups) continue;
                P.mean[(b0 + sub) * P.G + g0 + g] = first[i];
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

// dz of a thread's channels at one position, and x - mean; scale: rstd gamma.
template <typename T, int V>
__device__ __forceinline__ void gradient_at(float (&dz)[V], float (&far)[V], const u32x4 &x, const u32x4 &dy, const float (&mean)[V],
                                            const float (&scale)[V], const float (&beta)[V], int act)
{
    widened<T, V>(far, x);
    widened<T, V>(dz, dy);
#pragma unroll
    for (int e = 0; e < V; ++e) far[e] -= mean[e];
    if (act == HQML_ACT_NONE) return;
    float z[V];
#pragma unroll
    for (int e = 0; e < V; ++e) z[e] = __builtin_fmaf(far[e], scale[e], beta[e]);
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
    int each = 1;   // lanes of a sum
    while (each < 64 && each * 4 * width <= T_ && each < down) each <<= 1;
    const int lane = threadIdx.x & (each - 1);
    for (int i = (int)threadIdx.x / each; i < 2 * width; i += T_ / each) {
        const int q = i >= width, c = i - q * width;
        float sum = 0.0f;
#pragma unroll 4
        for (int l = lane; l < down; l += each) sum += lds[q * T_ * V + l * pitch + c];
        sum = lanes_sum(sum, each);
        if (lane) continue;
        if (P.part) {
            float *to = P.part + (row * 2 + q) * P.C + c0 + c;
            *to = P.add ? *to + sum : sum;
        } else if (q && P.dgamma) {
            narrow(sum, ((T *)P.dgamma)[c0 + c]);
        } else if (!q && P.dbeta) {
            narrow(sum, ((T *)P.dbeta)[c0 + c]);
        }
    }
}

template <typename T, int ROWS, int MOST>
__global__ __launch_bounds__(MOST) void k_resident_backward(Norm P)
{
    extern __shared__ float norm_lds[];
    constexpr int V = kVec<T>;
    const Map &m = P.map;
    const int c0 = blockIdx.y * m.width, width = P.C - c0 < m.width ? P.C - c0 : m.width, g0 = m.by_per(c0);
    const int sets = m.sets;
    const Place p = place<V>(m, width);
    float *groups = norm_lds + reduce_floats(blockDim.x, V);
    float gamma[V], beta[V], all[2][V] = {};
    int of[V];
    parameters<T, V>(gamma, P.gamma, c0 + p.c, p.n, 1.0f);
    parameters<T, V>(beta, P.beta, c0 + p.c, p.n, 0.0f);
    groups_of(of, m, p);
    const float inv = 1.0f / ((float)P.S * (float)m.per);
    for (long long b0 = (long long)blockIdx.x * m.subs; b0 < P.B; b0 += (long long)gridDim.x * m.subs) {
        const long long b = b0 + p.sub;
        const int S = b < P.B && p.n ? P.S : 0;
        const int beyond = rows_before_the_end<V>(P, b, c0 + p.c);
        const T *x = (const T *)P.x + b * P.S * P.ldx + c0 + p.c;
        const T *dy = (const T *)P.dy + b * P.S * P.lddy + c0 + p.c;
        u32x4 w[ROWS];
        float dz[ROWS][V], mean[V], rstd[V], scale[V];
        u32x4 d[ROWS];
#pragma unroll
        for (int k = 0; k < ROWS; ++k) {
            const int row = p.row + k * m.lanes;
            w[k] = d[k] = u32x4{0, 0, 0, 0};
            if (row < S) {
                w[k] = get<T, V>(x + row * P.ldx, p.n, row < beyond);
                d[k] = get<T, V>(dy + row * P.lddy, p.n, row < beyond);
            }
        }
#pragma unroll
        for (int e = 0; e < V; ++e) {
            const bool some = S > 0 && e < p.n;
            const long long g = b * P.G + g0 + m.by_per(p.c + e);
            mean[e] = some ? P.mean[g] : 0.0f;
            rstd[e] = some ? P.rstd[g] : 0.0f;
            scale[e] = rstd[e] * gamma[e];
        }
        float s[2][V] = {};
#pragma unroll
        for (int k = 0; k < ROWS; ++k) {
            float far[V];
            gradient_at<T, V>(dz[k], far, w[k], d[k], mean, scale, beta, P.act);
            const bool some = p.row + k * m.lanes < S;
#pragma unroll
            for (int e = 0; e < V; ++e) {
                s[0][e] += some ? dz[k][e] : 0.0f;
                s[1][e] += some ? dz[k][e] * far[e] : 0.0f;
            }
        }
#pragma unroll
        for (int e = 0; e < V; ++e) {
            s[1][e] *= rstd[e];
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
    if (P.dgamma || P.dbeta) parameter_sums<T, V>(P, p, all, c0, width, blockIdx.x, norm_lds);
}

// ---- chunks of positions ----

// Tickets lie in cache lines of their own: atomics on one line come one after the other (8 x 4096 positions of 512 channels fp32,
// statistics: eight tickets beside each other 27 us, apart 19.6; without any joining 13.7).
constexpr int kTicketStep = 32;

// Takes a ticket of sample b; whether this workgroup is the sample's last.  What it left before, as device-scope atomics, has
// arrived.
__device__ __forceinline__ bool last_of(const Norm &P, int b)
{
    __shared__ unsigned taken;
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // this wave's stores have arrived
    __syncthreads();                                   // every wave's have
    if (threadIdx.x == 0) taken = __hip_atomic_fetch_add(P.ticket + b * kTicketStep, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    __syncthreads();
    if (taken != (unsigned)P.chunks - 1) return false;
    if (threadIdx.x == 0) __hip_atomic_store(P.ticket + b * kTicketStep, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    return true;
}

using f32x2 = __attribute__((ext_vector_type(2))) float;

__device__ __forceinline__ void leave(float *to, float a, float b)
{
    __hip_atomic_store((unsigned long long *)to, __builtin_bit_cast(unsigned long long, f32x2{a, b}), __ATOMIC_RELAXED,
                       __HIP_MEMORY_SCOPE_AGENT);
}

__device__ __forceinline__ f32x2 fetch(const float *from)
{
    return __builtin_bit_cast(f32x2, __hip_atomic_load((const unsigned long long *)from, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT));
}

// What the chunks of a sample left for n groups from g0 on, put together in their order: threads across the groups and down the
// chunks.  take(value, pair, chunk) adds a chunk's to a thread's, join(value, other) one thread's to another's; a thread below n
// receives its group's.  lds: a value a thread.
template <class Value, class Take, class Join>
__device__ __forceinline__ Value over_chunks(const Norm &P, const float *stat, int g0, int n, Value *lds, Take take, Join join)
{
    const int parts = blockDim.x / n, part = threadIdx.x / n, g = g0 + threadIdx.x - part * n;
    constexpr int kAt = 8;   // loads under way together
    Value v{};
    if (part < parts)
        for (int i0 = part; i0 < P.chunks; i0 += parts * kAt) {
            f32x2 pair[kAt];
#pragma unroll
            for (int a = 0; a < kAt; ++a)
                if (i0 + a * parts < P.chunks) pair[a] = fetch(stat + ((long long)(i0 + a * parts) * P.G + g) * 2);
#pragma unroll
            for (int a = 0; a < kAt; ++a)
                if (i0 + a * parts < P.chunks) take(v, pair[a], i0 + a * parts);
        }
    __syncthreads();   // lds is free
    lds[threadIdx.x] = v;
    int h = 1;
    while (h < parts) h <<= 1;
    for (h >>= 1; h; h >>= 1) {
        __syncthreads();
        if (part < h && part + h < parts) {
            join(v, lds[threadIdx.x + h * n]);
            lds[threadIdx.x] = v;
        }
    }
    return v;
}

// Mean and squared distances from it of `count` values.
struct Moments {
    float count, mean, far;
};

__device__ __forceinline__ void join_moments(Moments &a, const Moments &b)
{
    if (b.count == 0.0f) return;
    const float all = a.count + b.count, share = b.count / all, d = b.mean - a.mean;
    a.far += __builtin_fmaf(d * d, a.count * share, b.far);
    a.mean = __builtin_fmaf(d, share, a.mean);
    a.count = all;
}

constexpr int kStep = 4;   // positions of a thread under way together

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
    const int beyond = rows_before_the_end<V>(P, b, p.c);
    float *first = norm_lds + reduce_floats(blockDim.x, V), *second = first + m.groups;
    // by channel: mean and squared distance of the positions so far, joined kStep at a time
    float mean[V] = {}, far[V] = {};
    float count = 0.0f;
    for (int r0 = s0 + p.row; r0 < s1 && p.n; r0 += kStep * m.lanes) {
        u32x4 w[kStep];
        int k_n = 0;
#pragma unroll
        for (int k = 0; k < kStep; ++k) {
            const int row = r0 + k * m.lanes;
            w[k] = u32x4{0, 0, 0, 0};
            if (row < s1) w[k] = get<T, V>(x + (long long)row * P.ldx, p.n, row < beyond), ++k_n;
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
    float sum[V];
#pragma unroll
    for (int e = 0; e < V; ++e) sum[e] = mean[e] * count;
    group_moments<V>(m, p, sum, far, count, s1 - s0, norm_lds, first);
    float *mine = P.stat + ((long long)b * P.chunks + chunk) * P.G * 2;
    for (int g = threadIdx.x; g < P.G; g += blockDim.x) {
        leave(mine + g * 2, first[g], second[g]);
    }
    if (!last_of(P, b)) return;
    const float *stat = P.stat + (long long)b * P.chunks * P.G * 2;
    for (int g0 = 0; g0 < P.G; g0 += blockDim.x) {
        const int n = P.G - g0 < (int)blockDim.x ? P.G - g0 : (int)blockDim.x;
        const Moments v = over_chunks(
            P, stat, g0, n, (Moments *)norm_lds,
            [&](Moments &to, f32x2 pair, int i) {
                const int positions = i + 1 == P.chunks ? P.S - i * P.chunk : P.chunk;
                join_moments(to, {(float)positions * (float)m.per, pair.x, pair.y});
            },
            [](Moments &to, const Moments &from) { join_moments(to, from); });
        if ((int)threadIdx.x < n) {
            const long long at = (long long)b * P.G + g0 + threadIdx.x;
            P.mean[at] = v.mean;
            P.rstd[at] = 1.0f / sqrtf(v.far / ((float)P.S * (float)m.per) + P.eps);
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
    const int beyond = rows_before_the_end<V>(P, b, p.c);
    T *y = (T *)P.y + (long long)b * P.S * P.ldy + p.c;
    float a[V], beta[V], mean[V];
    parameters<T, V>(a, P.gamma, p.c, p.n, 1.0f);
    parameters<T, V>(beta, P.beta, p.c, p.n, 0.0f);
#pragma unroll
    for (int e = 0; e < V; ++e) {
        const long long g = (long long)b * P.G + m.by_per(p.c + (e < p.n ? e : 0));
        mean[e] = P.mean[g];
        a[e] *= P.rstd[g];
    }
    for (int r0 = s0 + p.row; r0 < s1; r0 += kStep * m.lanes) {
        u32x4 w[kStep];
#pragma unroll
        for (int k = 0; k < kStep; ++k) {
            const int row = r0 + k * m.lanes;
            w[k] = u32x4{0, 0, 0, 0};
            if (row < s1) w[k] = get<T, V>(x + (long long)row * P.ldx, p.n, row < beyond);
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

// Sums of a thread: after so many steps they go to LDS and begin anew, so that no chain of additions grows with the sample (2^28
// positions of one channel, 4,096 of a thread: equal values off by 6.1e-5, so by 1.3e-7).
constexpr int kSegment = 32;

// What a thread has put into LDS, if any, is added to its sums.
template <int V>
__device__ __forceinline__ void add_held(float (&s)[2][V], const float *lds, bool held)
{
    if (!held) return;
#pragma unroll
    for (int q = 0; q < 2; ++q)
#pragma unroll
        for (int e = 0; e < V; ++e) s[q][e] += lds[(q * V + e) * blockDim.x + threadIdx.x];
}

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
    const int beyond = rows_before_the_end<V>(P, b, p.c);
    const T *dy = (const T *)P.dy + (long long)b * P.S * P.lddy + p.c;
    float *groups = norm_lds + reduce_floats(blockDim.x, V);
    float gamma[V], beta[V], mean[V], rstd[V], scale[V], s[2][V] = {};
    parameters<T, V>(gamma, P.gamma, p.c, p.n, 1.0f);
    parameters<T, V>(beta, P.beta, p.c, p.n, 0.0f);
#pragma unroll
    for (int e = 0; e < V; ++e) {
        const long long g = (long long)b * P.G + m.by_per(p.c + e);
        mean[e] = e < p.n ? P.mean[g] : 0.0f;
        rstd[e] = e < p.n ? P.rstd[g] : 0.0f;
        scale[e] = rstd[e] * gamma[e];
    }
    bool held = false;
    for (int r0 = s0 + p.row; p.n;) {
        const int end = s1 - r0 < kSegment * kStepBack * m.lanes ? s1 : r0 + kSegment * kStepBack * m.lanes;
        for (; r0 < end; r0 += kStepBack * m.lanes) {
            u32x4 w[kStepBack], d[kStepBack];
#pragma unroll
            for (int k = 0; k < kStepBack; ++k) {
                const int row = r0 + k * m.lanes;
                w[k] = d[k] = u32x4{0, 0, 0, 0};
                if (row < s1) {
                    w[k] = get<T, V>(x + (long long)row * P.ldx, p.n, row < beyond);
                    d[k] = get<T, V>(dy + (long long)row * P.lddy, p.n, row < beyond);
                }
            }
#pragma unroll
            for (int k = 0; k < kStepBack; ++k) {
                if (r0 + k * m.lanes >= s1) continue;
                float dz[V], far[V];
                gradient_at<T, V>(dz, far, w[k], d[k], mean, scale, beta, P.act);
#pragma unroll
                for (int e = 0; e < V; ++e) s[0][e] += dz[e], s[1][e] = __builtin_fmaf(dz[e], far[e], s[1][e]);
            }
        }
        if (r0 >= s1) break;
        add_held<V>(s, norm_lds, held);
        held = true;
#pragma unroll
        for (int q = 0; q < 2; ++q)
#pragma unroll
            for (int e = 0; e < V; ++e) norm_lds[(q * V + e) * blockDim.x + threadIdx.x] = s[q][e], s[q][e] = 0.0f;
    }
    add_held<V>(s, norm_lds, held);
#pragma unroll
    for (int e = 0; e < V; ++e) s[1][e] *= rstd[e];
    if (P.part) parameter_sums<T, V>(P, p, s, 0, P.C, (long long)b * P.chunks + chunk, norm_lds);
    if (!P.dx) return;
#pragma unroll
    for (int e = 0; e < V; ++e) s[0][e] *= gamma[e], s[1][e] *= gamma[e];
    __syncthreads();
    group_sums<V, 2>(m, p, s, norm_lds, groups);
    float *mine = P.stat + ((long long)b * P.chunks + chunk) * P.G * 2;
    for (int g = threadIdx.x; g < P.G; g += blockDim.x) {
        leave(mine + g * 2, groups[g], groups[m.groups + g]);
    }
    if (!last_of(P, b)) return;
    const float *stat = P.stat + (long long)b * P.chunks * P.G * 2;
    const float inv = 1.0f / ((float)P.S * (float)m.per);
    for (int g0 = 0; g0 < P.G; g0 += blockDim.x) {
        const int n = P.G - g0 < (int)blockDim.x ? P.G - g0 : (int)blockDim.x;
        const f32x2 v = over_chunks(
            P, stat, g0, n, (f32x2 *)norm_lds, [](f32x2 &to, f32x2 pair, int) { to += pair; },
            [](f32x2 &to, const f32x2 &from) { to += from; });
        if ((int)threadIdx.x < n) {
            float *to = P.group + ((long long)b * P.G + g0 + threadIdx.x) * 2;
            to[0] = v.x * inv, to[1] = v.y * inv;
        }
        __syncthreads();
    }
}

// dgamma and dbeta: the sums over `rows` partial ones, eight channels of one of them a workgroup, its other threads down the
// rows.
template <typename T>
__device__ __forceinline__ void reduce_parameters(const Norm &P, int block)
{
    __shared__ float held[128][8];
    const int lane = threadIdx.x & 7, down = threadIdx.x >> 3, across = blockDim.x >> 3, blocks = (P.C + 7) / 8;
    const int q = block / blocks, c = (block - q * blocks) * 8 + lane;
    float s = 0.0f;
    constexpr int kSome = 64;   // rows of a thread whose sum is its own, for short chains
    for (int r0 = 0; r0 < P.rows && c < P.C; r0 += kSome * across) {
        const int end = P.rows - r0 < kSome * across ? P.rows : r0 + kSome * across;
        float some = 0.0f;
#pragma unroll 8
        for (int r = r0 + down; r < end; r += across) some += P.part[((long long)r * 2 + q) * P.C + c];
        s += some;
    }
    held[down][lane] = s;
    int h = 64;   // the rows' threads, of which there are 32 to 128
    while (h >= across) h >>= 1;
    for (; h; h >>= 1) {
        __syncthreads();
        if (down < h && down + h < across) held[down][lane] += held[down + h][lane];
    }
    if (down || c >= P.C) return;
    T *to = (T *)(q ? P.dgamma : P.dbeta);
    if (to) narrow(held[0][lane], to[c]);
}

template <typename T>
__global__ __launch_bounds__(1024) void k_parameters(Norm P)
{
    reduce_parameters<T>(P, blockIdx.x);
}

// dx by chunks; the first `extra` workgroups, if any, form dgamma and dbeta.
template <typename T>
__global__ __launch_bounds__(1024) void k_apply_backward(Norm P)
{
    if ((int)blockIdx.x < P.extra) {
        reduce_parameters<T>(P, blockIdx.x);
        return;
    }
    constexpr int V = kVec<T>;
    const Map &m = P.map;
    const Place p = place<V>(m, P.C);
    const int id = gridDim.x - 1 - blockIdx.x, b = id / P.chunks, chunk = id - b * P.chunks;
    const int s0 = chunk * P.chunk, s1 = P.S - s0 < P.chunk ? P.S : s0 + P.chunk;
    if (!p.n) return;
    const T *x = (const T *)P.x + (long long)b * P.S * P.ldx + p.c;
    const int beyond = rows_before_the_end<V>(P, b, p.c);
    const T *dy = (const T *)P.dy + (long long)b * P.S * P.lddy + p.c;
    T *dx = (T *)P.dx + (long long)b * P.S * P.lddx + p.c;
    float gamma[V], beta[V], mean[V], scale[V], one[V], two[V];
    parameters<T, V>(gamma, P.gamma, p.c, p.n, 1.0f);
    parameters<T, V>(beta, P.beta, p.c, p.n, 0.0f);
#pragma unroll
    for (int e = 0; e < V; ++e) {
        const long long g = (long long)b * P.G + m.by_per(p.c + (e < p.n ? e : 0));
        mean[e] = P.mean[g];
        const float rstd = P.rstd[g];
        scale[e] = rstd * gamma[e];   // dx = scale dz - one - (x - mean) two
        one[e] = rstd * P.group[g * 2], two[e] = rstd * (rstd * P.group[g * 2 + 1]);   // rstd^2 may overflow
    }
    for (int r0 = s0 + p.row; r0 < s1; r0 += kStepBack * m.lanes) {
        u32x4 w[kStepBack], d[kStepBack];
#pragma unroll
        for (int k = 0; k < kStepBack; ++k) {
            const int row = r0 + k * m.lanes;
            w[k] = d[k] = u32x4{0, 0, 0, 0};
            if (row < s1) {
                w[k] = get<T, V>(x + (long long)row * P.ldx, p.n, row < beyond);
                d[k] = get<T, V>(dy + (long long)row * P.lddy, p.n, row < beyond);
            }
        }
#pragma unroll
        for (int k = 0; k < kStepBack; ++k) {
            const int row = r0 + k * m.lanes;
            if (row >= s1) continue;
            float dz[V], far[V];
            gradient_at<T, V>(dz, far, w[k], d[k], mean, scale, beta, P.act);
#pragma unroll
            for (int e = 0; e < V; ++e) dz[e] = __builtin_fmaf(scale[e], dz[e], -__builtin_fmaf(far[e], two[e], one[e]));
            put<T, V>(dx + (long long)row * P.lddx, dz, p.n);
        }
    }
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
// Workgroups that a split call aims at (32 x 4096 x 512 bf16, both passes, 512 / 1024 / 2048: 209 / 214 / 224 us; 8 x 4096 x 512 fp32
// 106 / 110 / 122).
constexpr int kSplitGroups = 512;
constexpr int kSampleChunks = 256;   // chunks of a sample, at most
// Workspace of the samples that are split at once, and how many they are at least; more go in rounds, whose ends leave compute units
// idle: rounds of 2,000 samples, 82 MB of x, cost 6 to 10 % (4000 x 5 x 4096 bf16 forward 134 / 144 us, backward 339 / 360), of 1,334
// 24 % (166) and 11 % (377).  Without rounds that call's workspace is 0.8 of x, with one channel a group 2.4.
constexpr size_t kRoundBytes = 64ull << 20;
constexpr int kRoundSamples = 2048;
// Workgroups of a span in a resident pass, of up to 256 threads; others: a third.  Backward fewer, since each leaves sums of all
// parameters (1000 x 784 fp32 forward 768 / 1024: 10.2 / 9.6 us; 3000 x 4 x 96 fp32 backward 12.3 / 15.3).
constexpr int kResidentForward = 1024, kResidentBackward = 768;
// Samples of a workgroup's sums in one launch, so that no chain of additions grows with the batch (2^20 x 2048 fp32, 2,048 samples of a
// workgroup in one: equal values off by 2.9e-5, so by 1.6e-6).
constexpr int kRun = 256;
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

// The most positions of a thread, by the size of the workgroup: what its registers hold (backward: x, and dz in 32 bits) with
// room for another workgroup's on the compute unit.
template <typename T>
constexpr int kMostForward = sizeof(T) == 2 ? 4 : 16;
template <typename T>
constexpr int kMostBackward = sizeof(T) == 2 ? 4 : 8;
constexpr int kMostOf1024 = 4;
// Threads of the workgroups that small samples share: in the backward pass each leaves sums of all parameters.
constexpr int kTogetherForward = 256, kTogetherBackward = 1024;

// What follows from a map's widths, for workgroups of `threads`.
template <typename T>
void complete(Map &m, int threads)
{
    constexpr int V = kVec<T>;
    const bool whole = m.per % V == 0;
    m.wide = whole ? 1 : V;
    m.pitch = m.vecs * m.wide;
    m.mine = whole ? m.per / V : m.per;
    m.channels = whole ? (float)V : 1.0f;
    m.sets = m.subs * m.groups;
    m.each = 1;
    while (m.each < 64 && m.each * 2 * m.sets <= threads && m.each < m.mine * m.lanes) m.each <<= 1;
    m.by_vecs = Div(m.vecs), m.by_lanes = Div(m.lanes), m.by_per = Div(m.per), m.by_groups = Div(m.groups), m.by_mine = Div(m.mine);
}

struct Resident {
    bool fits;
    int threads, rows, spans;
    Map map;
};

// most: positions that a thread holds; together: threads that small samples share.
template <typename T>
Resident resident(int B, int S, int C, int G, int most, int together)
{
    constexpr int V = kVec<T>;
    const int per = C / G;
    Resident r{};
    Map &m = r.map;
    // spans of whole groups: as many as give every compute unit one workgroup, of at least kMinSegment bytes of a row
    const bool small = (long long)B * S * C * (int)sizeof(T) <= kSmallArray;
    const int least = small ? per : std::max(1, ceil_div(kMinSegment / (int)sizeof(T), per)) * per;
    int unit = 1;   // groups that fill whole vectors
    while (unit * per % V) ++unit;
    int all = 0;    // threads down the positions that there can be
    for (int spans = std::min(ceil_div(kUnits, B), std::max(1, C / least));; ++spans) {
        int each = ceil_div(G, std::min(spans, G));   // groups of a span
        if (each > unit) each = each / unit * unit;
        r.spans = ceil_div(G, each);
        m.width = each * per;
        m.groups = each;
        m.vecs = ceil_div(m.width, V);
        int threads = m.vecs <= 512 ? 512 : 1024;
        // smaller workgroups where there are many: a compute unit holds more of them, one waiting while another computes
        if (m.vecs <= 256 && (long long)B * r.spans >= kUnits && (long long)(256 / m.vecs) * most >= S) threads = 256;
        all = threads / m.vecs;
        const long long room = (long long)all * (threads <= 512 ? most : kMostOf1024);
        if (room >= S) break;
        if (m.width <= least || spans >= G) return r;   // does not fit
    }
    // Spans beside each other in a second round, or few workgroups with much each, cost more than reading x twice in whole rows
    // (256 x 196 positions of 512 channels bf16, 768 workgroups: 67 us against 38; 5 x 589 of 172 fp32, 20 of 101 KB: 18.3 against
    // 13.6; 16 x 1024 of 512 fp32, 256 workgroups: 22 against 37).  Samples of few positions are never split.
    const long long wgs = (long long)B * r.spans, slab = (long long)S * m.width * (long long)sizeof(T);
    const bool better = (r.spans == 1 || wgs <= kUnits) && (wgs >= kUnits / 4 || slab <= 65536);
    if (!better && S > split_lanes<T>(C) * kMostOf1024) return r;
    r.fits = true;
    m.per = per;
    r.rows = ceil_div(S, all);
    m.lanes = ceil_div(S, r.rows);
    // but no fewer workgroups than half the compute units
    const int most_subs = (int)std::min<long long>(B, std::max<long long>(1, 2 * (long long)B * r.spans / kUnits));
    m.subs = std::max(1, std::min((r.rows == 1 ? together : 256) / (m.vecs * m.lanes), most_subs));
    r.threads = ceil_div(m.vecs * m.lanes * m.subs, 64) * 64;
    complete<T>(m, r.threads);
    return r;
}

// Workgroups of a span: what the compute units hold together; each goes on to other samples, with its parameters (and, backward,
// their sums) in registers.
int resident_groups(const Resident &r, int B, int most)
{
    return std::min(ceil_div(B, r.map.subs), r.threads <= 256 ? most : most / 3);
}

Norm common(const NormCall &a, int V)
{
    Norm P{};
    P.B = a.B, P.S = a.S, P.C = a.C, P.G = a.G;
    P.x = a.x, P.gamma = a.gamma, P.beta = a.beta, P.dy = a.dy;
    P.ldx = a.ldx, P.ldy = a.ldy, P.lddy = a.lddy, P.lddx = a.lddx;
    P.y = a.y, P.dx = a.dx;
    P.mean = a.mean, P.rstd = a.rstd;
    P.act = a.act, P.eps = a.eps;
    P.ahead = ceil_div(V, a.C);
    return P;
}

// Cuts a split call whose rounds have up to `samples`; the threads of its workgroups.
template <typename T>
int cut(Norm &P, const NormWorkspace &ws, int samples)
{
    Map &m = P.map;
    m.width = P.C;
    m.vecs = ceil_div(P.C, kVec<T>);
    m.lanes = split_lanes<T>(P.C);
    m.subs = 1;
    m.per = P.C / P.G;
    m.groups = P.G;
    complete<T>(m, split_threads<T>(P.C));
    // kSplitGroups chunks in all or, where those leave compute units with one more than others, up to twice as many; of one size,
    // and no more of a sample than its last workgroup joins quickly
    int most = std::max(1, kSplitGroups / samples);
    auto rounds = [&](int n) { return (float)ceil_div((long long)samples * n, kUnits) / (float)n; };
    for (int n = most + 1; n <= 2 * kSplitGroups / samples; ++n)
        if (rounds(n) < 0.9f * rounds(most)) most = n;
    most = std::min(most, kSampleChunks);
    P.chunk = std::min(P.S, std::max(m.lanes * kStep, ceil_div(P.S, most)));
    P.chunks = ceil_div(P.S, P.chunk);
    P.stat = ws.part;
    P.group = ws.group;
    P.ticket = ws.ticket;
    return split_threads<T>(P.C);
}

// The most samples of a round: each has two sums a channel, two values a group of its own and of a chunk's, and a ticket.
int round_samples(int C, int G)
{
    const size_t each = (2 * (size_t)C + 4 * (size_t)G + kTicketStep) * 4;
    return std::max((int)(kRoundBytes / each), kRoundSamples);
}

// What a round of a split call of up to `rows` positions in all takes at most: samples, and chunks of all of them.  A sample that
// is split has more positions than any resident workgroup holds across all channels.
template <typename T>
void split_most(long long rows, int C, int G, long long &samples, long long &chunks)
{
    samples = std::min<long long>(rows / (split_lanes<T>(C) * kMostOf1024 + 1), round_samples(C, G));
    chunks = samples ? std::max<long long>(2 * kSplitGroups, samples) : 0;
}

// The samples of a call from b on, n of them.
template <typename T>
NormCall samples_of(const NormCall &a, int b, int n)
{
    NormCall c = a;
    const long long at = (long long)b * a.S, g = (long long)b * a.G;
    auto from = [&](const void *p, long long ld) { return p ? (void *)((T *)p + at * ld) : nullptr; };
    c.B = n;
    c.x = from(a.x, a.ldx), c.dy = from(a.dy, a.lddy);
    c.y = from(a.y, a.ldy), c.dx = from(a.dx, a.lddx);
    if (a.mean) c.mean += g, c.rstd += g;
    return c;
}

// Calls f(samples, first, last) for the rounds of a call, of at most `most` samples, of one size up to the last.
template <typename T, typename F>
hipError_t in_rounds(const NormCall &a, long long most, F f)
{
    const int each = ceil_div(a.B, ceil_div(a.B, most));
    for (int b = 0; b < a.B;) {
        const int n = std::min(each, a.B - b);
        const hipError_t e = f(samples_of<T>(a, b, n), b == 0, b + n == a.B);
        if (e != hipSuccess) return e;
        b += n;
    }
    return hipSuccess;
}

bool fits(const Norm &P, const NormWorkspace &ws, bool parameters)
{
    const size_t chunks = (size_t)P.B * P.chunks;
    return chunks * (2 * P.G + (parameters ? 2 * P.C : 0)) * 4 <= ws.part_bytes && (size_t)P.B * P.G * 8 <= ws.group_bytes &&
           (size_t)P.B * kTicketStep * sizeof(unsigned) <= ws.ticket_bytes;
}

size_t lds_bytes(int threads, int V, int sets) { return (size_t)(reduce_floats(threads, V) + 2 * sets) * 4; }

template <typename T>
hipError_t forward(const NormCall &a, const NormWorkspace &ws, hipStream_t s)
{
    Norm P = common(a, kVec<T>);
    const Resident r = resident<T>(a.B, a.S, a.C, a.G, kMostForward<T>, kTogetherForward);
    if (r.fits) {
        P.map = r.map;
        const dim3 grid((unsigned)resident_groups(r, a.B, kResidentForward), (unsigned)r.spans);
        const size_t lds = lds_bytes(r.threads, kVec<T>, r.map.subs * r.map.groups);
        if (r.rows <= 1) k_resident_forward<T, 1, 1024><<<grid, r.threads, lds, s>>>(P);
        else if (r.threads > 512) k_resident_forward<T, kMostOf1024, 1024><<<grid, r.threads, lds, s>>>(P);
        else if (r.rows <= 4) k_resident_forward<T, 4, 512><<<grid, r.threads, lds, s>>>(P);
        else k_resident_forward<T, kMostForward<T>, 512><<<grid, r.threads, lds, s>>>(P);
        return hipGetLastError();
    }
    int most = 0;   // samples of a round
    return in_rounds<T>(a, round_samples(a.C, a.G), [&](const NormCall &c, bool first, bool) {
        if (first) most = c.B;
        Norm P = common(c, kVec<T>);
        const int threads = cut<T>(P, ws, most);
        if (!fits(P, ws, false)) return hipErrorInvalidValue;
        if (!P.mean) P.mean = ws.group, P.rstd = ws.group + (size_t)c.B * c.G;
        const unsigned grid = (unsigned)c.B * (unsigned)P.chunks;
        k_stats<T><<<grid, threads, lds_bytes(threads, kVec<T>, c.G), s>>>(P);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        k_apply_forward<T><<<grid, threads, 0, s>>>(P);
        return hipGetLastError();
    });
}

template <typename T>
hipError_t backward(const NormCall &a, const NormWorkspace &ws, hipStream_t s)
{
    const bool parameters = a.dgamma || a.dbeta;
    const int blocks = 2 * ceil_div(a.C, 8);   // of reduce_parameters
    const Resident r = resident<T>(a.B, a.S, a.C, a.G, kMostBackward<T>, kTogetherBackward);
    if (r.fits) {
        const dim3 grid((unsigned)resident_groups(r, a.B, kResidentBackward), (unsigned)r.spans);
        return in_rounds<T>(a, (long long)kRun * grid.x * r.map.subs, [&](const NormCall &c, bool first, bool last) {
            Norm P = common(c, kVec<T>);
            P.dgamma = a.dgamma, P.dbeta = a.dbeta;
            P.map = r.map;
            if (parameters && grid.x > 1) {
                P.rows = (int)grid.x;
                P.part = ws.part;
                P.add = !first;
                if ((size_t)P.rows * 2 * a.C * 4 > ws.part_bytes) return hipErrorInvalidValue;
            }
            const size_t lds = lds_bytes(r.threads, kVec<T>, r.map.subs * r.map.groups);
            if (r.rows <= 1) k_resident_backward<T, 1, 1024><<<grid, r.threads, lds, s>>>(P);
            else if (r.threads > 512) k_resident_backward<T, kMostOf1024, 1024><<<grid, r.threads, lds, s>>>(P);
            else if (r.rows <= 4) k_resident_backward<T, 4, 512><<<grid, r.threads, lds, s>>>(P);
            else k_resident_backward<T, kMostBackward<T>, 512><<<grid, r.threads, lds, s>>>(P);
            const hipError_t e = hipGetLastError();
            if (e != hipSuccess || !P.rows || !last) return e;
            k_parameters<T><<<blocks, 512, 0, s>>>(P);
            return hipGetLastError();
        });
    }
    int most = 0, rows = 0;   // samples of a round, its partial sums of parameters
    return in_rounds<T>(a, round_samples(a.C, a.G), [&](const NormCall &c, bool first, bool last) {
        if (first) most = c.B;
        Norm P = common(c, kVec<T>);
        P.dgamma = a.dgamma, P.dbeta = a.dbeta;
        const int threads = cut<T>(P, ws, most);
        if (!fits(P, ws, parameters)) return hipErrorInvalidValue;
        const unsigned grid = (unsigned)c.B * (unsigned)P.chunks;
        if (first) rows = (int)grid;   // no later round has more
        if (parameters) P.rows = rows, P.part = ws.part + (size_t)rows * 2 * a.G, P.add = !first;
        k_sums<T><<<grid, threads, lds_bytes(threads, kVec<T>, c.G), s>>>(P);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        const bool reduce = parameters && last;
        if (c.dx) {
            P.extra = reduce ? blocks : 0;
            k_apply_backward<T><<<grid + P.extra, threads, 0, s>>>(P);
        } else if (reduce) {   // as many threads: the sums' order, and so their last bit, is the same
            k_parameters<T><<<blocks, threads, 0, s>>>(P);
        }
        return hipGetLastError();
    });
}

// More dynamic LDS than 64 KB has to be allowed.
template <typename T>
hipError_t configure()
{
    const void *kernels[] = {(const void *)k_resident_forward<T, 1, 1024>,          (const void *)k_resident_forward<T, 4, 512>,
                             (const void *)k_resident_forward<T, kMostForward<T>, 512>, (const void *)k_resident_forward<T, kMostOf1024, 1024>,
                             (const void *)k_resident_backward<T, 1, 1024>,         (const void *)k_resident_backward<T, 4, 512>,
                             (const void *)k_resident_backward<T, kMostBackward<T>, 512>,
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
    split_most<T>(c.max_rows, c.channels, c.groups, samples, chunks);
    const size_t C = (size_t)c.channels, G = (size_t)c.groups;
    ws.part_bytes = std::max((size_t)chunks * (2 * G + 2 * C), std::min<size_t>(kResidentBackward, (size_t)c.max_rows) * 2 * C) * 4;
    ws.group_bytes = (size_t)samples * G * 8;
    ws.ticket_bytes = (size_t)samples * kTicketStep * sizeof(unsigned);
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
