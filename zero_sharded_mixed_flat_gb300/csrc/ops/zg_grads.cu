// The gradients of many tensors, clipped by their common norm.
//
// A list is cut into parts of at most kGradPart elements of one tensor, a block to
// each: the first pass leaves the sum of a part's squares, one block adds the
// sums up in a fixed order, and the second pass writes (scale * coefficient) * g.
//
// Bound by memory: every gradient is read for the norm, and again and written once the
// norm is known, the second time in the opposite order, since what was read last is still in
// L2. A thread has kAhead units of 16 bytes in flight.
#include "zg_launch.h"
#include "zg_ops.h"
#include "zg_rows.cuh"

namespace zg {
namespace {

constexpr int kThreads = 256;
constexpr int kAhead = 8;

__device__ __forceinline__ double sum_of_warp(double x)
{
#pragma unroll
    for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// The sum of all parts, of any number of threads in the order of 1,024 of them: each adds up every
// 1024-th sum, then 32 neighbours, then those 32.
__device__ double total_of(const double *sums, int64_t count)
{
    __shared__ double part[32];
    for (int64_t t = threadIdx.x; t < 1024; t += blockDim.x) {
        double s = 0.0;
        int64_t i = t;
        for (; i + 3 * 1024 < count; i += 4 * 1024) s += (sums[i] + sums[i + 1024]) + (sums[i + 2048] + sums[i + 3072]);
        for (; i < count; i += 1024) s += sums[i];
        s = sum_of_warp(s);
        if (t % 32 == 0) part[t / 32] = s;
    }
    __syncthreads();
    double s = 0.0;
#pragma unroll
    for (int i = 0; i < 32; ++i) s += part[i];
    return s;
}
__device__ __forceinline__ float2 stats_of(double sum, float max_norm, float eps, bool write)
{
    const double norm = sqrt(sum);
    return make_float2(float(norm),
                       write && isfinite(norm) ? float(fmin(1.0, double(max_norm) / (norm + double(eps)))) : 1.0f);
}

// The squares of a part, in units from the 16-byte boundary at or before it; what a unit has
// outside the part counts as zero.
template <class T>
__device__ __forceinline__ float squares(const GradPart &p, float scale)
{
    constexpr int N = Unit<T>::kN;
    const T *const g = static_cast<const T *>(p.grad);
    const int head = int((reinterpret_cast<uintptr_t>(g) & 15u) / sizeof(T)), end = head + p.n, units = (end + N - 1) / N;
    const uint4 *const from = reinterpret_cast<const uint4 *>(g - head);
    float2 sum = make_float2(0.0f, 0.0f);
    const float2 k = make_float2(scale, scale);
    auto add = [&](uint4 w, int u) {
        Unit<T> x;
        x.w = w;
        float2 v[N / 2];
        x.get(v);
        if (u * N < head || (u + 1) * N > end) {
#pragma unroll
            for (int i = 0; i < N / 2; ++i) {
                const int e = u * N + 2 * i;
                if (e < head || e >= end) v[i].x = 0.0f;
                if (e + 1 < head || e + 1 >= end) v[i].y = 0.0f;
            }
        }
#pragma unroll
        for (int i = 0; i < N / 2; ++i) {
            v[i] = mul_f32x2(v[i], k);
            sum = fma_f32x2(v[i], v[i], sum);
        }
    };
    int u = threadIdx.x;
    for (; u + (kAhead - 1) * kThreads < units; u += kAhead * kThreads) {
        uint4 w[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) w[i] = from[u + i * kThreads];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) add(w[i], u + i * kThreads);
    }
    for (; u < units; u += kThreads) add(from[u], u);
    return sum.x + sum.y;
}

__global__ void __launch_bounds__(kThreads) squares_kernel(const GradPart *parts, double *sums, float scale)
{
    pdl_trigger();
    const GradPart p = parts[blockIdx.x];
    __shared__ double part[kThreads / 32];
    const double mine = sum_of_warp(p.dtype == ZG_DTYPE_BF16 ? squares<uint16_t>(p, scale) : squares<float>(p, scale));
    if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = mine;
    __syncthreads();
    if (threadIdx.x) return;
    double total = 0.0;
    for (int i = 0; i < kThreads / 32; ++i) total += part[i];
    sums[blockIdx.x] = total;
}

__global__ void __launch_bounds__(1024) finish_kernel(const double *sums, int64_t count, float max_norm, float eps,
                                                      bool write, float *stats)
{
    pdl_trigger();
    pdl_wait();
    const double s = total_of(sums, count);
    if (threadIdx.x) return;
    const float2 found = stats_of(s, max_norm, eps, write);
    stats[0] = found.x;
    stats[1] = found.y;
}

// Eight neighbouring elements of either type.
template <class T>
struct Eight {
    float2 v[4];
    __device__ __forceinline__ void load(const T *p)
    {
        constexpr int N = Unit<T>::kN;
#pragma unroll
        for (int i = 0; i < 8 / N; ++i) {
            Unit<T> x;
            x.w = __ldcs(reinterpret_cast<const uint4 *>(p) + i);
            float2 f[N / 2];
            x.get(f);
#pragma unroll
            for (int j = 0; j < N / 2; ++j) v[i * N / 2 + j] = f[j];
        }
    }
    __device__ __forceinline__ void store(T *p) const
    {
        constexpr int N = Unit<T>::kN;
#pragma unroll
        for (int i = 0; i < 8 / N; ++i) {
            float2 f[N / 2];
#pragma unroll
            for (int j = 0; j < N / 2; ++j) f[j] = v[i * N / 2 + j];
            Unit<T> x;
            x.set(f);
            __stcs(reinterpret_cast<uint4 *>(p) + i, x.w);
        }
    }
};

template <class T, class O>
__device__ __forceinline__ void write_part(const GradPart &p, float k)
{
    const T *const g = static_cast<const T *>(p.grad);
    O *const out = static_cast<O *>(p.out);
    // whole eights where both lie on 16 bytes after as many elements; the rest one by one
    const int head = int((16 - (reinterpret_cast<uintptr_t>(g) & 15u)) % 16 / sizeof(T));
    const bool alike = (reinterpret_cast<uintptr_t>(out + head) & 15u) == 0;
    const int first = alike ? min(head, p.n) : p.n, eights = (p.n - first) / 8;
    auto one = [&](int i) { store1(out + i, load1(g + i) * k); };
    int u = threadIdx.x;
    for (; u + kThreads < eights; u += 2 * kThreads) {
        Eight<T> x, y;
        x.load(g + first + u * 8);
        y.load(g + first + (u + kThreads) * 8);
        Eight<O> a, b;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            a.v[i] = mul_f32x2(x.v[i], make_float2(k, k));
            b.v[i] = mul_f32x2(y.v[i], make_float2(k, k));
        }
        a.store(out + first + u * 8);
        b.store(out + first + (u + kThreads) * 8);
    }
    for (; u < eights; u += kThreads) {
        Eight<T> x;
        x.load(g + first + u * 8);
        Eight<O> a;
#pragma unroll
        for (int i = 0; i < 4; ++i) a.v[i] = mul_f32x2(x.v[i], make_float2(k, k));
        a.store(out + first + u * 8);
    }
    for (int i = first + eights * 8 + threadIdx.x; i < p.n; i += kThreads) one(i);
    int i = threadIdx.x;
    for (; i + 7 * kThreads < first; i += 8 * kThreads) {
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = load1(g + i + j * kThreads);
#pragma unroll
        for (int j = 0; j < 8; ++j) store1(out + i + j * kThreads, v[j] * k);
    }
    for (; i < first; i += kThreads) one(i);
}

// `sums`: every block adds the parts up itself, and the first writes stats; otherwise they are known.
__global__ void __launch_bounds__(kThreads) write_kernel(const GradPart *parts, const double *sums, int64_t count, float max_norm,
                                                         float eps, float *stats, float scale)
{
    const GradPart p = parts[gridDim.x - 1 - blockIdx.x];
    pdl_wait();
    float coefficient;
    if (sums) {
        const float2 found = stats_of(total_of(sums, count), max_norm, eps, true);
        coefficient = found.y;
        if (blockIdx.x == 0 && threadIdx.x == 0) {
            stats[0] = found.x;
            stats[1] = found.y;
        }
    } else {
        coefficient = stats[1];
    }
    const float k = scale * coefficient;
    if (p.dtype == ZG_DTYPE_BF16) {
        if (p.out_dtype == ZG_DTYPE_BF16)
            write_part<uint16_t, uint16_t>(p, k);
        else
            write_part<uint16_t, float>(p, k);
    } else {
        if (p.out_dtype == ZG_DTYPE_BF16)
            write_part<float, uint16_t>(p, k);
        else
            write_part<float, float>(p, k);
    }
}

}  // namespace

cudaError_t launch_grads_norm(const GradPart *parts, int64_t count, double *sums, float scale, float max_norm, float eps,
                              float *stats, bool write, cudaStream_t st)
{
    if (count) squares_kernel<<<unsigned(count), kThreads, 0, st>>>(parts, sums, scale);
    if (cudaError_t e = cudaGetLastError()) return e;
    // up to 1,024 parts are added up by each block that writes: a launch less (54 parts: 14.5 us for 10.5)
    const bool alone = write && count > 0 && count <= 1024;
    if (!alone)
        if (cudaError_t e = launch_dependent(&finish_kernel, 1, 1024, 0, st, sums, count, max_norm, eps,
                                             write, stats))
            return e;
    if (!write || !count) return cudaSuccess;
    return launch_dependent(&write_kernel, int(count), kThreads, 0, st, parts, static_cast<const double *>(alone ? sums : nullptr),
                            count, max_norm, eps, stats, scale);
}

}  // namespace zg
