// The gradients of many tensors, clipped by their common norm.
//
// A list is cut into parts of some thousand elements of one tensor (up to 32,768), a block to
// each: the first pass leaves the sum of a part's squares, one block adds the
// sums up in a fixed order, and the second pass writes (scale * coefficient) * g. Squares are
// binary32's, and binary64's in a part where those overflow or vanish.
//
// Bound by memory: every gradient is read for the norm, and again and written once the
// norm is known, the second time in the opposite order, since what was read last is still in
// L2. A thread has kAhead units of 16 bytes in flight.
//
// Measured: 124 M gradients of 148 tensors, matrices in bf16 and vectors in binary32, into a flat bf16 one, 112 us (249 MB read
// twice and written once: 6.7 TB/s; the squares 38 us, 6.5 TB/s); 0.6 M in binary32 6 us. Where a part and its output lie
// differently (a tensor of odd size before it in a flat output), elements are read and written one by one the second
// time: the same list behind a vector of 50257 bf16 elements 141 us, of binary32 into binary32 246 for 240.
#include "zg_launch.h"
#include "zg_ops.h"
#include "zg_rows.cuh"

namespace zg {
namespace {

constexpr int kThreads = 256;
constexpr int kAhead = 8;   // units of a thread at a time in the first pass
constexpr int kEights = 4;  // eights of elements in the second

template <class F>
__device__ __forceinline__ F sum_of_warp(F x)
{
#pragma unroll
    for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// The sum of all parts, for the block's first thread, in one order: a thread adds up every kThreads-th, then
// warps, then those. (binary64 is slow here: what every thread repeats of it shows.)
__device__ double total_of(const double *sums, int64_t count)
{
    __shared__ double part[kThreads / 32];
    double s = 0.0;
    int64_t i = threadIdx.x;
    for (; i + 7 * kThreads < count; i += 8 * kThreads) {
        double v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = sums[i + j * kThreads];
#pragma unroll
        for (int j = 0; j < 8; ++j) s += v[j];
    }
    for (; i < count; i += kThreads) s += sums[i];
    s = sum_of_warp(s);
    if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = s;
    __syncthreads();
    if (threadIdx.x) return 0.0;
    for (int w = 1; w < kThreads / 32; ++w) s += part[w];
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
__device__ __forceinline__ float squares(const GradPart &p, float scale, uint32_t &bits)
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
        bits |= w.x | w.y | w.z | w.w;
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
    for (int u = threadIdx.x; u < units; u += kAhead * kThreads) {
        uint4 w[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) w[i] = from[min(u + i * kThreads, units - 1)];
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
            if (u + i * kThreads < units) add(w[i], u + i * kThreads);
    }
    bits &= sizeof(T) == 2 ? 0x7fff7fffu : 0x7fffffffu;  // zeros of either sign
    return sum.x + sum.y;
}
// A thread's squares of the same part in binary64, which holds every finite one of theirs.
template <class T>
__device__ double wide_squares(const GradPart &p, float scale)
{
    const T *const g = static_cast<const T *>(p.grad);
    double s = 0.0;
    for (int i = threadIdx.x; i < p.n; i += kThreads) {
        const double v = double(load1(g + i)) * double(scale);
        s = fma(v, v, s);
    }
    return s;
}

// Sums of squares below this may have lost some of them: of a part's 2^15 squares each is off by at most
// 2^-150 where it is not normal, 2^-25 of such a sum in all.
constexpr float kLeastSum = 7.7e-34f;  // 2^-110

// A part whose sum has left binary32's range is added up again in binary64: one exploded
// element must not keep a list of finite ones from being clipped. `large` is for the sums that overflow; those
// that vanish though an element is not zero are always made good. The rest pay for the question alone (an or of
// every unit's bits: the norm of 124 M gradients 43 us with it and without).
__global__ void __launch_bounds__(kThreads) squares_kernel(const GradPart *parts, double *sums, float scale, bool large)
{
    pdl_trigger();
    __shared__ float part[kThreads / 32];
    __shared__ double wide[kThreads / 32];
    uint32_t bits = 0;
    const GradPart p = parts[blockIdx.x];
    const float mine =
        sum_of_warp(p.dtype == ZG_DTYPE_BF16 ? squares<uint16_t>(p, scale, bits) : squares<float>(p, scale, bits));
    if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = mine;
    const bool any = __syncthreads_or(bits != 0);
    double total = 0.0;
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < kThreads / 32; ++i) sum += part[i];
    if ((any && sum < kLeastSum) || (large && !isfinite(sum))) {
        const GradPart q = parts[blockIdx.x];  // read again: kept, it would cost the first look registers
        const double again =
            sum_of_warp(q.dtype == ZG_DTYPE_BF16 ? wide_squares<uint16_t>(q, scale) : wide_squares<float>(q, scale));
        if (threadIdx.x % 32 == 0) wide[threadIdx.x / 32] = again;
        __syncthreads();
        for (int i = 0; i < kThreads / 32; ++i) total += wide[i];
    } else if (threadIdx.x == 0) {
#pragma unroll
        for (int i = 0; i < kThreads / 32; ++i) total += part[i];
    }
    if (threadIdx.x == 0) sums[blockIdx.x] = total;
}

__global__ void __launch_bounds__(kThreads) finish_kernel(const double *sums, int64_t count, float max_norm, float eps,
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
    for (int u = threadIdx.x; u < eights; u += kEights * kThreads) {
        Eight<T> x[kEights];
#pragma unroll
        for (int i = 0; i < kEights; ++i) x[i].load(g + first + min(u + i * kThreads, eights - 1) * 8);
#pragma unroll
        for (int i = 0; i < kEights; ++i) {
            if (u + i * kThreads >= eights) break;
            Eight<O> y;
#pragma unroll
            for (int j = 0; j < 4; ++j) y.v[j] = mul_f32x2(x[i].v[j], make_float2(k, k));
            y.store(out + first + (u + i * kThreads) * 8);
        }
    }
    for (int i = first + eights * 8 + threadIdx.x; i < p.n; i += kThreads) one(i);
    for (int i = threadIdx.x; i < first; i += 8 * kThreads) {
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = load1(g + min(i + j * kThreads, first - 1));
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (i + j * kThreads < first) store1(out + i + j * kThreads, v[j] * k);
    }
}

// `sums`: every block adds the parts up itself, and the first writes stats; otherwise they are known.
__global__ void __launch_bounds__(kThreads) write_kernel(const GradPart *parts, const double *sums, int64_t count, float max_norm,
                                                         float eps, float *stats, float scale)
{
    const GradPart p = parts[gridDim.x - 1 - blockIdx.x];
    pdl_wait();
    __shared__ float coefficient;
    if (sums) {
        const double s = total_of(sums, count);
        if (threadIdx.x == 0) {
            const float2 found = stats_of(s, max_norm, eps, true);
            coefficient = found.y;
            if (blockIdx.x == 0) {
                stats[0] = found.x;
                stats[1] = found.y;
            }
        }
        __syncthreads();
    } else {
        if (threadIdx.x == 0) coefficient = stats[1];
        __syncthreads();
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
    if (count) squares_kernel<<<unsigned(count), kThreads, 0, st>>>(parts, sums, scale, write);
    if (cudaError_t e = cudaGetLastError()) return e;
    // up to 1,024 parts are added up by each block that writes: a launch less
    const bool alone = write && count > 0 && count <= 1024;
    if (!alone)
        if (cudaError_t e = launch_dependent(&finish_kernel, 1, kThreads, 0, st, sums, count, max_norm, eps,
                                             write, stats))
            return e;
    if (!write || !count) return cudaSuccess;
    return launch_dependent(&write_kernel, int(count), kThreads, 0, st, parts, static_cast<const double *>(alone ? sums : nullptr),
                            count, max_norm, eps, stats, scale);
}

}  // namespace zg
