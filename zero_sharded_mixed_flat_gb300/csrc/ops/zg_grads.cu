// The gradients of many tensors, clipped by their common norm.
//
// A list is cut into parts of at most kGradPart elements of one tensor, a block to
// each: the first pass leaves the sum of a part's squares, one block adds the
// sums up in a fixed order, and the second pass writes (scale * coefficient) * g.
#include "zg_ops.h"
#include "zg_rows.cuh"

namespace zg {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ float element(const void *p, int dtype, int i)
{
    return dtype == ZG_DTYPE_BF16 ? load1(static_cast<const uint16_t *>(p) + i) : load1(static_cast<const float *>(p) + i);
}

template <int THREADS>
__device__ __forceinline__ double sum_of_block(double x)
{
    __shared__ double part[THREADS / 32];
#pragma unroll
    for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = x;
    __syncthreads();
    double s = 0.0;
    for (int i = 0; i < THREADS / 32; ++i) s += part[i];
    return s;
}

__global__ void __launch_bounds__(kThreads) squares_kernel(const GradPart *parts, double *sums, float scale)
{
    const GradPart p = parts[blockIdx.x];
    float s = 0.0f;
    for (int i = threadIdx.x; i < p.n; i += kThreads) {
        const float g = element(p.grad, p.dtype, i) * scale;
        s = fmaf(g, g, s);
    }
    const double total = sum_of_block<kThreads>(s);
    if (threadIdx.x == 0) sums[blockIdx.x] = total;
}

__global__ void __launch_bounds__(1024) finish_kernel(const double *sums, int64_t count, float max_norm, float eps,
                                                      bool write, float *stats)
{
    double s = 0.0;
    for (int64_t i = threadIdx.x; i < count; i += 1024) s += sums[i];
    s = sum_of_block<1024>(s);
    if (threadIdx.x) return;
    const double norm = sqrt(s);
    stats[0] = float(norm);
    stats[1] = write && isfinite(norm) ? float(fmin(1.0, double(max_norm) / (norm + double(eps)))) : 1.0f;
}

__global__ void __launch_bounds__(kThreads) write_kernel(const GradPart *parts, const float *stats, float scale)
{
    const GradPart p = parts[blockIdx.x];
    const float k = scale * stats[1];
    for (int i = threadIdx.x; i < p.n; i += kThreads) {
        const float v = element(p.grad, p.dtype, i) * k;
        if (p.out_dtype == ZG_DTYPE_BF16)
            store1(static_cast<uint16_t *>(p.out) + i, v);
        else
            store1(static_cast<float *>(p.out) + i, v);
    }
}

}  // namespace

cudaError_t launch_grads_norm(const GradPart *parts, int64_t count, double *sums, float scale, float max_norm, float eps,
                              float *stats, bool write, cudaStream_t st)
{
    if (count) squares_kernel<<<unsigned(count), kThreads, 0, st>>>(parts, sums, scale);
    finish_kernel<<<1, 1024, 0, st>>>(sums, count, max_norm, eps, write, stats);
    if (write && count) write_kernel<<<unsigned(count), kThreads, 0, st>>>(parts, stats, scale);
    return cudaGetLastError();
}

}  // namespace zg
