// The distillation loss from a teacher's top logits, and its gradient.
#include <cuda_bf16.h>

#include "zg_launch.h"
#include "zg_ops.h"

namespace zg {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ float load1(const float *p) { return *p; }
__device__ __forceinline__ float load1(const uint16_t *p) { return __uint_as_float(uint32_t(*p) << 16); }
__device__ __forceinline__ void store1(float *p, float v) { *p = v; }
__device__ __forceinline__ void store1(uint16_t *p, float v) { *p = __bfloat16_as_ushort(__float2bfloat16_rn(v)); }

__device__ float block_sum(float v, float *red)
{
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    __syncthreads();
    if (threadIdx.x % 32 == 0) red[threadIdx.x / 32] = v;
    __syncthreads();
    v = red[0];
    for (int w = 1; w < kThreads / 32; ++w) v += red[w];
    return v;
}

// fmaxf drops a NaN; this keeps it.
__device__ __forceinline__ float max_nan(float a, float b) { return a != a ? a : b != b ? b : fmaxf(a, b); }

__device__ float block_max(float v, float *red)
{
    for (int o = 16; o; o >>= 1) v = max_nan(v, __shfl_xor_sync(0xffffffffu, v, o));
    __syncthreads();
    if (threadIdx.x % 32 == 0) red[threadIdx.x / 32] = v;
    __syncthreads();
    v = red[0];
    for (int w = 1; w < kThreads / 32; ++w) v = max_nan(v, red[w]);
    return v;
}

template <class T, class E>
__global__ void __launch_bounds__(kThreads) distill_kernel(DistillArgs a)
{
    __shared__ float red[kThreads / 32];
    __shared__ float p[ZG_TOPK_MAX];
    __shared__ int at[ZG_TOPK_MAX];
    const float rt = 1.0f / a.temperature;
    const int tid = threadIdx.x;
    for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
        const T *z = static_cast<const T *>(a.logits) + r * a.row_stride;
        T *dz = static_cast<T *>(a.dlogits) + r * a.drow_stride;
        __syncthreads();
        float t = -INFINITY;
        int i = -1;
        if (tid < a.k) {
            i = a.t_index[r * a.k + tid];
            if (i < 0 || i >= a.vocab) i = -1;
            at[tid] = i;
            if (i >= 0) t = load1(static_cast<const E *>(a.t_logits) + r * a.k + tid) * rt;
        }
        const float tm = block_max(t, red);
        if (tm == -INFINITY) {
            if (tid == 0 && a.loss) a.loss[r] = 0.0f;
            if (tid == 0 && a.lse) a.lse[r] = 0.0f;
            if (a.dlogits)
                for (int v = tid; v < a.vocab; v += kThreads) store1(dz + v, 0.0f);
            continue;
        }
        const float e = i >= 0 ? expf(t - tm) : 0.0f;
        const float total = block_sum(e, red);
        const float pk = e / total;
        if (tid < a.k) p[tid] = pk;
        float lse;
        if (a.lse_in) {
            lse = a.lse_in[r];
        } else {
            float m = -INFINITY;
            for (int v = tid; v < a.vocab; v += kThreads) m = max_nan(m, load1(z + v) * rt);
            m = block_max(m, red);
            float s = 0.0f;
            for (int v = tid; v < a.vocab; v += kThreads) s += expf(load1(z + v) * rt - m);
            s = block_sum(s, red);
            lse = m + logf(s);
            float term = 0.0f;
            if (i >= 0 && pk != 0.0f) term = pk * ((t - tm - logf(total)) - (load1(z + i) * rt - lse));
            term = block_sum(term, red);
            if (tid == 0 && a.loss) a.loss[r] = a.temperature * a.temperature * term;
            if (tid == 0 && a.lse) a.lse[r] = lse;
        }
        if (!a.dlogits) continue;
        const float g = a.scale * a.temperature * (a.dloss ? a.dloss[r] : 1.0f);
        // the entries' gradients, before their logits are overwritten; the
        // first entry of an index answers for all of them
        __syncthreads();
        float patch = 0.0f;
        bool mine = i >= 0;
        if (mine) {
            float sum = 0.0f;
            for (int j = 0; j < a.k; ++j)
                if (at[j] == i) {
                    if (j < tid) mine = false;
                    sum += p[j];
                }
            patch = (expf(load1(z + i) * rt - lse) - sum) * g;
        }
        __syncthreads();
        for (int v = tid; v < a.vocab; v += kThreads) store1(dz + v, expf(load1(z + v) * rt - lse) * g);
        __syncthreads();
        if (mine) store1(dz + i, patch);
    }
}

}  // namespace

cudaError_t launch_distill(const DistillArgs &a, cudaStream_t st)
{
    const unsigned blocks = unsigned(a.rows < 65535 ? a.rows : 65535);
    const bool bf = a.dtype == ZG_DTYPE_BF16, tbf = a.t_dtype == ZG_DTYPE_BF16;
    if (bf && tbf) distill_kernel<uint16_t, uint16_t><<<blocks, kThreads, 0, st>>>(a);
    else if (bf) distill_kernel<uint16_t, float><<<blocks, kThreads, 0, st>>>(a);
    else if (tbf) distill_kernel<float, uint16_t><<<blocks, kThreads, 0, st>>>(a);
    else distill_kernel<float, float><<<blocks, kThreads, 0, st>>>(a);
    return cudaGetLastError();
}

}  // namespace zg
