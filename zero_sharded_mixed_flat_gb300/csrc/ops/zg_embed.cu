// The token embedding and its gradient.
//
// Lookup: out row i = scale * table row tokens[i]. Gradient: dtable row v = add
// row v + scale * the sum of the drows rows whose token is v, in the order of
// the tokens.
#include "zg_ops.h"
#include "zg_rows.cuh"

namespace zg {
namespace {

constexpr int kThreads = 256;

template <class I>
__device__ __forceinline__ int64_t token_of(const EmbedArgs &a, int64_t i)
{
    const int64_t t = static_cast<const I *>(a.tokens)[i];
    return t >= 0 && t < a.vocab ? t : -1;
}

template <class T, class I>
__global__ void __launch_bounds__(kThreads) lookup_kernel(EmbedArgs a)
{
    for (int64_t i = blockIdx.x; i < a.n; i += gridDim.x) {
        const int64_t t = token_of<I>(a, i);
        T *const out = static_cast<T *>(a.out) + i * a.out_stride;
        const T *const row = static_cast<const T *>(a.table) + t * a.table_stride;
        for (int c = threadIdx.x; c < a.width; c += kThreads) store1(out + c, t < 0 ? 0.0f : load1(row + c) * a.scale);
    }
}

// A block to a row of the table, which looks all tokens through.
template <class T, class D, class I>
__global__ void __launch_bounds__(kThreads) gradient_kernel(EmbedArgs a)
{
    __shared__ int found[kThreads];
    __shared__ int count;
    for (int64_t v = blockIdx.x; v < a.vocab; v += gridDim.x) {
        const T *const add = a.table ? static_cast<const T *>(a.table) + v * a.table_stride : nullptr;
        T *const out = static_cast<T *>(a.out) + v * a.out_stride;
        for (int c0 = 0; c0 < a.width; c0 += kThreads) {
            const int c = c0 + threadIdx.x;
            float sum = 0.0f;
            bool any = false;
            for (int64_t i0 = 0; i0 < a.n; i0 += kThreads) {
                const bool hit = i0 + threadIdx.x < a.n && token_of<I>(a, i0 + threadIdx.x) == v;
                if (!__syncthreads_or(hit)) continue;
                any = true;
                found[threadIdx.x] = hit;
                __syncthreads();
                if (threadIdx.x == 0) {
                    count = 0;
                    for (int j = 0; j < kThreads; ++j)
                        if (found[j]) found[count++] = j;
                }
                __syncthreads();
                if (c < a.width)
                    for (int j = 0; j < count; ++j)
                        sum += load1(static_cast<const D *>(a.drows) + (i0 + found[j]) * a.drow_stride + c);
                __syncthreads();
            }
            if (c < a.width && (any || add != out)) store1(out + c, fmaf(a.scale, sum, add ? load1(add + c) : 0.0f));
        }
    }
}

unsigned blocks_of(int64_t n) { return unsigned(n < (1 << 30) ? n : 1 << 30); }

template <class T, class I>
cudaError_t gradient_of(const EmbedArgs &a, cudaStream_t st)
{
    if (a.drow_dtype == ZG_DTYPE_BF16)
        gradient_kernel<T, uint16_t, I><<<blocks_of(a.vocab), kThreads, 0, st>>>(a);
    else
        gradient_kernel<T, float, I><<<blocks_of(a.vocab), kThreads, 0, st>>>(a);
    return cudaGetLastError();
}

template <class T, class I>
cudaError_t lookup_of(const EmbedArgs &a, cudaStream_t st)
{
    lookup_kernel<T, I><<<blocks_of(a.n), kThreads, 0, st>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_embed(const EmbedArgs &a, cudaStream_t st)
{
    const bool wide = a.token_bytes == 8;
    if (a.dtype == ZG_DTYPE_BF16) return wide ? lookup_of<uint16_t, int64_t>(a, st) : lookup_of<uint16_t, int32_t>(a, st);
    return wide ? lookup_of<float, int64_t>(a, st) : lookup_of<float, int32_t>(a, st);
}

int64_t embed_grad_workspace(int64_t, int64_t, int64_t) { return 16; }

cudaError_t launch_embed_grad(const EmbedArgs &a, cudaStream_t st)
{
    const bool wide = a.token_bytes == 8;
    if (a.dtype == ZG_DTYPE_BF16)
        return wide ? gradient_of<uint16_t, int64_t>(a, st) : gradient_of<uint16_t, int32_t>(a, st);
    return wide ? gradient_of<float, int64_t>(a, st) : gradient_of<float, int32_t>(a, st);
}

}  // namespace zg
