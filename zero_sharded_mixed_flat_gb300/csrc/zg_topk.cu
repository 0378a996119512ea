// The k largest of each row of logits, largest first, ties to the lowest index.
#include <cuda_bf16.h>

#include "zg_launch.h"
#include "zg_ops.h"

namespace zg {
namespace {

constexpr int kThreads = 256;

// An unsigned key in the order of the values: NaN above everything, -0 = +0.
__device__ __forceinline__ uint32_t key_of(uint32_t bits)
{
    if ((bits & 0x7fffffffu) > 0x7f800000u) return 0xffffffffu;
    if (bits == 0x80000000u) bits = 0u;
    return (bits & 0x80000000u) ? ~bits : (bits | 0x80000000u);
}
__device__ __forceinline__ uint32_t bits_at(const float *p) { return __float_as_uint(*p); }
__device__ __forceinline__ uint32_t bits_at(const uint16_t *p) { return uint32_t(*p) << 16; }

// One block per row takes the largest (key, lowest index) below the last one taken, k times.
template <class T>
__global__ void __launch_bounds__(kThreads) topk_kernel(const T *logits, int64_t rows, int vocab, int64_t stride, int k, T *values, int32_t *index)
{
    __shared__ uint64_t best[kThreads / 32];
    for (int64_t r = blockIdx.x; r < rows; r += gridDim.x) {
        const T *row = logits + r * stride;
        uint64_t last = ~uint64_t(0);
        for (int j = 0; j < k; ++j) {
            uint64_t m = 0;
            for (int v = threadIdx.x; v < vocab; v += kThreads) {
                const uint64_t key = (uint64_t(key_of(bits_at(row + v))) << 32) | uint32_t(0x7fffffff - v);
                if (key < last && key > m) m = key;
            }
            for (int o = 16; o; o >>= 1) {
                const uint64_t n = __shfl_xor_sync(0xffffffffu, m, o);
                m = n > m ? n : m;
            }
            __syncthreads();
            if (threadIdx.x % 32 == 0) best[threadIdx.x / 32] = m;
            __syncthreads();
            m = best[0];
            for (int w = 1; w < kThreads / 32; ++w) m = best[w] > m ? best[w] : m;
            last = m;
            if (threadIdx.x == 0) {
                const int v = 0x7fffffff - int(uint32_t(m));
                values[r * k + j] = row[v];
                index[r * k + j] = v;
            }
        }
    }
}

}  // namespace

cudaError_t launch_topk(const void *logits, int dtype, int64_t rows, int vocab, int64_t stride, int k, void *values,
                        int32_t *index, cudaStream_t st)
{
    const unsigned blocks = unsigned(rows < 65535 ? rows : 65535);
    if (dtype == ZG_DTYPE_BF16)
        topk_kernel<<<blocks, kThreads, 0, st>>>(static_cast<const uint16_t *>(logits), rows, vocab, stride, k,
                                                 static_cast<uint16_t *>(values), index);
    else
        topk_kernel<<<blocks, kThreads, 0, st>>>(static_cast<const float *>(logits), rows, vocab, stride, k,
                                                 static_cast<float *>(values), index);
    return cudaGetLastError();
}

}  // namespace zg
