// The norms around a block in bf16.
#include "zg_block.cuh"

namespace zg {

int64_t block_norm_workspace(int64_t rows, int64_t width, int64_t groups)
{
    const int64_t one = shares_of(rows, groups, kBlocks).blocks, two = shares_of(rows, groups, 2 * kBlocks).blocks;
    return 2 * (one > two ? one : two) * width * 4;
}

cudaError_t launch_block_norm_bf16(const BlockArgs &a, cudaStream_t st) { return of_type<uint16_t, false>(a, st); }

cudaError_t launch_block_norm_grad_bf16(const BlockArgs &a, cudaStream_t st) { return of_type<uint16_t, true>(a, st); }

}  // namespace zg
