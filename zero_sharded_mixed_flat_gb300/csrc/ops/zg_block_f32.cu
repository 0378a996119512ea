// The norms around a block in binary32.
#include "zg_block.cuh"

namespace zg {

cudaError_t launch_block_norm_f32(const BlockArgs &a, cudaStream_t st) { return of_type<float, false>(a, st); }

cudaError_t launch_block_norm_grad_f32(const BlockArgs &a, cudaStream_t st) { return of_type<float, true>(a, st); }

}  // namespace zg
