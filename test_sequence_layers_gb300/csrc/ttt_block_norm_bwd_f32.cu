// ttt_block_norm_bwd_f32.cu -- the backward kernels of ttt_block_norm.cuh for fp32 tensors.
#include "ttt_block_norm.cuh"

namespace ttt {

int norm_bwd_f32(const NormBwdParams &p, const NormShape &s, int group, int limit, cudaStream_t st, int *blocks)
{
    return norm_bwd<float>(p, s, group, limit, st, blocks);
}

}  // namespace ttt
