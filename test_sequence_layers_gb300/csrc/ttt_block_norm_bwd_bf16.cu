// ttt_block_norm_bwd_bf16.cu -- the backward kernels of ttt_block_norm.cuh for bf16 tensors.
#include "ttt_block_norm.cuh"

namespace ttt {

int norm_bwd_bf16(const NormBwdParams &p, const NormShape &s, int group, int limit, cudaStream_t st, int *blocks)
{
    return norm_bwd<__nv_bfloat16>(p, s, group, limit, st, blocks);
}

}  // namespace ttt
