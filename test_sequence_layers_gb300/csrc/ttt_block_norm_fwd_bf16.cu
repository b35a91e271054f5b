// ttt_block_norm_fwd_bf16.cu -- the forward kernels of ttt_block_norm.cuh for bf16 tensors.
#include "ttt_block_norm.cuh"

namespace ttt {

int norm_fwd_bf16(const NormFwdParams &p, const NormShape &s, int group, cudaStream_t st)
{
    return norm_fwd<__nv_bfloat16>(p, s, group, st);
}

}  // namespace ttt
