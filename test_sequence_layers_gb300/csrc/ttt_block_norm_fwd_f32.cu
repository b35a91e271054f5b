// ttt_block_norm_fwd_f32.cu -- the forward kernels of ttt_block_norm.cuh for fp32 tensors.
#include "ttt_block_norm.cuh"

namespace ttt {

int norm_fwd_f32(const NormFwdParams &p, const NormShape &s, int group, cudaStream_t st)
{
    return norm_fwd<float>(p, s, group, st);
}

}  // namespace ttt
