// Norms around a block, backward: bf16 tensors around an fp32 residual.
#include "dn_block_bwd.cuh"

namespace dn {

cudaError_t block_bwd_bf16_f32(const BlockParams &p, bool bias, cudaStream_t stream, int *blocks) {
    return block_bwd_of<__nv_bfloat16, float>(p, bias, stream, blocks);
}

}  // namespace dn
