// Norms around a block, backward: bf16 tensors.
#include "dn_block_bwd.cuh"

namespace dn {

cudaError_t block_bwd_bf16(const BlockParams &p, bool bias, cudaStream_t stream, int *blocks) {
    return block_bwd_of<__nv_bfloat16, __nv_bfloat16>(p, bias, stream, blocks);
}

}  // namespace dn
