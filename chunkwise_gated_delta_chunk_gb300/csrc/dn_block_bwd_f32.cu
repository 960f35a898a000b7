// Norms around a block, backward: fp32 tensors.
#include "dn_block_bwd.cuh"

namespace dn {

cudaError_t block_bwd_f32(const BlockParams &p, bool bias, cudaStream_t stream, int *blocks) {
    return block_bwd_of<float, float>(p, bias, stream, blocks);
}

}  // namespace dn
