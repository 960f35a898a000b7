// Norms around a block, backward: the choice of types and the gradients of the vectors.
#include "dn_block.cuh"

namespace dn {
namespace {

// The gradients of the vectors from the blocks' rows of sums: 32 columns and 32 slices of the rows per
// block; S0 and S2 by one row of blocks, S1 and S3 by the other.
__global__ void __launch_bounds__(1024) block_bwd_sums(BlockParams p, int blocks, int planes) {
    __shared__ float red[2][32][33];
    wait_for_launches();
    const int c = blockIdx.x * 32 + threadIdx.x, y = blockIdx.y;
    float a[2] = {0.f, 0.f};
    if (c < p.D)
#pragma unroll 8
        for (int b = threadIdx.y; b < blocks; b += 32) {
            const float *row = p.partial + (long long)b * planes * p.D + c;
            a[0] += row[(long long)y * p.D];
            if (planes == 4) a[1] += row[(long long)(y + 2) * p.D];
        }
#pragma unroll
    for (int q = 0; q < 2; ++q) red[q][threadIdx.y][threadIdx.x] = a[q];
    __syncthreads();
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        a[q] = red[q][threadIdx.x][threadIdx.y];  // column threadIdx.y, slice threadIdx.x
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) a[q] += __shfl_xor_sync(0xffffffffu, a[q], off);
    }
    const int o = blockIdx.x * 32 + threadIdx.y;
    if (threadIdx.x != 0 || o >= p.D) return;
    if (y == 0) {
        if (p.dweight) p.dweight[o] = a[0];
        if (p.dbias) p.dbias[o] = a[1];
        return;
    }
    const float sc = p.scale ? p.scale[o] : 1.f;
    if (p.dpost_weight) p.dpost_weight[o] = sc * a[0];
    if (p.dpost_bias) p.dpost_bias[o] = sc * a[1];
    if (p.dscale) {
        const float v = (p.post_weight ? p.post_weight[o] : 1.f) * a[0];
        p.dscale[o] = p.post_bias ? fmaf(p.post_bias[o], a[1], v) : v;
    }
}

// of one type each, in files of their own (they compile side by side)
cudaError_t of_type(const BlockParams &p, bool bias, cudaStream_t stream, int *blocks) {
    if (!p.bf16) return block_bwd_f32(p, bias, stream, blocks);
    return p.res_f32 ? block_bwd_bf16_f32(p, bias, stream, blocks) : block_bwd_bf16(p, bias, stream, blocks);
}

}  // namespace

cudaError_t block_bwd_sums_launch(const BlockParams &p, int blocks, int planes, cudaStream_t stream) {
    return launch_after(block_bwd_sums, dim3((p.D + 31) / 32, 2), dim3(32, 32), 0, stream, p, blocks, planes);
}

cudaError_t block_bwd_launch(const BlockParams &p, cudaStream_t stream, const char **name) {
    if (p.rows == 0) *name = "block_bwd_sums";
    else if (p.partial) *name = p.bf16 ? "block_bwd+block_bwd_sums<bf16>" : "block_bwd+block_bwd_sums<f32>";
    else *name = p.bf16 ? "block_bwd<bf16>" : "block_bwd<f32>";
    return of_type(p, p.dbias || p.dpost_bias || p.post_bias, stream, nullptr);
}

size_t block_bwd_workspace(long long rows, int D, bool bf16, bool res_f32) {
    BlockParams p{};
    p.rows = rows;
    p.D = D;
    p.bf16 = bf16;
    p.res_f32 = res_f32;
    int with = 0, without = 0;
    of_type(p, true, nullptr, &with);
    of_type(p, false, nullptr, &without);
    const int most = 4 * with > 2 * without ? 4 * with : 2 * without;
    return (size_t)(most > 4 ? most : 4) * (size_t)D * 4u;
}

}  // namespace dn
