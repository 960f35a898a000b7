// Norms around a block, forward: y = norm(h) w2 + b2 with h = residual + scale sigmoid(z) p,
// p = norm(x) w1 + b1 (or x w1 + b1), in one pass over x, z and the residual stream.
//
// A row is held in registers by R threads as in the layer norm; h stays there between the
// two norms, so every tensor is read once and written once, and y is normed from the h that
// is not yet rounded to the residual's type.  Bound by memory.
#include "dn_block.cuh"

namespace dn {
namespace {

extern __shared__ __align__(16) char s_ring[];

template <typename T, typename TR, int V, int K, int R, bool FULL>
__global__ void __launch_bounds__(Row<T, V, K, R>::kThreads, 65536 / (kBlockFwdRegs * Row<T, V, K, R>::kThreads)) block_fwd(BlockParams p) {
    using L = BlockRow<T, V, K, R, FULL>;
    using G = BlockRing<T, TR, V, K, R, FULL, 1, 2, 1, kBlockFwdRegs>;
    constexpr int P = L::P, kBuf = 2 * (R / 32);
    __shared__ __align__(16) float buf[2 * kBuf + 4];  // consecutive norms in turn
    const float inv = 1.f / (float)p.D;
    const long long step = (long long)gridDim.x * L::kRows;
    long long row = (long long)blockIdx.x * L::kRows + threadIdx.x / R;
    G ring;
    ring.a[0] = static_cast<const T *>(p.x);
    ring.a[1] = static_cast<const T *>(p.z);
    ring.b[0] = static_cast<const TR *>(p.residual);
#pragma unroll
    for (int s = 0; s < G::S; ++s) ring.issue(s_ring, s, row + s * step, p.rows, p.D);
    // a single vector a thread: the fp32 vectors stay in registers
    Kept<L, V, K, K == 1> w2, w1, sc;
    Kept<L, V, K, false> b2, b1;
    w2.init(p.weight, p.D);
    w1.init(p.post_weight, p.D);
    sc.init(p.scale, p.D);
    b2.init(p.bias, p.D);
    b1.init(p.post_bias, p.D);
    int stage = 0, turn = 0;
    for (long long first = (long long)blockIdx.x * L::kRows; first < p.rows; first += step, row += step) {
        f2 hs[1][K][P];
        f2 (&h)[K][P] = hs[0];
        ring.wait();
#pragma unroll
        for (int k = 0; k < K; ++k) ring.get_a(h[k], s_ring, stage, 0, k, row, p.rows, p.D);
        auto norm = [&] {  // h becomes its deviations over their root mean square
            float m[1], r[1];
            row_stats<L, V, K, R>(hs, p.rms, p.eps, inv, p.D, buf + turn * kBuf, m, r);
            turn ^= 1;
            const f2 rr = both(r[0]);
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const f2 mm = L::inside(k, -m[0], p.D);
#pragma unroll
                for (int i = 0; i < P; ++i) h[k][i] = mul2(add2(h[k][i], mm), rr);
            }
        };
        if (p.post) norm();
#pragma unroll
        for (int k = 0; k < K; ++k) {
            w1.times(h[k], k, p.D);
            b1.plus(h[k], k, p.D);
            if (p.z) {
                f2 z[P];
                ring.get_a(z, s_ring, stage, 1, k, row, p.rows, p.D);
#pragma unroll
                for (int i = 0; i < P; ++i) h[k][i] = mul2(h[k][i], sigmoid2(z[i]));
            }
            sc.times(h[k], k, p.D);
            f2 r[P];
            ring.get_b(r, s_ring, stage, 0, k, row, p.rows, p.D);
#pragma unroll
            for (int i = 0; i < P; ++i) h[k][i] = add2(h[k][i], r[i]);
        }
        ring.issue(s_ring, stage, row + G::S * step, p.rows, p.D);
        stage = stage + 1 == G::S ? 0 : stage + 1;
        if (L::live(row, p.rows))
#pragma unroll
            for (int k = 0; k < K; ++k) store_row<L, V>(static_cast<TR *>(p.residual_out) + row * p.D, h[k], k, p.D);
        norm();
        if (L::live(row, p.rows))
#pragma unroll
            for (int k = 0; k < K; ++k) {
                w2.times(h[k], k, p.D);
                b2.plus(h[k], k, p.D);
                store_row<L, V>(static_cast<T *>(p.y) + row * p.D, h[k], k, p.D);
            }
    }
}

struct Launch {
    const BlockParams &p;
    cudaStream_t stream;
    template <typename T, typename TR, int V, int K, int R, bool FULL>
    cudaError_t operator()() const {
        constexpr int kThreads = Row<T, V, K, R>::kThreads;
        constexpr int bytes = BlockRing<T, TR, V, K, R, FULL, 1, 2, 1, kBlockFwdRegs>::kBytes;
        const cudaError_t err = allow_smem<block_fwd<T, TR, V, K, R, FULL>>(bytes);
        if (err != cudaSuccess) return err;
        block_fwd<T, TR, V, K, R, FULL><<<norm_blocks(p.rows, kThreads, Row<T, V, K, R>::kRows, kBlockFwdRegs), kThreads, bytes, stream>>>(p);
        return cudaGetLastError();
    }
};

}  // namespace

cudaError_t block_fwd_launch(const BlockParams &p, cudaStream_t stream, const char **name) {
    *name = p.bf16 ? "block_fwd<bf16>" : "block_fwd<f32>";
    const Launch f{p, stream};
    if (!p.bf16) return block_dispatch<float, float, 8>(p.D, f);
    return p.res_f32 ? block_dispatch<__nv_bfloat16, float, 8>(p.D, f) : block_dispatch<__nv_bfloat16, __nv_bfloat16, 8>(p.D, f);
}

}  // namespace dn
