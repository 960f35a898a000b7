// Norms around a block, backward.  With hhat and xhat the rows' deviations over their
// root mean squares (rh, rx the factors), s = sigmoid(z):
//
//     d = dy w2,  dh = dresidual_out + rh (d - mean(d) - hhat mean(d hhat)),  dresidual = dh
//     dscale = sum dh s p,  dz = dh scale p s (1 - s),  dp = dh scale s
//     e = dp w1,  dx = rx (e - mean(e) - xhat mean(e xhat))   (or e, without the norm after the block)
//     dw2 = sum dy hhat,  db2 = sum dy,  dw1 = sum dp xhat,  db1 = sum dp
// (no mean(d), mean(e) for the root-mean-square form).
//
// h is computed again from x, z and the residual, as in the forward; every tensor is read
// once.  The sums over rows stay in registers over all rows of a block, whose threads
// write one row of partial sums each; a second kernel adds these in a fixed order.
#include "dn_block.cuh"

namespace dn {
namespace {

constexpr int kSums = 5;  // dw2, db2, dw1, db1, dscale

extern __shared__ __align__(16) char s_ring[];

template <typename T, typename TR, int V, int K, int R>
__global__ void __launch_bounds__(Row<T, V, K, R>::kThreads) block_bwd(BlockParams p) {
    using L = Row<T, V, K, R>;
    using G = BlockRing<T, TR, V, K, R, 3, 2, block_bwd_regs<Row<T, V, K, R>::kThreads>()>;
    constexpr int P = L::P, kWarps = R / 32;
    __shared__ __align__(16) float buf[8 * kWarps];
    const float inv = 1.f / (float)p.D;
    const Norm norm{p.D, p.eps, p.rms};
    const long long step = (long long)gridDim.x * L::kRows;
    long long row = (long long)blockIdx.x * L::kRows + threadIdx.x / R;
    G ring;
    ring.a[0] = static_cast<const T *>(p.x);
    ring.a[1] = static_cast<const T *>(p.z);
    ring.a[2] = static_cast<const T *>(p.dy);
    ring.b[0] = static_cast<const TR *>(p.residual);
    ring.b[1] = static_cast<const TR *>(p.dresidual_out);
#pragma unroll
    for (int s = 0; s < G::S; ++s) ring.issue(s_ring, s, row + s * step, p.rows, p.D);
    Kept<L, V, K> w2, w1, sc;
    w2.init(p.weight, p.D, 1.f);
    w1.init(p.post_weight, p.D, 1.f);
    sc.init(p.scale, p.D, 1.f);
    f2 sums[kSums][K][P];
#pragma unroll
    for (int q = 0; q < kSums; ++q)
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int i = 0; i < P; ++i) sums[q][k][i] = 0ull;
    // the two means of a norm's gradient, over (d, hat)
    auto means = [&](f2 t0, f2 t1, float *b, float &c1, float &c2) {
        if (p.rms) {
            float s[1] = {sum_of(t0)};
            row_sum<R>(s, b);
            c1 = s[0] * inv;
            c2 = 0.f;
        } else {
            float s[2] = {sum_of(t0), sum_of(t1)};
            row_sum<R>(s, b);
            c1 = s[0] * inv;
            c2 = s[1] * inv;
        }
    };
    int stage = 0;
    for (long long first = (long long)blockIdx.x * L::kRows; first < p.rows; first += step, row += step) {
        typename L::Pairs a, h, g, sg;
        const bool live = row < p.rows;
        ring.wait();
#pragma unroll
        for (int k = 0; k < K; ++k) ring.get_a(a[k], s_ring, stage, 0, k, row, p.rows, p.D);
        float rx = 1.f;
        if (p.post) rx = normalise<L, V, K, R>(a, norm, inv, buf);
#pragma unroll
        for (int k = 0; k < K; ++k) {
            f2 r[P];
#pragma unroll
            for (int i = 0; i < P; ++i) h[k][i] = a[k][i];
            w1.times(h[k], k, p.D);
            affine<L, V>(h[k], nullptr, p.post_bias, k, p.D);
            if (p.z) {
                ring.get_a(sg[k], s_ring, stage, 1, k, row, p.rows, p.D);
#pragma unroll
                for (int i = 0; i < P; ++i) {
                    sg[k][i] = sigmoid2(sg[k][i]);
                    h[k][i] = mul2(h[k][i], sg[k][i]);
                }
            }
            sc.times(h[k], k, p.D);
            ring.get_b(r, s_ring, stage, 0, k, row, p.rows, p.D);
#pragma unroll
            for (int i = 0; i < P; ++i) h[k][i] = add2(h[k][i], r[i]);
        }
        const float rh = normalise<L, V, K, R>(h, norm, inv, buf + 2 * kWarps);
        f2 t0 = 0ull, t1 = 0ull;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            ring.get_a(g[k], s_ring, stage, 2, k, row, p.rows, p.D);
            if (live)
#pragma unroll
                for (int i = 0; i < P; ++i) {
                    sums[0][k][i] = fma2(g[k][i], h[k][i], sums[0][k][i]);
                    sums[1][k][i] = add2(sums[1][k][i], g[k][i]);
                }
            w2.times(g[k], k, p.D);
#pragma unroll
            for (int i = 0; i < P; ++i) {
                t0 = fma2(g[k][i], h[k][i], t0);
                t1 = add2(t1, g[k][i]);
            }
        }
        float c1, c2;
        means(t0, t1, buf + 4 * kWarps, c1, c2);
        f2 rr = both(rh), r1 = both(-rh * c1);
        t0 = t1 = 0ull;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            f2 r[P];
            // columns behind D stay 0: they count in the sums below
            const f2 r2 = pair(L::in(k, 0, p.D) ? -rh * c2 : 0.f, L::in(k, 1, p.D) ? -rh * c2 : 0.f);
            ring.get_b(r, s_ring, stage, 1, k, row, p.rows, p.D);
#pragma unroll
            for (int i = 0; i < P; ++i) g[k][i] = add2(r[i], fma2(h[k][i], r1, fma2(g[k][i], rr, r2)));  // dh
            if (!live) continue;
            store_row<L, V>(static_cast<TR *>(p.dresidual) + row * p.D, g[k], k, p.D);
            f2 q[P];  // p
#pragma unroll
            for (int i = 0; i < P; ++i) q[i] = a[k][i];
            w1.times(q, k, p.D);
            affine<L, V>(q, nullptr, p.post_bias, k, p.D);
            if (p.z) {
                f2 out[P];
                const f2 one = both(1.f), (&s)[P] = sg[k];
#pragma unroll
                for (int i = 0; i < P; ++i) {
                    const f2 dp = mul2(g[k][i], q[i]);
                    g[k][i] = mul2(g[k][i], s[i]);
                    sums[4][k][i] = fma2(dp, s[i], sums[4][k][i]);
                    // dh p s (1 - s)
                    out[i] = mul2(mul2(dp, s[i]), fma2(s[i], both(-1.f), one));
                }
                sc.times(out, k, p.D);
                store_row<L, V>(static_cast<T *>(p.dz) + row * p.D, out, k, p.D);
            } else {
#pragma unroll
                for (int i = 0; i < P; ++i) sums[4][k][i] = fma2(g[k][i], q[i], sums[4][k][i]);
            }
            sc.times(g[k], k, p.D);  // dp
#pragma unroll
            for (int i = 0; i < P; ++i) {
                sums[2][k][i] = fma2(g[k][i], a[k][i], sums[2][k][i]);
                sums[3][k][i] = add2(sums[3][k][i], g[k][i]);
            }
            w1.times(g[k], k, p.D);  // e
#pragma unroll
            for (int i = 0; i < P; ++i) {
                t0 = fma2(g[k][i], a[k][i], t0);
                t1 = add2(t1, g[k][i]);
            }
        }
        ring.issue(s_ring, stage, row + G::S * step, p.rows, p.D);
        stage = stage + 1 == G::S ? 0 : stage + 1;
        if (p.post) {
            means(t0, t1, buf + 6 * kWarps, c1, c2);
            rr = both(rx), r1 = both(-rx * c1);
            const f2 r2 = both(-rx * c2);
#pragma unroll
            for (int k = 0; k < K; ++k)
#pragma unroll
                for (int i = 0; i < P; ++i) g[k][i] = fma2(a[k][i], r1, fma2(g[k][i], rr, r2));
        }
        if (live)
#pragma unroll
            for (int k = 0; k < K; ++k) store_row<L, V>(static_cast<T *>(p.dx) + row * p.D, g[k], k, p.D);
    }
    if (!p.partial) return;
    float *part = p.partial + (long long)blockIdx.x * kSums * p.D;
#pragma unroll
    for (int q = 0; q < kSums; ++q)
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int i = 0; i < P; ++i) {
                float v[2];
                split(sums[q][k][i], v[0], v[1]);
                if constexpr (R == 32) {  // the rows of a block, one per warp
                    __shared__ float red[4][2][32];
                    __syncthreads();
                    red[threadIdx.x >> 5][0][threadIdx.x & 31] = v[0];
                    red[threadIdx.x >> 5][1][threadIdx.x & 31] = v[1];
                    __syncthreads();
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        v[e] = (red[0][e][threadIdx.x & 31] + red[1][e][threadIdx.x & 31]) +
                               (red[2][e][threadIdx.x & 31] + red[3][e][threadIdx.x & 31]);
                }
                if (threadIdx.x < R)
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        if (L::in(k, 2 * i + e, p.D)) part[(long long)q * p.D + L::col(k, 2 * i + e)] = v[e];
            }
}

// The sums over rows from the blocks' rows: 32 columns and 32 slices of the rows per block.
__global__ void __launch_bounds__(1024) block_bwd_sums(BlockParams p, int blocks) {
    __shared__ float red[32][33];
    wait_for_launches();
    float *const outs[kSums] = {p.dweight, p.dbias, p.dpost_weight, p.dpost_bias, p.dscale};
    float *out = outs[blockIdx.y];
    if (!out) return;
    const int c = blockIdx.x * 32 + threadIdx.x;
    float a = 0.f;
    if (c < p.D)
#pragma unroll 8
        for (int b = threadIdx.y; b < blocks; b += 32) a += p.partial[((long long)b * kSums + blockIdx.y) * p.D + c];
    red[threadIdx.y][threadIdx.x] = a;
    __syncthreads();
    float v = red[threadIdx.x][threadIdx.y];
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    const int o = blockIdx.x * 32 + threadIdx.y;
    if (threadIdx.x == 0 && o < p.D) out[o] = v;
}

struct Launch {
    const BlockParams &p;
    cudaStream_t stream;
    int *blocks;  // the size of the grid only
    template <typename T, typename TR, int V, int K, int R>
    cudaError_t operator()() const {
        constexpr int kThreads = Row<T, V, K, R>::kThreads;
        const int grid = norm_blocks(p.rows, kThreads, Row<T, V, K, R>::kRows, block_bwd_regs<kThreads>());
        if (blocks) {
            *blocks = grid;
            return cudaSuccess;
        }
        if (grid > 0) {
            constexpr int bytes = BlockRing<T, TR, V, K, R, 3, 2, block_bwd_regs<Row<T, V, K, R>::kThreads>()>::kBytes;
            cudaError_t err = allow_smem<block_bwd<T, TR, V, K, R>>(bytes);
            if (err != cudaSuccess) return err;
            block_bwd<T, TR, V, K, R><<<grid, kThreads, bytes, stream>>>(p);
            err = cudaGetLastError();
            if (err != cudaSuccess) return err;
        }
        if (!p.partial) return cudaSuccess;
        return launch_after(block_bwd_sums, dim3((p.D + 31) / 32, kSums), dim3(32, 32), 0, stream, p, grid);
    }
};

}  // namespace

cudaError_t block_bwd_launch(const BlockParams &p, cudaStream_t stream, const char **name) {
    if (p.rows == 0) *name = "block_bwd_sums";
    else if (p.partial) *name = p.bf16 ? "block_bwd+block_bwd_sums<bf16>" : "block_bwd+block_bwd_sums<f32>";
    else *name = p.bf16 ? "block_bwd<bf16>" : "block_bwd<f32>";
    return block_types(p, Launch{p, stream, nullptr});
}

size_t block_bwd_workspace(long long rows, int D, bool bf16, bool res_f32) {
    BlockParams p{};
    p.rows = rows;
    p.D = D;
    p.bf16 = bf16;
    p.res_f32 = res_f32;
    int blocks = 0;
    block_types(p, Launch{p, nullptr, &blocks});
    return (size_t)(blocks > 0 ? blocks : 1) * kSums * (size_t)D * 4u;
}

}  // namespace dn
