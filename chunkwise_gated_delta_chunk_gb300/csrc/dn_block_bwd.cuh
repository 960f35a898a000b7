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
// once from memory (x and z twice from shared memory, where they wait, which costs fewer registers
// than what comes of them).  With t = dh s the sums over rows are four, the last two only for biases:
//     S0 = sum dy hhat,  S1 = sum t xhat,  S2 = sum dy,  S3 = sum t
//     dw2 = S0,  db2 = S2,  dw1 = scale S1,  db1 = scale S3,  dscale = w1 S1 + b1 S3
// They stay in registers over all rows of a block, which writes a row of them; a second
// kernel adds these up in a fixed order.
#pragma once

#include "dn_block.cuh"

namespace dn {
namespace {

extern __shared__ __align__(16) char s_ring[];

template <typename T, typename TR, int V, int K, int R, bool FULL, int N, bool BIAS>
__global__ void __launch_bounds__(Row<T, V, K, R>::kThreads, 65536 / (block_bwd_regs(Row<T, V, K, R>::kThreads) * Row<T, V, K, R>::kThreads))
block_bwd(BlockParams p) {
    using L = BlockRow<T, V, K, R, FULL, N>;
    using G = BlockRing<T, TR, V, K, R, FULL, N, 3, 2, block_bwd_regs(L::kThreads)>;
    constexpr int P = L::P, kWarps = R / 32, kSums = BIAS ? 4 : 2;
    __shared__ __align__(16) float buf[8 * N * kWarps];
    const float inv = 1.f / (float)p.D;
    // N neighbouring rows of a warp or block at a time
    const long long step = (long long)gridDim.x * L::kRows * N;
    long long row = ((long long)blockIdx.x * L::kRows + threadIdx.x / R) * N;
    G ring;
    ring.a[0] = static_cast<const T *>(p.x);
    ring.a[1] = static_cast<const T *>(p.z);
    ring.a[2] = static_cast<const T *>(p.dy);
    ring.b[0] = static_cast<const TR *>(p.residual);
    ring.b[1] = static_cast<const TR *>(p.dresidual_out);
#pragma unroll
    for (int s = 0; s < G::S; ++s) ring.issue(s_ring, s, row + s / N * step + s % N, p.rows, p.D);
    // scale p = xhat A + B with A = scale w1, B = scale b1: A stays in registers where there are enough, and w2
    // where no sums for biases take its place
    constexpr bool kRoomy = block_bwd_regs(L::kThreads) >= 128, kAll = kRoomy && (!BIAS || K * V <= 8);
    Kept<L, V, K, kAll> w2;
    Scaled<L, V, K, kAll || (kRoomy && L::kThreads <= 128)> A;
    Scaled<L, V, K, kAll && BIAS> B;
    w2.init(p.weight, p.D);
    A.init(p.post_weight, p.scale, p.D);
    B.init(p.post_bias, p.scale, p.D);
    f2 sums[kSums][K][P];
#pragma unroll
    for (int q = 0; q < kSums; ++q)
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int i = 0; i < P; ++i) sums[q][k][i] = 0ull;
    // the two means of a norm's gradient, over (d, hat)
    auto means = [&](const f2 (&t0)[N], const f2 (&t1)[N], float *b, float (&c1)[N], float (&c2)[N]) {
        if (p.rms) {
            float s[N];
#pragma unroll
            for (int n = 0; n < N; ++n) s[n] = sum_of(t0[n]);
            sum_row<R>(s, b);
#pragma unroll
            for (int n = 0; n < N; ++n) {
                c1[n] = s[n] * inv;
                c2[n] = 0.f;
            }
        } else {
            float s[2 * N];
#pragma unroll
            for (int n = 0; n < N; ++n) {
                s[2 * n] = sum_of(t0[n]);
                s[2 * n + 1] = sum_of(t1[n]);
            }
            sum_row<R>(s, b);
#pragma unroll
            for (int n = 0; n < N; ++n) {
                c1[n] = s[2 * n] * inv;
                c2[n] = s[2 * n + 1] * inv;
            }
        }
    };
    auto inside = [&](int k, float v) { return L::inside(k, v, p.D); };
    int stage = 0;
    for (long long first = (long long)blockIdx.x * L::kRows * N; first < p.rows; first += step, row += step) {
        f2 h[N][K][P], g[N][K][P];
        float mx[N], rx[N], mh[N], rh[N];  // means and factors
        ring.wait();
#pragma unroll
        for (int n = 0; n < N; ++n) {
            mx[n] = 0.f;
            rx[n] = 1.f;
#pragma unroll
            for (int k = 0; k < K; ++k) ring.get_a(h[n][k], s_ring, stage + n, 0, k, row + n, p.rows, p.D);
        }
        if (p.post) row_stats<L, V, K, R>(h, p.rms, p.eps, inv, p.D, buf, mx, rx);
        // xhat of vector k from x, as the forward takes it
        auto hat = [&](f2 (&x)[P], int n, int k) {
            if (!p.post) return;
            const f2 mm = inside(k, -mx[n]), rr = both(rx[n]);
#pragma unroll
            for (int i = 0; i < P; ++i) x[i] = mul2(add2(x[i], mm), rr);
        };
#pragma unroll
        for (int n = 0; n < N; ++n)
#pragma unroll
            for (int k = 0; k < K; ++k) {
                f2 r[P];
                hat(h[n][k], n, k);
                if (A.a || A.b) A.times(h[n][k], k, p.D);
                if (BIAS && B.a) B.plus(h[n][k], k, p.D);
                if (p.z) {
                    ring.get_a(r, s_ring, stage + n, 1, k, row + n, p.rows, p.D);
#pragma unroll
                    for (int i = 0; i < P; ++i) h[n][k][i] = mul2(h[n][k][i], sigmoid2(r[i]));
                }
                ring.get_b(r, s_ring, stage + n, 0, k, row + n, p.rows, p.D);
#pragma unroll
                for (int i = 0; i < P; ++i) h[n][k][i] = add2(h[n][k][i], r[i]);
            }
        row_stats<L, V, K, R>(h, p.rms, p.eps, inv, p.D, buf + 2 * N * kWarps, mh, rh);
        f2 t0[N], t1[N];
#pragma unroll
        for (int n = 0; n < N; ++n) {
            t0[n] = t1[n] = 0ull;
            const bool live = L::live(row + n, p.rows);
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const f2 mm = inside(k, -mh[n]), rr = both(rh[n]);
                ring.get_a(g[n][k], s_ring, stage + n, 2, k, row + n, p.rows, p.D);
#pragma unroll
                for (int i = 0; i < P; ++i) {
                    h[n][k][i] = mul2(add2(h[n][k][i], mm), rr);
                    if (live) {
                        sums[0][k][i] = fma2(g[n][k][i], h[n][k][i], sums[0][k][i]);
                        if (BIAS) sums[2 % kSums][k][i] = add2(sums[2 % kSums][k][i], g[n][k][i]);
                    }
                }
                w2.times(g[n][k], k, p.D);
#pragma unroll
                for (int i = 0; i < P; ++i) {
                    t0[n] = fma2(g[n][k][i], h[n][k][i], t0[n]);
                    t1[n] = add2(t1[n], g[n][k][i]);
                }
            }
        }
        float c1[N], c2[N];
        means(t0, t1, buf + 4 * N * kWarps, c1, c2);
#pragma unroll
        for (int n = 0; n < N; ++n) {
            t0[n] = t1[n] = 0ull;
            const bool live = L::live(row + n, p.rows);
            const long long at = (row + n) * p.D;
#pragma unroll
            for (int k = 0; k < K; ++k) {
                f2 r[P], s[P];
                // columns behind D stay 0: they count in the sums below
                const f2 rr = both(rh[n]), r1 = both(-rh[n] * c1[n]), r2 = inside(k, -rh[n] * c2[n]);
                ring.get_b(r, s_ring, stage + n, 1, k, row + n, p.rows, p.D);
#pragma unroll
                for (int i = 0; i < P; ++i) g[n][k][i] = add2(r[i], fma2(h[n][k][i], r1, fma2(g[n][k][i], rr, r2)));  // dh
                ring.get_a(h[n][k], s_ring, stage + n, 0, k, row + n, p.rows, p.D);
                hat(h[n][k], n, k);  // xhat from here on
                if (!live) continue;
                store_row<L, V>(static_cast<TR *>(p.dresidual) + at, g[n][k], k, p.D);
                if (p.z) {
                    ring.get_a(s, s_ring, stage + n, 1, k, row + n, p.rows, p.D);
                    const f2 one = both(1.f), minus = both(-1.f);
#pragma unroll
                    for (int i = 0; i < P; ++i) {
                        s[i] = sigmoid2(s[i]);
                        g[n][k][i] = mul2(g[n][k][i], s[i]);  // t
                        s[i] = fma2(s[i], minus, one);
                        r[i] = h[n][k][i];
                    }
                    if (A.a || A.b) A.times(r, k, p.D);
                    if (BIAS && B.a) B.plus(r, k, p.D);
#pragma unroll
                    for (int i = 0; i < P; ++i) r[i] = mul2(r[i], mul2(g[n][k][i], s[i]));
                    store_row<L, V>(static_cast<T *>(p.dz) + at, r, k, p.D);
                }
#pragma unroll
                for (int i = 0; i < P; ++i) {
                    sums[1][k][i] = fma2(g[n][k][i], h[n][k][i], sums[1][k][i]);
                    if (BIAS) sums[3 % kSums][k][i] = add2(sums[3 % kSums][k][i], g[n][k][i]);
                }
                if (A.a || A.b) A.times(g[n][k], k, p.D);  // e
#pragma unroll
                for (int i = 0; i < P; ++i) {
                    t0[n] = fma2(g[n][k][i], h[n][k][i], t0[n]);
                    t1[n] = add2(t1[n], g[n][k][i]);
                }
            }
        }
#pragma unroll
        for (int n = 0; n < N; ++n) ring.issue(s_ring, stage + n, row + G::S / N * step + n, p.rows, p.D);
        stage = stage + N == G::S ? 0 : stage + N;
        if (p.post) means(t0, t1, buf + 6 * N * kWarps, c1, c2);
#pragma unroll
        for (int n = 0; n < N; ++n) {
            const bool live = L::live(row + n, p.rows);
            const f2 rr = both(rx[n]), r1 = both(-rx[n] * c1[n]), r2 = both(-rx[n] * c2[n]);
#pragma unroll
            for (int k = 0; k < K; ++k) {
                if (p.post)
#pragma unroll
                    for (int i = 0; i < P; ++i) g[n][k][i] = fma2(h[n][k][i], r1, fma2(g[n][k][i], rr, r2));
                if (live) store_row<L, V>(static_cast<T *>(p.dx) + (row + n) * p.D, g[n][k], k, p.D);
            }
        }
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

template <bool BIAS, int N>
struct BlockBwd {
    const BlockParams &p;
    cudaStream_t stream;
    int *blocks;  // the size of the grid only
    template <typename T, typename TR, int V, int K, int R, bool FULL>
    cudaError_t operator()() const {
        constexpr int kThreads = Row<T, V, K, R>::kThreads, kRegs = block_bwd_regs(kThreads);
        const int grid = norm_blocks(p.rows, kThreads, Row<T, V, K, R>::kRows * N, kRegs);
        if (blocks) {
            *blocks = grid;
            return cudaSuccess;
        }
        if (grid > 0) {
            constexpr int bytes = BlockRing<T, TR, V, K, R, FULL, N, 3, 2, kRegs>::kBytes;
            cudaError_t err = allow_smem<block_bwd<T, TR, V, K, R, FULL, N, BIAS>>(bytes);
            if (err != cudaSuccess) return err;
            block_bwd<T, TR, V, K, R, FULL, N, BIAS><<<grid, kThreads, bytes, stream>>>(p);
            err = cudaGetLastError();
            if (err != cudaSuccess) return err;
        }
        if (!p.partial) return cudaSuccess;
        return block_bwd_sums_launch(p, grid, BIAS ? 4 : 2, stream);
    }
};

// Two rows at a time of 8 elements a thread, whose barriers and loads of the vectors are shared (16383 rows of
// 4096 with biases 213 us, 250 one by one); without biases and above 2048 columns one row of 16
// elements a thread, whose vectors stay in registers (the same rows 165 us, 188 by twos).
template <typename T, typename TR>
cudaError_t block_bwd_of(const BlockParams &p, bool bias, cudaStream_t stream, int *blocks) {
    constexpr int kWide = 2048;
    if (bias) return block_dispatch<T, TR, 8>(p.D, BlockBwd<true, 2>{p, stream, blocks});
    if (p.D <= kWide) return block_dispatch<T, TR, 8, 1, kWide>(p.D, BlockBwd<false, 2>{p, stream, blocks});
    return block_dispatch<T, TR, 16, kWide + 1>(p.D, BlockBwd<false, 1>{p, stream, blocks});
}

}  // namespace
}  // namespace dn
