// Layer norm of rows of D elements (or its root-mean-square form), with
// weight, bias and the gate silu(z); forward and backward.
//
//     xhat = (x - m) r,   n = xhat w + b,   y = n silu(z)
//     backward, dn = dy silu(z), d = dn w:
//     dx = r (d - mean(d) - xhat mean(d xhat)),  dw = sum dn xhat,  db = sum dn,  dz = dy n silu'(z)
// (no mean(d) for the root-mean-square form).
//
// A row is held in registers by R threads, K vectors of V elements each, so
// that every tensor is read once and the variance is taken about the mean.
// R <= 32: several rows per warp, sums by shuffles; larger R: one row per
// block, sums through shared memory.  Blocks walk rows; the vectors of the rows
// ahead come by asynchronous copies into each thread's own part of shared memory,
// so that the sums' latency and the barriers do not keep memory idle (loaded into
// registers row by row, the backward of 4096 columns reached 31 % of the memory
// rate).  The arithmetic is on pairs.  Short rows are bound by memory and issue, long ones
// in the backward by three barriers a row against 2 blocks an SM: measured
// (bf16) 131072 rows of 128, root mean square and gate, forward 20.6 us (4.9 TB/s),
// backward 33 us (5.0); 16383 rows of 4096, backward 94 us (4.3 TB/s).
//
// Backward: the sums of dw and db of a thread's columns stay in registers over all
// rows of its block; the threads that share a column are joined and the block writes
// one row of partial sums; a second kernel adds these rows in a fixed order.
#include "dn_norm.cuh"

namespace dn {
namespace {

// The vectors of A tensors' rows that a thread works on, S iterations ahead.
template <typename T, int V, int K, int R, int A>
struct Ring {
    using L = Row<T, V, K, R>;
    static constexpr int kStage = L::kWhole ? A * K * L::kThreads * 16 : 0;
    static constexpr int kFit = L::kWhole ? 65536 / kStage : 1;
    static constexpr int S = kFit < 1 ? 1 : kFit > 4 ? 4 : kFit;
    static constexpr int kBytes = L::kWhole ? S * kStage : 0;
    const T *base[A];
    __device__ __forceinline__ void issue(char *ring, int s, long long row, const NormParams &p) {
        if constexpr (L::kWhole) {
#pragma unroll
            for (int a = 0; a < A; ++a)
#pragma unroll
                for (int k = 0; k < K; ++k)
                    if (row < p.rows && L::in(k, 0, p.D)) {
                        const unsigned dst = (unsigned)__cvta_generic_to_shared(ring) + s * kStage +
                                             ((a * K + k) * L::kThreads + threadIdx.x) * 16;
                        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst),
                                     "l"(base[a] + row * p.D + L::col(k, 0))
                                     : "memory");
                    }
            asm volatile("cp.async.commit_group;" ::: "memory");
        }
    }
    __device__ __forceinline__ void wait() {
        if constexpr (L::kWhole) asm volatile("cp.async.wait_group %0;" ::"n"(S - 1) : "memory");
    }
    // vector k of tensor a as pairs; zeros where the row or the column does not exist
    __device__ __forceinline__ void get(f2 (&v)[L::P], const char *ring, int s, int a, int k, long long row,
                                        const NormParams &p) const {
        if constexpr (L::kWhole) {
            Pack<T, V> r;
            r.clear();
            if (row < p.rows && L::in(k, 0, p.D))
                r.load(reinterpret_cast<const T *>(ring + s * kStage + ((a * K + k) * L::kThreads + threadIdx.x) * 16));
#pragma unroll
            for (int i = 0; i < L::P; ++i) v[i] = pair(r[2 * i], r[2 * i + 1]);
        } else {
            v[0] = load_elements<L>(base[a] + row * p.D, k, row < p.rows ? p.D : 0);
        }
    }
};

extern __shared__ __align__(16) char s_ring[];

template <typename T, int V, int K, int R, bool GATE>
__global__ void __launch_bounds__(Row<T, V, K, R>::kThreads) norm_fwd(NormParams p) {
    using L = Row<T, V, K, R>;
    using G = Ring<T, V, K, R, GATE ? 2 : 1>;
    constexpr int P = L::P;
    __shared__ __align__(16) float buf[4 * (R / 32) + 4];  // of even and of odd rows: one sum may be all that separates them
    const int sub = threadIdx.x / R;
    const float inv = 1.f / (float)p.D;
    const long long step = (long long)gridDim.x * L::kRows;
    long long row = (long long)blockIdx.x * L::kRows + sub;
    G ring;
    ring.base[0] = static_cast<const T *>(p.x);
    if (GATE) ring.base[GATE ? 1 : 0] = static_cast<const T *>(p.z);
#pragma unroll
    for (int s = 0; s < G::S; ++s) ring.issue(s_ring, s, row + s * step, p);
    f2 w[P], b[P];
    auto vectors = [&](int k) {  // weight and bias of vector k
        if (p.weight) load_vec<L, V>(w, p.weight, k, p.D, 1.f);
        if (p.bias) load_vec<L, V>(b, p.bias, k, p.D, 0.f);
    };
    if (K == 1) vectors(0);  // the same for all rows
    int stage = 0, odd = 0;
    for (long long first = (long long)blockIdx.x * L::kRows; first < p.rows; first += step, row += step) {
        typename L::Pairs a, z;
        ring.wait();
#pragma unroll
        for (int k = 0; k < K; ++k) {
            ring.get(a[k], s_ring, stage, 0, k, row, p);
            if (GATE) ring.get(z[k], s_ring, stage, GATE ? 1 : 0, k, row, p);
        }
        ring.issue(s_ring, stage, row + G::S * step, p);
        stage = stage + 1 == G::S ? 0 : stage + 1;
        normalise<L, V, K, R>(a, Norm{p.D, p.eps, p.rms}, inv, buf + odd * 2 * (R / 32));
        odd ^= 1;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            if (row >= p.rows) continue;
            if (K > 1) vectors(k);
#pragma unroll
            for (int i = 0; i < P; ++i) {
                f2 n = a[k][i];
                if (p.weight) n = p.bias ? fma2(n, w[i], b[i]) : mul2(n, w[i]);
                else if (p.bias) n = add2(n, b[i]);
                if (GATE) n = mul2(n, mul2(z[k][i], sigmoid2(z[k][i])));
                a[k][i] = n;
            }
            store_row<L, V>(static_cast<T *>(p.y) + row * p.D, a[k], k, p.D);
        }
    }
}

template <typename T, int V, int K, int R, bool GATE>
__global__ void __launch_bounds__(Row<T, V, K, R>::kThreads) norm_bwd(NormParams p) {
    using L = Row<T, V, K, R>;
    using G = Ring<T, V, K, R, GATE ? 3 : 2>;
    constexpr int P = L::P;
    __shared__ __align__(16) float buf[4 * (R / 32) + 4];
    const int sub = threadIdx.x / R;
    const float inv = 1.f / (float)p.D;
    const long long step = (long long)gridDim.x * L::kRows;
    long long row = (long long)blockIdx.x * L::kRows + sub;
    G ring;
    ring.base[0] = static_cast<const T *>(p.x);
    ring.base[1] = static_cast<const T *>(p.dy);
    if (GATE) ring.base[GATE ? 2 : 0] = static_cast<const T *>(p.z);
#pragma unroll
    for (int s = 0; s < G::S; ++s) ring.issue(s_ring, s, row + s * step, p);
    typename L::Pairs w, sw, sb;
#pragma unroll
    for (int k = 0; k < K; ++k) {
        load_vec<L, V>(w[k], p.weight, k, p.D, 1.f);
#pragma unroll
        for (int i = 0; i < P; ++i) sw[k][i] = sb[k][i] = 0ull;
    }
    int stage = 0;
    for (long long first = (long long)blockIdx.x * L::kRows; first < p.rows; first += step, row += step) {
        typename L::Pairs a, g, z;
        ring.wait();
#pragma unroll
        for (int k = 0; k < K; ++k) {
            ring.get(a[k], s_ring, stage, 0, k, row, p);
            ring.get(g[k], s_ring, stage, 1, k, row, p);
            if (GATE) ring.get(z[k], s_ring, stage, GATE ? 2 : 0, k, row, p);
        }
        ring.issue(s_ring, stage, row + G::S * step, p);
        stage = stage + 1 == G::S ? 0 : stage + 1;
        const float r = normalise<L, V, K, R>(a, Norm{p.D, p.eps, p.rms}, inv, buf);
        f2 t0 = 0ull, t1 = 0ull;  // sums of d xhat and of d
#pragma unroll
        for (int k = 0; k < K; ++k) {
            if (row >= p.rows) continue;
            if (GATE) {
                f2 b[P], out[P];
                if (p.bias) load_vec<L, V>(b, p.bias, k, p.D, 0.f);
#pragma unroll
                for (int i = 0; i < P; ++i) {
                    const f2 n = p.bias ? fma2(a[k][i], w[k][i], b[i]) : mul2(a[k][i], w[k][i]);
                    const f2 u = z[k][i], s = sigmoid2(u), one = both(1.f);
                    // silu' = s (1 + u (1 - s))
                    out[i] = mul2(mul2(g[k][i], n), mul2(s, fma2(u, fma2(s, both(-1.f), one), one)));
                    g[k][i] = mul2(g[k][i], mul2(u, s));
                }
                store_row<L, V>(static_cast<T *>(p.dz) + row * p.D, out, k, p.D);
            }
#pragma unroll
            for (int i = 0; i < P; ++i) {
                sw[k][i] = fma2(g[k][i], a[k][i], sw[k][i]);
                sb[k][i] = add2(sb[k][i], g[k][i]);
                g[k][i] = mul2(g[k][i], w[k][i]);
                t0 = fma2(g[k][i], a[k][i], t0);
                t1 = add2(t1, g[k][i]);
            }
        }
        float c1, c2 = 0.f;
        if (p.rms) {
            float s[1] = {sum_of(t0)};
            row_sum<R>(s, buf + 2 * (R / 32));
            c1 = s[0] * inv;
        } else {
            float s[2] = {sum_of(t0), sum_of(t1)};
            row_sum<R>(s, buf + 2 * (R / 32));
            c1 = s[0] * inv;
            c2 = s[1] * inv;
        }
        const f2 rr = both(r), r1 = both(-r * c1), r2 = both(-r * c2);
#pragma unroll
        for (int k = 0; k < K; ++k) {
            if (row >= p.rows) continue;
#pragma unroll
            for (int i = 0; i < P; ++i) g[k][i] = fma2(a[k][i], r1, fma2(g[k][i], rr, r2));
            store_row<L, V>(static_cast<T *>(p.dx) + row * p.D, g[k], k, p.D);
        }
    }
    if (!p.partial) return;
    float *part = p.partial + (long long)blockIdx.x * 2 * p.D;
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int i = 0; i < P; ++i) {
                float v[2];
                split(h ? sb[k][i] : sw[k][i], v[0], v[1]);
                // the rows of a warp first, then its warps
#pragma unroll
                for (int off = R; off < 32; off <<= 1) {
                    v[0] += __shfl_xor_sync(0xffffffffu, v[0], off);
                    v[1] += __shfl_xor_sync(0xffffffffu, v[1], off);
                }
                if constexpr (R <= 32) {
                    __shared__ float red[4][2][32];
                    __syncthreads();
                    red[threadIdx.x >> 5][0][threadIdx.x & 31] = v[0];
                    red[threadIdx.x >> 5][1][threadIdx.x & 31] = v[1];
                    __syncthreads();
#pragma unroll
                    for (int q = 0; q < 2; ++q)
                        v[q] = (red[0][q][threadIdx.x & 31] + red[1][q][threadIdx.x & 31]) +
                               (red[2][q][threadIdx.x & 31] + red[3][q][threadIdx.x & 31]);
                }
                if (threadIdx.x < R)
#pragma unroll
                    for (int q = 0; q < 2; ++q)
                        if (L::in(k, 2 * i + q, p.D)) part[(long long)h * p.D + L::col(k, 2 * i + q)] = v[q];
            }
}

// dweight and dbias from the blocks' rows: 32 columns and 32 slices of the rows per block.
__global__ void __launch_bounds__(1024) norm_bwd_sums(NormParams p, int blocks) {
    __shared__ float red[32][33];
    wait_for_launches();
    const int c = blockIdx.x * 32 + threadIdx.x;
    const int h = blockIdx.y;
    float a = 0.f;
    if (c < p.D)
#pragma unroll 8
        for (int b = threadIdx.y; b < blocks; b += 32) a += p.partial[((long long)b * 2 + h) * p.D + c];
    red[threadIdx.y][threadIdx.x] = a;
    __syncthreads();
    float v = red[threadIdx.x][threadIdx.y];  // column threadIdx.y, slice threadIdx.x
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    float *out = h ? p.dbias : p.dweight;
    const int o = blockIdx.x * 32 + threadIdx.y;
    if (threadIdx.x == 0 && o < p.D && out) out[o] = v;
}

template <typename T, int V, int K, int R, bool GATE>
cudaError_t norm_launch_g(const NormParams &p, bool bwd, cudaStream_t stream) {
    constexpr int kRows = Row<T, V, K, R>::kRows, kThreads = Row<T, V, K, R>::kThreads;
    if (!bwd) {
        constexpr int bytes = Ring<T, V, K, R, GATE ? 2 : 1>::kBytes;
        const cudaError_t err = allow_smem<norm_fwd<T, V, K, R, GATE>>(bytes);
        if (err != cudaSuccess) return err;
        norm_fwd<T, V, K, R, GATE><<<norm_blocks(p.rows, kThreads, kRows, 64), kThreads, bytes, stream>>>(p);
    } else {
        const int grid = norm_blocks(p.rows, kThreads, kRows, 128);
        if (grid > 0) {
            constexpr int bytes = Ring<T, V, K, R, GATE ? 3 : 2>::kBytes;
            cudaError_t err = allow_smem<norm_bwd<T, V, K, R, GATE>>(bytes);
            if (err != cudaSuccess) return err;
            norm_bwd<T, V, K, R, GATE><<<grid, kThreads, bytes, stream>>>(p);
            err = cudaGetLastError();
            if (err != cudaSuccess) return err;
        }
        if (p.partial) return launch_after(norm_bwd_sums, dim3((p.D + 31) / 32, 2), dim3(32, 32), 0, stream, p, grid);
    }
    return cudaGetLastError();
}

template <typename T, int V, int K, int R>
cudaError_t norm_launch(const NormParams &p, bool bwd, cudaStream_t stream, int *blocks) {
    if (blocks) {  // the size of the backward's grid only
        *blocks = norm_blocks(p.rows, Row<T, V, K, R>::kThreads, Row<T, V, K, R>::kRows, 128);
        return cudaSuccess;
    }
    return p.z ? norm_launch_g<T, V, K, R, true>(p, bwd, stream) : norm_launch_g<T, V, K, R, false>(p, bwd, stream);
}

// Threads and vectors of a row by its length in vectors of 16 bytes.  The backward takes
// two vectors a thread where the forward takes one: its sums need the registers of fewer
// threads (2048 columns of bf16, 16384 rows: forward 29 us with one vector, 39 with two;
// backward 61 with one, 55 with two; a warp alone, 8 vectors: 54 and 97).
template <typename T>
cudaError_t norm_dispatch(const NormParams &p, bool bwd, cudaStream_t stream, int *blocks) {
    constexpr int V = 16 / sizeof(T);
    if (p.D % V == 0) {
        const int n = p.D / V;  // at most 4096 (fp32)
        if (n <= 8) return norm_launch<T, V, 1, 8>(p, bwd, stream, blocks);
        if (n <= 16) return norm_launch<T, V, 1, 16>(p, bwd, stream, blocks);
        if (n <= 32) return norm_launch<T, V, 1, 32>(p, bwd, stream, blocks);
        if (n <= 64) return norm_launch<T, V, 2, 32>(p, bwd, stream, blocks);
        if (n <= 128) return norm_launch<T, V, 1, 128>(p, bwd, stream, blocks);
        if (n <= 256) return bwd ? norm_launch<T, V, 2, 128>(p, bwd, stream, blocks) : norm_launch<T, V, 1, 256>(p, bwd, stream, blocks);
        if (n <= 512) return bwd ? norm_launch<T, V, 2, 256>(p, bwd, stream, blocks) : norm_launch<T, V, 1, 512>(p, bwd, stream, blocks);
        if (n <= 1024) return norm_launch<T, V, 2, 512>(p, bwd, stream, blocks);
        return norm_launch<T, V, 16 / V, 1024>(p, bwd, stream, blocks);
    }
    // rows that do not begin on 16 bytes: single elements
    if (p.D <= 32) return norm_launch<T, 2, 1, 16>(p, bwd, stream, blocks);
    if (p.D <= 128) return norm_launch<T, 2, 2, 32>(p, bwd, stream, blocks);
    if (p.D <= 512) return norm_launch<T, 2, 2, 128>(p, bwd, stream, blocks);
    if (p.D <= 2048) return norm_launch<T, 2, 4, 256>(p, bwd, stream, blocks);
    if (p.D <= 8192) return norm_launch<T, 2, 8, 512>(p, bwd, stream, blocks);
    return norm_launch<T, 2, 8, 1024>(p, bwd, stream, blocks);
}

}  // namespace

cudaError_t norm_fwd_launch(const NormParams &p, bool bf16, cudaStream_t stream, const char **name) {
    *name = bf16 ? "norm_fwd<bf16>" : "norm_fwd<f32>";
    return bf16 ? norm_dispatch<__nv_bfloat16>(p, false, stream, nullptr) : norm_dispatch<float>(p, false, stream, nullptr);
}

cudaError_t norm_bwd_launch(const NormParams &p, bool bf16, cudaStream_t stream, const char **name) {
    if (p.rows == 0) *name = "norm_bwd_sums";
    else if (p.partial) *name = bf16 ? "norm_bwd+norm_bwd_sums<bf16>" : "norm_bwd+norm_bwd_sums<f32>";
    else *name = bf16 ? "norm_bwd<bf16>" : "norm_bwd<f32>";
    return bf16 ? norm_dispatch<__nv_bfloat16>(p, true, stream, nullptr) : norm_dispatch<float>(p, true, stream, nullptr);
}

size_t norm_bwd_workspace(long long rows, int D, bool bf16) {
    NormParams p{};
    p.rows = rows;
    p.D = D;
    int blocks = 0;
    if (bf16) norm_dispatch<__nv_bfloat16>(p, true, nullptr, &blocks);
    else norm_dispatch<float>(p, true, nullptr, &blocks);
    return (size_t)(blocks > 0 ? blocks : 1) * 2u * (size_t)D * 4u;
}

}  // namespace dn
