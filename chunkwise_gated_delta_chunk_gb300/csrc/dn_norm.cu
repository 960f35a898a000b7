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
// block, sums through shared memory.  Both directions are bound by memory.
//
// Backward: a block walks rows with the sums of dw and db of its columns in
// registers, joins the threads that share a column and writes one row of
// partial sums; a second kernel adds these rows in a fixed order.
#include "dn_layer.cuh"

namespace dn {
namespace {

// Sum over the R threads of a row; every one of them gets it.  R > 32: `buf`
// has R / 32 floats, and two buffers are used in turn by consecutive sums.
template <int R, int S>
__device__ __forceinline__ void row_sum(float (&a)[S], float *buf) {
    constexpr int kIn = R < 32 ? R : 32;
#pragma unroll
    for (int off = kIn / 2; off > 0; off >>= 1)
#pragma unroll
        for (int s = 0; s < S; ++s) a[s] += __shfl_xor_sync(0xffffffffu, a[s], off);
    if constexpr (R > 32) {
        constexpr int kWarps = R / 32;
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        if (lane == 0)
#pragma unroll
            for (int s = 0; s < S; ++s) buf[s * kWarps + warp] = a[s];
        __syncthreads();
#pragma unroll
        for (int s = 0; s < S; ++s) {
            float v = lane < kWarps ? buf[s * kWarps + lane] : 0.f;
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
            a[s] = v;
        }
    }
}

// One row in registers: element (k, i) of a thread is column (k R + lane) V + i.
template <typename T, int V, int K, int R>
struct Row {
    static constexpr int kThreads = R < 128 ? 128 : R;
    static constexpr int kRows = kThreads / R;  // rows of a block
};

// Mean and reciprocal deviation; x becomes xhat.  Columns behind D hold 0.
template <int V, int K, int R>
__device__ __forceinline__ void normalise(float (&x)[K][V], int lane, int D, float eps, bool rms, float *buf,
                                          float &r) {
    const float inv = 1.f / (float)D;
    if (!rms) {
        float s[1] = {0.f};
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int i = 0; i < V; ++i) s[0] += x[k][i];
        row_sum<R>(s, buf);
        const float m = s[0] * inv;
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int i = 0; i < V; ++i) x[k][i] = (k * R + lane) * V + i < D ? x[k][i] - m : 0.f;
    }
    float q[1] = {0.f};
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
        for (int i = 0; i < V; ++i) q[0] = fmaf(x[k][i], x[k][i], q[0]);
    row_sum<R>(q, buf + 2 * (R / 32 + 1));
    r = 1.f / sqrtf(fmaf(q[0], inv, eps));
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
        for (int i = 0; i < V; ++i) x[k][i] *= r;
}

template <typename T, int V, int K, int R>
__global__ void __launch_bounds__(Row<T, V, K, R>::kThreads) norm_fwd(NormParams p) {
    __shared__ float buf[4 * (R / 32 + 1)];
    const int lane = threadIdx.x % R;
    const long long row = (long long)blockIdx.x * Row<T, V, K, R>::kRows + threadIdx.x / R;
    const bool in = row < p.rows;
    const T *x = static_cast<const T *>(p.x) + row * p.D;
    const T *z = p.z ? static_cast<const T *>(p.z) + row * p.D : nullptr;
    T *y = static_cast<T *>(p.y) + row * p.D;
    float a[K][V];
    Vec<T, V> gate[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int c = (k * R + lane) * V;
        Vec<T, V> l;
        zero(l);
        zero(gate[k]);
        if (in && c < p.D) {
            l.load(x + c);
            if (z) gate[k].load(z + c);
        }
#pragma unroll
        for (int i = 0; i < V; ++i) a[k][i] = l.v[i];
    }
    float r;
    normalise<V, K, R>(a, lane, p.D, p.eps, p.rms, buf, r);
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int c = (k * R + lane) * V;
        if (!in || c >= p.D) continue;
        Vec<float, V> w, b;
        if (p.weight) w.load(p.weight + c);
        if (p.bias) b.load(p.bias + c);
        Vec<T, V> out;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            float n = p.weight ? a[k][i] * w.v[i] : a[k][i];
            if (p.bias) n += b.v[i];
            out.v[i] = z ? n * silu_f(gate[k].v[i]) : n;
        }
        out.store(y + c);
    }
}

template <typename T, int V, int K, int R>
__global__ void __launch_bounds__(Row<T, V, K, R>::kThreads) norm_bwd(NormParams p) {
    constexpr int kRows = Row<T, V, K, R>::kRows;
    __shared__ float buf[8 * (R / 32 + 1)];
    const int lane = threadIdx.x % R;
    const int sub = threadIdx.x / R;
    const float inv = 1.f / (float)p.D;
    float sw[K][V], sb[K][V];
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
        for (int i = 0; i < V; ++i) sw[k][i] = sb[k][i] = 0.f;
    for (long long first = (long long)blockIdx.x * kRows; first < p.rows; first += (long long)gridDim.x * kRows) {
        const long long row = first + sub;
        const bool in = row < p.rows;
        const T *x = static_cast<const T *>(p.x) + row * p.D;
        const T *dy = static_cast<const T *>(p.dy) + row * p.D;
        const T *z = p.z ? static_cast<const T *>(p.z) + row * p.D : nullptr;
        float a[K][V];
        Vec<T, V> grad[K], gate[K];
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int c = (k * R + lane) * V;
            Vec<T, V> l;
            zero(l);
            zero(grad[k]);
            zero(gate[k]);
            if (in && c < p.D) {
                l.load(x + c);
                grad[k].load(dy + c);
                if (z) gate[k].load(z + c);
            }
#pragma unroll
            for (int i = 0; i < V; ++i) a[k][i] = l.v[i];
        }
        float r;
        normalise<V, K, R>(a, lane, p.D, p.eps, p.rms, buf, r);
        float s[2] = {0.f, 0.f};  // sums of d xhat and of d
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int c = (k * R + lane) * V;
            if (!in || c >= p.D) continue;
            Vec<float, V> w;
            if (p.weight) w.load(p.weight + c);
            if (z) {
                Vec<float, V> b;
                if (p.bias) b.load(p.bias + c);
                Vec<T, V> out;
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    float n = p.weight ? a[k][i] * w.v[i] : a[k][i];
                    if (p.bias) n += b.v[i];
                    const float u = gate[k].v[i], g = sigmoid_f(u);
                    out.v[i] = grad[k].v[i] * n * (g * fmaf(u, 1.f - g, 1.f));
                    grad[k].v[i] *= u * g;
                }
                out.store(static_cast<T *>(p.dz) + row * p.D + c);
            }
#pragma unroll
            for (int i = 0; i < V; ++i) {
                sw[k][i] = fmaf(grad[k].v[i], a[k][i], sw[k][i]);
                sb[k][i] += grad[k].v[i];
                if (p.weight) grad[k].v[i] *= w.v[i];
                s[0] = fmaf(grad[k].v[i], a[k][i], s[0]);
                s[1] += grad[k].v[i];
            }
        }
        row_sum<R>(s, buf + 4 * (R / 32 + 1));
        const float c1 = s[0] * inv, c2 = p.rms ? 0.f : s[1] * inv;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int c = (k * R + lane) * V;
            if (!in || c >= p.D) continue;
            Vec<T, V> out;
#pragma unroll
            for (int i = 0; i < V; ++i) out.v[i] = r * (grad[k].v[i] - c2 - a[k][i] * c1);
            out.store(static_cast<T *>(p.dx) + row * p.D + c);
        }
    }
    if (!p.partial) return;
    float *part = p.partial + (long long)blockIdx.x * 2 * p.D;
    if constexpr (kRows == 1) {
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int c = (k * R + lane) * V + i;
                if (c < p.D) {
                    part[c] = sw[k][i];
                    part[p.D + c] = sb[k][i];
                }
            }
    } else {
        __shared__ float red[kRows][R];
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int i = 0; i < V; ++i)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    __syncthreads();
                    red[sub][lane] = h ? sb[k][i] : sw[k][i];
                    __syncthreads();
                    const int c = (k * R + lane) * V + i;
                    if (sub == 0 && c < p.D) {
                        float v = 0.f;
#pragma unroll
                        for (int q = 0; q < kRows; ++q) v += red[q][lane];
                        part[(long long)h * p.D + c] = v;
                    }
                }
    }
}

// dweight and dbias from the blocks' rows: 32 columns and 8 slices of the rows per block.
__global__ void __launch_bounds__(256) norm_bwd_sums(NormParams p, int blocks) {
    __shared__ float red[8][32];
    const int c = blockIdx.x * 32 + threadIdx.x;
    const int h = blockIdx.y;
    float a = 0.f;
    if (c < p.D)
        for (int b = threadIdx.y; b < blocks; b += 8) a += p.partial[((long long)b * 2 + h) * p.D + c];
    red[threadIdx.y][threadIdx.x] = a;
    __syncthreads();
    float *out = h ? p.dbias : p.dweight;
    if (threadIdx.y == 0 && c < p.D && out) {
        float v = 0.f;
#pragma unroll
        for (int q = 0; q < 8; ++q) v += red[q][threadIdx.x];
        out[c] = v;
    }
}

// Blocks of the backward: enough to fill the GPU, no more than there are rows
// for them.  From the sizes alone, since every block has a row of workspace.
int norm_bwd_blocks(long long rows, int per_block) {
    const long long most = (rows + per_block - 1) / per_block;
    const long long fill = kSms * 4;
    return (int)(most < fill ? most : fill);
}

template <typename T, int V, int K, int R>
cudaError_t norm_launch(const NormParams &p, bool bwd, cudaStream_t stream, int *blocks) {
    constexpr int kRows = Row<T, V, K, R>::kRows, kThreads = Row<T, V, K, R>::kThreads;
    if (blocks) {  // the size of the backward's grid only
        *blocks = norm_bwd_blocks(p.rows, kRows);
        return cudaSuccess;
    }
    if (!bwd) {
        const long long grid = (p.rows + kRows - 1) / kRows;
        if (grid > 0x7fffffffLL) return cudaErrorInvalidValue;
        norm_fwd<T, V, K, R><<<(unsigned)grid, kThreads, 0, stream>>>(p);
    } else {
        const int grid = norm_bwd_blocks(p.rows, kRows);
        if (grid > 0) norm_bwd<T, V, K, R><<<grid, kThreads, 0, stream>>>(p);
        if (p.partial) norm_bwd_sums<<<dim3((p.D + 31) / 32, 2), dim3(32, 8), 0, stream>>>(p, grid);
    }
    return cudaGetLastError();
}

// Threads and vectors of a row by its length in vectors: as few threads as
// hold it in at most 4 vectors of 16 bytes each.
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
        if (n <= 256) return norm_launch<T, V, 2, 128>(p, bwd, stream, blocks);
        if (n <= 512) return norm_launch<T, V, 2, 256>(p, bwd, stream, blocks);
        if (n <= 1024) return norm_launch<T, V, 2, 512>(p, bwd, stream, blocks);
        return norm_launch<T, V, 16 / V * 2, 512>(p, bwd, stream, blocks);
    }
    // rows that do not begin on 16 bytes: single elements
    if (p.D <= 32) return norm_launch<T, 1, 1, 32>(p, bwd, stream, blocks);
    if (p.D <= 128) return norm_launch<T, 1, 4, 32>(p, bwd, stream, blocks);
    if (p.D <= 512) return norm_launch<T, 1, 4, 128>(p, bwd, stream, blocks);
    if (p.D <= 2048) return norm_launch<T, 1, 8, 256>(p, bwd, stream, blocks);
    if (p.D <= 8192) return norm_launch<T, 1, 16, 512>(p, bwd, stream, blocks);
    return norm_launch<T, 1, 32, 512>(p, bwd, stream, blocks);
}

}  // namespace

cudaError_t norm_fwd_launch(const NormParams &p, bool bf16, cudaStream_t stream, const char **name) {
    *name = bf16 ? "norm_fwd<bf16>" : "norm_fwd<f32>";
    return bf16 ? norm_dispatch<__nv_bfloat16>(p, false, stream, nullptr) : norm_dispatch<float>(p, false, stream, nullptr);
}

cudaError_t norm_bwd_launch(const NormParams &p, bool bf16, cudaStream_t stream, const char **name) {
    *name = bf16 ? "norm_bwd<bf16>" : "norm_bwd<f32>";
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
