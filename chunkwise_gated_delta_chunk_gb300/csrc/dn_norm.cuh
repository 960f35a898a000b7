// Rows of a norm on threads: where a row's vectors lie, its sums, its deviations over
// their root mean square.
#pragma once

#include "dn_layer.cuh"

namespace dn {

// Sum over the R threads of a row; every one of them gets it.  R > 32: `buf`
// has S R / 32 floats, and consecutive sums use buffers of their own in turn.
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
        for (int s = 0; s < S; ++s) {  // every thread adds all of them: shorter than shuffles
            float4 v = reinterpret_cast<const float4 *>(buf)[s * kWarps / 4];
#pragma unroll
            for (int w = 1; w < kWarps / 4; ++w) {
                const float4 o = reinterpret_cast<const float4 *>(buf)[s * kWarps / 4 + w];
                v.x += o.x; v.y += o.y; v.z += o.z; v.w += o.w;
            }
            a[s] = (v.x + v.y) + (v.z + v.w);
        }
    }
}

// How a row lies on threads: vector k of a thread is V neighbouring columns from
// (k R + lane) V on.  Rows that do not begin on 16 bytes are taken element by element
// (V = 2): there vector k is columns 2 k R + lane and (2 k + 1) R + lane.
template <typename T, int V, int K, int R>
struct Row {
    static_assert(R <= 32 || R % 128 == 0, "rows within a warp, or one row per block with sums of four warps' vectors");
    static constexpr int kThreads = R < 128 ? 128 : R;
    static constexpr int kRows = kThreads / R;  // rows of a block
    static constexpr int P = V / 2;             // pairs of a vector
    static constexpr bool kWhole = sizeof(T) * V == 16;
    typedef f2 Pairs[K][P];
    static __device__ __forceinline__ int col(int k, int i) {
        const int lane = threadIdx.x % R;
        return kWhole ? (k * R + lane) * V + i : (k * V + i) * R + lane;
    }
    // Whether element i of vector k exists (a whole vector does or does not).
    static __device__ __forceinline__ bool in(int k, int i, int D) { return col(k, kWhole ? 0 : i) < D; }
};

// Vector k of a row taken element by element, as one pair; zeros where it does not exist.
template <typename L, typename T>
__device__ __forceinline__ f2 load_elements(const T *src, int k, int D) {
    Vec<T, 1> a, b;
    a.v[0] = b.v[0] = 0.f;
    if (L::in(k, 0, D)) a.load(src + L::col(k, 0));
    if (L::in(k, 1, D)) b.load(src + L::col(k, 1));
    return pair(a.v[0], b.v[0]);
}
// Vector k of one of the fp32 vectors as pairs; `other` where it does not exist.
template <typename L, int V>
__device__ __forceinline__ void load_vec(f2 (&v)[V / 2], const float *src, int k, int D, float other) {
    if constexpr (L::kWhole) {
        Vec<float, V> r;
#pragma unroll
        for (int i = 0; i < V; ++i) r.v[i] = other;
        if (src && L::in(k, 0, D)) r.load(src + L::col(k, 0));
#pragma unroll
        for (int i = 0; i < V / 2; ++i) v[i] = pair(r.v[2 * i], r.v[2 * i + 1]);
    } else {
        v[0] = pair(src && L::in(k, 0, D) ? src[L::col(k, 0)] : other, src && L::in(k, 1, D) ? src[L::col(k, 1)] : other);
    }
}
template <typename L, int V, typename T>
__device__ __forceinline__ void store_row(T *dst, const f2 (&v)[V / 2], int k, int D) {
    Vec<T, L::kWhole ? V : 1> out;
    if constexpr (L::kWhole) {
#pragma unroll
        for (int i = 0; i < V / 2; ++i) split(v[i], out.v[2 * i], out.v[2 * i + 1]);
        if (L::in(k, 0, D)) out.store(dst + L::col(k, 0));
    } else {
        float lo, hi;
        split(v[0], lo, hi);
        out.v[0] = lo;
        if (L::in(k, 0, D)) out.store(dst + L::col(k, 0));
        out.v[0] = hi;
        if (L::in(k, 1, D)) out.store(dst + L::col(k, 1));
    }
}

// What the rows are normed with.
struct Norm {
    int D;
    float eps;
    bool rms;
};

// x becomes xhat; returns the reciprocal deviation.  Columns behind D hold 0.
template <typename L, int V, int K, int R>
__device__ __forceinline__ float normalise(f2 (&x)[K][V / 2], const Norm &p, float inv, float *buf) {
    constexpr int P = V / 2;
    if (!p.rms) {
        f2 t = 0ull;
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int i = 0; i < P; ++i) t = add2(t, x[k][i]);
        float s[1] = {sum_of(t)};
        row_sum<R>(s, buf);
        const float m = -s[0] * inv;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const f2 mm = pair(L::in(k, 0, p.D) ? m : 0.f, L::in(k, 1, p.D) ? m : 0.f);
#pragma unroll
            for (int i = 0; i < P; ++i) x[k][i] = add2(x[k][i], mm);
        }
    }
    f2 t = 0ull;
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
        for (int i = 0; i < P; ++i) t = fma2(x[k][i], x[k][i], t);
    float q[1] = {sum_of(t)};
    row_sum<R>(q, buf + R / 32);
    const float r = rsqrtf(fmaf(q[0], inv, p.eps));
    const f2 rr = both(r);
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
        for (int i = 0; i < P; ++i) x[k][i] = mul2(x[k][i], rr);
    return r;
}

// sigmoid of both halves
__device__ __forceinline__ f2 sigmoid2(f2 u) {
    float a, b;
    split(u, a, b);
    return pair(sigmoid_f(a), sigmoid_f(b));
}

// Blocks that walk the rows: as many as the GPU holds at once, no more than there are
// rows for them.  From the sizes alone, since every block of the backward has a row of
// workspace; all of them walk the same number of rows, or one less.
inline int norm_blocks(long long rows, int threads, int per_block, int regs) {
    const long long most = (rows + per_block - 1) / per_block;
    const long long fill = (long long)kSms * (65536 / (regs * threads) > 0 ? 65536 / (regs * threads) : 1);
    if (most <= fill) return (int)most;
    const long long each = (most + fill - 1) / fill;
    return (int)((most + each - 1) / each);
}

}  // namespace dn
