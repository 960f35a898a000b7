// The norms around a block in one pass: what both directions share.
//
//     p = norm(x) w1 + b1   (or x w1 + b1),   f = scale sigmoid(z),   h = residual + f p
//     y = norm(h) w2 + b2
#pragma once

#include "dn_norm.cuh"

namespace dn {

// The vectors of A tensors of T and of B tensors of TR that a thread works on, S
// iterations ahead, in shared memory by asynchronous copies.  Rows that do not begin on 16
// bytes, and those too long for a stage to fit, are loaded where they are used.  Tensors that are
// null are zeros.
template <typename T, typename TR, int V, int K, int R, int A, int B, int REGS>
struct BlockRing {
    using L = Row<T, V, K, R>;
    static constexpr int kRes = (int)sizeof(TR) * V;  // bytes of a vector of TR: 16 or 32
    static constexpr int kOne = K * L::kThreads;      // vectors of one tensor
    static constexpr int kStage = kOne * (A * 16 + B * kRes);
    // as many stages, up to 4, as leave room for the blocks that an SM's registers hold
    static constexpr int kBlocks = 65536 / (REGS * L::kThreads) < 1 ? 1 : 65536 / (REGS * L::kThreads);
    static constexpr int kRoom = 226 * 1024 / kBlocks - 2048;
    static constexpr bool kAhead = L::kWhole && kStage <= kRoom;
    static constexpr int kFit = kRoom / kStage;
    static constexpr int S = !kAhead || kFit < 1 ? 1 : kFit > 4 ? 4 : kFit;
    static constexpr int kBytes = kAhead ? S * kStage : 0;
    const T *a[A];
    const TR *b[B];
    static __device__ __forceinline__ void copy16(unsigned dst, const void *src) {
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
    }
    __device__ __forceinline__ void issue(char *ring, int s, long long row, long long rows, int D) {
        if constexpr (kAhead) {
            const unsigned base = (unsigned)__cvta_generic_to_shared(ring) + s * kStage;
#pragma unroll
            for (int k = 0; k < K; ++k) {
                if (row >= rows || !L::in(k, 0, D)) continue;
                const long long at = row * D + L::col(k, 0);
                const unsigned me = k * L::kThreads + threadIdx.x;
#pragma unroll
                for (int i = 0; i < A; ++i)
                    if (a[i]) copy16(base + (i * kOne + me) * 16, a[i] + at);
#pragma unroll
                for (int i = 0; i < B; ++i)
                    if (b[i])
#pragma unroll
                        for (int q = 0; q < kRes / 16; ++q)  // 16-byte parts apart from each other: no bank conflicts
                            copy16(base + A * kOne * 16 + ((i * (kRes / 16) + q) * kOne + me) * 16,
                                   reinterpret_cast<const char *>(b[i] + at) + 16 * q);
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        }
    }
    __device__ __forceinline__ void wait() {
        if constexpr (kAhead) asm volatile("cp.async.wait_group %0;" ::"n"(S - 1) : "memory");
    }
    // vector k of tensor i as pairs; zeros where the row or the column does not exist
    __device__ __forceinline__ void get_a(f2 (&v)[L::P], const char *ring, int s, int i, int k, long long row, long long rows,
                                          int D) const {
        if constexpr (L::kWhole) {
            Pack<T, V> r;
            r.clear();
            if (a[i] && row < rows && L::in(k, 0, D))
                r.load(kAhead ? reinterpret_cast<const T *>(ring + s * kStage + (i * kOne + k * L::kThreads + threadIdx.x) * 16)
                              : a[i] + row * D + L::col(k, 0));
#pragma unroll
            for (int q = 0; q < L::P; ++q) v[q] = pair(r[2 * q], r[2 * q + 1]);
        } else {
            v[0] = load_elements<L>(a[i] + row * D, k, a[i] && row < rows ? D : 0);
        }
    }
    __device__ __forceinline__ void get_b(f2 (&v)[L::P], const char *ring, int s, int i, int k, long long row, long long rows,
                                          int D) const {
        if constexpr (L::kWhole) {
            constexpr int W = 16 / sizeof(TR);  // elements of 16 bytes
            const bool here = b[i] && row < rows && L::in(k, 0, D);
#pragma unroll
            for (int q = 0; q < kRes / 16; ++q) {
                Pack<TR, W> r;
                r.clear();
                if (here)
                    r.load(kAhead ? reinterpret_cast<const TR *>(ring + s * kStage + A * kOne * 16 +
                                                                 ((i * (kRes / 16) + q) * kOne + k * L::kThreads + threadIdx.x) * 16)
                                  : b[i] + row * D + L::col(k, 0) + q * W);
#pragma unroll
                for (int e = 0; e < W / 2; ++e) v[q * (W / 2) + e] = pair(r[2 * e], r[2 * e + 1]);
            }
        } else {
            v[0] = load_elements<L>(b[i] + row * D, k, b[i] && row < rows ? D : 0);
        }
    }
};

// One of the fp32 vectors: of a single vector a thread the values stay in registers for all rows
// (loaded for every row they cost more time than memory does: 8192 rows of 2048 in the backward
// 148 us), else they are loaded where they are used.
template <typename L, int V, int K>
struct Kept {
    static constexpr int P = V / 2;
    static constexpr bool kKeep = K == 1;
    const float *src;
    f2 v[kKeep ? P : 1];
    __device__ __forceinline__ void init(const float *from, int D, float other) {
        src = from;
        if constexpr (kKeep) load_vec<L, V>(v, from, 0, D, other);
    }
    __device__ __forceinline__ void times(f2 (&x)[P], int k, int D) const {
        if (!src) return;
        f2 t[P];
        get(t, k, D, 1.f);
#pragma unroll
        for (int i = 0; i < P; ++i) x[i] = mul2(x[i], t[i]);
    }
    __device__ __forceinline__ void plus(f2 (&x)[P], int k, int D) const {
        if (!src) return;
        f2 t[P];
        get(t, k, D, 0.f);
#pragma unroll
        for (int i = 0; i < P; ++i) x[i] = add2(x[i], t[i]);
    }

private:
    __device__ __forceinline__ void get(f2 (&t)[P], int k, int D, float other) const {
        if constexpr (kKeep) {
#pragma unroll
            for (int i = 0; i < P; ++i) t[i] = v[i];
        } else {
            load_vec<L, V>(t, src, k, D, other);
        }
    }
};

// w v + b of one vector, where given.
template <typename L, int V>
__device__ __forceinline__ void affine(f2 (&v)[V / 2], const float *w, const float *b, int k, int D) {
    f2 t[V / 2];
    if (w) {
        load_vec<L, V>(t, w, k, D, 1.f);
#pragma unroll
        for (int i = 0; i < V / 2; ++i) v[i] = mul2(v[i], t[i]);
    }
    if (b) {
        load_vec<L, V>(t, b, k, D, 0.f);
#pragma unroll
        for (int i = 0; i < V / 2; ++i) v[i] = add2(v[i], t[i]);
    }
}

// Threads and vectors of a row: about one vector of 16 bytes a thread up to 512 of them, then
// more.  F is given the types and sizes.
template <typename T, typename TR, typename F>
cudaError_t block_dispatch(int D, F &&f) {
    constexpr int V = 16 / sizeof(T);
    if (D % V == 0) {
        const int n = D / V;  // at most 4096 (fp32)
        if (n <= 32) return f.template operator()<T, TR, V, 1, 32>();
        if (n <= 128) return f.template operator()<T, TR, V, 1, 128>();
        if (n <= 256) return f.template operator()<T, TR, V, 1, 256>();
        if (n <= 512) return f.template operator()<T, TR, V, 1, 512>();
        if (n <= 1024) return f.template operator()<T, TR, V, 2, 512>();
        return f.template operator()<T, TR, V, 16 / V, 1024>();
    }
    if (D <= 128) return f.template operator()<T, TR, 2, 2, 32>();
    if (D <= 512) return f.template operator()<T, TR, 2, 2, 128>();
    if (D <= 2048) return f.template operator()<T, TR, 2, 4, 256>();
    if (D <= 8192) return f.template operator()<T, TR, 2, 8, 512>();
    return f.template operator()<T, TR, 2, 8, 1024>();
}

template <typename F>
cudaError_t block_types(const BlockParams &p, F &&f) {
    if (!p.bf16) return block_dispatch<float, float>(p.D, f);
    return p.res_f32 ? block_dispatch<__nv_bfloat16, float>(p.D, f) : block_dispatch<__nv_bfloat16, __nv_bfloat16>(p.D, f);
}

// Registers that a thread of the backward may have, and with it the blocks of its grid: from the
// sizes alone, since every block has a row of workspace.
template <int kThreads>
constexpr int block_bwd_regs() { return kThreads <= 512 ? 128 : 65536 / kThreads; }
constexpr int kBlockFwdRegs = 64;

}  // namespace dn
