// The norms around a block in one pass: what both directions share.
//
//     p = norm(x) w1 + b1   (or x w1 + b1),   f = scale sigmoid(z),   h = residual + f p
//     y = norm(h) w2 + b2
#pragma once

#include "dn_norm.cuh"

namespace dn {

// A row on threads that it fills exactly (FULL: D = R K V, as most widths do) needs no checks of columns;
// one row a block at a time none of rows.  N: rows that a thread works on at a time.
template <typename T, int V, int K, int R, bool FULL, int N = 1>
struct BlockRow : Row<T, V, K, R> {
    using B = Row<T, V, K, R>;
    static __device__ __forceinline__ bool in(int k, int i, int D) { return FULL || B::in(k, i, D); }
    static __device__ __forceinline__ bool live(long long row, long long rows) { return (B::kRows == 1 && N == 1) || row < rows; }
    // v in the columns that exist, 0 elsewhere
    static __device__ __forceinline__ f2 inside(int k, float v, int D) {
        return FULL ? both(v) : pair(in(k, 0, D) ? v : 0.f, in(k, 1, D) ? v : 0.f);
    }
};

// The vectors of A tensors of T and of B tensors of TR that a thread works on, of N rows at a time, S
// rows ahead in all, in shared memory by asynchronous copies.  Rows that do not begin on 16
// bytes, and those too long for a stage to fit, are loaded where they are used.  Tensors that are
// null are zeros.
template <typename T, typename TR, int V, int K, int R, bool FULL, int N, int A, int B, int REGS>
struct BlockRing {
    using L = BlockRow<T, V, K, R, FULL, N>;
    static constexpr int kRes = (int)sizeof(TR) * V;  // bytes of a vector of TR: 16 or 32
    static constexpr int kOne = K * L::kThreads;      // vectors of one tensor
    static constexpr int kStage = kOne * (A * 16 + B * kRes);
    // as many stages, up to 4, as leave room for the blocks that an SM's registers hold
    static constexpr int kBlocks = 65536 / (REGS * L::kThreads) < 1 ? 1 : 65536 / (REGS * L::kThreads);
    static constexpr int kRoom = 226 * 1024 / kBlocks - 2048;
    static constexpr bool kAhead = L::kWhole && N * kStage <= kRoom;
    static constexpr int kFit = kRoom / kStage / N * N;
    static constexpr int S = !kAhead || kFit < N ? N : kFit > 4 ? 4 : kFit;
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
        if constexpr (kAhead) asm volatile("cp.async.wait_group %0;" ::"n"(S - N) : "memory");
    }
    // vector k of tensor i as pairs; zeros where the row or the column does not exist
    __device__ __forceinline__ void get_a(f2 (&v)[L::P], const char *ring, int s, int i, int k, long long row, long long rows,
                                          int D) const {
        if constexpr (L::kWhole) {
            Pack<T, V> r;
            r.clear();
            if (a[i] && L::live(row, rows) && L::in(k, 0, D))
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
            const bool here = b[i] && L::live(row, rows) && L::in(k, 0, D);
#pragma unroll
            for (int q = 0; q < kRes / 16; ++q) {
                const TR *src = kAhead ? reinterpret_cast<const TR *>(ring + s * kStage + A * kOne * 16 +
                                                                      ((i * (kRes / 16) + q) * kOne + k * L::kThreads + threadIdx.x) * 16)
                                       : b[i] + row * D + L::col(k, 0) + q * W;
                if constexpr (sizeof(TR) == 4) {
                    ulonglong2 r = make_ulonglong2(0ull, 0ull);
                    if (here) r = *reinterpret_cast<const ulonglong2 *>(src);
                    v[2 * q] = r.x;
                    v[2 * q + 1] = r.y;
                } else {
                    Pack<TR, W> r;
                    r.clear();
                    if (here) r.load(src);
#pragma unroll
                    for (int e = 0; e < W / 2; ++e) v[q * (W / 2) + e] = pair(r[2 * e], r[2 * e + 1]);
                }
            }
        } else {
            v[0] = load_elements<L>(b[i] + row * D, k, b[i] && row < rows ? D : 0);
        }
    }
};

// Sums of S = 1, 2 or 4 values over the R threads of a row; every one of them gets them.  The values share the
// shuffles, each on its part of a warp (one after the other the sums were a third of the backward's
// instructions).  R > 32: `buf` has S R / 32 floats, and consecutive sums use buffers of their own in turn.
template <int R, int S>
__device__ __forceinline__ void sum_row(float (&a)[S], float *buf) {
    static_assert(R == 32 || R % 128 == 0, "a row on a warp, or one row per block");
    constexpr int kPart = 32 / S, W = R / 32;  // lanes of a value; warps
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = lane % kPart, which = lane / kPart;
    float t;
    auto add = [&](float mine, float theirs, int x) { return mine + __shfl_xor_sync(0xffffffffu, theirs, x); };
    if constexpr (S == 4) {
        const bool low = lane < 16, even = !(lane & 8);
        const float u = add(low ? a[0] : a[2], low ? a[2] : a[0], 16), v = add(low ? a[1] : a[3], low ? a[3] : a[1], 16);
        t = add(even ? u : v, even ? v : u, 8);
    } else if constexpr (S == 2) {
        t = add(lane < 16 ? a[0] : a[1], lane < 16 ? a[1] : a[0], 16);
    } else {
        t = add(a[0], a[0], 16);
    }
#pragma unroll
    for (int x = S == 1 ? 8 : kPart / 2; x > 0; x >>= 1) t = add(t, t, x);
    if constexpr (R > 32) {
        if (sub == 0) buf[which * W + warp] = t;
        __syncthreads();
        if constexpr (W <= kPart) {
            t = buf[which * W + sub % W];
#pragma unroll
            for (int x = W / 2; x > 0; x >>= 1) t = add(t, t, x);
        } else {
            t = buf[which * W + sub];
#pragma unroll
            for (int i = kPart; i < W; i += kPart) t += buf[which * W + sub + i];
#pragma unroll
            for (int x = kPart / 2; x > 0; x >>= 1) t = add(t, t, x);
        }
    }
    if constexpr (S == 1) {
        a[0] = t;
    } else {
#pragma unroll
        for (int i = 0; i < S; ++i) a[i] = __shfl_sync(0xffffffffu, t, i * kPart);
    }
}

// Means m (0 for the root-mean-square form) and reciprocal deviations r of N rows; columns behind D hold 0.
// buf: 2 N R / 32 floats.
template <typename L, int V, int K, int R, int N>
__device__ __forceinline__ void row_stats(const f2 (&x)[N][K][V / 2], bool rms, float eps, float inv, int D, float *buf, float (&m)[N],
                                          float (&r)[N]) {
    constexpr int P = V / 2;
    float s[N];
#pragma unroll
    for (int n = 0; n < N; ++n) m[n] = 0.f;
    if (!rms) {
#pragma unroll
        for (int n = 0; n < N; ++n) {
            f2 t = 0ull;
#pragma unroll
            for (int k = 0; k < K; ++k)
#pragma unroll
                for (int i = 0; i < P; ++i) t = add2(t, x[n][k][i]);
            s[n] = sum_of(t);
        }
        sum_row<R>(s, buf);
#pragma unroll
        for (int n = 0; n < N; ++n) m[n] = s[n] * inv;
    }
#pragma unroll
    for (int n = 0; n < N; ++n) {
        f2 t = 0ull;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const f2 mm = L::inside(k, -m[n], D);
#pragma unroll
            for (int i = 0; i < P; ++i) {
                const f2 d = add2(x[n][k][i], mm);
                t = fma2(d, d, t);
            }
        }
        s[n] = sum_of(t);
    }
    sum_row<R>(s, buf + N * (R / 32));
#pragma unroll
    for (int n = 0; n < N; ++n) r[n] = rsqrtf(fmaf(s[n], inv, eps));
}

// Vector k of one of the fp32 vectors; 0 where the column does not exist.
template <typename L, int V>
__device__ __forceinline__ void load_given(f2 (&t)[V / 2], const float *w, int k, int D) {
    if constexpr (L::kWhole) {
#pragma unroll
        for (int i = 0; i < V / 4; ++i) {
            ulonglong2 r = make_ulonglong2(0ull, 0ull);
            if (L::in(k, 0, D)) r = reinterpret_cast<const ulonglong2 *>(w + L::col(k, 0))[i];
            t[2 * i] = r.x;
            t[2 * i + 1] = r.y;
        }
    } else {
        t[0] = pair(L::in(k, 0, D) ? w[L::col(k, 0)] : 0.f, L::in(k, 1, D) ? w[L::col(k, 1)] : 0.f);
    }
}

// One of the fp32 vectors, where it is given.  KEEP: its values stay in registers for all rows; else they
// are loaded where they are used (which few warps cannot hide).
template <typename L, int V, int K, bool KEEP>
struct Kept {
    static constexpr int P = V / 2;
    const float *src;
    f2 v[KEEP ? K : 1][KEEP ? P : 1];
    __device__ __forceinline__ void init(const float *from, int D) {
        src = from;
        if constexpr (KEEP)
            if (from)
#pragma unroll
                for (int k = 0; k < K; ++k) load_given<L, V>(v[k], from, k, D);
    }
    __device__ __forceinline__ void times(f2 (&x)[P], int k, int D) const {
        if (!src) return;
        f2 t[P];
        get(t, k, D);
#pragma unroll
        for (int i = 0; i < P; ++i) x[i] = mul2(x[i], t[i]);
    }
    __device__ __forceinline__ void plus(f2 (&x)[P], int k, int D) const {
        if (!src) return;
        f2 t[P];
        get(t, k, D);
#pragma unroll
        for (int i = 0; i < P; ++i) x[i] = add2(x[i], t[i]);
    }

private:
    __device__ __forceinline__ void get(f2 (&t)[P], int k, int D) const {
        if constexpr (KEEP) {
#pragma unroll
            for (int i = 0; i < P; ++i) t[i] = v[k][i];
        } else {
            load_given<L, V>(t, src, k, D);
        }
    }
};

// The product of two of the fp32 vectors, either of which may be absent (one).
template <typename L, int V, int K, bool KEEP>
struct Scaled {
    static constexpr int P = V / 2;
    const float *a, *b;
    f2 v[KEEP ? K : 1][KEEP ? P : 1];
    __device__ __forceinline__ void init(const float *x, const float *y, int D) {
        a = x;
        b = y;
        if constexpr (KEEP)
#pragma unroll
            for (int k = 0; k < K; ++k) load(v[k], k, D);
    }
    __device__ __forceinline__ void times(f2 (&x)[P], int k, int D) const {
        f2 t[P];
        get(t, k, D);
#pragma unroll
        for (int i = 0; i < P; ++i) x[i] = mul2(x[i], t[i]);
    }
    __device__ __forceinline__ void plus(f2 (&x)[P], int k, int D) const {
        f2 t[P];
        get(t, k, D);
#pragma unroll
        for (int i = 0; i < P; ++i) x[i] = add2(x[i], t[i]);
    }

private:
    __device__ __forceinline__ void load(f2 (&t)[P], int k, int D) const {
#pragma unroll
        for (int i = 0; i < P; ++i) t[i] = both(1.f);
        if (a) load_given<L, V>(t, a, k, D);
        if (b) {
            f2 u[P];
            load_given<L, V>(u, b, k, D);
#pragma unroll
            for (int i = 0; i < P; ++i) t[i] = mul2(t[i], u[i]);
        }
    }
    __device__ __forceinline__ void get(f2 (&t)[P], int k, int D) const {
        if constexpr (KEEP) {
#pragma unroll
            for (int i = 0; i < P; ++i) t[i] = v[k][i];
        } else {
            load(t, k, D);
        }
    }
};

constexpr int kBlockMaxCols = 16384;

// Threads and vectors of a row: E elements a thread where that fills at least a block of 128.  F is given the
// types and sizes; it is called for widths from MIN to MAX, and only what these reach is compiled.
template <typename T, typename TR, int E, int MIN = 1, int MAX = 1 << 30, typename F>
cudaError_t block_dispatch(int D, F &&f) {
    constexpr int V = 16 / sizeof(T), K = E / V;
    // a row of `w` columns, and the rows of up to `w` behind those of up to `below`
#define DN_BLOCK_FULL(w, R) \
    if constexpr (w >= MIN && w <= MAX)  \
        if (D == w) return f.template operator()<T, TR, V, K, R, true>();
#define DN_BLOCK_UP_TO(w, below, V, K, R) \
    if constexpr (w >= MIN && below < MAX) \
        if (D <= w) return f.template operator()<T, TR, V, K, R, false>();
    if (D % V == 0) {
        DN_BLOCK_FULL(128 * E, 128)
        DN_BLOCK_FULL(256 * E, 256)
        DN_BLOCK_FULL(512 * E, 512)
        DN_BLOCK_UP_TO(32 * E, 0, V, K, 32)
        DN_BLOCK_UP_TO(128 * E, 32 * E, V, K, 128)
        DN_BLOCK_UP_TO(256 * E, 128 * E, V, K, 256)
        DN_BLOCK_UP_TO(512 * E, 256 * E, V, K, 512)
        DN_BLOCK_UP_TO(kBlockMaxCols, 512 * E, V, 16 / V, 1024)
    } else {
        DN_BLOCK_UP_TO(128, 0, 2, 2, 32)
        DN_BLOCK_UP_TO(512, 128, 2, 2, 128)
        DN_BLOCK_UP_TO(2048, 512, 2, 4, 256)
        DN_BLOCK_UP_TO(8192, 2048, 2, 8, 512)
        DN_BLOCK_UP_TO(kBlockMaxCols, 8192, 2, 8, 1024)
    }
#undef DN_BLOCK_FULL
#undef DN_BLOCK_UP_TO
    return cudaErrorInvalidValue;
}

// Registers that a thread may have, and with it the blocks of a grid: in the backward from the sizes
// alone, since every block has a row of workspace.
constexpr int kBlockFwdRegs = 64;
// (blocks of 128 threads: three an SM, with more rows in flight each, not four)
constexpr int block_bwd_regs(int threads) { return threads <= 128 ? 168 : threads <= 512 ? 128 : 65536 / threads; }

// The backward, of one type each; the grid's size alone where `blocks` is not null.
cudaError_t block_bwd_f32(const BlockParams &p, bool bias, cudaStream_t stream, int *blocks);
cudaError_t block_bwd_bf16(const BlockParams &p, bool bias, cudaStream_t stream, int *blocks);
cudaError_t block_bwd_bf16_f32(const BlockParams &p, bool bias, cudaStream_t stream, int *blocks);
cudaError_t block_bwd_sums_launch(const BlockParams &p, int blocks, int planes, cudaStream_t stream);

}  // namespace dn
