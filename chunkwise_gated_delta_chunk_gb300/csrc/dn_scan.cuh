// What the selective scan's kernels share: softplus, the channels of a block
// (all of one group: they read the same rows of Bm and Cm), loads of rows, and
// the sums over lanes.
#pragma once

#include "dn_layer.cuh"

namespace dn {
namespace scan {

constexpr int kS = 4;  // states in one access: those of a thread in the backward and the single-token kernel

// log(1 + e^v) = max(v, 0) + log(1 + e^-|v|) without loss on either side (for v << 0
// it is e^v).  With q = e^-|v| in (0, 1], log(1 + q) = 2 atanh(s), s = q / (2 + q) in
// (0, 1/3]: the series s + s^3 / 3 + ... to s^13 / 13, whose rest is below s^15 / 15 /
// (1 - s^2) = 5.3e-9, 1.5e-8 of the sum.  The exponential's argument is split in two
// so that its rounding does not grow with |v|.
__device__ __forceinline__ float softplus(float v) {
    const float u = fmaxf(-fabsf(v), -104.f), m = u * kLog2e;  // below, q is 0 beside 1
    const float rest = fmaf(u, kLog2e, -m) + u * 1.9259629911e-8f;  // u log2(e) - m
    const float e = ex2(m);
    const float q = fmaf(e * 0.6931471806f, rest, e);
    const float s = q * rcp(2.f + q), w = s * s;
    float r = fmaf(w, 1.f / 13.f, 1.f / 11.f);
    r = fmaf(r, w, 1.f / 9.f);
    r = fmaf(r, w, 1.f / 7.f);
    r = fmaf(r, w, 1.f / 5.f);
    r = fmaf(r, w, 1.f / 3.f);
    r = fmaf(r * w, s, s);
    return v != v ? v : fmaxf(v, 0.f) + (r + r);
}

// softplus of both halves: the same steps, most of them on pairs.
__device__ __forceinline__ f2 softplus2(f2 v) {
    float v0, v1;
    split(v, v0, v1);
    const f2 u = pair(fmaxf(-fabsf(v0), -104.f), fmaxf(-fabsf(v1), -104.f));
    const f2 m = mul2(u, both(kLog2e));
    const f2 rest = fma2(u, both(1.9259629911e-8f), fma2(u, both(kLog2e), mul2(u, both(-kLog2e))));
    float m0, m1, d0, d1;
    split(m, m0, m1);
    const f2 e = pair(ex2(m0), ex2(m1));
    const f2 q = fma2(mul2(e, both(0.6931471806f)), rest, e);
    split(add2(q, both(2.f)), d0, d1);
    const f2 s = mul2(q, pair(rcp(d0), rcp(d1))), w = mul2(s, s);
    f2 r = fma2(w, both(1.f / 13.f), both(1.f / 11.f));
    r = fma2(r, w, both(1.f / 9.f));
    r = fma2(r, w, both(1.f / 7.f));
    r = fma2(r, w, both(1.f / 5.f));
    r = fma2(r, w, both(1.f / 3.f));
    r = fma2(mul2(r, w), s, s);
    r = fma2(r, both(2.f), pair(fmaxf(v0, 0.f), fmaxf(v1, 0.f)));
    float r0, r1;
    split(r, r0, r1);
    return pair(v0 != v0 ? v0 : r0, v1 != v1 ? v1 : r1);
}

// A in units of log2; an infinite one becomes the largest finite one, so that a
// token without a step (delta = 0) keeps the state.
__device__ __forceinline__ float log2_rate(float A) {
    const float v = A * kLog2e;
    return isinf(v) ? copysignf(3.402823466e38f, v) : v;
}

// Channels of a block: tile `ct` of the groups' tiles, CH channels each.
struct Channels {
    int g, d0, n;  // group, first channel, channels (<= CH)
};
template <int CH>
__device__ __forceinline__ Channels channels_of(const ScanParams &p, int ct) {
    const int dg = p.D / p.G;
    const int per = (dg + CH - 1) / CH;
    Channels r;
    r.g = ct / per;
    const int o = (ct - r.g * per) * CH;
    r.d0 = r.g * dg + o;
    r.n = dg - o < CH ? dg - o : CH;
    return r;
}
template <int CH>
inline int channel_tiles(int D, int G) {
    return G * ((D / G + CH - 1) / CH);
}

// Four neighbouring channels of one token as they lie in memory; absent ones are 0.
// VEC: rows and tiles begin on a multiple of four elements.  (Else they stay apart until
// they are used: joining them would wait for their loads.)
template <typename T, bool VEC>
struct Four {
    Pack<T, VEC ? 4 : 1> p[VEC ? 1 : 4];
    __device__ __forceinline__ void load(const void *base, long long row, int D, int d, int n, bool in) {
#pragma unroll
        for (int i = 0; i < (VEC ? 1 : 4); ++i) {
            p[i].clear();
            if (in && i < n) p[i].load(static_cast<const T *>(base) + row * D + d + i);
        }
    }
    __device__ __forceinline__ float operator[](int i) const { return VEC ? p[0][VEC ? i : 0] : p[VEC ? 0 : i][0]; }
};

template <typename T, bool VEC>
__device__ __forceinline__ void store4(T *dst, int n, const float (&v)[4]) {
    if constexpr (VEC) {
        Vec<T, 4> a;
#pragma unroll
        for (int i = 0; i < 4; ++i) a.v[i] = v[i];
        a.store(dst);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i < n) {
                Vec<T, 1> a;
                a.v[0] = v[i];
                a.store(dst + i);
            }
    }
}

// What a thread reads of each tile, fetched S tiles ahead: K vectors of four
// elements by asynchronous copies into its own part of shared memory (a thread
// reads only what it copied itself: no barrier).
template <typename T, int K, int NT, int S>
struct Ahead {
    static constexpr int kB = 4 * (int)sizeof(T);
    static constexpr int kBytes = S * K * NT * kB;
    static __device__ __forceinline__ int at(int s, int k) { return ((s * K + k) * NT + (int)threadIdx.x) * kB; }
    // vector k of the tile in stage s
    __device__ __forceinline__ void issue(char *ring, int s, int k, const T *src, bool in) {
        if (!in) return;
        const unsigned dst = (unsigned)__cvta_generic_to_shared(ring) + at(s, k);
        if constexpr (kB == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
        else asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
    }
    __device__ __forceinline__ void commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
    // Waits for the oldest of the S tiles in flight.
    __device__ __forceinline__ void wait() { asm volatile("cp.async.wait_group %0;" ::"n"(S - 1) : "memory"); }
    // A vector that was not issued holds anything.
    __device__ __forceinline__ Pack<T, 4> get(const char *ring, int s, int k) const {
        Pack<T, 4> r;
        r.load(reinterpret_cast<const T *>(ring + at(s, k)));
        return r;
    }
};

// Sum over the lanes that differ in bit `bit` of R values each, the lower half
// of the values staying with the lane whose bit is 0: R / 2 shuffles.
template <int R>
__device__ __forceinline__ void fold(float (&v)[R], int bit, bool upper) {
#pragma unroll
    for (int i = 0; i < R / 2; ++i) {
        const float give = upper ? v[i] : v[i + R / 2];
        const float keep = upper ? v[i + R / 2] : v[i];
        v[i] = keep + __shfl_xor_sync(0xffffffffu, give, bit);
    }
}

// Of four values per lane, the sums over a channel's L lanes: lane l of the
// channel ends with value l & 3.
template <int L>
__device__ __forceinline__ float sum4(float (&v)[4], int lane) {
    // bit 1 picks the upper pair, bit 0 the odd one of it
    fold<4>(v, 2, lane & 2);
    float w[2] = {v[0], v[1]};
    fold<2>(w, 1, lane & 1);
    float s = w[0];
#pragma unroll
    for (int bit = 4; bit < L; bit <<= 1) s += __shfl_xor_sync(0xffffffffu, s, bit);
    return s;
}

}  // namespace scan

// The shortest chunk worth its part in the walk over a sequence's chunks: a token of a
// chunk takes about 0.3 us in each of two kernels, a chunk 0.1 us in that walk, so that
// the sum is least near 0.4 sqrt(tokens).
inline int scan_least_chunk(long long tokens) {
    int len = 16;
    while (6LL * len * len < tokens) len += 16;
    return len;
}

// Steps the states over the chunks of every sequence: hs[c] becomes the state at
// the start of chunk c; bwd: gs[c] also becomes the gradient of the state at the
// end of chunk c, and dh0 that of h0.
cudaError_t scan_combine_launch(const ScanParams &p, bool bwd, cudaStream_t stream);

}  // namespace dn
