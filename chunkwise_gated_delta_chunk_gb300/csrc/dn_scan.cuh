// What the selective scan's kernels share: how channels and states lie on
// threads, the tiles of tokens in shared memory, and the sums over lanes.
//
// Every thread holds 4 of a channel's N states, so a channel takes
// L = N / 4 neighbouring lanes and a warp 32 / L channels.  A block works on
// channels of one group (they read the same rows of Bm and Cm).
#pragma once

#include "dn_layer.cuh"

namespace dn {
namespace scan {

constexpr int kS = 4;  // states of a thread

// log(1 + e^v) without loss on either side: for v << 0 it is e^v.
__device__ __forceinline__ float softplus(float v) { return fmaxf(v, 0.f) + log1pf(expf(-fabsf(v))); }

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

// Four neighbouring channels of one token as fp32; absent ones are 0.
// VEC: rows and tiles begin on a multiple of four elements.
template <typename T, bool VEC>
__device__ __forceinline__ void load4(const void *base, long long row, int D, int d, int n, bool in, float (&v)[4]) {
    v[0] = v[1] = v[2] = v[3] = 0.f;
    if (!in || n <= 0) return;
    const T *src = static_cast<const T *>(base) + row * D + d;
    if constexpr (VEC) {
        Vec<T, 4> a;
        a.load(src);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = a.v[i];
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i < n) {
                Vec<T, 1> a;
                a.load(src + i);
                v[i] = a.v[0];
            }
    }
}

template <typename T, bool VEC>
__device__ __forceinline__ void store4(void *base, long long row, int D, int d, int n, bool in, const float (&v)[4]) {
    if (!in || n <= 0) return;
    T *dst = static_cast<T *>(base) + row * D + d;
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

// Steps the states over the chunks of every sequence: hs[c] becomes the state at
// the start of chunk c; bwd: gs[c] also becomes the gradient of the state at the
// end of chunk c, and dh0 that of h0.
cudaError_t scan_combine_launch(const ScanParams &p, bool bwd, cudaStream_t stream);

}  // namespace dn
