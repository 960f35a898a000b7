// Device helpers of the operators around the recurrence: loads and stores of
// V consecutive elements, the tiles of packed sequences, silu.
#pragma once

#include <cuda_bf16.h>

#include "dn_layer.h"

namespace dn {

// V consecutive elements of T in one access (V = 1, or a power of two whose
// bytes are the pointer's alignment), as fp32.
template <typename T, int V>
struct Vec;

template <int V>
struct Vec<float, V> {
    float v[V];
    __device__ __forceinline__ void load(const float *p) {
        if constexpr (V == 1) {
            v[0] = *p;
        } else {
#pragma unroll
            for (int i = 0; i < V; i += 4) {
                const float4 r = *reinterpret_cast<const float4 *>(p + i);
                v[i] = r.x; v[i + 1] = r.y; v[i + 2] = r.z; v[i + 3] = r.w;
            }
        }
    }
    __device__ __forceinline__ void store(float *p) const {
        if constexpr (V == 1) {
            *p = v[0];
        } else {
#pragma unroll
            for (int i = 0; i < V; i += 4)
                *reinterpret_cast<float4 *>(p + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
        }
    }
};

template <int V>
struct Vec<__nv_bfloat16, V> {
    float v[V];
    static __device__ __forceinline__ void unpack(unsigned u, float &lo, float &hi) {
        lo = __uint_as_float(u << 16);
        hi = __uint_as_float(u & 0xffff0000u);
    }
    static __device__ __forceinline__ unsigned pack(float lo, float hi) {
        const __nv_bfloat162 r = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const unsigned *>(&r);
    }
    __device__ __forceinline__ void load(const __nv_bfloat16 *p) {
        if constexpr (V == 1) {
            v[0] = __bfloat162float(*p);
        } else if constexpr (V == 2) {
            unpack(*reinterpret_cast<const unsigned *>(p), v[0], v[1]);
        } else if constexpr (V == 4) {
            const uint2 r = *reinterpret_cast<const uint2 *>(p);
            unpack(r.x, v[0], v[1]);
            unpack(r.y, v[2], v[3]);
        } else {
#pragma unroll
            for (int i = 0; i < V; i += 8) {
                const uint4 r = *reinterpret_cast<const uint4 *>(p + i);
                unpack(r.x, v[i], v[i + 1]);
                unpack(r.y, v[i + 2], v[i + 3]);
                unpack(r.z, v[i + 4], v[i + 5]);
                unpack(r.w, v[i + 6], v[i + 7]);
            }
        }
    }
    __device__ __forceinline__ void store(__nv_bfloat16 *p) const {
        if constexpr (V == 1) {
            *p = __float2bfloat16_rn(v[0]);
        } else if constexpr (V == 2) {
            *reinterpret_cast<unsigned *>(p) = pack(v[0], v[1]);
        } else if constexpr (V == 4) {
            *reinterpret_cast<uint2 *>(p) = make_uint2(pack(v[0], v[1]), pack(v[2], v[3]));
        } else {
#pragma unroll
            for (int i = 0; i < V; i += 8)
                *reinterpret_cast<uint4 *>(p + i) = make_uint4(pack(v[i], v[i + 1]), pack(v[i + 2], v[i + 3]),
                                                               pack(v[i + 4], v[i + 5]), pack(v[i + 6], v[i + 7]));
        }
    }
};

template <typename T, int V>
__device__ __forceinline__ void zero(Vec<T, V> &a) {
#pragma unroll
    for (int i = 0; i < V; ++i) a.v[i] = 0.f;
}

// One tile of a sequence (see tile_slots).  `ok` is false where the slot holds
// none; every access a tile leads to is inside the tensors whatever the
// offsets hold.
struct SeqTile {
    int n;               // sequence
    int c;               // tile of the sequence
    long long bos, eos;  // the sequence's tokens
    long long t0, t1;    // the tile's tokens
    bool ok;
};

__device__ __forceinline__ SeqTile seq_tile(const SeqView &s, long long slot, int len) {
    SeqTile r;
    if (!s.cu) {
        const long long per = s.T > 0 ? ((long long)s.T + len - 1) / len : 1;
        r.n = (int)(slot / per);
        r.c = (int)(slot - r.n * per);
        r.bos = (long long)r.n * s.T;
        r.eos = r.bos + s.T;
        r.ok = r.n < s.N;
    } else {
        int lo = 0, hi = s.N - 1;  // the last sequence whose first slot is not behind this one
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (s.cu[mid] / len + mid <= slot) lo = mid;
            else hi = mid - 1;
        }
        r.n = lo;
        r.bos = s.cu[lo];
        r.eos = s.cu[lo + 1];
        r.ok = r.bos >= 0 && r.eos >= r.bos && r.eos <= s.tokens;
        const long long c = slot - (r.bos / len + lo);
        r.ok = r.ok && c >= 0 && (c == 0 || r.bos + c * len < r.eos);
        r.c = r.ok ? (int)c : 0;
    }
    r.t0 = r.bos + (long long)r.c * len;
    r.t1 = r.t0 + len < r.eos ? r.t0 + len : r.eos;
    return r;
}

// A whole sequence as one tile.
__device__ __forceinline__ SeqTile seq_whole(const SeqView &s, int n) {
    SeqTile r;
    r.n = n;
    r.c = 0;
    r.bos = s.cu ? s.cu[n] : (long long)n * s.T;
    r.eos = s.cu ? s.cu[n + 1] : r.bos + s.T;
    r.ok = r.bos >= 0 && r.eos >= r.bos && r.eos <= s.tokens;
    r.t0 = r.bos;
    r.t1 = r.eos;
    return r;
}

// The offsets' own check, by the threads of one block: a bad value anywhere
// goes to the status word.
__device__ __forceinline__ void check_offsets(const SeqView &s, int thread, int threads) {
    if (!s.cu) return;
    bool bad = thread == 0 && s.cu[0] != 0;
    for (int i = thread; i < s.N; i += threads) bad |= s.cu[i + 1] < s.cu[i] || s.cu[i + 1] > s.tokens;
    if (bad) atomicOr(s.status, kStatusBadSeq);
}

// 1 / (1 + e^-u): __expf and __fdividef are within a few units of fp32's last
// place here, far below the rounding of a bf16 result.
__device__ __forceinline__ float sigmoid_f(float u) { return __fdividef(1.f, 1.f + __expf(-u)); }
__device__ __forceinline__ float silu_f(float u) { return __fdividef(u, 1.f + __expf(-u)); }
// d silu(u) / du = s (1 + u (1 - s)), s = sigmoid(u)
__device__ __forceinline__ float silu_grad_f(float u) {
    const float s = sigmoid_f(u);
    return s * fmaf(u, 1.f - s, 1.f);
}

}  // namespace dn
