// Device helpers of the operators around the recurrence: loads and stores of
// V consecutive elements, the tiles of packed sequences, silu.
#pragma once

#include <cuda_bf16.h>

#include <atomic>

#include "dn_layer.h"

namespace dn {

// Launch of a kernel that works on what the launch before it in the stream wrote.  It may
// be set up while that one still runs; the kernel itself calls wait_for_launches() before
// it touches anything.
template <typename... P, typename... A>
inline cudaError_t launch_after(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream, A... args) {
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, P(args)...);
}
__device__ __forceinline__ void wait_for_launches() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Lets a kernel have `bytes` of dynamic shared memory beside a few KB of its own: nothing
// to do up to 32 KB (48 KB in all need no leave), else
// once for every device (the attribute stays).
template <auto kKernel>
inline cudaError_t allow_smem(int bytes) {
    static std::atomic<unsigned long long> done{0};
    if (bytes <= 32 * 1024) return cudaSuccess;
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess) return err;
    const unsigned long long bit = dev < 64 ? 1ull << dev : 0;
    if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
    err = cudaFuncSetAttribute(kKernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (err == cudaSuccess) err = cudaFuncSetAttribute(kKernel, cudaFuncAttributePreferredSharedMemoryCarveout, 100);
    if (err == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
    return err;
}

// Lets a kernel be launched in clusters of more than 8 blocks, once for every device.
template <auto kKernel>
inline cudaError_t allow_wide_cluster() {
    static std::atomic<unsigned long long> done{0};
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess) return err;
    const unsigned long long bit = dev < 64 ? 1ull << dev : 0;
    if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
    err = cudaFuncSetAttribute(kKernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (err == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
    return err;
}

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
        } else if constexpr (V == 2) {
            const float2 r = *reinterpret_cast<const float2 *>(p);
            v[0] = r.x; v[1] = r.y;
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
        } else if constexpr (V == 2) {
            *reinterpret_cast<float2 *>(p) = make_float2(v[0], v[1]);
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

// The same V elements as they lie in memory: what a load in flight holds (half
// the registers of Vec for bf16).
template <typename T, int V>
struct Pack {
    static constexpr int kWords = V * (int)sizeof(T) / 4 > 0 ? V * (int)sizeof(T) / 4 : 1;
    unsigned w[kWords];
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int i = 0; i < kWords; ++i) w[i] = 0u;
    }
    __device__ __forceinline__ void load(const T *p) {
        if constexpr (sizeof(T) * V == 2) {
            w[0] = *reinterpret_cast<const unsigned short *>(p);
        } else if constexpr (kWords == 1) {
            w[0] = *reinterpret_cast<const unsigned *>(p);
        } else if constexpr (kWords == 2) {
            const uint2 r = *reinterpret_cast<const uint2 *>(p);
            w[0] = r.x; w[1] = r.y;
        } else {
#pragma unroll
            for (int i = 0; i < kWords; i += 4) {
                const uint4 r = reinterpret_cast<const uint4 *>(p)[i / 4];
                w[i] = r.x; w[i + 1] = r.y; w[i + 2] = r.z; w[i + 3] = r.w;
            }
        }
    }
    __device__ __forceinline__ void store(T *p) const {
        if constexpr (sizeof(T) * V == 2) {
            *reinterpret_cast<unsigned short *>(p) = (unsigned short)w[0];
        } else if constexpr (kWords == 1) {
            *reinterpret_cast<unsigned *>(p) = w[0];
        } else if constexpr (kWords == 2) {
            *reinterpret_cast<uint2 *>(p) = make_uint2(w[0], w[1]);
        } else {
#pragma unroll
            for (int i = 0; i < kWords; i += 4)
                reinterpret_cast<uint4 *>(p)[i / 4] = make_uint4(w[i], w[i + 1], w[i + 2], w[i + 3]);
        }
    }
    __device__ __forceinline__ float operator[](int i) const {
        if constexpr (sizeof(T) == 4) return __uint_as_float(w[i]);
        else return __uint_as_float(i & 1 ? w[i >> 1] & 0xffff0000u : w[i >> 1] << 16);
    }
};

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

__device__ __forceinline__ SeqTile seq_tile(const SeqView &s, unsigned slot, int len) {
    SeqTile r;
    if (!s.cu) {
        const unsigned per = s.T > 0 ? ((unsigned)s.T + len - 1) / len : 1;
        const unsigned n = slot / per;
        r.n = (int)n;
        r.c = (int)(slot - n * per);
        r.bos = (long long)r.n * s.T;
        r.eos = r.bos + s.T;
        r.ok = n < (unsigned)s.N;
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
        const long long c = (long long)slot - (r.bos / len + lo);
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

constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float rcp(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// 1 / (1 + e^-u), from the two approximate instructions (each within two units
// of fp32's last place; the exponent's rounding adds |u| 2^-24 of the value).
// Below u = -87.3 it is 0, and so is silu, whose value there is above -1.2e-36.
__device__ __forceinline__ float sigmoid_f(float u) { return rcp(1.f + ex2(-kLog2e * u)); }
__device__ __forceinline__ float silu_f(float u) { return u * sigmoid_f(u); }
// d silu(u) / du = s (1 + u (1 - s)), s = sigmoid(u)
__device__ __forceinline__ float silu_grad_f(float u) {
    const float s = sigmoid_f(u);
    return s * fmaf(u, 1.f - s, 1.f);
}

// Two fp32 values in one register pair, and the instructions that work on both
// (beside memory, the number of instructions is what most of these kernels pay for).
typedef unsigned long long f2;
__device__ __forceinline__ f2 pair(float lo, float hi) {
    f2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void split(f2 v, float &lo, float &hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ f2 both(float x) { return pair(x, x); }
__device__ __forceinline__ float sum_of(f2 v) {
    float lo, hi;
    split(v, lo, hi);
    return lo + hi;
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
    f2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
    f2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f2 add2(f2 a, f2 b) {
    f2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

}  // namespace dn
