// The ring cache of keys and values, and attention of one new token of every
// sequence over it.
//
//     o = sum_j p_j v_j,  p = softmax(scale q . k_j)  over the sinks, the window's
//     tokens in the cache, and the new token itself
//
// The positions that are seen are walked as one list: the sinks, then the window
// (consecutive slots of the ring, wrapping once), then the new token, whose key and value
// are read from the call's own arguments.  The slot that the new token goes to held the
// position `ring` before it, which is outside the window (ring >= window): no block reads it.
#include "dn_window.cuh"

namespace dn {
namespace {

// The list of positions that the token at position `had` sees, without itself.
struct Seen {
    int sinks, n;          // sinks in the cache; all that are seen
    int first, ring, base; // ring slot of the window's first token; base: the ring's first slot
    __device__ __forceinline__ Seen(long long had, const CacheParams &p) {
        base = p.sinks;
        ring = p.ring;
        sinks = had < p.sinks ? (int)had : p.sinks;
        long long lo = had - p.window + 1;
        if (lo < p.sinks) lo = p.sinks;
        const long long w = had - lo;
        n = sinks + (w > 0 ? (int)w : 0);
        first = w > 0 ? (int)((lo - p.sinks) % p.ring) : 0;
    }
    __device__ __forceinline__ int slot(int i) const {
        if (i < sinks) return i;
        const int r = first + i - sinks;
        return base + (r < ring ? r : r - ring);
    }
};

__device__ __forceinline__ int slot_of(long long pos, const CacheParams &p) {
    return pos < p.sinks ? (int)pos : p.sinks + (int)((pos - p.sinks) % p.ring);
}

template <typename T, int D>
__global__ void __launch_bounds__(128) step_simple(CacheParams p) {
    constexpr int E = D / 32;
    const int h = blockIdx.x % p.Nq, n = blockIdx.x / p.Nq;
    const int G = p.Nq / p.Nk, hk = h / G;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const long long had = p.lengths[n];
    if (had < 0) {
        if (threadIdx.x == 0) atomicOr(p.status, kStatusBadSeq);
        return;
    }
    const long long cache = ((long long)n * p.Nk + hk) * (p.sinks + p.ring);
    const T *kc = static_cast<const T *>(p.kc) + cache * D, *vc = static_cast<const T *>(p.vc) + cache * D;
    const T *kn = static_cast<const T *>(p.k) + ((long long)n * p.Nk + hk) * D;
    const T *vn = static_cast<const T *>(p.v) + ((long long)n * p.Nk + hk) * D;
    const Seen seen(had, p);
    const float c = p.scale * kLog2e;
    Vec<T, E> q;
    q.load(static_cast<const T *>(p.q) + ((long long)n * p.Nq + h) * D + lane * E);
    float m = -CUDART_INF_F, l = 0.f, acc[E];
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = 0.f;
    for (int i = warp; i <= seen.n; i += 4) {
        const long long at = i < seen.n ? (long long)seen.slot(i) * D : 0;
        Vec<T, E> k, v;
        k.load((i < seen.n ? kc + at : kn) + lane * E);
        v.load((i < seen.n ? vc + at : vn) + lane * E);
        float s = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) s = fmaf(q.v[e], k.v[e], s);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        s *= c;
        const float top = fmaxf(m, s), base = top == -CUDART_INF_F ? 0.f : top;
        const float f = ex2(m - base), w = ex2(s - base);
        m = top;
        l = l * f + w;
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] = acc[e] * f + w * v.v[e];
    }
    __shared__ float sm[4], sl[4], so[4][D];
    if (lane == 0) sm[warp] = m, sl[warp] = l;
#pragma unroll
    for (int e = 0; e < E; ++e) so[warp][lane * E + e] = acc[e];
    __syncthreads();
    if (threadIdx.x < D) {
        float top = fmaxf(fmaxf(sm[0], sm[1]), fmaxf(sm[2], sm[3]));
        top = top == -CUDART_INF_F ? 0.f : top;
        float sum = 0.f, o = 0.f;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            const float f = ex2(sm[w] - top);
            sum += sl[w] * f;
            o += so[w][threadIdx.x] * f;
        }
        Vec<T, 1> y;
        y.v[0] = o / sum;
        y.store(static_cast<T *>(p.o) + ((long long)n * p.Nq + h) * D + threadIdx.x);
    }
    if (h % G == 0) {
        const long long at = (cache + slot_of(had, p)) * D;
        for (int i = threadIdx.x; i < D; i += 128) {
            static_cast<T *>(p.kc)[at + i] = kn[i];
            static_cast<T *>(p.vc)[at + i] = vn[i];
        }
    }
}

// Tokens of the prompts into the caches: a tile of 32 tokens of one sequence per block,
// 16 bytes a thread at a time.
constexpr int kFillTile = 32;

template <typename T, int D>
__global__ void __launch_bounds__(256) fill(CacheParams p, long long slots) {
    constexpr int V = 16 / sizeof(T), C = D / V;
    if (blockIdx.x == 0) check_offsets(p.seq, threadIdx.x, 256);
    for (long long b = blockIdx.x; b < slots; b += gridDim.x) {
        const SeqTile s = seq_tile(p.seq, (unsigned)b, kFillTile);
        if (!s.ok || s.t0 >= s.t1) continue;
        const long long had = p.lengths ? p.lengths[s.n] : 0;
        if (had < 0) {
            if (threadIdx.x == 0) atomicOr(p.status, kStatusBadSeq);
            continue;
        }
        const long long end = had + (s.eos - s.bos);
        const int per = p.Nk * C, n = (int)(s.t1 - s.t0) * per;
        for (int i = threadIdx.x; i < n; i += 256) {
            const long long t = s.t0 + i / per;
            const int h = i % per / C, c = i % C * V;
            const long long pos = had + t - s.bos;
            if (pos >= p.sinks && pos < end - p.ring) continue;
            const long long from = (t * p.Nk + h) * D + c;
            const long long to = (((long long)s.n * p.Nk + h) * (p.sinks + p.ring) + slot_of(pos, p)) * D + c;
            Pack<T, V> k, v;
            k.load(static_cast<const T *>(p.k) + from);
            v.load(static_cast<const T *>(p.v) + from);
            k.store(static_cast<T *>(p.kc) + to);
            v.store(static_cast<T *>(p.vc) + to);
        }
    }
}

}  // namespace

cudaError_t window_fill_launch(const CacheParams &p, bool bf16, cudaStream_t stream, const char **name) {
    *name = bf16 ? "window_fill<bf16>" : "window_fill<f32>";
    const long long slots = tile_slots(p.seq, kFillTile);
    const unsigned grid = (unsigned)(slots < 65536 ? slots : 65536);
    if (grid == 0) return cudaSuccess;
    if (bf16 && p.d == 64) fill<__nv_bfloat16, 64><<<grid, 256, 0, stream>>>(p, slots);
    else if (bf16) fill<__nv_bfloat16, 128><<<grid, 256, 0, stream>>>(p, slots);
    else if (p.d == 64) fill<float, 64><<<grid, 256, 0, stream>>>(p, slots);
    else fill<float, 128><<<grid, 256, 0, stream>>>(p, slots);
    return cudaGetLastError();
}

cudaError_t window_step_launch(const CacheParams &p, bool bf16, cudaStream_t stream, const char **name) {
    *name = bf16 ? "window_step<bf16>" : "window_step<f32>";
    const unsigned grid = (unsigned)p.N * p.Nq;
    if (grid == 0) return cudaSuccess;
    if (bf16 && p.d == 64) step_simple<__nv_bfloat16, 64><<<grid, 128, 0, stream>>>(p);
    else if (bf16) step_simple<__nv_bfloat16, 128><<<grid, 128, 0, stream>>>(p);
    else if (p.d == 64) step_simple<float, 64><<<grid, 128, 0, stream>>>(p);
    else step_simple<float, 128><<<grid, 128, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace dn
