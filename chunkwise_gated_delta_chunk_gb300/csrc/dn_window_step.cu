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
//
// A warp takes 16 positions at a time, with a running maximum and sum of its own; the warps of a
// block, and the blocks of a cluster that share a sequence where there are few of them, join
// these at the end through shared memory.  Every position on the list is seen, so there is
// nothing to mask but the end of the list.
#include <type_traits>

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

constexpr int kWarps = 4;   // of a block
constexpr int kKeys = 16;   // positions that a warp takes at a time

__device__ __forceinline__ unsigned smem_at(const void *p) { return (unsigned)__cvta_generic_to_shared(p); }
// 16 bytes into shared memory; zeros where not `in`
__device__ __forceinline__ void copy16(unsigned dst, const void *src, bool in) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(in ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ unsigned cluster_rank() {
    unsigned r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ float remote(const float *p, unsigned rank) {  // the same place in another block of the cluster
    unsigned at;
    float v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_at(p)), "r"(rank));
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(at) : "memory");
    return v;
}

// One block's sequence, key head and rows of queries.
template <typename T, int D>
struct Job {
    int n, hk, row0, rows;  // query heads hk G + row0 + 0..rows-1
    long long had;
    const T *kc, *vc, *kn, *vn;
    bool ok;
    __device__ __forceinline__ Job(const CacheParams &p, unsigned block, int tile) {
        const int G = p.Nq / p.Nk, tiles = (G + tile - 1) / tile;
        row0 = block % tiles * tile;
        rows = G - row0 < tile ? G - row0 : tile;
        hk = block / tiles % p.Nk;
        n = block / tiles / p.Nk;
        had = p.lengths[n];
        const long long cache = ((long long)n * p.Nk + hk) * (p.sinks + p.ring) * D, one = ((long long)n * p.Nk + hk) * D;
        kc = static_cast<const T *>(p.kc) + cache;
        vc = static_cast<const T *>(p.vc) + cache;
        kn = static_cast<const T *>(p.k) + one;
        vn = static_cast<const T *>(p.v) + one;
        ok = had >= 0;
        if (!ok) {
            if (threadIdx.x == 0) atomicOr(p.status, kStatusBadSeq);
            had = 0;
        }
    }
    __device__ __forceinline__ long long query(const CacheParams &p, int r) const {
        return ((long long)n * p.Nq + hk * (p.Nq / p.Nk) + row0 + r) * D;
    }
    // rows i of the list: key and value, and whether there is such a row
    __device__ __forceinline__ bool row(const Seen &seen, int i, const T *&k, const T *&v) const {
        const long long at = i < seen.n ? (long long)seen.slot(i) * D : 0;
        k = i < seen.n ? kc + at : kn;
        v = i < seen.n ? vc + at : vn;
        return i <= seen.n;
    }
    // the new token's own slot (see above: no block of this launch reads it)
    __device__ __forceinline__ void keep(const CacheParams &p) const {
        constexpr int V = 16 / sizeof(T);
        const long long at = (long long)slot_of(had, p) * D;
        for (int i = threadIdx.x * V; i < 2 * D; i += 32 * kWarps * V) {
            Pack<T, V> x;
            x.load(i < D ? kn + i : vn + i - D);
            x.store(const_cast<T *>(i < D ? kc + at + i : vc + at + i - D));
        }
    }
};

// Joins what the warps of a cluster's blocks found: for every row a maximum m (of scores times
// log2 e), the sum l of the weights and the weighted values o, all in shared memory.  First within the block,
// then every block adds up its share of the columns over all blocks, in their order.
template <typename T, int D, int ROWS>
__device__ __forceinline__ void join(const CacheParams &p, const Job<T, D> &job, const float *o, int stride, float (&m)[kWarps][ROWS],
                                     float (&l)[kWarps][ROWS], float *sum, float (&top)[ROWS], float (&all)[ROWS], unsigned blocks) {
    constexpr int NT = 32 * kWarps;
    auto best = [&](int r) { return fmaxf(fmaxf(m[0][r], m[1][r]), fmaxf(m[2][r], m[3][r])); };
    __syncthreads();
    for (int i = threadIdx.x; i < job.rows * D; i += NT) {
        const int r = i / D;
        const float t = best(r), base = t == -CUDART_INF_F ? 0.f : t;
        float a = 0.f, s = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float f = ex2(m[w][r] - base);
            a = fmaf(f, o[w * stride + i], a);
            s = fmaf(f, l[w][r], s);
        }
        sum[i] = a;
        if (i % D == 0) {
            top[r] = t;
            all[r] = s;
        }
    }
    if (blocks > 1) cluster_sync();
    else __syncthreads();
    const unsigned rank = blocks > 1 ? cluster_rank() : 0;
    auto add_up = [&](auto count) {  // all blocks' numbers are asked for at once
        constexpr int N = decltype(count)::value;
        for (int i = rank * NT + threadIdx.x; i < job.rows * D; i += NT * N) {
            const int r = i / D;
            float a, s;
            if constexpr (N > 1) {
                float ms[N], os[N], ls[N], t = -CUDART_INF_F;
#pragma unroll
                for (int b = 0; b < N; ++b) {
                    ms[b] = remote(&top[r], b);
                    os[b] = remote(sum + i, b);
                    ls[b] = remote(&all[r], b);
                }
#pragma unroll
                for (int b = 0; b < N; ++b) t = fmaxf(t, ms[b]);
                const float base = t == -CUDART_INF_F ? 0.f : t;
                a = s = 0.f;
#pragma unroll
                for (int b = 0; b < N; ++b) {
                    const float f = ex2(ms[b] - base);
                    a = fmaf(f, os[b], a);
                    s = fmaf(f, ls[b], s);
                }
            } else {
                a = sum[i];
                s = all[r];
            }
            Vec<T, 1> y;
            y.v[0] = a / s;
            y.store(static_cast<T *>(p.o) + job.query(p, 0) + i);
        }
    };
    if (job.ok) {
        if (blocks == 1) add_up(std::integral_constant<int, 1>());
        else if (blocks == 2) add_up(std::integral_constant<int, 2>());
        else if (blocks == 4) add_up(std::integral_constant<int, 4>());
        else if (blocks == 8) add_up(std::integral_constant<int, 8>());
        else add_up(std::integral_constant<int, 16>());
    }
    if (blocks > 1) cluster_sync();  // a block's shared memory stays until the others have read it
}

// ---- bf16 -------------------------------------------------------------------

__device__ __forceinline__ void ldmatrix4(unsigned (&r)[4], unsigned at) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];" : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at) : "memory");
}
__device__ __forceinline__ void ldmatrix4t(unsigned (&r)[4], unsigned at) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(at)
                 : "memory");
}
__device__ __forceinline__ void mma16816(float (&c)[4], const unsigned (&a)[4], unsigned b0, unsigned b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ unsigned transposed(unsigned x) {  // an 8 x 8 matrix of 16 bits, a pair of a row a lane
    unsigned y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

template <int D, int ROWS>
struct StepSmem {
    static constexpr int kStage = 2 * kKeys * D * 2;  // keys and values
    static constexpr int kStages = 3;
    static constexpr int kWarp = kStages * kStage;
    static constexpr int kPart = ROWS * D * 4;  // a warp's o, over its stages
    static_assert(kPart <= kWarp, "a warp's sums lie over its stages");
    static constexpr int kBytes = kWarps * kWarp + kPart;
};

extern __shared__ __align__(128) char s_step[];

// Tensor-core form (mma.sync): keys and values are the operands with 16 rows, the query heads of a key
// head the one with 8 columns, twice where there are more than 8 (the other way round, 8 heads fill
// half of 16 rows, and the products alone took as long as memory):
//     S^T = K q^T,   O^T += V^T P^T,   P^T from S^T by two 8 x 8 transpositions.
// The weights are rounded to bf16 for the second product, by half a step of each; their sum takes them unrounded.
// The reference that weights are relative to moves up only when a score exceeds it by 2^8, so that a
// group of positions needs no reduction but a vote.  Bound by memory: three stages of asynchronous copies a
// warp keep the positions' 2 x 16 x d values coming; no warp waits for another before the end.
template <int D, int ROWS>
__global__ void __launch_bounds__(32 * kWarps, 2) step_bf16(const __grid_constant__ CacheParams p, unsigned blocks) {
    using T = __nv_bfloat16;
    using S = StepSmem<D, ROWS>;
    constexpr int C = D / 8, NK = D / 16, NT = ROWS / 8, PER = C / 2;  // 16-byte chunks of a row; steps of 16 columns; tiles of heads; rows that a lane copies
    __shared__ float sm[kWarps][ROWS], sl[kWarps][ROWS], top[ROWS], all[ROWS];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const Job<T, D> job(p, blockIdx.x / blocks, ROWS);
    const Seen seen(job.had, p);
    const int total = job.ok ? (seen.n + kKeys) / kKeys : 0;  // groups of positions, the new token among them
    const int first = (int)(blockIdx.x % blocks) * kWarps + warp, step = (int)blocks * kWarps;
    char *mine = s_step + warp * S::kWarp;
    const unsigned base = smem_at(mine);
    auto fetch = [&](int g, int stage) {
        if (g < total) {
#pragma unroll
            for (int j = 0; j < PER; ++j) {
                const int r = lane / C + (32 / C) * j, c = lane % C;
                const T *k, *v;
                const bool in = job.row(seen, g * kKeys + r, k, v);
                const unsigned to = base + stage * S::kStage + r * D * 2 + ((c ^ (r & 7)) << 4);
                copy16(to, k + 8 * c, in);
                copy16(to + kKeys * D * 2, v + 8 * c, in);
            }
        }
        copy_commit();
    };
    for (int s = 0; s < S::kStages - 1; ++s) fetch(first + s * step, s);
    unsigned q[NT][NK][2];  // heads lane / 4 (and 8 behind it), columns 2 (lane % 4) and 8 behind them of every step
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        const int r = lane / 4 + 8 * t;
        const T *src = static_cast<const T *>(p.q) + job.query(p, r < job.rows ? r : 0) + (lane % 4) * 2;
#pragma unroll
        for (int i = 0; i < NK; ++i)
#pragma unroll
            for (int e = 0; e < 2; ++e) q[t][i][e] = r < job.rows ? *reinterpret_cast<const unsigned *>(src + i * 16 + 8 * e) : 0u;
    }
    const float c = p.scale * kLog2e;
    float m[NT][2], l[NT][2];  // heads 2 (lane % 4) and the next one: reference; this lane's part of the sum
    float o[NT][NK][4];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            m[t][e] = -CUDART_INF_F;
            l[t][e] = 0.f;
        }
#pragma unroll
        for (int i = 0; i < NK; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[t][i][e] = 0.f;
    }
    int stage = 0;
    for (int g = first; g < total; g += step) {
        fetch(g + (S::kStages - 1) * step, stage + S::kStages - 1 >= S::kStages ? stage - 1 : stage + S::kStages - 1);
        copy_wait<S::kStages - 1>();
        __syncwarp();
        const unsigned ks = base + stage * S::kStage, vs = ks + kKeys * D * 2;
        float s[NT][2][4] = {};  // even and odd steps apart: half the chain
        {
            // matrices: keys 0-7 and 8-15, columns 0-7 and 8-15 of the step
            const int r = lane & 15, cc = lane >> 4;
#pragma unroll
            for (int i = 0; i < NK; ++i) {
                unsigned a[4];
                ldmatrix4(a, ks + r * D * 2 + (((2 * i + cc) ^ (r & 7)) << 4));
#pragma unroll
                for (int t = 0; t < NT; ++t) mma16816(s[t][i & 1], a, q[t][i][0], q[t][i][1]);
            }
        }
        // keys lane / 4 (elements 0, 1) and 8 behind it (2, 3); positions behind the list weigh nothing
        const int left = seen.n + 1 - g * kKeys - lane / 4;
        bool above = false;
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                s[t][0][e] = (e >> 1) * 8 < left ? (s[t][0][e] + s[t][1][e]) * c : -CUDART_INF_F;
                above |= s[t][0][e] > m[t][e & 1] + 8.f;
            }
        if (__any_sync(0xffffffffu, above)) {
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float best = fmaxf(m[t][e], fmaxf(s[t][0][e], s[t][0][e + 2]));
#pragma unroll
                    for (int x = 4; x < 32; x <<= 1) best = fmaxf(best, __shfl_xor_sync(0xffffffffu, best, x));
                    const float f = ex2(m[t][e] - (best == -CUDART_INF_F ? 0.f : best));
                    m[t][e] = best;
                    l[t][e] *= f;
#pragma unroll
                    for (int i = 0; i < NK; ++i) {
                        o[t][i][e] *= f;
                        o[t][i][e + 2] *= f;
                    }
                }
        }
        unsigned w[NT][2];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            float x[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                x[e] = ex2(s[t][0][e] - (m[t][e & 1] == -CUDART_INF_F ? 0.f : m[t][e & 1]));
                l[t][e & 1] += x[e];
            }
            w[t][0] = transposed(Vec<T, 2>::pack(x[0], x[1]));
            w[t][1] = transposed(Vec<T, 2>::pack(x[2], x[3]));
        }
        {
            // transposed: columns 0-7 and 8-15 of the step, keys 0-7 and 8-15
            const int r = (lane & 7) + (lane >> 4) * 8, cc = lane >> 3 & 1;
#pragma unroll
            for (int i = 0; i < NK; ++i) {
                unsigned a[4];
                ldmatrix4t(a, vs + r * D * 2 + (((2 * i + cc) ^ (r & 7)) << 4));
#pragma unroll
                for (int t = 0; t < NT; ++t) mma16816(o[t][i], a, w[t][0], w[t][1]);
            }
        }
        __syncwarp();
        stage = stage + 1 == S::kStages ? 0 : stage + 1;
    }
    copy_wait<0>();
    __syncwarp();
    float *part = reinterpret_cast<float *>(mine);
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int r = 8 * t + 2 * (lane & 3) + e;
#pragma unroll
            for (int x = 4; x < 32; x <<= 1) l[t][e] += __shfl_xor_sync(0xffffffffu, l[t][e], x);
            if (lane < 4) {
                sm[warp][r] = m[t][e];
                sl[warp][r] = l[t][e];
            }
#pragma unroll
            for (int i = 0; i < NK; ++i) {
                part[r * D + i * 16 + lane / 4] = o[t][i][e];
                part[r * D + i * 16 + lane / 4 + 8] = o[t][i][e + 2];
            }
        }
    if (job.ok && job.row0 == 0 && blockIdx.x % blocks == 0) job.keep(p);
    join<T, D, ROWS>(p, job, reinterpret_cast<const float *>(s_step), S::kWarp / 4, sm, sl,
                     reinterpret_cast<float *>(s_step + kWarps * S::kWarp), top, all, blocks);
}

// ---- fp32 -------------------------------------------------------------------

// CUDA-core form: a lane takes one position's score over half of the columns (two lanes a position)
// for ROWS query heads, then D / 32 columns of the weighted values.
template <int D, int ROWS>
struct StepSmem32 {
    static constexpr int kRow = D + 4;  // floats: rows 16 bytes apart on the banks
    static constexpr int kStage = 2 * kKeys * kRow * 4;
    static constexpr int kStages = 2;
    static constexpr int kWarp = kStages * kStage;
    static constexpr int kPart = ROWS * D * 4;
    static_assert(kPart <= kWarp, "a warp's sums lie over its stages");
    static constexpr int kBytes = kWarps * kWarp + 2 * kPart;  // and the queries
};

template <int D, int ROWS>
__global__ void __launch_bounds__(32 * kWarps) step_f32(const __grid_constant__ CacheParams p, unsigned blocks) {
    using S = StepSmem32<D, ROWS>;
    constexpr int C = D / 4, E = D / 32;  // 16-byte chunks of a row; columns of a lane
    __shared__ float sm[kWarps][ROWS], sl[kWarps][ROWS], top[ROWS], all[ROWS];
    __shared__ __align__(16) float weight[kWarps][kKeys][ROWS];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const Job<float, D> job(p, blockIdx.x / blocks, ROWS);
    const Seen seen(job.had, p);
    const int total = job.ok ? (seen.n + kKeys) / kKeys : 0;
    const int first = (int)(blockIdx.x % blocks) * kWarps + warp, step = (int)blocks * kWarps;
    char *mine = s_step + warp * S::kWarp;
    float *qs = reinterpret_cast<float *>(s_step + kWarps * S::kWarp);
    const unsigned base = smem_at(mine);
    auto fetch = [&](int g, int stage) {
        if (g < total) {
#pragma unroll
            for (int j = 0; j < kKeys * C / 32; ++j) {
                const int r = (lane + 32 * j) / C, c = (lane + 32 * j) % C;
                const float *k, *v;
                const bool in = job.row(seen, g * kKeys + r, k, v);
                const unsigned to = base + stage * S::kStage + r * S::kRow * 4 + 16 * c;
                copy16(to, k + 4 * c, in);
                copy16(to + kKeys * S::kRow * 4, v + 4 * c, in);
            }
        }
        copy_commit();
    };
    for (int s = 0; s < S::kStages - 1; ++s) fetch(first + s * step, s);
    for (int i = threadIdx.x; i < ROWS * D; i += 32 * kWarps)
        qs[i] = i < job.rows * D ? static_cast<const float *>(p.q)[job.query(p, 0) + i] : 0.f;
    __syncthreads();
    const float c = p.scale * kLog2e;
    const int key = lane & 15, half = lane >> 4;
    float m[ROWS], l[ROWS], o[ROWS][E];
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
        m[r] = -CUDART_INF_F;
        l[r] = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) o[r][e] = 0.f;
    }
    int stage = 0;
    for (int g = first; g < total; g += step) {
        fetch(g + (S::kStages - 1) * step, stage ^ 1);
        copy_wait<S::kStages - 1>();
        __syncwarp();
        const float *ks = reinterpret_cast<const float *>(mine + stage * S::kStage), *vs = ks + kKeys * S::kRow;
        f2 acc[ROWS];
#pragma unroll
        for (int r = 0; r < ROWS; ++r) acc[r] = 0ull;
#pragma unroll 4
        for (int i = 0; i < D / 2; i += 4) {
            const ulonglong2 k = *reinterpret_cast<const ulonglong2 *>(ks + key * S::kRow + half * (D / 2) + i);
#pragma unroll
            for (int r = 0; r < ROWS; ++r) {
                const ulonglong2 x = *reinterpret_cast<const ulonglong2 *>(qs + r * D + half * (D / 2) + i);
                acc[r] = fma2(x.y, k.y, fma2(x.x, k.x, acc[r]));
            }
        }
        const bool in = g * kKeys + key <= seen.n;
#pragma unroll
        for (int r = 0; r < ROWS; ++r) {
            float s = sum_of(acc[r]);
            s += __shfl_xor_sync(0xffffffffu, s, 16);
            s = in ? s * c : -CUDART_INF_F;
            float t = fmaxf(m[r], s);
#pragma unroll
            for (int x = 8; x > 0; x >>= 1) t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, x));
            const float from = t == -CUDART_INF_F ? 0.f : t;
            const float f = ex2(m[r] - from), w = ex2(s - from);
            m[r] = t;
            l[r] = l[r] * f + (half ? 0.f : w);
#pragma unroll
            for (int e = 0; e < E; ++e) o[r][e] *= f;
            if (!half) weight[warp][key][r] = w;
        }
        __syncwarp();
#pragma unroll 4
        for (int k = 0; k < kKeys; ++k) {
            Vec<float, E> v;
            v.load(vs + k * S::kRow + lane * E);
#pragma unroll
            for (int r = 0; r < ROWS; ++r)
#pragma unroll
                for (int e = 0; e < E; ++e) o[r][e] = fmaf(weight[warp][k][r], v.v[e], o[r][e]);
        }
        __syncwarp();
        stage ^= 1;
    }
    copy_wait<0>();
    __syncwarp();
    float *part = reinterpret_cast<float *>(mine);
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
#pragma unroll
        for (int x = 16; x > 0; x >>= 1) l[r] += __shfl_xor_sync(0xffffffffu, l[r], x);
        if (lane == 0) {
            sm[warp][r] = m[r];
            sl[warp][r] = l[r];
        }
#pragma unroll
        for (int e = 0; e < E; ++e) part[r * D + lane * E + e] = o[r][e];
    }
    if (job.ok && job.row0 == 0 && blockIdx.x % blocks == 0) job.keep(p);
    join<float, D, ROWS>(p, job, reinterpret_cast<const float *>(s_step), S::kWarp / 4, sm, sl, qs + ROWS * D, top, all, blocks);
}

// Tokens of the prompts into the caches.  Of a sequence's tokens those stay that are sinks, and the last
// `ring` ones; a block takes kFillTile of these, with four loads of 16 bytes of keys and of values in flight
// a thread (a tile of 32 tokens of the prompt a block, one load after the other: packed prompts of 8
// sequences 24 us instead of 15; ring slots by one division of 64 bits a block, not one a load: 16.4 to 14.7).
// Bound by memory and by the chain of loads of a block (offsets, length, rows).
constexpr int kFillTile = 8, kFillUnits = 4;

template <typename T, int D>
__global__ void __launch_bounds__(256) fill(const __grid_constant__ CacheParams p, long long tiles, unsigned per_seq) {
    constexpr int V = 16 / sizeof(T), C = D / V;
    if (blockIdx.x == 0) check_offsets(p.seq, threadIdx.x, 256);
    for (long long b = blockIdx.x; b < tiles; b += gridDim.x) {
        const int n = (int)(b / per_seq);
        const long long had = p.lengths ? p.lengths[n] : 0;
        const SeqTile s = seq_whole(p.seq, n);
        if (!s.ok) continue;
        const int len = (int)(s.eos - s.bos);
        if (had < 0 || had > INT64_MAX - len) {
            if (threadIdx.x == 0) atomicOr(p.status, kStatusBadSeq);
            continue;
        }
        const int head = had >= p.sinks ? 0 : p.sinks - had < len ? (int)(p.sinks - had) : len;  // tokens that are sinks
        const int tail = len - p.ring > head ? len - p.ring : head;                              // the first of the others that stays
        const int i0 = (int)(b % per_seq) * kFillTile, kept = head + len - tail;
        const int count = kept - i0 < kFillTile ? kept - i0 : kFillTile;
        if (count <= 0) continue;
        const int slots = p.sinks + p.ring;
        // ring slot of the first token behind the sinks: one division of 64 bits a block
        const unsigned first = (unsigned)((had + head - p.sinks) % p.ring);
        const T *ks = static_cast<const T *>(p.k) + s.bos * p.Nk * D, *vs = static_cast<const T *>(p.v) + s.bos * p.Nk * D;
        T *kc = static_cast<T *>(p.kc) + (long long)n * p.Nk * slots * D, *vc = static_cast<T *>(p.vc) + (long long)n * p.Nk * slots * D;
        const unsigned per = p.Nk * C, units = count * per;
        for (unsigned u0 = threadIdx.x; u0 < units; u0 += 256 * kFillUnits) {
            Pack<T, V> k[kFillUnits], v[kFillUnits];
            long long to[kFillUnits];
#pragma unroll
            for (int e = 0; e < kFillUnits; ++e) {
                const unsigned u = u0 + 256 * e;
                if (u >= units) continue;
                const unsigned r = u / per, w = u - r * per;  // token of the tile; 16 bytes of its heads
                const int i = i0 + (int)r, t = i < head ? i : tail + i - head;
                const unsigned slot = t < head ? (unsigned)had + t : p.sinks + (first + (unsigned)(t - head)) % (unsigned)p.ring;
                const long long from = (long long)t * p.Nk * D + w * V;
                to[e] = ((long long)(w / C) * slots + slot) * D + w % C * V;
                k[e].load(ks + from);
                v[e].load(vs + from);
            }
#pragma unroll
            for (int e = 0; e < kFillUnits; ++e) {
                if (u0 + 256 * e >= units) continue;
                k[e].store(kc + to[e]);
                v[e].store(vc + to[e]);
            }
        }
    }
}

}  // namespace

cudaError_t window_fill_launch(const CacheParams &p, bool bf16, cudaStream_t stream, const char **name) {
    *name = bf16 ? "window_fill<bf16>" : "window_fill<f32>";
    // no sequence keeps more than the cache holds, or than there are tokens
    const long long most = (long long)p.sinks + p.ring < p.seq.T ? (long long)p.sinks + p.ring : p.seq.T;
    const long long per = (most + kFillTile - 1) / kFillTile, tiles = per * p.N;
    const unsigned grid = (unsigned)(tiles < 1 << 20 ? tiles : 1 << 20);
    if (grid == 0) return cudaSuccess;
    const unsigned per_seq = (unsigned)per;
    if (bf16 && p.d == 64) fill<__nv_bfloat16, 64><<<grid, 256, 0, stream>>>(p, tiles, per_seq);
    else if (bf16) fill<__nv_bfloat16, 128><<<grid, 256, 0, stream>>>(p, tiles, per_seq);
    else if (p.d == 64) fill<float, 64><<<grid, 256, 0, stream>>>(p, tiles, per_seq);
    else fill<float, 128><<<grid, 256, 0, stream>>>(p, tiles, per_seq);
    return cudaGetLastError();
}

namespace {

// Blocks of a cluster, that share a sequence's positions: as many as it takes to put a block on every
// SM, while each warp still has two groups of positions (twice as many, 256 jobs of 2048 positions
// took 47 us instead of 42).
template <auto kKernel>
cudaError_t step_launch(const CacheParams &p, int rows, int bytes, cudaStream_t stream) {
    const int G = p.Nq / p.Nk;
    const long long jobs = (long long)p.N * p.Nk * ((G + rows - 1) / rows);
    const long long most = (long long)p.sinks + p.window;
    unsigned blocks = 1;
    while (blocks < 16 && jobs * blocks < kSms && most > (long long)blocks * kWarps * kKeys * 2) blocks *= 2;
    if (jobs * blocks > 0x7fffffffll) return cudaErrorInvalidValue;
    cudaError_t err = allow_smem<kKernel>(bytes);
    if (err == cudaSuccess && blocks > 8) err = allow_wide_cluster<kKernel>();
    if (err != cudaSuccess) return err;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = blocks;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(jobs * blocks));
    cfg.blockDim = dim3(32 * kWarps);
    cfg.dynamicSmemBytes = bytes;
    cfg.stream = stream;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kKernel, p, blocks);
}

template <int D>
cudaError_t step_f32_launch(const CacheParams &p, cudaStream_t stream) {
    const int G = p.Nq / p.Nk;
    if (G == 1) return step_launch<step_f32<D, 1>>(p, 1, StepSmem32<D, 1>::kBytes, stream);
    if (G == 2) return step_launch<step_f32<D, 2>>(p, 2, StepSmem32<D, 2>::kBytes, stream);
    if (G <= 4) return step_launch<step_f32<D, 4>>(p, 4, StepSmem32<D, 4>::kBytes, stream);
    return step_launch<step_f32<D, 8>>(p, 8, StepSmem32<D, 8>::kBytes, stream);
}

}  // namespace

cudaError_t window_step_launch(const CacheParams &p, bool bf16, cudaStream_t stream, const char **name) {
    *name = bf16 ? "window_step<bf16>" : "window_step<f32>";
    if (p.N == 0) return cudaSuccess;
    if (!bf16) return p.d == 64 ? step_f32_launch<64>(p, stream) : step_f32_launch<128>(p, stream);
    if (p.Nq / p.Nk <= 8)
        return p.d == 64 ? step_launch<step_bf16<64, 8>>(p, 8, StepSmem<64, 8>::kBytes, stream)
                         : step_launch<step_bf16<128, 8>>(p, 8, StepSmem<128, 8>::kBytes, stream);
    return p.d == 64 ? step_launch<step_bf16<64, 16>>(p, 16, StepSmem<64, 16>::kBytes, stream)
                     : step_launch<step_bf16<128, 16>>(p, 16, StepSmem<128, 16>::kBytes, stream);
}

}  // namespace dn
