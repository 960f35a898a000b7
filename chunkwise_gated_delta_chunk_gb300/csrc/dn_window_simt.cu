// Attention over a sliding window with sinks on CUDA cores: fp32 tensors, and the
// tiles that the tensor-core kernels marked (REDO).
//
//     forward   s = scale q . k over the visible pairs, p = e^{s - m}, o = sum p v / sum p,
//               with the maximum m and the sum carried along from tile to tile of keys
//     backward  p = e^{s - lse},  dS = p (dO . v - sum dO o)
//               dq = scale sum_k dS k,   dk = scale sum_q dS q,   dv = sum_q p dO
//
// Tiles of 64 queries and 64 keys, 256 threads; a thread holds 4 x 4 scores and 4 rows of
// d / 16 columns of each output in registers.  Both products' operands are rows in shared
// memory, read four columns at a time; the arithmetic is on pairs.  The next tile comes by
// asynchronous copies while one is worked on.  Bound by the fp32 pipes where there are many
// tiles (7 ragged sequences of 600 tokens, 6 heads of 64 columns, window 101: 39, 53 and 70 us for the three
// kernels, 0.4 to 0.46 of the issue slots).  The backward takes dq (by query tiles) and dk, dv (by key tiles) in launches of
// their own, so that nothing is added by atomics: 7 products instead of 5, the same bits
// in every call.
//
// REDO: the tensor-core kernels, and these without REDO, give masked pairs of a visited
// tile the weight 0, and 0 times an infinite or NaN value is NaN.  Rows (forward) and tiles
// (backward) that come out with a NaN are marked and taken again here with masked pairs
// skipped.  Unmarked ones cost a look at the mark.
#include "dn_window.cuh"

namespace dn {
namespace {

constexpr int BT = 64;       // queries and keys of a tile
constexpr int NT = 256;      // threads
constexpr int PS = BT + 4;   // row stride of scores in shared memory

template <int D>
struct Smem {
    static constexpr int kRow = D + 4;  // rows a multiple of 16 bytes apart, 8 of them on different banks
    static constexpr int kTile = BT * kRow;
    static constexpr int kFwd = (4 * kTile + BT * PS) * 4;       // q, two of k, v, p
    static constexpr int kDq = (5 * kTile + BT * PS) * 4;        // q, do, two of k, v, ds
    static constexpr int kDkv = (5 * kTile + 2 * BT * PS) * 4;   // k, v, two of q, do, p, ds
    static_assert(kDkv <= 227 * 1024, "exceeds the 227 KB of shared memory per CTA");
};

extern __shared__ __align__(16) float s_win[];

// Rows [t0, t0 + 64) of head h of a [tokens, H, D] tensor as fp32; zeros from token `end` on.  fp32 tensors come by
// asynchronous copies, one group of them per call; landed<N>() waits for all but the last N groups.
template <typename T, int D>
__device__ __forceinline__ void load_rows(float *dst, const T *src, long long t0, long long end, int H, int h) {
    constexpr int V = 16 / sizeof(T);
#pragma unroll 4
    for (int i = threadIdx.x; i < BT * (D / V); i += NT) {
        const int r = i / (D / V), c = (i % (D / V)) * V;
        const bool in = t0 + r < end;
        const T *from = src + ((in ? t0 + r : t0) * H + h) * D + c;
        float *to = dst + r * Smem<D>::kRow + c;
        if constexpr (sizeof(T) == 4) {
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"((unsigned)__cvta_generic_to_shared(to)), "l"(from),
                         "r"(in ? 16 : 0)
                         : "memory");
        } else {
            Vec<T, V> x;
            Vec<float, V> y;
            if (in) x.load(from);
#pragma unroll
            for (int e = 0; e < V; ++e) y.v[e] = in ? x.v[e] : 0.f;
            y.store(to);
        }
    }
    if constexpr (sizeof(T) == 4) asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void landed() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// s[i][j] = a_{4 ty + i} . b_{tx + 16 j} over D columns.
template <int D>
__device__ __forceinline__ void dot_rows(float (&s)[4][4], const float *a, const float *b, int ty, int tx) {
    constexpr int R = Smem<D>::kRow;
    f2 acc[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = 0ull;
#pragma unroll 4
    for (int c = 0; c < D; c += 4) {
        ulonglong2 x[4], y[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = *reinterpret_cast<const ulonglong2 *>(a + (4 * ty + i) * R + c);
#pragma unroll
        for (int j = 0; j < 4; ++j) y[j] = *reinterpret_cast<const ulonglong2 *>(b + (tx + 16 * j) * R + c);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[i][j] = fma2(x[i].y, y[j].y, fma2(x[i].x, y[j].x, acc[i][j]));
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) s[i][j] = sum_of(acc[i][j]);
}

// acc[i][.] += sum_k w_{4 ty + i, k} b_k over the tile's 64 rows b_k; columns 4 tx + 64 u + (0..3).
// SKIP(i, k): the pair is left out (not weighted 0).
template <int D, bool REDO, typename Skip>
__device__ __forceinline__ void add_rows(f2 (&acc)[4][D / 32], const float *w, const float *b, int ty, int tx, Skip skip) {
    constexpr int R = Smem<D>::kRow, U = D / 64;
#pragma unroll 2
    for (int k = 0; k < BT; k += 4) {
        float4 p[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) p[i] = *reinterpret_cast<const float4 *>(w + (4 * ty + i) * PS + k);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            ulonglong2 y[U];
#pragma unroll
            for (int u = 0; u < U; ++u) y[u] = *reinterpret_cast<const ulonglong2 *>(b + (k + e) * R + 4 * tx + 64 * u);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (REDO && skip(i, k + e)) continue;
                const f2 pp = both(e == 0 ? p[i].x : e == 1 ? p[i].y : e == 2 ? p[i].z : p[i].w);
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    acc[i][2 * u] = fma2(pp, y[u].x, acc[i][2 * u]);
                    acc[i][2 * u + 1] = fma2(pp, y[u].y, acc[i][2 * u + 1]);
                }
            }
        }
    }
}

// Row 4 ty + i of an output, scaled; true where it holds a NaN.
template <typename T, int D>
__device__ __forceinline__ bool store_cols(T *row, const f2 (&acc)[D / 32], float f, int tx, bool write) {
    bool nan = false;
#pragma unroll
    for (int u = 0; u < D / 64; ++u) {
        Vec<T, 4> y;
        split(acc[2 * u], y.v[0], y.v[1]);
        split(acc[2 * u + 1], y.v[2], y.v[3]);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            y.v[e] *= f;
            nan |= isnan(y.v[e]);
        }
        if (write) y.store(row + 4 * tx + 64 * u);
    }
    return nan;
}

__device__ __forceinline__ float max16(float x) {
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
    return x;
}
__device__ __forceinline__ float sum16(float x) {
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// Item of a grid: half a slot of kWinTile tokens, and a head.
struct Half {
    SeqTile s;
    long long flag;  // its place among the slots' halves
    int head, t0, t1;
    bool ok;
    __device__ __forceinline__ Half(const SeqView &seq, long long item, int heads) {
        head = (int)(item % heads);
        flag = item / heads;
        s = seq_tile(seq, (unsigned)(flag >> 1), kWinTile);
        t0 = s.c * kWinTile + (int)(flag & 1) * BT;
        const int L = (int)(s.eos - s.bos);
        t1 = t0 + BT < L ? t0 + BT : L;
        ok = s.ok && t0 < t1;
    }
};

// What a block of a grid does: item after item, or (REDO) a look at many marks at a time and only the
// marked ones.  `marked(i)`: thread-wise, is group i of `group` items marked anywhere.
template <bool REDO, typename Marked, typename Work>
__device__ __forceinline__ void walk(unsigned block, unsigned blocks, long long items, int group, Marked marked, Work work) {
    if constexpr (!REDO) {
        for (long long item = block; item < items; item += blocks) work(item);
    } else {
        for (long long g = block; g * group < items; g += blocks) {
            if (!__syncthreads_or(marked(g))) continue;
            for (int i = 0; i < group && g * group + i < items; ++i) work(g * group + i);
        }
    }
}

template <typename T, int D, bool REDO>
__global__ void __launch_bounds__(NT, D == 64 ? 2 : 1) simt_fwd(WindowParams p, long long items) {
    const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
    const Sight sight{p.window, p.sinks};
    const float c = p.scale * kLog2e;
    constexpr int kTile = Smem<D>::kTile;
    float *Qs = s_win, *Kb = Qs + kTile, *Vs = Kb + 2 * kTile, *Ps = Vs + kTile;
    wait_for_launches();
    if (REDO && blockIdx.x == 0) check_offsets(p.seq, threadIdx.x, NT);  // the last kernel of every forward
    // a group: the heads of half a slot
    auto marked = [&](long long g) {
        const Half it(p.seq, g * p.Nq, p.Nq);
        bool any = false;
        if (it.ok)
            for (int i = threadIdx.x; i < (it.t1 - it.t0) * p.Nq; i += NT)
                any |= is_redo(p.lse[(it.s.bos + it.t0) * p.Nq + i]);
        return any;
    };
    walk<REDO>(blockIdx.x, gridDim.x, items, p.Nq, marked, [&](long long item) {
        const Half it(p.seq, item, p.Nq);
        if (!it.ok) return;
        const long long bos = it.s.bos;
        float *lse = p.lse + bos * p.Nq + it.head;
        bool write[4];
        bool any = false;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int t = it.t0 + 4 * ty + i;
            write[i] = t < it.t1 && (!REDO || is_redo(lse[(long long)t * p.Nq]));
            any |= write[i];
        }
        if (REDO && !__syncthreads_or(any)) return;
        const int hk = it.head / (p.Nq / p.Nk);
        load_rows<T, D>(Qs, static_cast<const T *>(p.q), bos + it.t0, it.s.eos, p.Nq, it.head);
        f2 acc[4][D / 32];
        float m[4], l[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            m[i] = -CUDART_INF_F;
            l[i] = 0.f;
#pragma unroll
            for (int u = 0; u < D / 32; ++u) acc[i][u] = 0ull;
        }
        const KeyTiles kt(it.t0, it.t1, BT, sight);
        auto keys = [&](int n) {
            load_rows<T, D>(Kb + (n & 1) * kTile, static_cast<const T *>(p.k), bos + (long long)kt.tile(n) * BT, it.s.eos, p.Nk, hk);
        };
        keys(0);
        for (int n = 0; n < kt.count(); ++n) {
            const int k0 = kt.tile(n) * BT;
            landed<0>();
            __syncthreads();
            load_rows<T, D>(Vs, static_cast<const T *>(p.v), bos + k0, it.s.eos, p.Nk, hk);
            const bool more = n + 1 < kt.count();
            if (more) keys(n + 1);
            float s[4][4];
            dot_rows<D>(s, Qs, Kb + (n & 1) * kTile, ty, tx);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int t = it.t0 + 4 * ty + i;
                float top = m[i];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    s[i][j] = sight.sees(t, k0 + tx + 16 * j) ? s[i][j] * c : -CUDART_INF_F;
                    // fmaxf drops a NaN; the weights below bring it back
                    top = fmaxf(top, s[i][j]);
                }
                top = max16(top);
                const float base = top == -CUDART_INF_F ? 0.f : top;
                const float f = ex2(m[i] - base);
                m[i] = top;
                float sum = 0.f;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    s[i][j] = ex2(s[i][j] - base);
                    sum += s[i][j];
                    Ps[(4 * ty + i) * PS + tx + 16 * j] = s[i][j];
                }
                l[i] = l[i] * f + sum;
#pragma unroll
                for (int u = 0; u < D / 32; ++u) acc[i][u] = mul2(acc[i][u], both(f));
            }
            if (more) landed<1>();
            else landed<0>();
            __syncthreads();
            add_rows<D, REDO>(acc, Ps, Vs, ty, tx, [&](int i, int k) { return !sight.sees(it.t0 + 4 * ty + i, k0 + k); });
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int t = it.t0 + 4 * ty + i;
            const float sum = sum16(l[i]);
            T *row = static_cast<T *>(p.o) + ((bos + t) * p.Nq + it.head) * D;
            bool nan = store_cols<T, D>(row, acc[i], 1.f / sum, tx, write[i]);
            nan = __ballot_sync(0xffffffffu, nan) & (0xffffu << (threadIdx.x & 16));
            if (write[i] && tx == 0)
                lse[(long long)t * p.Nq] = !REDO && nan ? redo_mark() : (m[i] + log2f(sum)) * 0.6931471805599453f;
        }
        __syncthreads();
    });
}

// Weights p and score gradients dS of a tile: s holds q . k, g holds dO . v; rows (i) and
// columns (j) are queries and keys or the other way round.
__device__ __forceinline__ void weights(float &s, float &g, bool seen, float c, float lse2, float dsum) {
    const float w = seen ? ex2(s * c - lse2) : 0.f;
    g = seen ? w * (g - dsum) : 0.f;
    s = w;
}

template <typename T, int D, bool REDO>
__device__ __forceinline__ void work_dq(const WindowParams &p, unsigned block, unsigned blocks, long long items) {
    const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
    const Sight sight{p.window, p.sinks};
    const float c = p.scale * kLog2e;
    constexpr int kTile = Smem<D>::kTile;
    float *Qs = s_win, *Gs = Qs + kTile, *Kb = Gs + kTile, *Vs = Kb + 2 * kTile, *Ss = Vs + kTile;
    if (!REDO && block == 0) check_offsets(p.seq, threadIdx.x, NT);
    auto marked = [&](long long g) {
        const long long i = g * NT + threadIdx.x;
        return i < items && p.redo[i / p.Nq * (p.Nq + p.Nk) + i % p.Nq] != 0;
    };
    walk<REDO>(block, blocks, items, NT, marked, [&](long long item) {
        const Half it(p.seq, item, p.Nq);
        unsigned *flag = p.redo + it.flag * (p.Nq + p.Nk) + it.head;
        if (REDO) {
            if (!it.ok || !*flag) return;
        } else if (!it.ok) {
            if (threadIdx.x == 0) *flag = 0;
            return;
        }
        const long long bos = it.s.bos;
        const int hk = it.head / (p.Nq / p.Nk);
        load_rows<T, D>(Qs, static_cast<const T *>(p.q), bos + it.t0, it.s.eos, p.Nq, it.head);
        load_rows<T, D>(Gs, static_cast<const T *>(p.dout), bos + it.t0, it.s.eos, p.Nq, it.head);
        if (!REDO) load_rows<T, D>(Vs, static_cast<const T *>(p.o), bos + it.t0, it.s.eos, p.Nq, it.head);
        const KeyTiles kt(it.t0, it.t1, BT, sight);
        auto keys = [&](int n) {
            load_rows<T, D>(Kb + (n & 1) * kTile, static_cast<const T *>(p.k), bos + (long long)kt.tile(n) * BT, it.s.eos, p.Nk, hk);
        };
        auto values = [&](int n) {
            load_rows<T, D>(Vs, static_cast<const T *>(p.v), bos + (long long)kt.tile(n) * BT, it.s.eos, p.Nk, hk);
        };
        landed<0>();
        __syncthreads();
        keys(0);
        f2 acc[4][D / 32];
        float lse2[4], dsum[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = 4 * ty + i, t = it.t0 + r;
            const long long at = (bos + t) * p.Nq + it.head;
            lse2[i] = t < it.t1 ? p.lse[at] * kLog2e : 0.f;
            if (REDO) {
                dsum[i] = t < it.t1 ? p.dsum[at] : 0.f;
            } else {
                float a = 0.f;
#pragma unroll
                for (int u = 0; u < D / 16; ++u) a = fmaf(Gs[r * Smem<D>::kRow + tx + 16 * u], Vs[r * Smem<D>::kRow + tx + 16 * u], a);
                dsum[i] = sum16(a);
                if (tx == 0 && t < it.t1) p.dsum[at] = dsum[i];
            }
#pragma unroll
            for (int u = 0; u < D / 32; ++u) acc[i][u] = 0ull;
        }
        __syncthreads();
        values(0);
        for (int n = 0; n < kt.count(); ++n) {
            const int k0 = kt.tile(n) * BT;
            const float *Ks = Kb + (n & 1) * kTile;
            const bool more = n + 1 < kt.count();
            landed<0>();
            __syncthreads();
            if (more) keys(n + 1);
            float s[4][4], g[4][4];
            dot_rows<D>(s, Qs, Ks, ty, tx);
            dot_rows<D>(g, Gs, Vs, ty, tx);
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    weights(s[i][j], g[i][j], sight.sees(it.t0 + 4 * ty + i, k0 + tx + 16 * j), c, lse2[i], dsum[i]);
                    Ss[(4 * ty + i) * PS + tx + 16 * j] = g[i][j];
                }
            __syncthreads();
            if (more) values(n + 1);
            add_rows<D, REDO>(acc, Ss, Ks, ty, tx, [&](int i, int k) { return !sight.sees(it.t0 + 4 * ty + i, k0 + k); });
        }
        bool nan = false;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int t = it.t0 + 4 * ty + i;
            T *row = static_cast<T *>(p.dq) + ((bos + t) * p.Nq + it.head) * D;
            nan |= store_cols<T, D>(row, acc[i], p.scale, tx, t < it.t1) && t < it.t1;
        }
        if (!REDO) {
            nan = __syncthreads_or(nan);
            if (threadIdx.x == 0) *flag = nan;
        } else {
            __syncthreads();
        }
    });
}

// What the rows of a key tile's sums go to.
//   whole: dk and dv of all query heads and tiles
//   by head (p.head_part): an item for each query head, summed up by simt_head_sums: where there
//   are too few key tiles to fill the GPU
// Of the first key tile of a sequence the query tiles behind its window see the sinks alone; they are taken by
// items of their own (p.parts, as in the tensor-core kernels), which leave fp32 sums of the sinks' rows.
struct KeyItem {
    SeqTile s;
    long long flag, place;  // its mark; its place among the parts
    int hk, h0, heads, k0, k1, first, last, L;
    bool ok, part, split;
    template <bool REDO>
    static __device__ __forceinline__ KeyItem of(const WindowParams &p, long long item, long long main_items, long long part_slots) {
        KeyItem u;
        const int G = p.Nq / p.Nk;
        const Sight sight{p.window, p.sinks};
        u.part = !REDO && item >= main_items;
        if (u.part) {
            item -= main_items;
            const int half = (int)(item & 1), per = p.Nq / p.part_heads;
            u.place = item >> 1;
            u.h0 = (int)(u.place % p.part_heads) * per;
            u.hk = u.h0 / G;
            u.heads = per;
            u.s = seq_tile(p.seq, (unsigned)(u.place / p.part_heads), p.part_tiles * kWinTile);
            u.k0 = half * BT;
        } else {
            const bool by_head = !REDO && p.head_part;
            const int n = by_head ? p.Nq : p.Nk, head = (int)(item % n);
            const long long half = item / n;
            u.hk = by_head ? head / G : head;
            u.h0 = by_head ? head : head * G;
            u.heads = by_head ? 1 : G;
            u.flag = half * (p.Nq + p.Nk) + p.Nq + u.hk;
            u.s = seq_tile(p.seq, (unsigned)(half >> 1), kWinTile);
            u.k0 = u.s.c * kWinTile + (int)(half & 1) * BT;
            u.place = part_slots * p.part_heads + (long long)u.s.n * p.Nk + u.hk;
        }
        u.L = (int)(u.s.eos - u.s.bos);
        u.k1 = u.k0 + BT < u.L ? u.k0 + BT : u.L;
        u.ok = u.s.ok && u.k0 < u.k1;
        if (!u.ok) return u;
        // the queries behind the window of the first tile of kWinTile keys, where any are
        const QueryTiles far(0, kWinTile < u.L ? kWinTile : u.L, u.L, kWinTile, sight);
        u.split = !REDO && p.parts && u.k0 < p.sinks && far.end > far.last;
        const QueryTiles qt(u.k0, u.k1, u.L, BT, sight);
        u.first = qt.first;
        u.last = u.k0 < p.sinks ? (u.split ? 2 * far.last + 1 : qt.end) : qt.last;
        if (u.part) {
            const int from = u.s.c * p.part_tiles, to = (int)(u.s.t1 - u.s.bos - 1) / kWinTile;
            u.first = 2 * (from > far.last + 1 ? from : far.last + 1);
            u.last = 2 * to + 1;
            u.ok = u.split && u.first <= u.last;
        }
        if (u.last > qt.end) u.last = qt.end;
        return u;
    }
};

template <typename T, int D, bool REDO>
__device__ __forceinline__ void work_dkv(const WindowParams &p, unsigned block, unsigned blocks, long long items, long long main_items,
                                         long long part_slots) {
    const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
    const Sight sight{p.window, p.sinks};
    const float c = p.scale * kLog2e;
    constexpr int kTile = Smem<D>::kTile;
    float *Ks = s_win, *Vs = Ks + kTile, *Qb = Vs + kTile, *Gs = Qb + 2 * kTile, *Ps = Gs + kTile, *Ss = Ps + BT * PS;
    auto marked = [&](long long g) {
        const long long i = g * NT + threadIdx.x;
        return i < items && p.redo[i / p.Nk * (p.Nq + p.Nk) + p.Nq + i % p.Nk] != 0;
    };
    walk<REDO>(block, blocks, items, NT, marked, [&](long long item) {
        const KeyItem u = KeyItem::of<REDO>(p, item, main_items, part_slots);
        const bool by_head = !REDO && p.head_part && !u.part;
        if (REDO) {
            if (!u.ok || !p.redo[u.flag]) return;
        } else if (!u.ok) {
            if (threadIdx.x == 0 && !u.part && !by_head) p.redo[u.flag] = 0;
            return;
        }
        const long long bos = u.s.bos;
        const int L = u.L, k0 = u.k0, tiles = u.last - u.first + 1, rounds = tiles * u.heads;
        load_rows<T, D>(Ks, static_cast<const T *>(p.k), bos + k0, u.s.eos, p.Nk, u.hk);
        load_rows<T, D>(Vs, static_cast<const T *>(p.v), bos + k0, u.s.eos, p.Nk, u.hk);
        auto queries = [&](int n) {
            load_rows<T, D>(Qb + (n & 1) * kTile, static_cast<const T *>(p.q), bos + (long long)(u.first + n % tiles) * BT, u.s.eos, p.Nq,
                            u.h0 + n / tiles);
        };
        auto gradients = [&](int n) {
            load_rows<T, D>(Gs, static_cast<const T *>(p.dout), bos + (long long)(u.first + n % tiles) * BT, u.s.eos, p.Nq, u.h0 + n / tiles);
        };
        queries(0);
        gradients(0);
        f2 dk[4][D / 32], dv[4][D / 32];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int e = 0; e < D / 32; ++e) dk[i][e] = dv[i][e] = 0ull;
        for (int n = 0; n < rounds; ++n) {
            const int h = u.h0 + n / tiles, q0 = (u.first + n % tiles) * BT;
            const float *Qs = Qb + (n & 1) * kTile;
            const bool more = n + 1 < rounds;
            landed<0>();
            __syncthreads();
            if (more) queries(n + 1);
            float s[4][4], g[4][4];
            dot_rows<D>(s, Ks, Qs, ty, tx);
            dot_rows<D>(g, Vs, Gs, ty, tx);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int t = q0 + tx + 16 * j;
                const long long at = (bos + t) * p.Nq + h;
                const float lse2 = t < L ? p.lse[at] * kLog2e : 0.f, dsum = t < L ? p.dsum[at] : 0.f;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    weights(s[i][j], g[i][j], t < L && sight.sees(t, k0 + 4 * ty + i), c, lse2, dsum);
                    Ps[(4 * ty + i) * PS + tx + 16 * j] = s[i][j];
                    Ss[(4 * ty + i) * PS + tx + 16 * j] = g[i][j];
                }
            }
            __syncthreads();
            auto skip = [&](int i, int k) { return q0 + k >= L || !sight.sees(q0 + k, k0 + 4 * ty + i); };
            add_rows<D, REDO>(dv, Ps, Gs, ty, tx, skip);
            __syncthreads();
            if (more) gradients(n + 1);
            add_rows<D, REDO>(dk, Ss, Qs, ty, tx, skip);
        }
        bool nan = false;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int j = k0 + 4 * ty + i;
            const bool in = j < u.k1;
            if (by_head) {
                float *to = p.head_part + ((bos + j) * p.Nq + u.h0) * 2 * D;
                store_cols<float, D>(to, dv[i], 1.f, tx, in);
                store_cols<float, D>(to + D, dk[i], p.scale, tx, in);
            } else if (u.part || (u.split && j < p.sinks)) {
                float *to = p.sink_part + (u.place * 2 * p.sinks + j) * D;
                store_cols<float, D>(to, dv[i], 1.f, tx, j < p.sinks && in);
                store_cols<float, D>(to + (long long)p.sinks * D, dk[i], p.scale, tx, j < p.sinks && in);
            } else {
                const long long at = ((bos + j) * p.Nk + u.hk) * D;
                nan |= store_cols<T, D>(static_cast<T *>(p.dk) + at, dk[i], p.scale, tx, in) && in;
                nan |= store_cols<T, D>(static_cast<T *>(p.dv) + at, dv[i], 1.f, tx, in) && in;
            }
        }
        nan = __syncthreads_or(nan);
        if (!REDO && threadIdx.x == 0 && !u.part && !by_head) p.redo[u.flag] = nan;
    });
}

template <typename T, int D>
__global__ void __launch_bounds__(NT) simt_dq(WindowParams p, long long items) {
    wait_for_launches();
    work_dq<T, D, false>(p, blockIdx.x, gridDim.x, items);
}
template <typename T, int D>
__global__ void __launch_bounds__(NT) simt_dkv(WindowParams p, long long items, long long main_items, long long part_slots) {
    wait_for_launches();
    work_dkv<T, D, false>(p, blockIdx.x, gridDim.x, items, main_items, part_slots);
}
// The marked tiles of both: the first `dq_blocks` blocks look at those of queries, the others at those of keys.
template <typename T, int D>
__global__ void __launch_bounds__(NT) simt_bwd_redo(WindowParams p, unsigned dq_blocks, long long dq_items, long long dkv_items) {
    wait_for_launches();
    if (blockIdx.x < dq_blocks) work_dq<T, D, true>(p, blockIdx.x, dq_blocks, dq_items);
    else work_dkv<T, D, true>(p, blockIdx.x - dq_blocks, gridDim.x - dq_blocks, dkv_items, dkv_items, 0);
}

// The query heads' sums of a key tile, in order.
template <typename T, int D>
__global__ void __launch_bounds__(NT) simt_head_sums(WindowParams p, long long items, long long part_slots) {
    wait_for_launches();
    const int G = p.Nq / p.Nk;
    WindowParams whole = p;
    whole.head_part = nullptr;
    for (long long item = blockIdx.x; item < items; item += gridDim.x) {
        const KeyItem u = KeyItem::of<false>(whole, item, items, part_slots);
        bool nan = false;
        if (u.ok)
            for (int i = threadIdx.x; i < (u.k1 - u.k0) * (D / 2); i += NT) {  // four columns of dv or dk
                const int j = u.k0 + i / (D / 2), w = i / (D / 4) % 2, col = i % (D / 4) * 4;
                const float *from = p.head_part + (((u.s.bos + j) * p.Nq + u.h0) * 2 + w) * D + col;
                float4 v = *reinterpret_cast<const float4 *>(from);
                for (int h = 1; h < G; ++h) {
                    const float4 a = *reinterpret_cast<const float4 *>(from + (long long)h * 2 * D);
                    v.x += a.x; v.y += a.y; v.z += a.z; v.w += a.w;
                }
                if (u.split && j < p.sinks) {
                    *reinterpret_cast<float4 *>(p.sink_part + ((u.place * 2 + w) * p.sinks + j) * D + col) = v;
                } else {
                    nan |= isnan(v.x) | isnan(v.y) | isnan(v.z) | isnan(v.w);
                    Vec<T, 4> y;
                    y.v[0] = v.x; y.v[1] = v.y; y.v[2] = v.z; y.v[3] = v.w;
                    y.store(static_cast<T *>(w == 0 ? p.dv : p.dk) + ((u.s.bos + j) * p.Nk + u.hk) * D + col);
                }
            }
        nan = __syncthreads_or(nan);
        if (threadIdx.x == 0) p.redo[u.flag] = nan;
    }
}

template <auto kKernel, bool REDO, typename... A>
cudaError_t launch_items(int bytes, long long items, int group, cudaStream_t stream, const WindowParams &p, A... rest) {
    if (items <= 0) return cudaSuccess;
    const cudaError_t err = allow_smem<kKernel>(bytes);
    if (err != cudaSuccess) return err;
    // looks at marks: one block an SM; else one block an item, up to where blocks walk on
    const long long most = REDO ? kSms : kSms * 64, want = REDO ? (items + group - 1) / group : items;
    const unsigned grid = (unsigned)(want < most ? want : most);
    return launch_after(kKernel, dim3(grid), dim3(NT), bytes, stream, p, items, rest...);
}

template <typename T, int D>
cudaError_t bwd(const WindowParams &p, cudaStream_t stream) {
    const long long halves = 2 * tile_slots(p.seq, kWinTile);
    cudaError_t err = launch_items<simt_dq<T, D>, false>(Smem<D>::kDq, halves * p.Nq, NT, stream, p);
    if (err != cudaSuccess) return err;
    const long long part_slots = p.parts ? tile_slots(p.seq, p.part_tiles * kWinTile) : 0;
    const long long main_items = halves * (p.head_part ? p.Nq : p.Nk), items = main_items + part_slots * p.part_heads * 2;
    err = launch_items<simt_dkv<T, D>, false>(Smem<D>::kDkv, items, NT, stream, p, main_items, part_slots);
    if (err == cudaSuccess && p.head_part) err = launch_items<simt_head_sums<T, D>, false>(0, halves * p.Nk, 1, stream, p, part_slots);
    return err == cudaSuccess ? window_sink_sums(p, sizeof(T) == 2, stream) : err;
}

template <typename T, int D>
cudaError_t bwd_redo(const WindowParams &p, cudaStream_t stream) {
    const long long halves = 2 * tile_slots(p.seq, kWinTile), dq_items = halves * p.Nq, dkv_items = halves * p.Nk;
    constexpr int bytes = Smem<D>::kDq > Smem<D>::kDkv ? Smem<D>::kDq : Smem<D>::kDkv;
    const cudaError_t err = allow_smem<simt_bwd_redo<T, D>>(bytes);
    if (err != cudaSuccess) return err;
    auto blocks = [](long long items) { return (unsigned)((items + NT - 1) / NT < kSms ? (items + NT - 1) / NT : kSms); };
    return launch_after(simt_bwd_redo<T, D>, dim3(blocks(dq_items) + blocks(dkv_items)), dim3(NT), bytes, stream, p, blocks(dq_items), dq_items,
                        dkv_items);
}

template <typename T, int D, bool REDO>
cudaError_t fwd(const WindowParams &p, cudaStream_t stream) {
    const long long items = 2 * tile_slots(p.seq, kWinTile) * p.Nq;
    return launch_items<simt_fwd<T, D, REDO>, REDO>(Smem<D>::kFwd, items, p.Nq, stream, p);
}

}  // namespace

cudaError_t window_simt_fwd(const WindowParams &p, cudaStream_t stream) {
    return p.d == 64 ? fwd<float, 64, false>(p, stream) : fwd<float, 128, false>(p, stream);
}

cudaError_t window_fwd_redo(const WindowParams &p, bool bf16, cudaStream_t stream) {
    if (bf16) return p.d == 64 ? fwd<__nv_bfloat16, 64, true>(p, stream) : fwd<__nv_bfloat16, 128, true>(p, stream);
    return p.d == 64 ? fwd<float, 64, true>(p, stream) : fwd<float, 128, true>(p, stream);
}

cudaError_t window_simt_bwd(const WindowParams &p, cudaStream_t stream) {
    return p.d == 64 ? bwd<float, 64>(p, stream) : bwd<float, 128>(p, stream);
}

cudaError_t window_bwd_redo(const WindowParams &p, bool bf16, cudaStream_t stream) {
    if (bf16) return p.d == 64 ? bwd_redo<__nv_bfloat16, 64>(p, stream) : bwd_redo<__nv_bfloat16, 128>(p, stream);
    return p.d == 64 ? bwd_redo<float, 64>(p, stream) : bwd_redo<float, 128>(p, stream);
}

}  // namespace dn
