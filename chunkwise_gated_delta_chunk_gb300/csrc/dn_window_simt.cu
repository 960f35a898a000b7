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
// memory, read four columns at a time; the arithmetic is on pairs.  Bound by the fp32
// pipes.  The backward takes dq (by query tiles) and dk, dv (by key tiles) in launches of
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
    static constexpr int kFwd = (2 * kTile + BT * PS) * 4;
    static constexpr int kDq = (4 * kTile + BT * PS) * 4;
    static constexpr int kDkv = (4 * kTile + 2 * BT * PS) * 4;
};

extern __shared__ __align__(16) float s_win[];

// Rows [t0, t0 + 64) of head h of a [tokens, H, D] tensor as fp32; zeros from token `end` on.
template <typename T, int D>
__device__ __forceinline__ void load_rows(float *dst, const T *src, long long t0, long long end, int H, int h) {
    constexpr int V = 16 / sizeof(T);
    for (int i = threadIdx.x; i < BT * (D / V); i += NT) {
        const int r = i / (D / V), c = (i % (D / V)) * V;
        Vec<T, V> x;
        if (t0 + r < end) {
            x.load(src + ((t0 + r) * H + h) * D + c);
        } else {
#pragma unroll
            for (int e = 0; e < V; ++e) x.v[e] = 0.f;
        }
        Vec<float, V> y;
#pragma unroll
        for (int e = 0; e < V; ++e) y.v[e] = x.v[e];
        y.store(dst + r * Smem<D>::kRow + c);
    }
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
__device__ __forceinline__ void walk(long long items, int group, Marked marked, Work work) {
    if constexpr (!REDO) {
        for (long long item = blockIdx.x; item < items; item += gridDim.x) work(item);
    } else {
        for (long long g = blockIdx.x; g * group < items; g += gridDim.x) {
            if (!__syncthreads_or(marked(g))) continue;
            for (int i = 0; i < group && g * group + i < items; ++i) work(g * group + i);
        }
    }
}

template <typename T, int D, bool REDO>
__global__ void __launch_bounds__(NT, 2) simt_fwd(WindowParams p, long long items) {
    const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
    const Sight sight{p.window, p.sinks};
    const float c = p.scale * kLog2e;
    float *Qs = s_win, *Ks = Qs + Smem<D>::kTile, *Ps = Ks + Smem<D>::kTile;
    wait_for_launches();
    if (!REDO && blockIdx.x == 0) check_offsets(p.seq, threadIdx.x, NT);
    // a group: the heads of half a slot
    auto marked = [&](long long g) {
        const Half it(p.seq, g * p.Nq, p.Nq);
        bool any = false;
        if (it.ok)
            for (int i = threadIdx.x; i < (it.t1 - it.t0) * p.Nq; i += NT)
                any |= is_redo(p.lse[(it.s.bos + it.t0) * p.Nq + i]);
        return any;
    };
    walk<REDO>(items, p.Nq, marked, [&](long long item) {
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
        for (int n = 0; n < kt.count(); ++n) {
            const int k0 = kt.tile(n) * BT;
            load_rows<T, D>(Ks, static_cast<const T *>(p.k), bos + k0, it.s.eos, p.Nk, hk);
            __syncthreads();
            float s[4][4];
            dot_rows<D>(s, Qs, Ks, ty, tx);
            __syncthreads();
            load_rows<T, D>(Ks, static_cast<const T *>(p.v), bos + k0, it.s.eos, p.Nk, hk);
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
            __syncthreads();
            add_rows<D, REDO>(acc, Ps, Ks, ty, tx, [&](int i, int k) { return !sight.sees(it.t0 + 4 * ty + i, k0 + k); });
            __syncthreads();
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
__global__ void __launch_bounds__(NT) simt_dq(WindowParams p, long long items) {
    const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
    const Sight sight{p.window, p.sinks};
    const float c = p.scale * kLog2e;
    constexpr int kTile = Smem<D>::kTile;
    float *Qs = s_win, *Gs = Qs + kTile, *Ks = Gs + kTile, *Vs = Ks + kTile, *Ss = Vs + kTile;
    wait_for_launches();
    if (!REDO && blockIdx.x == 0) check_offsets(p.seq, threadIdx.x, NT);
    auto marked = [&](long long g) {
        const long long i = g * NT + threadIdx.x;
        return i < items && p.redo[i / p.Nq * (p.Nq + p.Nk) + i % p.Nq] != 0;
    };
    walk<REDO>(items, NT, marked, [&](long long item) {
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
        load_rows<T, D>(Ks, static_cast<const T *>(p.o), bos + it.t0, it.s.eos, p.Nq, it.head);
        __syncthreads();
        f2 acc[4][D / 32];
        float lse2[4], dsum[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = 4 * ty + i, t = it.t0 + r;
            float a = 0.f;
#pragma unroll
            for (int u = 0; u < D / 16; ++u) a = fmaf(Gs[r * Smem<D>::kRow + tx + 16 * u], Ks[r * Smem<D>::kRow + tx + 16 * u], a);
            dsum[i] = sum16(a);
            lse2[i] = t < it.t1 ? p.lse[(bos + t) * p.Nq + it.head] * kLog2e : 0.f;
            if (!REDO && tx == 0 && t < it.t1) p.dsum[(bos + t) * p.Nq + it.head] = dsum[i];
#pragma unroll
            for (int u = 0; u < D / 32; ++u) acc[i][u] = 0ull;
        }
        __syncthreads();
        const KeyTiles kt(it.t0, it.t1, BT, sight);
        for (int n = 0; n < kt.count(); ++n) {
            const int k0 = kt.tile(n) * BT;
            load_rows<T, D>(Ks, static_cast<const T *>(p.k), bos + k0, it.s.eos, p.Nk, hk);
            load_rows<T, D>(Vs, static_cast<const T *>(p.v), bos + k0, it.s.eos, p.Nk, hk);
            __syncthreads();
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
            add_rows<D, REDO>(acc, Ss, Ks, ty, tx, [&](int i, int k) { return !sight.sees(it.t0 + 4 * ty + i, k0 + k); });
            __syncthreads();
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

template <typename T, int D, bool REDO>
__global__ void __launch_bounds__(NT) simt_dkv(WindowParams p, long long items) {
    const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
    const Sight sight{p.window, p.sinks};
    const float c = p.scale * kLog2e;
    const int G = p.Nq / p.Nk;
    constexpr int kTile = Smem<D>::kTile;
    float *Ks = s_win, *Vs = Ks + kTile, *Qs = Vs + kTile, *Gs = Qs + kTile, *Ps = Gs + kTile, *Ss = Ps + BT * PS;
    wait_for_launches();
    auto marked = [&](long long g) {
        const long long i = g * NT + threadIdx.x;
        return i < items && p.redo[i / p.Nk * (p.Nq + p.Nk) + p.Nq + i % p.Nk] != 0;
    };
    walk<REDO>(items, NT, marked, [&](long long item) {
        const Half it(p.seq, item, p.Nk);
        unsigned *flag = p.redo + it.flag * (p.Nq + p.Nk) + p.Nq + it.head;
        if (REDO) {
            if (!it.ok || !*flag) return;
        } else if (!it.ok) {
            if (threadIdx.x == 0) *flag = 0;
            return;
        }
        const long long bos = it.s.bos;
        const int L = (int)(it.s.eos - bos), k0 = it.t0;
        load_rows<T, D>(Ks, static_cast<const T *>(p.k), bos + k0, it.s.eos, p.Nk, it.head);
        load_rows<T, D>(Vs, static_cast<const T *>(p.v), bos + k0, it.s.eos, p.Nk, it.head);
        f2 dk[4][D / 32], dv[4][D / 32];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int u = 0; u < D / 32; ++u) dk[i][u] = dv[i][u] = 0ull;
        const QueryTiles qt(k0, it.t1, L, BT, sight);
        const int last = k0 < p.sinks ? qt.end : qt.last;
        for (int hg = 0; hg < G; ++hg) {
            const int h = it.head * G + hg;
            for (int n = qt.first; n <= last; ++n) {
                const int q0 = n * BT;
                load_rows<T, D>(Qs, static_cast<const T *>(p.q), bos + q0, it.s.eos, p.Nq, h);
                load_rows<T, D>(Gs, static_cast<const T *>(p.dout), bos + q0, it.s.eos, p.Nq, h);
                __syncthreads();
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
                add_rows<D, REDO>(dk, Ss, Qs, ty, tx, skip);
                __syncthreads();
            }
        }
        bool nan = false;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int j = k0 + 4 * ty + i;
            const long long at = ((bos + j) * p.Nk + it.head) * D;
            const bool in = j < it.t1;
            nan |= store_cols<T, D>(static_cast<T *>(p.dk) + at, dk[i], p.scale, tx, in) && in;
            nan |= store_cols<T, D>(static_cast<T *>(p.dv) + at, dv[i], 1.f, tx, in) && in;
        }
        if (!REDO) {
            nan = __syncthreads_or(nan);
            if (threadIdx.x == 0) *flag = nan;
        } else {
            __syncthreads();
        }
    });
}

template <auto kKernel, bool REDO>
cudaError_t launch_items(int bytes, long long items, int group, const WindowParams &p, cudaStream_t stream) {
    if (items <= 0) return cudaSuccess;
    const cudaError_t err = allow_smem<kKernel>(bytes);
    if (err != cudaSuccess) return err;
    // looks at marks: one block an SM; else one block an item, up to where blocks walk on
    const long long most = REDO ? kSms : kSms * 64, want = REDO ? (items + group - 1) / group : items;
    const unsigned grid = (unsigned)(want < most ? want : most);
    return launch_after(kKernel, dim3(grid), dim3(NT), bytes, stream, p, items);
}

template <typename T, int D, bool REDO>
cudaError_t bwd(const WindowParams &p, cudaStream_t stream) {
    const long long halves = 2 * tile_slots(p.seq, kWinTile);
    const cudaError_t err = launch_items<simt_dq<T, D, REDO>, REDO>(Smem<D>::kDq, halves * p.Nq, NT, p, stream);
    if (err != cudaSuccess) return err;
    return launch_items<simt_dkv<T, D, REDO>, REDO>(Smem<D>::kDkv, halves * p.Nk, NT, p, stream);
}

template <typename T, int D>
cudaError_t fwd(const WindowParams &p, bool redo, cudaStream_t stream) {
    const long long items = 2 * tile_slots(p.seq, kWinTile) * p.Nq;
    return redo ? launch_items<simt_fwd<T, D, true>, true>(Smem<D>::kFwd, items, p.Nq, p, stream)
                : launch_items<simt_fwd<T, D, false>, false>(Smem<D>::kFwd, items, p.Nq, p, stream);
}

}  // namespace

cudaError_t window_simt_fwd(const WindowParams &p, bool bf16, bool redo, cudaStream_t stream) {
    if (bf16) return p.d == 64 ? fwd<__nv_bfloat16, 64>(p, redo, stream) : fwd<__nv_bfloat16, 128>(p, redo, stream);
    return p.d == 64 ? fwd<float, 64>(p, redo, stream) : fwd<float, 128>(p, redo, stream);
}

cudaError_t window_simt_bwd(const WindowParams &p, bool bf16, bool redo, cudaStream_t stream) {
    auto go = [&](auto t) {
        using T = decltype(t);
        if (p.d == 64) return redo ? bwd<T, 64, true>(p, stream) : bwd<T, 64, false>(p, stream);
        return redo ? bwd<T, 128, true>(p, stream) : bwd<T, 128, false>(p, stream);
    };
    return bf16 ? go(__nv_bfloat16{}) : go(float{});
}

}  // namespace dn
