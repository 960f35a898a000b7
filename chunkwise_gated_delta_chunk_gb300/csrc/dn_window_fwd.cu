// Attention over a sliding window with sinks, forward, bf16: tcgen05 / TMEM / TMA.
//
//     S = Q K^T,  p = e^{scale s - m},  O += P V,  o = O / sum p,  lse = m + log sum p
//
// tile by tile of 128 keys with the running maximum m and sum of every row.  A CTA works on
// two tiles of 128 queries at once that share their keys: two query heads of one key head
// where its group is even, else two neighbouring tiles of tokens of one head.  While one
// tile's scores go through the softmax, the tensor cores work for the other.
//
// Warps 0-3 and 4-7: softmax of the first and the second query tile, one row a thread;
// warp 8: TMA loads of Q, K and V; warp 9: issues the MMAs (one thread).
// Tensor memory: scores of both tiles (128 fp32 columns each; the weights P overwrite them
// as bf16) and both O (d columns each).
// For every key tile j the issuer does, for the first and then the second query tile,
//     wait P(j);  O += P V(j);  S = Q K(j+1)
// so S(j+1) of one tile is ready when the softmax of the other has just begun.
//
// O is rescaled only when a row's maximum has grown by more than 2^8 since the last time:
// weights stay below 2^8, sums in fp32 lose nothing (and P in bf16 has the same relative
// rounding at every size).  Masks cost selects only in tiles that the window's or the
// sequence's border crosses.  The sinks in front of the window are a tile of 32 keys where
// they fit in one.  P is rounded to bf16 for the product; the sum takes it unrounded.
//
// CTAs are persistent, one an SM; every wait is bounded (dn_tc_sync.cuh).
#include "dn_window_tc.cuh"

namespace dn {
namespace {

using namespace ptx;
using namespace tcs;

constexpr int kThreads = 320;

template <int D>
struct Lay {
    static constexpr uint32_t kPanel = 128 * 128;            // 128 rows of 64 columns
    static constexpr uint32_t kTile = (D / 64) * kPanel;     // 128 rows of D
    static constexpr int NS = D == 64 ? 4 : 2;               // stages of K and of V
    static constexpr uint32_t kQ = 0, kK = 2 * kTile, kV = kK + NS * kTile, kBar = kV + NS * kTile;
    // barriers
    static constexpr int bQFull = 0, bQEmpty = 1, bKFull = 2, bKEmpty = bKFull + NS, bVFull = bKEmpty + NS,
                         bVEmpty = bVFull + NS, bS = bVEmpty + NS, bP = bS + 2, bO = bP + 2, bOEmpty = bO + 2, bDrain = bOEmpty + 2,
                         kBars = bDrain + 1;
    static constexpr uint32_t kMisc = kBar + 8 * kBars, kAlloc = kMisc + 16 + 1024;
    static_assert(kAlloc <= 232448, "exceeds the 227 KB of shared memory per CTA");
    // tensor memory columns
    static constexpr uint32_t tS = 0, tO = 256, kCols = 512;
};

constexpr uint32_t kIdS = idesc_bf16(128, 128, 0, 0), kIdSNarrow = idesc_bf16(128, kSinkCols, 0, 0);

// One work item: two query tiles and the key tiles that either sees.
struct Plan {
    long long bos;
    int L, hk;
    int h[2], t0[2], first[2], last[2];
    bool act[2];
    bool sink, narrow;  // the list begins with the sinks' tile; as kSinkCols keys
    int lo, n;          // the first of the other tiles, and the length of the list
    int sinks;
    __device__ __forceinline__ int tile(int i) const { return sink ? (i == 0 ? 0 : lo + i - 1) : lo + i; }
    __device__ __forceinline__ bool small(int i) const { return narrow && i == 0; }
    // whether query tile q looks at place i of the list
    __device__ __forceinline__ bool takes(int q, int i) const {
        const int k = tile(i);
        return act[q] && ((k >= first[q] && k <= last[q]) || (k == 0 && sinks > 0));
    }
    __device__ __forceinline__ int next(int q, int i) const {
        for (++i; i < n; ++i)
            if (takes(q, i)) return i;
        return n;
    }
};

// Items are numbered with a key head's pairs next to each other and late tiles first: under a
// causal mask these are the long ones.
__device__ __forceinline__ bool plan(Plan &u, const WindowParams &p, unsigned item, long long slots) {
    const int G = p.Nq / p.Nk;
    const bool by_head = G % 2 == 0;
    const int pairs = by_head ? G / 2 : G;
    const int pr = item % pairs;
    u.hk = item / pairs % p.Nk;
    const unsigned slot = (unsigned)(slots - 1 - item / pairs / p.Nk);
    const SeqTile s = seq_tile(p.seq, slot, by_head ? 128 : 256);
    if (!s.ok || s.t0 >= s.t1) return false;
    u.bos = s.bos;
    u.L = (int)(s.eos - s.bos);
    u.sinks = p.sinks;
    const Sight sight{p.window, p.sinks};
    const int t0 = (int)(s.t0 - s.bos);
    u.lo = 1 << 30;
    int hi = -1;
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        u.h[q] = u.hk * G + (by_head ? 2 * pr + q : pr);
        u.t0[q] = t0 + (by_head ? 0 : 128 * q);
        u.act[q] = u.t0[q] < u.L;
        const int t1 = u.t0[q] + 128 < u.L ? u.t0[q] + 128 : u.L;
        const KeyTiles kt(u.t0[q], u.act[q] ? t1 : u.t0[q] + 1, 128, sight);
        u.first[q] = kt.first;
        u.last[q] = kt.last;
        if (u.act[q]) {
            u.lo = kt.first < u.lo ? kt.first : u.lo;
            hi = kt.last > hi ? kt.last : hi;
        }
    }
    u.sink = u.lo > 0 && p.sinks > 0;
    u.narrow = u.sink && p.sinks <= kSinkCols;
    u.n = hi - u.lo + 1 + (u.sink ? 1 : 0);
    return true;
}

template <int D>
struct Fwd {
    using Y = Lay<D>;
    Ctx x;
    const WindowParams &p;
    unsigned items;
    long long slots;
    uint32_t tm;

    __device__ __forceinline__ uint32_t bar(int i) const { return x.base + Y::kBar + 8u * i; }

    // ---- TMA ------------------------------------------------------------------
    __device__ void load(const CUtensorMap *mq, const CUtensorMap *mk, const CUtensorMap *mv, const CUtensorMap *mks,
                         const CUtensorMap *mvs) {
        unsigned kv = 0, qn = 0;
        bool fine = true;
        for (unsigned item = blockIdx.x; fine && item < items; item += gridDim.x) {
            Plan u;
            if (!plan(u, p, item, slots)) continue;
            if (!wait(x, bar(Y::bQEmpty), (qn & 1) ^ 1)) break;
            mbar_arrive_expect_tx(bar(Y::bQFull), (u.act[0] + u.act[1]) * Y::kTile);
            for (int q = 0; q < 2; ++q)
                if (u.act[q])
                    for (int c = 0; c < D / 64; ++c)
                        tma_load_3d(x.base + Y::kQ + q * Y::kTile + c * Y::kPanel, mq, bar(Y::bQFull), 64 * c, u.h[q],
                                    (int)(u.bos + u.t0[q]));
            ++qn;
            for (int i = 0; i < u.n; ++i, ++kv) {
                const int s = kv % Y::NS;
                const uint32_t ph = ((kv / Y::NS) & 1) ^ 1;
                const bool small = u.small(i);
                const uint32_t bytes = small ? kSinkCols * D * 2 : Y::kTile;
                const int row = (int)(u.bos + (long long)u.tile(i) * 128);
                if (!(fine = wait(x, bar(Y::bKEmpty + s), ph))) break;
                mbar_arrive_expect_tx(bar(Y::bKFull + s), bytes);
                for (int c = 0; c < D / 64; ++c)
                    tma_load_3d(x.base + Y::kK + s * Y::kTile + c * Y::kPanel, small ? mks : mk, bar(Y::bKFull + s), 64 * c, u.hk, row);
                if (!(fine = wait(x, bar(Y::bVEmpty + s), ph))) {
                    wait_drain(bar(Y::bKFull + s), ph ^ 1);
                    break;
                }
                mbar_arrive_expect_tx(bar(Y::bVFull + s), bytes);
                for (int c = 0; c < D / 64; ++c)
                    tma_load_3d(x.base + Y::kV + s * Y::kTile + c * Y::kPanel, small ? mvs : mv, bar(Y::bVFull + s), 64 * c, u.hk, row);
            }
        }
        // copies still in flight land before the CTA ends
        if (qn) wait_drain(bar(Y::bQFull), (qn - 1) & 1);
        for (unsigned i = kv > Y::NS ? kv - Y::NS : 0; i < kv; ++i) {
            wait_drain(bar(Y::bKFull + i % Y::NS), (i / Y::NS) & 1);
            wait_drain(bar(Y::bVFull + i % Y::NS), (i / Y::NS) & 1);
        }
    }

    // ---- MMA ------------------------------------------------------------------
    __device__ __forceinline__ bool issue_s(const Plan &u, int q, int i, unsigned kv) {
        const unsigned k = kv + i;
        if (!wait(x, bar(Y::bKFull + k % Y::NS), (k / Y::NS) & 1)) return false;
        tc_fence_after();
        const uint32_t a = x.base + Y::kQ + q * Y::kTile, b = x.base + Y::kK + (k % Y::NS) * Y::kTile;
        const uint32_t id = u.small(i) ? kIdSNarrow : kIdS;
#pragma unroll
        for (int c = 0; c < D / 64; ++c)
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
                mma_ss(tm + Y::tS + 128 * q, sdesc(a + c * Y::kPanel + kk * 32, 16, 1024),
                       sdesc(b + c * Y::kPanel + kk * 32, 16, 1024), id, (c | kk) != 0);
        mma_commit(bar(Y::bS + q));
        mma_commit(bar(Y::bKEmpty + k % Y::NS));
        return true;
    }

    __device__ bool mma_item(const Plan &u, unsigned kv, unsigned qn, unsigned (&ns)[2], unsigned (&no)[2]) {
        if (!wait(x, bar(Y::bQFull), qn & 1)) return false;
        int at[2];
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            at[q] = u.next(q, -1);
            if (at[q] < u.n && !issue_s(u, q, at[q], kv)) return false;
        }
        bool first[2] = {true, true}, q_free = false;
        for (int i = 0; i < u.n; ++i) {
            const unsigned k = kv + i;
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                if (at[q] != i) {  // not this one's: its share of the stage is free
                    mbar_arrive(bar(Y::bKEmpty + k % Y::NS));
                    continue;
                }
                if (!wait(x, bar(Y::bVFull + k % Y::NS), (k / Y::NS) & 1)) return false;
                if (first[q] && !wait(x, bar(Y::bOEmpty + q), (no[q] & 1) ^ 1)) return false;
                if (!wait(x, bar(Y::bP + q), ns[q] & 1)) return false;
                ++ns[q];
                tc_fence_after();
                const uint32_t b = x.base + Y::kV + (k % Y::NS) * Y::kTile;
                const int steps = u.small(i) ? kSinkCols / 16 : 8;
                for (int kk = 0; kk < steps; ++kk)
                    mma_ts(tm + Y::tO + D * q, tm + Y::tS + 128 * q + kk * 8, sdesc(b + kk * 2048, Y::kPanel, 1024),
                           idesc_bf16(128, D, 0, 1), !(first[q] && kk == 0));
                first[q] = false;
                at[q] = u.next(q, i);
                if (at[q] < u.n) {
                    if (!issue_s(u, q, at[q], kv)) return false;
                } else {
                    mma_commit(bar(Y::bO + q));
                    ++no[q];
                }
            }
            mma_commit(bar(Y::bVEmpty + k % Y::NS));
            // all scores of the item are issued: Q may change when they are done
            if (!q_free && at[0] >= u.n && at[1] >= u.n) {
                mma_commit(bar(Y::bQEmpty));
                q_free = true;
            }
        }
        return true;
    }

    __device__ void mma() {
        unsigned kv = 0, qn = 0, ns[2] = {0, 0}, no[2] = {0, 0};
        for (unsigned item = blockIdx.x; item < items; item += gridDim.x) {
            Plan u;
            if (!plan(u, p, item, slots)) continue;
            if (!mma_item(u, kv, qn, ns, no)) break;
            kv += u.n;
            ++qn;
        }
        mma_commit(bar(Y::bDrain));
        wait_drain(bar(Y::bDrain), 0);
    }

    // ---- softmax of query tile q ------------------------------------------------
    __device__ void softmax(int q) {
        const int warp = threadIdx.x >> 5, row = threadIdx.x & 127;
        const uint32_t ts = lane_base(tm, warp) + Y::tS + 128 * q, to = lane_base(tm, warp) + Y::tO + D * q;
        const float c = p.scale * kLog2e;
        const Sight sight{p.window, p.sinks};
        unsigned ns = 0, no = 0;
        for (unsigned item = blockIdx.x; item < items; item += gridDim.x) {
            Plan u;
            if (!plan(u, p, item, slots)) continue;
            if (!u.act[q]) continue;
            const int t = u.t0[q] + row;
            float m = -CUDART_INF_F, l = 0.f;  // maximum of the raw scores that O is scaled by; sum of the weights
            bool first = true;
            for (int i = 0; i < u.n; ++i) {
                if (!u.takes(q, i)) continue;
                const int k0 = u.tile(i) * 128;
                if (!wwait(x, bar(Y::bS + q), ns & 1)) return;
                ++ns;
                tc_fence_after();
                uint32_t s[4][32];
                const int parts = u.small(i) ? 1 : 4;
#pragma unroll
                for (int g = 0; g < 4; ++g)
                    if (g < parts) tmem_ld32(ts + 32 * g, s[g]);
                tmem_wait_ld();
#pragma unroll
                for (int g = 0; g < 4; ++g) tmem_ld_dep(s[g]);
                // some row of the tile does not see some key of it
                const bool edge = k0 + 127 > u.t0[q] || u.t0[q] + 127 - k0 >= p.window;
                float top = -CUDART_INF_F;
#pragma unroll
                for (int g = 0; g < 4; ++g)
                    if (g < parts) {
                        if (edge) {
                            const uint32_t mask = seen32(t, k0 + 32 * g, sight);
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                s[g][e] = mask >> e & 1 ? s[g][e] : 0xff800000u;
                        }
#pragma unroll
                        for (int e = 0; e < 32; e += 2)
                            top = fmaxf(top, fmaxf(__uint_as_float(s[g][e]), __uint_as_float(s[g][e + 1])));
                    }
                if ((top - m) * c > 8.f || m == -CUDART_INF_F) {
                    const float f = ex2((m - top) * c);  // 0 where there was no maximum
                    const bool scale = !first && m != -CUDART_INF_F;
                    m = top;
                    if (scale) l *= f;
                    top = scale ? f : 1.f;
                } else {
                    top = 1.f;
                }
                if (__any_sync(0xffffffffu, top != 1.f)) {
#pragma unroll
                    for (int g = 0; g < D / 16; ++g) {
                        uint32_t o[16];
                        tmem_ld16(to + 16 * g, o);
                        tmem_wait_ld_dep16(o);
#pragma unroll
                        for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * top);
                        tmem_st16(to + 16 * g, o);
                    }
                }
                first = false;
                const float mc = m == -CUDART_INF_F ? 0.f : -m * c;
                const f2 cc = both(c), mm = both(mc);
                f2 sum[2] = {0ull, 0ull};
#pragma unroll
                for (int g = 0; g < 4; ++g)
                    if (g < parts) {
                        uint32_t w[16];
#pragma unroll
                        for (int e = 0; e < 32; e += 2) {
                            float a, b;
                            split(fma2(pair(__uint_as_float(s[g][e]), __uint_as_float(s[g][e + 1])), cc, mm), a, b);
                            a = ex2(a);
                            b = ex2(b);
                            sum[(e >> 1) & 1] = add2(sum[(e >> 1) & 1], pair(a, b));
                            w[e / 2] = pack_bf16(a, b);
                        }
                        tmem_st16(ts + 16 * g, w);
                    }
                l += sum_of(add2(sum[0], sum[1]));
                tmem_wait_st();
                tc_fence_before();
                warp_arrive(bar(Y::bP + q));
            }
            if (!wwait(x, bar(Y::bO + q), no & 1)) return;
            ++no;
            tc_fence_after();
            const float f = 1.f / l;
            bool nan = false;
            __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(p.o) + ((u.bos + t) * p.Nq + u.h[q]) * D;
#pragma unroll
            for (int g = 0; g < D / 64; ++g) {
                uint32_t o[2][32];
                tmem_ld32(to + 64 * g, o[0]);
                tmem_ld32(to + 64 * g + 32, o[1]);
                tmem_wait_ld();
                tmem_ld_dep(o[0]);
                tmem_ld_dep(o[1]);
                if (g + 1 == D / 64) {  // all of O is read
                    tc_fence_before();
                    warp_arrive(bar(Y::bOEmpty + q));
                }
#pragma unroll
                for (int h = 0; h < 4; ++h) {
                    uint32_t w[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float a = __uint_as_float(o[h / 2][(h & 1) * 16 + 2 * e]) * f;
                        const float b = __uint_as_float(o[h / 2][(h & 1) * 16 + 2 * e + 1]) * f;
                        nan |= isnan(a) | isnan(b);
                        w[e] = pack_bf16(a, b);
                    }
                    if (t < u.L) store32(out + 64 * g + 16 * h, w);
                }
            }
            if (t < u.L) p.lse[(u.bos + t) * p.Nq + u.h[q]] = nan ? redo_mark() : m * p.scale + log2f(l) * 0.6931471805599453f;
        }
    }
};

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
window_fwd(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv,
           const __grid_constant__ CUtensorMap mks, const __grid_constant__ CUtensorMap mvs, const __grid_constant__ WindowParams p,
           unsigned items, long long slots) {
    using Y = Lay<D>;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    Ctx x;
    x.base = (raw + 1023u) & ~1023u;
    x.gbase = smem_raw + (x.base - raw);
    x.abort_flag = reinterpret_cast<volatile int *>(x.gbase + Y::kMisc + 4);
    x.status = p.seq.status;
    const int warp = threadIdx.x >> 5;
    auto bar = [&](int i) { return x.base + Y::kBar + 8u * i; };
    if (threadIdx.x == 0) {
        mbar_init(bar(Y::bQFull), 1);
        mbar_init(bar(Y::bQEmpty), 1);
        for (int s = 0; s < Y::NS; ++s) {
            mbar_init(bar(Y::bKFull + s), 1);
            mbar_init(bar(Y::bKEmpty + s), 2);  // both query tiles
            mbar_init(bar(Y::bVFull + s), 1);
            mbar_init(bar(Y::bVEmpty + s), 1);
        }
        for (int q = 0; q < 2; ++q) {
            mbar_init(bar(Y::bS + q), 1);
            mbar_init(bar(Y::bP + q), 4);
            mbar_init(bar(Y::bO + q), 1);
            mbar_init(bar(Y::bOEmpty + q), 4);
        }
        mbar_init(bar(Y::bDrain), 1);
        *x.abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == 9) {
        tmem_alloc(x.base + Y::kMisc, Y::kCols);
        tmem_relinquish();
    }
    fence_proxy_async_smem();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    Fwd<D> f{x, p, items, slots, *reinterpret_cast<volatile uint32_t *>(x.gbase + Y::kMisc)};
    wait_for_launches();
    if (warp == 8) {
        if (blockIdx.x == 0) check_offsets(p.seq, threadIdx.x & 31, 32);
        __syncwarp();
        if ((threadIdx.x & 31) == 0) f.load(&mq, &mk, &mv, &mks, &mvs);
        __syncwarp();
    } else if (warp == 9) {
        if ((threadIdx.x & 31) == 0) f.mma();
        __syncwarp();
    } else {
        f.softmax(warp >> 2);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 9) tmem_dealloc(f.tm, Y::kCols);
}

template <int D>
cudaError_t launch(const WindowParams &p, cudaStream_t stream) {
    const int G = p.Nq / p.Nk;
    const long long slots = tile_slots(p.seq, G % 2 == 0 ? 128 : 256);
    const long long items = slots * p.Nk * (G % 2 == 0 ? G / 2 : G);
    if (items <= 0) return cudaSuccess;
    if (items > 0x7fffffffll) return cudaErrorInvalidValue;
    CUtensorMap mq, mk, mv, mks, mvs;
    const uint64_t tokens = (uint64_t)p.seq.tokens;
    if (!make_tmap_rows_heads_d(&mq, p.q, tokens, p.Nq, D, 64, 128) || !make_tmap_rows_heads_d(&mk, p.k, tokens, p.Nk, D, 64, 128) ||
        !make_tmap_rows_heads_d(&mv, p.v, tokens, p.Nk, D, 64, 128) || !make_tmap_rows_heads_d(&mks, p.k, tokens, p.Nk, D, 64, kSinkCols) ||
        !make_tmap_rows_heads_d(&mvs, p.v, tokens, p.Nk, D, 64, kSinkCols))
        return cudaErrorInvalidValue;
    const cudaError_t err = allow_smem<window_fwd<D>>((int)Lay<D>::kAlloc);
    if (err != cudaSuccess) return err;
    const unsigned grid = (unsigned)(items < kSms ? items : kSms);
    return launch_after(window_fwd<D>, dim3(grid), dim3(kThreads), Lay<D>::kAlloc, stream, mq, mk, mv, mks, mvs, p, (unsigned)items, slots);
}

}  // namespace

cudaError_t window_tc_fwd(const WindowParams &p, cudaStream_t stream) {
    return p.d == 64 ? launch<64>(p, stream) : launch<128>(p, stream);
}

}  // namespace dn
