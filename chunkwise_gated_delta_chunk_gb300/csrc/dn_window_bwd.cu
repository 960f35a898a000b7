// Attention over a sliding window with sinks, backward, bf16: tcgen05 / TMEM / TMA.
//
//     p = e^{scale q . k - lse},  dp = do . v,  ds = p (dp - D),  D = sum do o
//     dq = scale ds k     (window_dq:  tiles of 128 queries, one head; keys stream by)
//     dk = scale ds^T q,  dv = p^T do   (window_dkv: tiles of 128 keys, one key head; the
//                                        group's heads' queries and do stream by)
//
// p and ds are rounded to bf16 for their products, by half a step of each; D and the recomputed weights are fp32.
//
// Two kernels, so that no sum is added by atomics: every sum stays in tensor memory until it is
// done, in a fixed order, for 8 products of 128 x 128 x d a tile instead of 5.
//
// D.  Taken from the rounded o it is off by about half a step of a bf16 of its terms, which at windows
// of a few keys is more than the roundings of p and ds make (dq and dk 1.5 to 2.7 times as far off
// as rounding the result alone; 1.42 with an exact D).  So a first pass over o and do (window_dsum) gives
// an approximate D', and window_dq sums the exact D = sum p dp of its rows beside its products, along with
// C = sum p k:
//     dq = scale (sum p (dp - D') k + (D' - D) C)
// and leaves D for window_dkv.
//
// Warps 0-3 and 4-7: the first and the second 64 columns of every tile of scores, one row a
// thread; warp 8: TMA loads, and the plans of the items; warp 9: the MMAs; warp 10 (window_dkv): the
// columns' lse and D into shared memory.
//
// Tensor memory: S and dP of a tile (128 columns each; P and dS overwrite the first half of each half of
// them as bf16), and two accumulators of d columns.  The products alternate with the threads' work on the
// other matrix:
//     threads   P(n)        dS(n)                     P(n+1)
//     MMAs      ...         C(n) or dV(n), S(n+1)     dQ(n) or dK(n), dP(n+1)
// (window_dkv has the transposed tiles: rows are keys.)
//
// All queries see the sinks.  Query tiles behind the window of the first key tile are taken
// in parts (a run of part_tiles tiles each) by items of their own, which leave fp32 sums of
// the sinks' rows; window_sink_sums (dn_window.cu) adds them up in order.
//
// Measured (4 x 2048 tokens, window 512, 16 heads of 128 columns): window_dsum 12 us, window_dq 78, window_dkv 80, the
// tensor pipe at work 45 to 49 % of the time.  Bound by the threads' phases and the products taking turns, and by the
// accumulators' way out between items, when the tensor cores wait.
#include "dn_window_tc.cuh"

namespace dn {
namespace {

using namespace ptx;
using namespace tcs;

constexpr int kThreads = 352;
constexpr uint32_t kPanel = 128 * 128;  // 128 rows of 64 columns of bf16

constexpr int kPlans = 4;  // items whose plans are kept

// Shared memory of both kernels: two tiles that stay, and two rings of tiles that stream by, NX and NY
// deep, each freed as soon as its own last reader is done.  window_dq: keys (read until dQ of their tile) and
// values (until dP).  window_dkv: q (until dK) and do (until dV).
template <int D, bool DQ>
struct Lay {
    static constexpr uint32_t kTile = (D / 64) * kPanel;
    static constexpr int NX = DQ ? (D == 64 ? 6 : 3) : (D == 64 ? 4 : 2), NY = D == 64 ? 4 : 2;
    static constexpr uint32_t kA = 0, kB = kTile, kX = 2 * kTile, kY = kX + NX * kTile, kEnd = kY + NY * kTile;
    static constexpr uint32_t kCols = kEnd;  // window_dkv: lse and D of the queries
    static constexpr uint32_t kPlan = kCols + (DQ ? 0 : NX * 1024), kBar = kPlan + kPlans * 64;
    static constexpr int bHold = 0, bHoldEmpty = 1, bX = 2, bXEmpty = bX + NX, bY = bXEmpty + NX, bYEmpty = bY + NY, bCol = bYEmpty + NY,
                         bS = bCol + NX, bDP = bS + 1, bP = bDP + 1, bDS = bP + 1, bOut = bDS + 1, bOutEmpty = bOut + 1,
                         bPlan = bOutEmpty + 1, bDrain = bPlan + kPlans, bPair = bDrain + 1, bTaken = bPair + 4, bItem = bTaken + 4, kBars = bItem + 1;
    static constexpr uint32_t kBox = (kBar + 8 * kBars + 15) / 16 * 16, kMisc = kBox + (DQ ? 2 * 128 * 4 : 0), kAlloc = kMisc + 32 + 1024;
    static_assert(kAlloc <= 232448, "exceeds the 227 KB of shared memory per CTA");
};

template <int D, bool DQ, typename Plan>
struct Base {
    using Y = Lay<D, DQ>;
    static_assert(sizeof(Plan) <= 64, "a plan's place in shared memory");
    Ctx x;
    const WindowParams &p;
    uint32_t tm;
    __device__ __forceinline__ uint32_t bar(int i) const { return x.base + Y::kBar + 8u * i; }

    __device__ __forceinline__ Items items() const { return Items{bar(Y::bItem), x.base + Y::kMisc + 16}; }
    // The TMA warp works out the plans and leaves the n-th item's in shared memory: when all scores of
    // item n - 1 are done, and every other warp is past item n - 4, whose place it takes.  A plan of
    // no rounds: no item is left.
    __device__ __forceinline__ void put_plan(const Plan &u, unsigned n) const {
        *reinterpret_cast<Plan *>(x.gbase + Y::kPlan + n % kPlans * 64) = u;
        mbar_arrive(bar(Y::bPlan + n % kPlans));
    }
    __device__ __forceinline__ bool next_plan(Plan &u, unsigned n) const {
        if (!hold(x, bar(Y::bPlan + n % kPlans), n / kPlans & 1)) return false;
        u = *reinterpret_cast<const Plan *>(x.gbase + Y::kPlan + n % kPlans * 64);
        return u.rounds > 0;
    }
    // use k of a ring of N: whether its tile has landed; whether its place is free
    __device__ __forceinline__ bool full_x(unsigned k) const { return hold(x, bar(Y::bX + k % Y::NX), (k / Y::NX) & 1); }
    __device__ __forceinline__ bool full_y(unsigned k) const { return hold(x, bar(Y::bY + k % Y::NY), (k / Y::NY) & 1); }
    __device__ __forceinline__ bool free_x(unsigned k) const { return wait(x, bar(Y::bXEmpty + k % Y::NX), ((k / Y::NX) & 1) ^ 1); }
    __device__ __forceinline__ bool free_y(unsigned k) const { return wait(x, bar(Y::bYEmpty + k % Y::NY), ((k / Y::NY) & 1) ^ 1); }
    static __device__ __forceinline__ uint32_t at_x(unsigned k) { return Y::kX + k % Y::NX * Y::kTile; }
    static __device__ __forceinline__ uint32_t at_y(unsigned k) { return Y::kY + k % Y::NY * Y::kTile; }
    // Copies still in flight land before the CTA ends: uses up to k of both rings.
    __device__ __forceinline__ void drain(unsigned kx, unsigned ky, unsigned holds) const {
        if (holds) wait_drain(bar(Y::bHold), (holds - 1) & 1);
        for (unsigned i = kx > Y::NX ? kx - Y::NX : 0; i < kx; ++i) wait_drain(bar(Y::bX + i % Y::NX), (i / Y::NX) & 1);
        for (unsigned i = ky > Y::NY ? ky - Y::NY : 0; i < ky; ++i) wait_drain(bar(Y::bY + i % Y::NY), (i / Y::NY) & 1);
    }
    // rows of 128 x D by panels
    __device__ __forceinline__ void tma_tile(uint32_t at, const CUtensorMap *m, uint32_t b, int head, int row) const {
        for (int c = 0; c < D / 64; ++c) tma_load_3d(x.base + at + c * kPanel, m, b, 64 * c, head, row);
    }
    // C[128 x n] = A[128 x D] B[n x D]^T, both rows in shared memory
    __device__ __forceinline__ void mma_rows(uint32_t lead, uint32_t c, uint32_t at_a, uint32_t at_b, uint32_t id) const {
        const uint32_t a = rows_of(x.base + at_a), b = rows_of(x.base + at_b);
#pragma unroll
        for (int s = 0; s < D / 64; ++s)
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
                mma_ss_by(lead, tm + c, a + (s * kPanel + kk * 32) / 16, b + (s * kPanel + kk * 32) / 16, id, (s | kk) != 0);
    }
    // the warp's byte in the mark of its half of the rows (two warps of each column half)
    __device__ __forceinline__ void mark(bool nan, long long flag) const {
        const int warp = threadIdx.x >> 5;
        nan = __any_sync(0xffffffffu, nan);
        unsigned char *m = reinterpret_cast<unsigned char *>(p.redo + flag + (warp >> 1 & 1) * (p.Nq + p.Nk));
        if ((threadIdx.x & 31) == 0) m[2 * (warp >> 2) + (warp & 1)] = nan;
    }
    // N columns of an accumulator times f, to bf16; true where one of the lane's row is not finite.  `to`: the
    // lane's row, of a tensor with `stride` elements from row to row; of the warp's 32 rows those from
    // from_row up to rows are written.
    // ADD: plus f2nd times the accumulator at `second`.
    template <int N, bool ADD = false>
    __device__ __forceinline__ bool store_cols(uint32_t from, __nv_bfloat16 *to, long long stride, int from_row, int rows, float f,
                                               uint32_t second = 0, float f2nd = 0.f) const {
        f2 bad = 0ull;
        const f2 ff = both(f);
#pragma unroll 1
        for (int c = 0; c < N; c += 64) {
            uint32_t w[4][8];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint32_t o[32], a[ADD ? 32 : 1];
                tmem_ld32(from + c + 32 * h, o);
                if constexpr (ADD) tmem_ld32(second + c + 32 * h, a);
                tmem_wait_ld();
                tmem_ld_dep(o);
                if constexpr (ADD) tmem_ld_dep(a);
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    f2 v = mul2(pair(__uint_as_float(o[2 * e]), __uint_as_float(o[2 * e + 1])), ff);
                    if constexpr (ADD) v = fma2(pair(__uint_as_float(a[2 * e]), __uint_as_float(a[2 * e + 1])), both(f2nd), v);
                    bad = fma2(v, 0ull, bad);  // 0 times infinity or NaN stays
                    float lo, hi;
                    split(v, lo, hi);
                    w[2 * h + (e >> 3)][e & 7] = pack_bf16(lo, hi);
                }
            }
            store_rows<64>(to + c, stride, from_row, rows, w);
        }
        const int r = threadIdx.x & 31;
        return isnan(sum_of(bad)) && r >= from_row && r < rows;
    }
};

struct QueryPlan {
    long long bos, flag;
    int L, h, hk, t0, rounds;
    KeyTiles kt;
    bool narrow;
    __device__ __forceinline__ bool small(int i) const { return narrow && i == 0; }
};

template <int D>
struct Dq : Base<D, true, QueryPlan> {
    using B = Base<D, true, QueryPlan>;
    using Y = typename B::Y;
    using Plan = QueryPlan;
    using B::bar;
    using B::p;
    using B::tm;
    using B::x;
    long long slots;
    static constexpr uint32_t tS = 0, tDP = 128, tDQ = 256, tC = 384;

    // late tiles first
    __device__ __forceinline__ bool plan(Plan &u, unsigned item) const {
        u.h = item % p.Nq;
        const unsigned slot = slot_in_order(p.seq, item / p.Nq, (unsigned)slots, false);
        u.flag = (long long)slot * 2 * (p.Nq + p.Nk) + u.h;
        const SeqTile s = seq_tile(p.seq, slot, 128);
        if (!s.ok || s.t0 >= s.t1) return false;
        u.bos = s.bos;
        u.L = (int)(s.eos - s.bos);
        u.hk = u.h / (p.Nq / p.Nk);
        u.t0 = (int)(s.t0 - s.bos);
        u.kt = KeyTiles(u.t0, (int)(s.t1 - s.bos), 128, Sight{p.window, p.sinks});
        u.narrow = u.kt.sink_end > 0 && p.sinks <= kSinkCols;
        u.rounds = u.kt.count();
        return true;
    }

    __device__ void load(const CUtensorMap *mq, const CUtensorMap *mg, const CUtensorMap *mk, const CUtensorMap *mv,
                         const CUtensorMap *mks, const CUtensorMap *mvs) {
        unsigned kx = 0, ky = 0, qn = 0;
        bool fine = true;
        Items next = B::items();
        for (; fine; fine = fine && next.next(x)) {
            Plan u;
            if (!next.any) {
                u.rounds = 0;
            } else if (!plan(u, next.item)) {
                p.redo[u.flag] = p.redo[u.flag + (p.Nq + p.Nk)] = 0;  // no tile there
                continue;
            }
            if (!(fine = wait(x, bar(Y::bHoldEmpty), (qn & 1) ^ 1))) break;
            B::put_plan(u, qn);
            if (u.rounds == 0) break;
            mbar_arrive_expect_tx(bar(Y::bHold), 2 * Y::kTile);
            B::tma_tile(Y::kA, mq, bar(Y::bHold), u.h, (int)(u.bos + u.t0));
            B::tma_tile(Y::kB, mg, bar(Y::bHold), u.h, (int)(u.bos + u.t0));
            ++qn;
            for (int i = 0; i < u.rounds; ++i) {
                const int row = (int)(u.bos + (long long)u.kt.tile(i) * 128);
                const uint32_t bytes = u.small(i) ? kSinkCols * D * 2 : Y::kTile;
                if (i + 2 >= u.rounds) next.ask();
                if (!(fine = B::free_x(kx))) break;
                mbar_arrive_expect_tx(bar(Y::bX + kx % Y::NX), bytes);
                B::tma_tile(B::at_x(kx), u.small(i) ? mks : mk, bar(Y::bX + kx % Y::NX), u.hk, row);
                ++kx;
                if (!(fine = B::free_y(ky))) break;
                mbar_arrive_expect_tx(bar(Y::bY + ky % Y::NY), bytes);
                B::tma_tile(B::at_y(ky), u.small(i) ? mvs : mv, bar(Y::bY + ky % Y::NY), u.hk, row);
                ++ky;
            }
        }
        next.drain();
        B::drain(kx, ky, qn);
    }

    __device__ __forceinline__ bool issue_s(uint32_t lead, bool small, unsigned k) const {
        if (!B::full_x(k)) return false;
        tc_fence_after();
        B::mma_rows(lead, tS, Y::kA, B::at_x(k), small ? idesc_bf16(128, kSinkCols, 0, 0) : idesc_bf16(128, 128, 0, 0));
        commit_by(lead, bar(Y::bS));
        return true;
    }
    __device__ __forceinline__ bool issue_dp(uint32_t lead, bool small, unsigned k) const {
        if (!B::full_y(k)) return false;
        tc_fence_after();
        B::mma_rows(lead, tDP, Y::kB, B::at_y(k), small ? idesc_bf16(128, kSinkCols, 0, 0) : idesc_bf16(128, 128, 0, 0));
        commit_by(lead, bar(Y::bDP));
        commit_by(lead, bar(Y::bYEmpty + k % Y::NY));
        return true;
    }
    // acc += a K, the bf16 halves of a 64 columns apart
    __device__ __forceinline__ void issue_acc(uint32_t lead, uint32_t acc, uint32_t a, unsigned k, bool small, bool more) const {
        const uint32_t b = cols_of(x.base + B::at_x(k));
        constexpr uint32_t id = idesc_bf16(128, D, 0, 1);
        mma_ts_by(lead, tm + acc, tm + a, b, id, more);
        mma_ts_by(lead, tm + acc, tm + a + 8, b + 128, id, 1);
        if (!small)
#pragma unroll
            for (int kk = 2; kk < 8; ++kk) mma_ts_by(lead, tm + acc, tm + a + 64 * (kk >> 2) + 8 * (kk & 3), b + 128 * kk, id, 1);
    }

    __device__ void mma() {
        const uint32_t lead = elect();
        unsigned k = 0, qn = 0;
        bool fine = true;
        Plan u;
        for (; fine && B::next_plan(u, qn); ++qn) {
            const int n = u.rounds;
            if (!(fine = hold(x, bar(Y::bHold), qn & 1) && issue_s(lead, u.small(0), k) && issue_dp(lead, u.small(0), k))) break;
            if (n == 1) commit_by(lead, bar(Y::bHoldEmpty));
            if (!(fine = hold(x, bar(Y::bOutEmpty), (qn & 1) ^ 1))) break;
#pragma unroll 1
            for (int i = 0; i < n; ++i, ++k) {
                const bool small = u.small(i);
                if (!(fine = hold(x, bar(Y::bP), k & 1))) break;
                tc_fence_after();
                issue_acc(lead, tC, tS, k, small, i > 0);
                if (i + 1 < n && !(fine = issue_s(lead, false, k + 1))) break;
                if (!(fine = hold(x, bar(Y::bDS), k & 1))) break;
                tc_fence_after();
                issue_acc(lead, tDQ, tDP, k, small, i > 0);
                commit_by(lead, bar(Y::bXEmpty + k % Y::NX));
                if (i + 1 < n) {
                    if (!(fine = issue_dp(lead, false, k + 1))) break;
                    if (i + 2 == n) commit_by(lead, bar(Y::bHoldEmpty));  // the last that read q and do
                } else {
                    commit_by(lead, bar(Y::bOut));
                }
            }
        }
        commit_by(lead, bar(Y::bDrain));
        wait_drain(bar(Y::bDrain), 0);
    }

    __device__ void threads() {
        const int warp = threadIdx.x >> 5, row = threadIdx.x & 127, w = warp >> 2;
        const uint32_t lane = lane_base(tm, warp);
        const float c = p.scale * kLog2e;
        const Sight sight{p.window, p.sinks};
        unsigned k = 0, qn = 0;
        Plan u;
        for (; B::next_plan(u, qn); ++qn) {
            const int t = u.t0 + row;
            const bool live = t < u.L;
            const long long at = (u.bos + t) * p.Nq + u.h;
            const float lse2 = live ? p.lse[at] * kLog2e : 0.f;
            const float dsum = live ? p.dsum[at] : 0.f;
            const f2 cc = both(c), ll = both(-lse2), dd = both(-dsum);
            f2 exact = 0ull;  // this thread's part of sum p dp
            for (int i = 0; i < u.rounds; ++i, ++k) {
                const int k0 = u.kt.tile(i) * 128 + 64 * w;
                const int cols = u.small(i) ? (w == 0 ? 1 : 0) : 2;  // groups of 32 columns
                const bool edge = k0 + 63 > u.t0 || u.t0 + 127 - k0 >= p.window;
                if (!hold(x, bar(Y::bS), k & 1)) return;
                tc_fence_after();
                uint32_t s[2][32];
#pragma unroll
                for (int q = 0; q < 2; ++q)
                    if (q < cols) tmem_ld32(lane + tS + 64 * w + 32 * q, s[q]);
                tmem_wait_ld();
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    tmem_ld_dep(s[q]);
                    if (q >= cols) continue;
                    const uint32_t mask = edge ? seen32(t, k0 + 32 * q, sight) : 0xffffffffu;
                    uint32_t v[16];
#pragma unroll
                    for (int e = 0; e < 32; e += 2) {
                        float a, b;
                        split(fma2(pair(__uint_as_float(s[q][e]), __uint_as_float(s[q][e + 1])), cc, ll), a, b);
                        a = ex2(a);
                        b = ex2(b);
                        if (edge) {
                            a = mask >> e & 1 ? a : 0.f;
                            b = mask >> (e + 1) & 1 ? b : 0.f;
                        }
                        s[q][e] = __float_as_uint(a);
                        s[q][e + 1] = __float_as_uint(b);
                        v[e / 2] = pack_bf16(a, b);
                    }
                    tmem_st16(lane + tS + 64 * w + 16 * q, v);
                }
                tmem_wait_st();
                tc_fence_before();
                warp_arrive(bar(Y::bP));
                if (!hold(x, bar(Y::bDP), k & 1)) return;
                tc_fence_after();
#pragma unroll
                for (int q = 0; q < 2; ++q) {  // one after the other: both do not fit beside p
                    if (q >= cols) continue;
                    uint32_t g[32], v[16];
                    tmem_ld32(lane + tDP + 64 * w + 32 * q, g);
                    tmem_wait_ld_dep(g);
                    if (edge) {  // a masked value may be anything
                        const uint32_t mask = seen32(t, k0 + 32 * q, sight);
#pragma unroll
                        for (int e = 0; e < 32; ++e) g[e] = mask >> e & 1 ? g[e] : 0u;
                    }
#pragma unroll
                    for (int e = 0; e < 32; e += 2) {
                        const f2 w2 = pair(__uint_as_float(s[q][e]), __uint_as_float(s[q][e + 1]));
                        const f2 dp = pair(__uint_as_float(g[e]), __uint_as_float(g[e + 1]));
                        exact = fma2(w2, dp, exact);
                        float a, b;
                        split(mul2(w2, add2(dp, dd)), a, b);
                        v[e / 2] = pack_bf16(a, b);
                    }
                    tmem_st16(lane + tDP + 64 * w + 16 * q, v);
                }
                tmem_wait_st();
                tc_fence_before();
                warp_arrive(bar(Y::bDS));
            }
            // D of the row from its two threads
            volatile float *box = reinterpret_cast<float *>(x.gbase + Y::kBox) + row;
            const float mine = sum_of(exact);
            if (!hold(x, bar(Y::bTaken + (warp & 3)), (qn & 1) ^ 1)) return;  // the last ones are read
            box[128 * w] = mine;
            warp_arrive(bar(Y::bPair + (warp & 3)));
            if (!hold(x, bar(Y::bPair + (warp & 3)), qn & 1)) return;
            const float full = mine + box[128 * (w ^ 1)];
            warp_arrive(bar(Y::bTaken + (warp & 3)));
            if (w == 0 && live) p.dsum[at] = full;
            if (!hold(x, bar(Y::bOut), qn & 1)) return;
            tc_fence_after();
            bool nan = false;
            if (D == 128 || w == 0) {
                const float off = dsum - full;
                nan = B::template store_cols<64, true>(lane + tDQ + 64 * w, static_cast<__nv_bfloat16 *>(p.dq) + at * D + 64 * w,
                                                       (long long)p.Nq * D, 0, u.L - (t & ~31), p.scale, lane + tC + 64 * w, off * p.scale);
            }
            tc_fence_before();
            warp_arrive(bar(Y::bOutEmpty));
            B::mark(nan, u.flag);
        }
    }
};

// ---- dk and dv ------------------------------------------------------------------

// Items: (parts) a run of query tiles that see the sinks of a sequence alone; then a key tile of 128 tokens and a
// key head.
struct KeyPlan {
    long long bos, flag;
    long long place;   // of the sinks' rows of this item among the parts
    int L, hk, k0, first, tiles, rounds;  // query tiles [first, first + tiles) of each of the group's heads
    bool part, split;  // split: the sinks' rows are summed over parts
};

struct Parts {  // how the query tiles behind the window are cut
    long long slots;  // of part_tiles x 128 tokens
    int tiles;
};

__device__ __forceinline__ bool key_plan(KeyPlan &u, const WindowParams &p, long long slots, const Parts &parts, unsigned item) {
    const Sight sight{p.window, p.sinks};
    // the parts first: they are long
    const unsigned part_items = (unsigned)(parts.slots * p.Nk);
    u.hk = item % p.Nk;
    u.part = item < part_items;
    const unsigned slot = u.part ? item / p.Nk : slot_in_order(p.seq, (item - part_items) / p.Nk, (unsigned)slots, true);
    u.flag = (long long)slot * 2 * (p.Nq + p.Nk) + p.Nq + u.hk;
    const SeqTile s = seq_tile(p.seq, slot, u.part ? parts.tiles * 128 : 128);
    if (!s.ok || s.t0 >= s.t1) return false;
    u.bos = s.bos;
    u.L = (int)(s.eos - s.bos);
    u.k0 = u.part ? 0 : (int)(s.t0 - s.bos);
    const QueryTiles qt(u.k0, u.k0 + 128 < u.L ? u.k0 + 128 : u.L, u.L, 128, sight);
    u.split = u.k0 < p.sinks && qt.end > qt.last;
    if (u.part) {
        const int from = s.c * parts.tiles, to = (int)(s.t1 - s.bos - 1) / 128;
        u.first = from > qt.last + 1 ? from : qt.last + 1;
        u.tiles = to - u.first + 1;
        u.place = slot;
        u.rounds = u.tiles * (p.Nq / p.Nk);
        return u.split && u.tiles > 0;
    }
    u.first = qt.first;
    u.tiles = qt.last - qt.first + 1;
    u.place = parts.slots + s.n;
    u.rounds = u.tiles * (p.Nq / p.Nk);
    return true;
}

template <int D>
struct Dkv : Base<D, false, KeyPlan> {
    using B = Base<D, false, KeyPlan>;
    using Y = typename B::Y;
    using B::bar;
    using B::p;
    using B::tm;
    using B::x;
    long long slots;
    Parts parts;
    static constexpr uint32_t tS = 0, tDP = 128, tDV = 256, tDK = 384;

    // The rounds of an item: its query tiles for the first of the group's heads, then the next one.
    struct Round {
        int h, tile, left;
        __device__ __forceinline__ Round(const KeyPlan &u, int G) : h(u.hk * G), tile(u.first), left(u.tiles) {}
        __device__ __forceinline__ void step(const KeyPlan &u) {
            ++tile;
            if (--left == 0) {
                ++h;
                tile = u.first;
                left = u.tiles;
            }
        }
    };

    __device__ void load(const CUtensorMap *mq, const CUtensorMap *mg, const CUtensorMap *mk, const CUtensorMap *mv) {
        unsigned kx = 0, ky = 0, kn = 0;
        bool fine = true;
        Items next = B::items();
        for (; fine; fine = fine && next.next(x)) {
            KeyPlan u;
            if (!next.any) {
                u.rounds = 0;
            } else if (!key_plan(u, p, slots, parts, next.item)) {
                if (!u.part) p.redo[u.flag] = p.redo[u.flag + (p.Nq + p.Nk)] = 0;  // no tile there
                continue;
            }
            if (!(fine = wait(x, bar(Y::bHoldEmpty), (kn & 1) ^ 1))) break;
            B::put_plan(u, kn);
            if (u.rounds == 0) break;
            mbar_arrive_expect_tx(bar(Y::bHold), 2 * Y::kTile);
            B::tma_tile(Y::kA, mk, bar(Y::bHold), u.hk, (int)(u.bos + u.k0));
            B::tma_tile(Y::kB, mv, bar(Y::bHold), u.hk, (int)(u.bos + u.k0));
            ++kn;
            Round r(u, p.Nq / p.Nk);
            for (int i = 0; i < u.rounds; ++i, r.step(u)) {
                const int row = (int)(u.bos + r.tile * 128);
                if (i + 2 >= u.rounds) next.ask();
                if (!(fine = B::free_x(kx))) break;
                mbar_arrive_expect_tx(bar(Y::bX + kx % Y::NX), Y::kTile);
                B::tma_tile(B::at_x(kx), mq, bar(Y::bX + kx % Y::NX), r.h, row);
                ++kx;
                if (!(fine = B::free_y(ky))) break;
                mbar_arrive_expect_tx(bar(Y::bY + ky % Y::NY), Y::kTile);
                B::tma_tile(B::at_y(ky), mg, bar(Y::bY + ky % Y::NY), r.h, row);
                ++ky;
            }
        }
        next.drain();
        B::drain(kx, ky, kn);
    }

    // lse (times log2 e) and D of the streamed queries, a stage ahead like their tiles
    __device__ void columns() {
        const int lane = threadIdx.x & 31;
        unsigned qs = 0, kn = 0;
        KeyPlan u;
        for (; B::next_plan(u, kn); ++kn) {
            Round r(u, p.Nq / p.Nk);
            for (int i = 0; i < u.rounds; ++i, ++qs, r.step(u)) {
                const int s = qs % Y::NX;
                float a[4], b[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int t = r.tile * 128 + lane + 32 * e;
                    const long long at = (u.bos + t) * p.Nq + r.h;
                    a[e] = t < u.L ? -p.lse[at] * kLog2e : 0.f;
                    b[e] = t < u.L ? -p.dsum[at] : 0.f;
                }
                if (!hold(x, bar(Y::bXEmpty + s), ((qs / Y::NX) & 1) ^ 1)) return;
                float *to = reinterpret_cast<float *>(x.gbase + Y::kCols + s * 1024);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    to[lane + 32 * e] = a[e];
                    to[128 + lane + 32 * e] = b[e];
                }
                warp_arrive(bar(Y::bCol + s));
            }
        }
    }

    __device__ __forceinline__ void mma_acc(uint32_t lead, uint32_t acc, uint32_t a, uint32_t at_b, bool more) const {
        const uint32_t b = cols_of(x.base + at_b);
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)  // the two halves of the queries lie 64 columns apart
            mma_ts_by(lead, tm + acc, tm + a + 64 * (kk >> 2) + 8 * (kk & 3), b + 128 * kk, idesc_bf16(128, D, 0, 1), more || kk != 0);
    }

    __device__ void mma() {
        constexpr uint32_t id = idesc_bf16(128, 128, 0, 0);
        const uint32_t lead = elect();
        unsigned k = 0, kn = 0;
        bool fine = true;
        KeyPlan u;
        for (; fine && B::next_plan(u, kn); ++kn) {
            const int n = u.rounds;
            if (!(fine = hold(x, bar(Y::bHold), kn & 1) && B::full_x(k))) break;
            tc_fence_after();
            B::mma_rows(lead, tS, Y::kA, B::at_x(k), id);
            commit_by(lead, bar(Y::bS));
            if (!(fine = B::full_y(k))) break;
            tc_fence_after();
            B::mma_rows(lead, tDP, Y::kB, B::at_y(k), id);
            commit_by(lead, bar(Y::bDP));
            if (n == 1) commit_by(lead, bar(Y::bHoldEmpty));
            if (!(fine = hold(x, bar(Y::bOutEmpty), (kn & 1) ^ 1))) break;
#pragma unroll 1
            for (int i = 0; i < n; ++i, ++k) {
                if (!(fine = hold(x, bar(Y::bP), k & 1))) break;
                tc_fence_after();
                mma_acc(lead, tDV, tS, B::at_y(k), i > 0);
                commit_by(lead, bar(Y::bYEmpty + k % Y::NY));
                if (i + 1 < n) {
                    if (!(fine = B::full_x(k + 1))) break;
                    tc_fence_after();
                    B::mma_rows(lead, tS, Y::kA, B::at_x(k + 1), id);
                    commit_by(lead, bar(Y::bS));
                }
                if (!(fine = hold(x, bar(Y::bDS), k & 1))) break;
                tc_fence_after();
                mma_acc(lead, tDK, tDP, B::at_x(k), i > 0);
                commit_by(lead, bar(Y::bXEmpty + k % Y::NX));
                if (i + 1 < n) {
                    if (!(fine = B::full_y(k + 1))) break;
                    tc_fence_after();
                    B::mma_rows(lead, tDP, Y::kB, B::at_y(k + 1), id);
                    commit_by(lead, bar(Y::bDP));
                    if (i + 2 == n) commit_by(lead, bar(Y::bHoldEmpty));  // the last that read the keys and values
                } else {
                    commit_by(lead, bar(Y::bOut));
                }
            }
        }
        commit_by(lead, bar(Y::bDrain));
        wait_drain(bar(Y::bDrain), 0);
    }

    __device__ void threads() {
        const int warp = threadIdx.x >> 5, row = threadIdx.x & 127, w = warp >> 2;
        const uint32_t lane = lane_base(tm, warp);
        const float c = p.scale * kLog2e;
        const f2 cc = both(c);
        unsigned k = 0, kn = 0;
        KeyPlan u;
        for (; B::next_plan(u, kn); ++kn) {
            const int j = u.k0 + row;  // the thread's key
            Round r(u, p.Nq / p.Nk);
            for (int i = 0; i < u.rounds; ++i, ++k, r.step(u)) {
                const int q0 = r.tile * 128;
                const float *cols = reinterpret_cast<const float *>(x.gbase + Y::kCols + k % Y::NX * 1024) + 64 * w;
                // queries of the tile that see the key: [j, j + window - 1], or all behind j for a sink
                const long long far = j < p.sinks ? (long long)u.L - 1 : (long long)j + p.window - 1;
                const int lo = j - q0, hi = (int)((far < u.L - 1 ? far : u.L - 1) - q0);
                const bool edge = q0 < u.k0 + 127 || q0 + 127 >= u.L || (long long)q0 + 127 - u.k0 >= p.window;
                if (!hold(x, bar(Y::bCol + k % Y::NX), (k / Y::NX) & 1)) return;
                if (!hold(x, bar(Y::bS), k & 1)) return;
                tc_fence_after();
                uint32_t s[2][32];
                tmem_ld32(lane + tS + 64 * w, s[0]);
                tmem_ld32(lane + tS + 64 * w + 32, s[1]);
                tmem_wait_ld();
                tmem_ld_dep(s[0]);
                tmem_ld_dep(s[1]);
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const uint32_t mask = edge ? bit_range(lo - 64 * w - 32 * q, hi - 64 * w - 32 * q) : 0xffffffffu;
                    uint32_t v[16];
#pragma unroll
                    for (int e = 0; e < 32; e += 4) {
                        const ulonglong2 l = *reinterpret_cast<const ulonglong2 *>(cols + 32 * q + e);
                        float a[4];
                        split(fma2(pair(__uint_as_float(s[q][e]), __uint_as_float(s[q][e + 1])), cc, l.x), a[0], a[1]);
                        split(fma2(pair(__uint_as_float(s[q][e + 2]), __uint_as_float(s[q][e + 3])), cc, l.y), a[2], a[3]);
#pragma unroll
                        for (int f = 0; f < 4; ++f) {
                            a[f] = ex2(a[f]);
                            if (edge) a[f] = mask >> (e + f) & 1 ? a[f] : 0.f;
                            s[q][e + f] = __float_as_uint(a[f]);
                        }
                        v[e / 2] = pack_bf16(a[0], a[1]);
                        v[e / 2 + 1] = pack_bf16(a[2], a[3]);
                    }
                    tmem_st16(lane + tS + 64 * w + 16 * q, v);
                }
                tmem_wait_st();
                tc_fence_before();
                warp_arrive(bar(Y::bP));
                if (!hold(x, bar(Y::bDP), k & 1)) return;
                tc_fence_after();
                uint32_t g[2][32];
                tmem_ld32(lane + tDP + 64 * w, g[0]);
                tmem_ld32(lane + tDP + 64 * w + 32, g[1]);
                tmem_wait_ld();
                tmem_ld_dep(g[0]);
                tmem_ld_dep(g[1]);
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const uint32_t mask = edge ? bit_range(lo - 64 * w - 32 * q, hi - 64 * w - 32 * q) : 0xffffffffu;
                    uint32_t v[16];
#pragma unroll
                    for (int e = 0; e < 32; e += 4) {
                        const ulonglong2 d = *reinterpret_cast<const ulonglong2 *>(cols + 128 + 32 * q + e);
                        float a[4];
                        split(mul2(pair(__uint_as_float(s[q][e]), __uint_as_float(s[q][e + 1])),
                                   add2(pair(__uint_as_float(g[q][e]), __uint_as_float(g[q][e + 1])), d.x)), a[0], a[1]);
                        split(mul2(pair(__uint_as_float(s[q][e + 2]), __uint_as_float(s[q][e + 3])),
                                   add2(pair(__uint_as_float(g[q][e + 2]), __uint_as_float(g[q][e + 3])), d.y)), a[2], a[3]);
                        if (edge)
#pragma unroll
                            for (int f = 0; f < 4; ++f) a[f] = mask >> (e + f) & 1 ? a[f] : 0.f;
                        v[e / 2] = pack_bf16(a[0], a[1]);
                        v[e / 2 + 1] = pack_bf16(a[2], a[3]);
                    }
                    tmem_st16(lane + tDP + 64 * w + 16 * q, v);
                }
                tmem_wait_st();
                tc_fence_before();
                warp_arrive(bar(Y::bDS));
            }
            if (!hold(x, bar(Y::bOut), kn & 1)) return;
            tc_fence_after();
            // dv by the first four warps, dk by the others; sinks that parts add to as fp32
            const uint32_t from = lane + (w == 0 ? tDV : tDK);
            const float f = w == 0 ? 1.f : p.scale;
            const bool summed = u.split && j < p.sinks;
            __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(w == 0 ? p.dv : p.dk) + ((u.bos + j) * p.Nk + u.hk) * D;
            // rows of the warp that are this item's alone: [own0, own1)
            const int j0 = j & ~31, own0 = u.split ? p.sinks - j0 : 0, own1 = u.part ? 0 : u.L - j0;
            const bool nan = own0 < 32 && B::template store_cols<D>(from, out, (long long)p.Nk * D, own0, own1, f);
            if (u.split) {
                float *sum = p.sink_part + (((u.place * p.Nk + u.hk) * 2 + w) * p.sinks + row) * D;
#pragma unroll 1
                for (int q = 0; q < D / 16; ++q) {
                    uint32_t o[16];
                    tmem_ld16(from + 16 * q, o);
                    tmem_wait_ld_dep16(o);
                    if (summed)
#pragma unroll
                        for (int e = 0; e < 16; e += 4)
                            *reinterpret_cast<float4 *>(sum + 16 * q + e) =
                                make_float4(__uint_as_float(o[e]) * f, __uint_as_float(o[e + 1]) * f, __uint_as_float(o[e + 2]) * f,
                                            __uint_as_float(o[e + 3]) * f);
                }
            }
            tc_fence_before();
            warp_arrive(bar(Y::bOutEmpty));
            if (!u.part) B::mark(nan, u.flag);
        }
    }
};

template <typename F>
__device__ __forceinline__ void set_up(F &f, uint8_t *raw_smem, unsigned *status) {
    using Y = typename F::Y;
    const uint32_t raw = smem_u32(raw_smem);
    f.x.base = (raw + 1023u) & ~1023u;
    f.x.gbase = raw_smem + (f.x.base - raw);
    f.x.abort_flag = reinterpret_cast<volatile int *>(f.x.gbase + Y::kMisc + 4);
    f.x.status = status;
    if (threadIdx.x == 0) {
        mbar_init(f.bar(Y::bHold), 1);
        mbar_init(f.bar(Y::bHoldEmpty), 1);
        for (int s = 0; s < Y::NX; ++s) {
            mbar_init(f.bar(Y::bX + s), 1);
            mbar_init(f.bar(Y::bXEmpty + s), 1);
            mbar_init(f.bar(Y::bCol + s), 1);
        }
        for (int s = 0; s < Y::NY; ++s) {
            mbar_init(f.bar(Y::bY + s), 1);
            mbar_init(f.bar(Y::bYEmpty + s), 1);
        }
        mbar_init(f.bar(Y::bS), 1);
        mbar_init(f.bar(Y::bDP), 1);
        mbar_init(f.bar(Y::bP), 8);
        mbar_init(f.bar(Y::bDS), 8);
        mbar_init(f.bar(Y::bOut), 1);
        mbar_init(f.bar(Y::bOutEmpty), 8);
        for (int i = 0; i < kPlans; ++i) mbar_init(f.bar(Y::bPlan + i), 1);
        mbar_init(f.bar(Y::bDrain), 1);
        mbar_init(f.bar(Y::bItem), 1);
        for (int i = 0; i < 4; ++i) {
            mbar_init(f.bar(Y::bPair + i), 2);
            mbar_init(f.bar(Y::bTaken + i), 2);
        }
        *f.x.abort_flag = 0;
        fence_barrier_init();
    }
    if (threadIdx.x >> 5 == 9) {
        tmem_alloc(f.x.base + Y::kMisc, 512);
        tmem_relinquish();
    }
    fence_proxy_async_smem();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    f.tm = *reinterpret_cast<volatile uint32_t *>(f.x.gbase + Y::kMisc);
}

__device__ __forceinline__ void clear_up(uint32_t tm) {
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (threadIdx.x >> 5 == 9) tmem_dealloc(tm, 512);
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
window_dq(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mg, const __grid_constant__ CUtensorMap mk,
          const __grid_constant__ CUtensorMap mv, const __grid_constant__ CUtensorMap mks, const __grid_constant__ CUtensorMap mvs,
          const __grid_constant__ WindowParams p, long long slots) {
    extern __shared__ uint8_t smem_raw[];
    Dq<D> f{{Ctx{}, p, 0u}, slots};
    set_up(f, smem_raw, p.seq.status);
    wait_for_launches();
    const int warp = threadIdx.x >> 5;
    const bool one = (threadIdx.x & 31) == 0;
    if (warp == 8) {
        if (one) f.load(&mq, &mg, &mk, &mv, &mks, &mvs);
        __syncwarp();
    } else if (warp == 9) {
        f.mma();
    } else if (warp < 8) {
        f.threads();
    }
    clear_up(f.tm);
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
window_dkv(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mg, const __grid_constant__ CUtensorMap mk,
           const __grid_constant__ CUtensorMap mv, const __grid_constant__ WindowParams p, long long slots, Parts parts) {
    extern __shared__ uint8_t smem_raw[];
    Dkv<D> f{{Ctx{}, p, 0u}, slots, parts};
    set_up(f, smem_raw, p.seq.status);
    wait_for_launches();
    const int warp = threadIdx.x >> 5;
    const bool one = (threadIdx.x & 31) == 0;
    if (warp == 8) {
        if (one) f.load(&mq, &mg, &mk, &mv);
        __syncwarp();
    } else if (warp == 9) {
        f.mma();
    } else if (warp == 10) {
        f.columns();
    } else {
        f.threads();
    }
    clear_up(f.tm);
}

// D' = sum do o of every token and head: 16 bytes of both a thread, D / 8 threads a row.
template <int D>
__global__ void __launch_bounds__(256) window_dsum(WindowParams p, long long rows) {
    constexpr int L = D / 8, ROWS = 4;  // rows in flight of a thread
    wait_for_launches();
    if (blockIdx.x == 0) check_offsets(p.seq, threadIdx.x, 256);
    const __nv_bfloat16 *o = static_cast<const __nv_bfloat16 *>(p.o), *g = static_cast<const __nv_bfloat16 *>(p.dout);
    const int per = 256 / L, sub = threadIdx.x / L, at = threadIdx.x % L * 8;
    for (long long r0 = (long long)blockIdx.x * per * ROWS; r0 < rows; r0 += (long long)gridDim.x * per * ROWS) {
        Pack<__nv_bfloat16, 8> a[ROWS], b[ROWS];
#pragma unroll
        for (int i = 0; i < ROWS; ++i) {
            const long long r = r0 + i * per + sub;
            a[i].clear();
            b[i].clear();
            if (r < rows) {
                a[i].load(o + r * D + at);
                b[i].load(g + r * D + at);
            }
        }
#pragma unroll
        for (int i = 0; i < ROWS; ++i) {
            const long long r = r0 + i * per + sub;
            float s = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) s = fmaf(a[i][e], b[i][e], s);
#pragma unroll
            for (int x = L / 2; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
            if (at == 0 && r < rows) p.dsum[r] = s;
        }
    }
}

template <int D>
cudaError_t launch(const WindowParams &p, cudaStream_t stream) {
    const long long slots = tile_slots(p.seq, 128);
    if (slots <= 0) return cudaSuccess;
    const Parts parts{p.parts ? tile_slots(p.seq, p.part_tiles * 128) : 0, p.part_tiles};
    const long long qi = slots * p.Nq, ki = (slots + parts.slots) * p.Nk;
    if (qi > 0x7fffffffll || ki > 0x7fffffffll) return cudaErrorInvalidValue;
    CUtensorMap mq, mg, mk, mv, mks, mvs;
    const uint64_t tokens = (uint64_t)p.seq.tokens;
    if (!make_tmap_rows_heads_d(&mq, p.q, tokens, p.Nq, D, 64, 128) || !make_tmap_rows_heads_d(&mg, p.dout, tokens, p.Nq, D, 64, 128) ||
        !make_tmap_rows_heads_d(&mk, p.k, tokens, p.Nk, D, 64, 128) ||
        !make_tmap_rows_heads_d(&mv, p.v, tokens, p.Nk, D, 64, 128) ||
        !make_tmap_rows_heads_d(&mks, p.k, tokens, p.Nk, D, 64, kSinkCols) || !make_tmap_rows_heads_d(&mvs, p.v, tokens, p.Nk, D, 64, kSinkCols))
        return cudaErrorInvalidValue;
    constexpr int q_bytes = (int)Lay<D, true>::kAlloc, k_bytes = (int)Lay<D, false>::kAlloc;
    cudaError_t err = allow_smem<window_dq<D>>(q_bytes);
    if (err == cudaSuccess) err = allow_smem<window_dkv<D>>(k_bytes);
    if (err != cudaSuccess) return err;
    const long long rows = p.seq.tokens * p.Nq, blocks = (rows + 8192 / D - 1) / (8192 / D);
    err = launch_after(window_dsum<D>, dim3((unsigned)(blocks < kSms * 8 ? blocks : kSms * 8)), dim3(256), 0, stream, p, rows);
    if (err != cudaSuccess) return err;
    err = launch_after(window_dq<D>, dim3((unsigned)qi), dim3(kThreads), q_bytes, stream, mq, mg, mk, mv, mks, mvs, p, slots);
    if (err != cudaSuccess) return err;
    err = launch_after(window_dkv<D>, dim3((unsigned)ki), dim3(kThreads), k_bytes, stream, mq, mg, mk, mv, p, slots, parts);
    return err == cudaSuccess ? window_sink_sums(p, true, stream) : err;
}

}  // namespace

cudaError_t window_tc_bwd(const WindowParams &p, cudaStream_t stream) {
    return p.d == 64 ? launch<64>(p, stream) : launch<128>(p, stream);
}

}  // namespace dn
