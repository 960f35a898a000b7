// Attention over a sliding window with sinks, forward, bf16: tcgen05 / TMEM / TMA.
//
//     S = Q K^T,  p = e^{scale s - m},  O += P V,  o = O / sum p,  lse = m + log sum p
//
// tile by tile of 128 keys with the running maximum m and sum of every row.  A CTA works on
// two tiles of 128 queries at once that share their keys: two query heads of one key head
// where its group is even, else two neighbouring tiles of tokens of one head.  While one
// tile's scores go through the softmax, the tensor cores work for the other.
//
// Warps 0-7 and 8-15: softmax of the first and the second query tile, four warps for each
// half of the keys of a tile, two threads a row (one thread a row took 1900 cycles a tile, of which
// the tensor cores need 1024: a warp alone on its scheduler does not keep up the rate of the
// exponentials).  The two agree on the maximum through shared memory.
// Warp 16: TMA loads of Q, K and V; warp 17: the MMAs.
// Tensor memory: scores of both tiles (128 fp32 columns each; the weights P overwrite the
// first half of each half of them as bf16) and both O (d columns each).
// For every key tile j warp 17 does, for the first and then the second query tile,
//     wait P(j);  O += P V(j);  S = Q K(j+1)
// so S(j+1) of one tile is ready when the softmax of the other has just begun (with a warp for
// each, the two tiles fell into step: both in the softmax, then both on the tensor cores, 15 % slower).
//
// What a row's weights are relative to is the maximum of the first tile that it sees.  It moves up, and O and
// the sum are rescaled, only when the weights of half a tile have summed to more than 2^16, so that later
// tiles need no maximum: sums in fp32 lose nothing, P in bf16 has the same relative rounding at every
// size.  A row whose weights sum to 2^124 within half a tile (a score, in units of log 2, 124 above the reference)
// is marked.  Masks cost selects only in tiles that the window's or the
// sequence's border crosses.  The sinks in front of the window are a tile of 32 keys where they fit in
// one.  P is rounded to bf16 for the product, by half a step of each weight; the sum takes it unrounded.
//
// A masked pair weighs 0, and 0 times an infinite or NaN value is NaN.  Rows that come out so are marked in
// lse, and taken again by a kernel that leaves masked pairs out (dn_window_simt.cu).
//
// CTAs are persistent, one an SM, and take items as they get done (Items: 47 us for the training shape below, 56 with
// items at a fixed stride); every wait is bounded (dn_tc_sync.cuh).  Measured: one prompt of 32768
// tokens, window 4096, 32 heads on 8 of 128 columns, 1.35 ms, 1.45 in a run of calls under the power cap (1.09 at the
// measured rate of products in the pairs that are seen); 4 x 2048 tokens, window 512, 16 heads, 48 us, the tensor
// pipe at work 39 % of the time: an item's first and last tiles have nothing to overlap with.
#include "dn_window_tc.cuh"

namespace dn {
namespace {

using namespace ptx;
using namespace tcs;

constexpr int kThreads = 576;

constexpr int kPlans = 4;  // items whose plans are kept

template <int D>
struct Lay {
    static constexpr uint32_t kPanel = 128 * 128;            // 128 rows of 64 columns
    static constexpr uint32_t kTile = (D / 64) * kPanel;     // 128 rows of D
    static constexpr int NS = D == 64 ? 4 : 2;               // stages of keys and values
    static constexpr uint32_t kQ = 0, kK = 2 * kTile, kV = kK + NS * kTile, kBar = kV + NS * kTile;
    // barriers
    static constexpr int bQFull = 0, bQEmpty = 1, bFull = 2, bEmpty = bFull + NS, bS = bEmpty + NS, bP = bS + 2, bO = bP + 2,
                         bOEmpty = bO + 2, bDrain = bOEmpty + 2, bPair = bDrain + 1, bPlan = bPair + 8, bPlanEmpty = bPlan + kPlans,
                         bItem = bPlanEmpty + kPlans, kBars = bItem + 1;
    static constexpr uint32_t kBox = (kBar + 8 * kBars + 15) / 16 * 16, kWish = kBox + 2 * 2 * 2 * 128 * 4, kPlan = kWish + 2 * 2 * 2 * 128 * 4, kMisc = kPlan + kPlans * 96, kAlloc = kMisc + 32 + 1024;
    static_assert(kAlloc <= 232448, "exceeds the 227 KB of shared memory per CTA");
    // tensor memory columns
    static constexpr uint32_t tS = 0, tO = 256, kCols = 512;
};

// A tile's weights in a row, half of them, may sum to this before the row's reference moves up.
constexpr float kGrown = 65536.f;
// Above this they count as infinite, and so does a row's sum above twice as much (both halves), which marks the row: the
// approximate instructions flush what is below 2^-126 to 0, the reciprocal of a sum above 2^126 and the factor
// that such a rise of the reference scales by among it.
constexpr float kMost = 0x1p124f;

constexpr uint32_t kIdS = idesc_bf16(128, 128, 0, 0), kIdSNarrow = idesc_bf16(128, kSinkCols, 0, 0);

// One work item: two query tiles and the list of key tiles that either sees.  Places of the
// list that a query tile looks at: [from, to], and 0 where `zero`.
struct Span {
    int from, to, t0, h;
    bool zero, act;
    __device__ __forceinline__ bool has(int i) const { return i == 0 ? zero : i >= from && i <= to; }
};
struct __align__(16) Plan {
    Span q0, q1;
    long long bos;
    int L, hk;
    int lo, n;          // place i holds key tile lo + i (but the sinks' at 0); length of the list (0: no item is left)
    bool sink, narrow;  // the list begins with the sinks' tile; as kSinkCols keys
    __device__ __forceinline__ int tile(int i) const { return sink && i == 0 ? 0 : lo + i; }
    __device__ __forceinline__ bool small(int i) const { return narrow && i == 0; }
};

// Items are numbered with a key head's pairs next to each other and late tiles first.
__device__ __forceinline__ bool plan(Plan &u, const WindowParams &p, unsigned item, long long slots) {
    const int G = p.Nq / p.Nk;
    const bool by_head = G % 2 == 0;
    const int pairs = by_head ? G / 2 : G;
    const int pr = item % pairs;
    u.hk = item / pairs % p.Nk;
    const unsigned slot = slot_in_order(p.seq, item / pairs / p.Nk, (unsigned)slots, false);
    const SeqTile s = seq_tile(p.seq, slot, by_head ? 128 : 256);
    if (!s.ok || s.t0 >= s.t1) return false;
    u.bos = s.bos;
    u.L = (int)(s.eos - s.bos);
    const Sight sight{p.window, p.sinks};
    auto span = [&](int q, KeyTiles &kt) {
        Span v;
        v.h = u.hk * G + (by_head ? 2 * pr + q : pr);
        v.t0 = (int)(s.t0 - s.bos) + (by_head ? 0 : 128 * q);
        v.act = v.t0 < u.L;
        const int t1 = v.t0 + 128 < u.L ? v.t0 + 128 : u.L;
        kt = KeyTiles(v.t0, v.act ? t1 : v.t0 + 1, 128, sight);
        return v;
    };
    KeyTiles k0, k1;
    u.q0 = span(0, k0);  // always there
    u.q1 = span(1, k1);
    const int lo = k0.first, hi = u.q1.act ? k1.last : k0.last;
    u.sink = lo > 0 && p.sinks > 0;
    u.narrow = u.sink && p.sinks <= kSinkCols;
    u.lo = u.sink ? lo - 1 : lo;
    u.n = hi - u.lo + 1;
    auto places = [&](Span &v, const KeyTiles &kt) {
        v.from = kt.first - u.lo;
        v.to = kt.last - u.lo;
        v.zero = v.act && (v.from == 0 || (u.tile(0) == 0 && p.sinks > 0));
        if (!v.act) v.from = 1, v.to = 0;
    };
    places(u.q0, k0);
    places(u.q1, k1);
    return true;
}

static_assert(sizeof(Plan) <= 96, "a plan's place in shared memory");

template <int D>
struct Fwd {
    using Y = Lay<D>;
    Ctx x;
    const WindowParams &p;
    long long slots;
    uint32_t tm;

    __device__ __forceinline__ uint32_t bar(int i) const { return x.base + Y::kBar + 8u * i; }

    // ---- plans ----------------------------------------------------------------
    // The TMA warp works them out (a few hundred cycles of divisions and look-ups, and code that the other
    // roles would fetch anew for every item: 3000 cycles an item each) and leaves the n-th item's in
    // shared memory, when all scores of item n - 1 are issued and the other warps have read plan n - 4,
    // whose place it takes.  What a plan holds is copied at once.
    __device__ __forceinline__ Plan *place(unsigned n) const { return reinterpret_cast<Plan *>(x.gbase + Y::kPlan + n % kPlans * 96); }
    __device__ __forceinline__ bool next_plan(const Plan *&u, unsigned n) const {
        if (!hold(x, bar(Y::bPlan + n % kPlans), n / kPlans & 1)) return false;
        u = place(n);
        return u->n > 0;
    }
    __device__ __forceinline__ void read_plan(unsigned n) const { warp_arrive(bar(Y::bPlanEmpty + n % kPlans)); }

    // ---- TMA ------------------------------------------------------------------
    // Keys and values come in units: the keys of place 0; the values of place i with the keys
    // of place i + 1.
    __device__ void load(const CUtensorMap *mq, const CUtensorMap *mk, const CUtensorMap *mv, const CUtensorMap *mks,
                         const CUtensorMap *mvs) {
        unsigned un = 0, qn = 0;
        bool fine = true;
        Items next{bar(Y::bItem), x.base + Y::kMisc + 16};
        for (; fine; fine = fine && next.next(x)) {
            Plan u;
            if (!next.any) u.n = 0;
            else if (!plan(u, p, next.item, slots)) continue;
            if (!(fine = wait(x, bar(Y::bQEmpty), (qn & 1) ^ 1) && wait(x, bar(Y::bPlanEmpty + qn % kPlans), (qn / kPlans & 1) ^ 1))) break;
            *place(qn) = u;
            mbar_arrive(bar(Y::bPlan + qn % kPlans));
            if (u.n == 0) break;
            mbar_arrive_expect_tx(bar(Y::bQFull), u.q1.act ? 2 * Y::kTile : Y::kTile);
            for (int c = 0; c < D / 64; ++c) {
                tma_load_3d(x.base + Y::kQ + c * Y::kPanel, mq, bar(Y::bQFull), 64 * c, u.q0.h, (int)(u.bos + u.q0.t0));
                if (u.q1.act)
                    tma_load_3d(x.base + Y::kQ + Y::kTile + c * Y::kPanel, mq, bar(Y::bQFull), 64 * c, u.q1.h, (int)(u.bos + u.q1.t0));
            }
            ++qn;
            for (int i = 0; i <= u.n; ++i, ++un) {
                const int s = un % Y::NS;
                if (i + 1 >= u.n) next.ask();
                if (!(fine = wait(x, bar(Y::bEmpty + s), ((un / Y::NS) & 1) ^ 1))) break;
                const bool vs = i > 0 && u.small(i - 1), ks = u.small(i);
                uint32_t bytes = 0;
                if (i > 0) bytes += vs ? kSinkCols * D * 2 : Y::kTile;
                if (i < u.n) bytes += ks ? kSinkCols * D * 2 : Y::kTile;
                mbar_arrive_expect_tx(bar(Y::bFull + s), bytes);
                for (int c = 0; c < D / 64; ++c) {
                    if (i > 0)
                        tma_load_3d(x.base + Y::kV + s * Y::kTile + c * Y::kPanel, vs ? mvs : mv, bar(Y::bFull + s), 64 * c, u.hk,
                                    (int)(u.bos + (long long)u.tile(i - 1) * 128));
                    if (i < u.n)
                        tma_load_3d(x.base + Y::kK + s * Y::kTile + c * Y::kPanel, ks ? mks : mk, bar(Y::bFull + s), 64 * c, u.hk,
                                    (int)(u.bos + (long long)u.tile(i) * 128));
                }
            }
        }
        // copies still in flight land before the CTA ends
        next.drain();
        if (qn) wait_drain(bar(Y::bQFull), (qn - 1) & 1);
        for (unsigned i = un > Y::NS ? un - Y::NS : 0; i < un; ++i) wait_drain(bar(Y::bFull + i % Y::NS), (i / Y::NS) & 1);
    }

    // ---- MMAs -----------------------------------------------------------------
    __device__ __forceinline__ void issue_s(uint32_t lead, int q, unsigned unit, bool small) const {
        const uint32_t a = rows_of(x.base + Y::kQ + q * Y::kTile), b = rows_of(x.base + Y::kK + (unit % Y::NS) * Y::kTile);
        const uint32_t id = small ? kIdSNarrow : kIdS;
#pragma unroll
        for (int c = 0; c < D / 64; ++c)
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
                mma_ss_by(lead, tm + Y::tS + 128 * q, a + (c * Y::kPanel + kk * 32) / 16, b + (c * Y::kPanel + kk * 32) / 16, id,
                          (c | kk) != 0);
        commit_by(lead, bar(Y::bS + q));
    }
    __device__ __forceinline__ void issue_o(uint32_t lead, int q, unsigned unit, bool small, bool more) const {
        const uint32_t b = cols_of(x.base + Y::kV + (unit % Y::NS) * Y::kTile), d = tm + Y::tO + D * q, w = tm + Y::tS + 128 * q;
        constexpr uint32_t id = idesc_bf16(128, D, 0, 1);
        mma_ts_by(lead, d, w, b, id, more);
        mma_ts_by(lead, d, w + 8, b + 128, id, 1);
        static_assert(kSinkCols == 32, "two steps of 16 keys");
        if (!small)
#pragma unroll
            for (int kk = 2; kk < 8; ++kk)  // the keys' halves lie 64 columns apart
                mma_ts_by(lead, d, w + 64 * (kk >> 2) + 8 * (kk & 3), b + kk * 128, id, 1);
    }

    __device__ void mma() {
        const uint32_t lead = elect();
        unsigned un = 0, qn = 0, ns[2] = {0, 0}, no[2] = {0, 0};
        bool fine = true;
        for (const Plan *next; fine && next_plan(next, qn);) {
            const Plan u = *next;
            read_plan(qn);
            if (!(fine = hold(x, bar(Y::bQFull), qn & 1) && hold(x, bar(Y::bFull + un % Y::NS), (un / Y::NS) & 1))) break;
            tc_fence_after();
            if (u.q0.zero) issue_s(lead, 0, un, u.small(0));
            if (u.q1.zero) issue_s(lead, 1, un, u.small(0));
            commit_by(lead, bar(Y::bEmpty + un % Y::NS));
            if (u.n == 1) commit_by(lead, bar(Y::bQEmpty));
            ++un;
            bool more[2] = {false, false};
            for (int i = 0; i < u.n; ++i, ++un) {
                if (!(fine = hold(x, bar(Y::bFull + un % Y::NS), (un / Y::NS) & 1))) break;
                const bool small = u.small(i);
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const Span &v = q ? u.q1 : u.q0;
                    if (v.has(i)) {
                        if (!more[q] && !(fine = hold(x, bar(Y::bOEmpty + q), (no[q] & 1) ^ 1))) break;
                        if (!(fine = hold(x, bar(Y::bP + q), ns[q] & 1))) break;
                        ++ns[q];
                        tc_fence_after();
                        issue_o(lead, q, un, small, more[q]);
                        more[q] = true;
                        if (i == v.to) {
                            commit_by(lead, bar(Y::bO + q));
                            ++no[q];
                        }
                    }
                    if (v.has(i + 1)) issue_s(lead, q, un, false);
                }
                if (!fine) break;
                commit_by(lead, bar(Y::bEmpty + un % Y::NS));
                if (i + 2 == u.n) commit_by(lead, bar(Y::bQEmpty));  // the last scores are issued: Q may change after them
            }
            ++qn;
        }
        commit_by(lead, bar(Y::bDrain));
        wait_drain(bar(Y::bDrain), 0);
    }

    // ---- softmax of query tile q, the keys' half h ----------------------------------
    // Two threads share a row.  Each leaves a number for the other: what they agree on next.  Two boxes in turn: the
    // other thread may not have read the last one yet, but it has read the one before.
    __device__ __forceinline__ bool swap(int q, int h, float &mine, float &other, unsigned &n) const {
        const int row = threadIdx.x & 127, pairs = q * 4 + (row >> 5);
        volatile float *box = reinterpret_cast<float *>(x.gbase + Y::kBox) + (n & 1) * 512 + q * 256;
        box[h * 128 + row] = mine;
        warp_arrive(bar(Y::bPair + pairs));
        if (!hold(x, bar(Y::bPair + pairs), n & 1)) return false;
        ++n;
        other = box[(h ^ 1) * 128 + row];
        return true;
    }

    static __device__ __forceinline__ void hide(uint32_t (&s)[16], uint32_t mask) {  // what a row does not see
#pragma unroll
        for (int e = 0; e < 16; ++e) s[e] = mask >> e & 1 ? s[e] : 0xff800000u;
    }

    static __device__ __forceinline__ void scaled(const uint32_t (&s)[16], uint32_t (&w)[8], f2 ff, f2 &bads) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const f2 v = mul2(pair(__uint_as_float(s[2 * e]), __uint_as_float(s[2 * e + 1])), ff);
            bads = fma2(v, 0ull, bads);  // 0 times infinity or NaN stays
            float lo, hi;
            split(v, lo, hi);
            w[e] = pack_bf16(lo, hi);
        }
    }

    __device__ void softmax(int q, int h) {
        const int warp = threadIdx.x >> 5, row = threadIdx.x & 127;
        const uint32_t ts = lane_base(tm, warp) + Y::tS + 128 * q + 64 * h, to = lane_base(tm, warp) + Y::tO + D * q + D / 2 * h;
        // Wishes for a higher reference have two places, for tiles in turn: both threads of a row take up what tile j left in
        // tile j + 1, and whoever is done with that first may write before the other one has read.  (A write in every
        // tile costs 1 % of the kernel; one in two tiles from each new wish on, 3 %.)
        volatile float *wish = reinterpret_cast<float *>(x.gbase + Y::kWish) + q * 256 + row;
        const float c = p.scale * kLog2e;
        const Sight sight{p.window, p.sinks};
        unsigned ns = 0, no = 0, nx = 0, qn = 0;
        for (const Plan *next; next_plan(next, qn); ++qn) {
            const Plan &u = *next;
            const Span v = q ? u.q1 : u.q0;
            const int lo = u.lo, L = u.L;
            const bool sink = u.sink, narrow = u.narrow;
            const long long bos = u.bos;
            read_plan(qn);
            if (!v.act) continue;
            const int t = v.t0 + row;
            // what weights are relative to, times log2 e scale: -infinity until the row has seen a key; sum of the weights;
            // the highest reference that this thread has wished for
            float m = -CUDART_INF_F, l = 0.f, mine = -CUDART_INF_F;
            for (int i = v.zero ? 0 : v.from; i <= v.to; i = i + 1 < v.from ? v.from : i + 1) {
                const int k0 = (sink && i == 0 ? 0 : lo + i) * 128 + 64 * h;
                const int groups = narrow && i == 0 ? 2 - 2 * h : 4;  // of 16 keys
                // some row of the tile does not see some key of it
                const bool edge = k0 + 63 > v.t0 || v.t0 + 127 - k0 >= p.window;
                if (!hold(x, bar(Y::bS + q), ns & 1)) return;
                ++ns;
                tc_fence_after();
                uint32_t s[2][16];
                if (__any_sync(0xffffffffu, m == -CUDART_INF_F)) {
                    // the first tile that a row sees: its maximum
                    float top = -CUDART_INF_F, other;
#pragma unroll 1
                    for (int g = 0; g < groups; ++g) {
                        tmem_ld16(ts + 16 * g, s[0]);
                        tmem_wait_ld_dep16(s[0]);
                        if (edge) hide(s[0], seen32(t, k0 + 16 * g, sight));
#pragma unroll
                        for (int e = 0; e < 16; e += 2) top = max3(top, __uint_as_float(s[0][e]), __uint_as_float(s[0][e + 1]));
                    }
                    if (!swap(q, h, top, other, nx)) return;
                    if (m == -CUDART_INF_F) {
                        m = fmaxf(top, other) * c;
                    }
                } else {
                    // what the two threads left in the tile before
                    const float want = fmaxf(mine, wish[512 * (ns & 1) + 128 * (h ^ 1)]);
                    if (__any_sync(0xffffffffu, want > m)) {
                        const float f = want > m ? ex2(m - want) : 1.f;
                        m = want > m ? want : m;
                        l *= f;
#pragma unroll 1
                        for (int g = 0; g < D / 32; ++g) {
                            tmem_ld16(to + 16 * g, s[0]);
                            tmem_wait_ld_dep16(s[0]);
#pragma unroll
                            for (int e = 0; e < 16; ++e) s[0][e] = __float_as_uint(__uint_as_float(s[0][e]) * f);
                            tmem_st16(to + 16 * g, s[0]);
                        }
                    }
                }
                const f2 cc = both(c), mm = both(m == -CUDART_INF_F ? 0.f : -m);
                f2 sum[2] = {0ull, 0ull};
                // P lies over scores that are read by then.  Two groups a round, not all four unrolled: an item's code
                // that does not stay in the instruction cache costs more than the loop.
                if (groups) tmem_ld16(ts, s[0]);
#pragma unroll 1
                for (int r = 0; r < groups; r += 2) {
#pragma unroll
                    for (int g = 0; g < 2; ++g) {
                        tmem_wait_ld_dep16(s[g]);
                        if (g == 0 || r + 2 < groups) tmem_ld16(ts + 16 * (r + g + 1), s[g ^ 1]);
                        if (edge) hide(s[g], seen32(t, k0 + 16 * (r + g), sight));
                        uint32_t w[8];
#pragma unroll
                        for (int e = 0; e < 16; e += 2) {
                            float a, b;
                            split(fma2(pair(__uint_as_float(s[g][e]), __uint_as_float(s[g][e + 1])), cc, mm), a, b);
                            a = ex2(a);
                            b = ex2(b);
                            sum[(e >> 1) & 1] = add2(sum[(e >> 1) & 1], pair(a, b));
                            w[e / 2] = pack_bf16(a, b);
                        }
                        tmem_st8(ts + 8 * (r + g), w);
                    }
                }
                const float part = sum_of(add2(sum[0], sum[1]));
                l += part < kMost ? part : CUDART_INF_F;  // a NaN as well
                if (part > kGrown) mine = fmaxf(mine, m + lg2(part));
                wish[512 * ((ns & 1) ^ 1) + 128 * h] = mine;
                tmem_wait_st();
                tc_fence_before();
                warp_arrive(bar(Y::bP + q));
            }
            if (!hold(x, bar(Y::bO + q), no & 1)) return;
            ++no;
            tc_fence_after();
            float other;
            if (!swap(q, h, l, other, nx)) return;
            l += other;
            const float f = rcp(l);
            const long long at = (bos + t) * p.Nq + v.h;
            __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(p.o) + at * D + D / 2 * h;
            f2 bads = 0ull;
            const f2 ff = both(f);
            uint32_t w[4][D / 16];
#pragma unroll
            for (int g = 0; g < D / 32; ++g) {
                uint32_t s[16], v[8];
                tmem_ld16(to + 16 * g, s);
                tmem_wait_ld_dep16(s);
                scaled(s, v, ff, bads);
#pragma unroll
                for (int e = 0; e < 8; ++e) w[(8 * g + e) / (D / 16)][(8 * g + e) % (D / 16)] = v[e];
            }
            store_rows<D / 2>(out, (long long)p.Nq * D, 0, L - (t & ~31), w);
            tc_fence_before();
            warp_arrive(bar(Y::bOEmpty + q));
            float bad = sum_of(bads);
            if (!swap(q, h, bad, other, nx)) return;
            if (h == 0 && t < L)
                p.lse[at] = bad + other == 0.f && l <= 2.f * kMost ? (m + lg2(l)) * 0.6931471805599453f : redo_mark();
        }
    }
};

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
window_fwd(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv,
           const __grid_constant__ CUtensorMap mks, const __grid_constant__ CUtensorMap mvs, const __grid_constant__ WindowParams p,
           long long slots) {
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
            mbar_init(bar(Y::bFull + s), 1);
            mbar_init(bar(Y::bEmpty + s), 1);
        }
        for (int q = 0; q < 2; ++q) {
            mbar_init(bar(Y::bS + q), 1);
            mbar_init(bar(Y::bP + q), 8);
            mbar_init(bar(Y::bO + q), 1);
            mbar_init(bar(Y::bOEmpty + q), 8);
        }
        for (int i = 0; i < 8; ++i) mbar_init(bar(Y::bPair + i), 2);
        for (int i = 0; i < kPlans; ++i) {
            mbar_init(bar(Y::bPlan + i), 1);
            mbar_init(bar(Y::bPlanEmpty + i), 17);
        }
        mbar_init(bar(Y::bDrain), 1);
        mbar_init(bar(Y::bItem), 1);
        *x.abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == 17) {
        tmem_alloc(x.base + Y::kMisc, Y::kCols);
        tmem_relinquish();
    }
    fence_proxy_async_smem();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    Fwd<D> f{x, p, slots, *reinterpret_cast<volatile uint32_t *>(x.gbase + Y::kMisc)};
    wait_for_launches();
    if (warp == 16) {
        if ((threadIdx.x & 31) == 0) f.load(&mq, &mk, &mv, &mks, &mvs);
        __syncwarp();
    } else if (warp == 17) {
        f.mma();
    } else {
        f.softmax(warp >> 3, warp >> 2 & 1);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 17) tmem_dealloc(f.tm, Y::kCols);
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
    return launch_after(window_fwd<D>, dim3((unsigned)items), dim3(kThreads), Lay<D>::kAlloc, stream, mq, mk, mv, mks, mvs, p, slots);
}

}  // namespace

cudaError_t window_tc_fwd(const WindowParams &p, cudaStream_t stream) {
    return p.d == 64 ? launch<64>(p, stream) : launch<128>(p, stream);
}

}  // namespace dn
