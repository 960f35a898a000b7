// Selective state space scan, backward.
//
// With a_t[n] = e^{delta_t A[n]}, dyo = dy silu(z) and the states h of the forward:
//     g_t[n]  = C_t[n] dyo_t + a_{t+1}[n] g_{t+1}[n]        (the gradient of h_t)
//     s_t     = sum_n g_t[n] B_t[n],   q_t[n] = g_t[n] a_t[n] h_{t-1}[n]
//     dx      = delta s + Dskip dyo,   ddelta = x s + sum_n q[n] A[n],   ddt = ddelta softplus'(dt + dt_bias)
//     dA[n]   = sum_t delta q[n],      dB[n] = sum_d delta x g[n],       dC[n] = sum_d dyo h[n]
//     dDskip  = sum_t dyo x,           ddt_bias = sum_t ddt,             dz = dy (C.h + Dskip x) silu'(z)
//
// Every sequence is cut into chunks of 64 tokens (fewer in small calls), and all chunks
// are worked on at once:
//   1. scan_bwd_state  per chunk, in one walk: the state from zero at its end, the sum
//                      of delta, and the gradient that its own outputs send to the state
//                      at its start (with the running product of a);
//   2. scan_combine    steps both over the chunks, forward and back;
//   3. scan_bwd        per chunk: the states again from its start, then the reverse walk;
//   4. scan_bwd_bc, scan_bwd_sums  add the parts in a fixed order.
//
// The states of 4 tokens are kept in registers: the reverse walk takes the chunk in
// pieces of 8 tokens, a half at a time, and computes the states of a half again from the
// state at the piece's start, which a first walk over the chunk left in shared memory.
// The factors a_t[n] are computed each time they are used: no state and no factor is ever
// written per token.
//
// A thread holds 4 states of two neighbouring channels.  The sums over channels (dB, dC)
// are taken over its two channels, folded over the lanes that hold the warp's channels,
// joined over the warps in shared memory, and added there over the channel tiles of the
// block, which takes one chunk and a part of a group's channels and writes one row of 2 N
// sums per token.  (With one channel per thread the shared-memory pipe bounds it.)
//
// What bounds it: every factor is computed 4.4 times (once in step 1, then 7/8, 1/2, 1 and
// 1 times in step 3's walks), 1.2e9 exponentials of the shape below, 117 us of their pipe at
// 2.07 GHz; beside them about 30 paired fp32 instructions for every 4 states of a channel
// and token, 100 us of theirs; shuffles, shared memory and staging are as many instructions
// again, and 12 warps an SM (168 registers a thread) issue in 0.60 of the cycles.  With the
// states of 8 tokens in registers, 253 a thread and 8 warps, the reverse walk took 443 us.
// For N = 64 and 128 a block's tile is 16 and 8 channels, and each tile adds its sums of dB
// and dC to the block's row in global memory: no case of that width is timed.
//
// Measured (bf16, N = 16, gate, 4 x 2048 tokens of 2048 channels): 518 us (states 102,
// their steps 14, reverse walk 390, sums 12).
#include "dn_scan.cuh"

namespace dn {
namespace {

using namespace scan;

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kLen = 64;   // tokens of a chunk at most
constexpr int kPiece = 8;  // tokens staged at a time; step 3 keeps the state at the start of each piece

// One thread's place in a tile's rows: four channels of one token.
struct Place {
    int t, c, n;  // token of the tile, first channel, channels there (<= 0: none)
};

template <int CH>
__device__ __forceinline__ Place place_of(int tid, const Channels &cs) {
    constexpr int CV = CH / 4;
    Place r;
    r.t = tid / CV;
    r.c = (tid % CV) * 4;
    r.n = r.t < kPiece ? cs.n - r.c : 0;
    return r;
}

template <typename T, int N>
struct BcRows {
    static constexpr int kAll = kPiece * N / 2, kVecs = (kAll + kThreads - 1) / kThreads;
    Pack<T, 4> v[kVecs];
    __device__ __forceinline__ void fetch(const ScanParams &p, int g, long long t0, long long t1, bool c_too) {
#pragma unroll
        for (int k = 0; k < kVecs; ++k) {
            const int i = threadIdx.x + k * kThreads, which = i / (kPiece * N / 4), r = i % (kPiece * N / 4);
            const int t = r / (N / 4), c = (r % (N / 4)) * 4;
            if (i >= kAll || (which && !c_too)) continue;
            v[k].clear();
            if (t0 + t < t1) v[k].load(static_cast<const T *>(which ? p.Cm : p.Bm) + ((t0 + t) * p.G + g) * N + c);
        }
    }
    __device__ __forceinline__ void put(float *bc, bool c_too) {  // bc [2][kPiece][N]
#pragma unroll
        for (int k = 0; k < kVecs; ++k) {
            const int i = threadIdx.x + k * kThreads;
            if (i >= (c_too ? kAll : kAll / 2)) continue;
            *reinterpret_cast<float4 *>(bc + i * 4) = make_float4(v[k][0], v[k][1], v[k][2], v[k][3]);
        }
    }
};

// ---- 1: what a chunk does to the state, and its outputs to the state's gradient ------

// A thread holds 4 states of two neighbouring channels: what it reads of Bm and Cm, and
// (in step 3) its sums over channels, then serve both.
template <typename T, int L, bool VEC>
__global__ void __launch_bounds__(kThreads) scan_bwd_state(ScanParams p) {
    constexpr int N = kS * L, CH = 2 * kThreads / L;
    // two tiles in turn: a tile is written where the one before the last lay, which every
    // thread has left when it is behind the barrier of the last
    __shared__ __align__(16) float2 s_dx[2][kPiece][CH];
    __shared__ __align__(16) float s_g[2][kPiece][CH];
    __shared__ __align__(16) float s_bc[2][2 * kPiece * N];
    const int tid = threadIdx.x;
    const unsigned tiles = p.G * ((p.D / p.G + CH - 1) / CH);
    const unsigned slot = blockIdx.x / tiles;
    const int ct = blockIdx.x - slot * tiles;
    if (blockIdx.x == 0) check_offsets(p.seq, tid, kThreads);
    const SeqTile seq = seq_tile(p.seq, slot, p.chunk);
    if (!seq.ok) return;
    const Channels cs = channels_of<CH>(p, ct);
    const int ch = tid / L * 2, lane = tid % L;  // the first of this thread's channels
    const bool own[2] = {ch < cs.n, ch + 1 < cs.n};
    const long long dn = (long long)(cs.d0 + ch) * N + lane * kS, dn_at = (long long)slot * p.D * N + dn;
    f2 a[2][2], h[2][2], pr[2][2], rg[2][2];
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        a[c][0] = a[c][1] = 0ull;
        if (own[c]) {
            const float4 r = *reinterpret_cast<const float4 *>(p.A + dn + c * N);
            a[c][0] = pair(log2_rate(r.x), log2_rate(r.y));
            a[c][1] = pair(log2_rate(r.z), log2_rate(r.w));
        }
        h[c][0] = h[c][1] = rg[c][0] = rg[c][1] = 0ull;
        pr[c][0] = pr[c][1] = both(1.f);
    }
    const Place at = place_of<CH>(tid, cs);
    float bias[4], dsum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < 4; ++i) bias[i] = i < at.n && p.dt_bias ? p.dt_bias[cs.d0 + at.c + i] : 0.f;

    BcRows<T, N> bc;
    Four<T, VEC> fx, fd, fg, fz;
    auto fetch = [&](long long t0) {  // this thread's rows of a tile, one tile ahead
        const bool in = t0 + at.t < seq.t1;
        bc.fetch(p, cs.g, t0, seq.t1, true);
        fx.load(p.x, t0 + at.t, p.D, cs.d0 + at.c, at.n, in);
        fd.load(p.dt, t0 + at.t, p.D, cs.d0 + at.c, at.n, in);
        fg.load(p.dy, t0 + at.t, p.D, cs.d0 + at.c, at.n, in);
        if (p.z) fz.load(p.z, t0 + at.t, p.D, cs.d0 + at.c, at.n, in);
    };
    fetch(seq.t0);
    int turn = 0;
    for (long long t0 = seq.t0; t0 < seq.t1; t0 += kPiece, turn ^= 1) {
        if (at.t < kPiece) {
            const bool in = t0 + at.t < seq.t1;
            float g[4];
#pragma unroll
            for (int i = 0; i < 4; i += 2) {
                const f2 raw = pair(fd[i] + bias[i], fd[i + 1] + bias[i + 1]);
                float d0, d1;
                split(p.softplus ? softplus2(raw) : raw, d0, d1);
                d0 = in && i < at.n ? d0 : 0.f;
                d1 = in && i + 1 < at.n ? d1 : 0.f;
                *reinterpret_cast<float4 *>(&s_dx[turn][at.t][at.c + i]) = make_float4(d0, d0 * fx[i], d1, d1 * fx[i + 1]);
                dsum[i] += d0;
                dsum[i + 1] += d1;
                g[i] = p.z ? fg[i] * silu_f(fz[i]) : fg[i];
                g[i + 1] = p.z ? fg[i + 1] * silu_f(fz[i + 1]) : fg[i + 1];
            }
            *reinterpret_cast<float4 *>(&s_g[turn][at.t][at.c]) = make_float4(g[0], g[1], g[2], g[3]);
        }
        bc.put(s_bc[turn], true);
        __syncthreads();
        if (t0 + kPiece < seq.t1) fetch(t0 + kPiece);
#pragma unroll
        for (int t = 0; t < kPiece; ++t) {
            const float4 dx = *reinterpret_cast<const float4 *>(&s_dx[turn][t][ch]);
            const float2 go = *reinterpret_cast<const float2 *>(&s_g[turn][t][ch]);
            const ulonglong2 b = *reinterpret_cast<const ulonglong2 *>(s_bc[turn] + t * N + lane * kS);
            const ulonglong2 cv = *reinterpret_cast<const ulonglong2 *>(s_bc[turn] + (kPiece + t) * N + lane * kS);
            const f2 bb[2] = {b.x, b.y}, cc[2] = {cv.x, cv.y};
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const f2 d2 = both(c ? dx.z : dx.x), x2 = both(c ? dx.w : dx.y), g2 = both(c ? go.y : go.x);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    float e0, e1;
                    split(mul2(d2, a[c][i]), e0, e1);
                    const f2 e = pair(ex2(e0), ex2(e1));
                    h[c][i] = fma2(e, h[c][i], mul2(x2, bb[i]));
                    pr[c][i] = mul2(pr[c][i], e);
                    rg[c][i] = fma2(pr[c][i], mul2(cc[i], g2), rg[c][i]);
                }
            }
        }
    }
    // A sum that is not finite: the product of the decays may have left fp32 (rates above zero, or
    // a decay below it beside an infinite d_y) where the gradient itself does not.  It is taken
    // again as it is defined, from the last token back; only such calls pay for it.
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        float r[4], w[4];
        split(rg[c][0], r[0], r[1]);
        split(rg[c][1], r[2], r[3]);
        if (!own[c] || (r[0] - r[0]) + (r[1] - r[1]) + (r[2] - r[2]) + (r[3] - r[3]) == 0.f) continue;
        split(a[c][0], w[0], w[1]);
        split(a[c][1], w[2], w[3]);
        r[0] = r[1] = r[2] = r[3] = 0.f;
        const int d = cs.d0 + ch + c;
#pragma unroll 1
        for (long long t = seq.t1 - 1; t >= seq.t0; --t) {
            Vec<T, 1> dt, dy, z;
            Vec<T, 4> cv;
            dt.load(static_cast<const T *>(p.dt) + t * p.D + d);
            dy.load(static_cast<const T *>(p.dy) + t * p.D + d);
            cv.load(static_cast<const T *>(p.Cm) + (t * p.G + cs.g) * N + lane * kS);
            float go = dy.v[0];
            if (p.z) {
                z.load(static_cast<const T *>(p.z) + t * p.D + d);
                go *= silu_f(z.v[0]);
            }
            const float raw = dt.v[0] + (p.dt_bias ? p.dt_bias[d] : 0.f), delta = p.softplus ? softplus(raw) : raw;
#pragma unroll
            for (int i = 0; i < 4; ++i) r[i] = fmaf(cv.v[i], go, r[i]) * ex2(delta * w[i]);
        }
        rg[c][0] = pair(r[0], r[1]);
        rg[c][1] = pair(r[2], r[3]);
    }
#pragma unroll
    for (int c = 0; c < 2; ++c)
        if (own[c]) {
            *reinterpret_cast<ulonglong2 *>(p.hs + dn_at + c * N) = make_ulonglong2(h[c][0], h[c][1]);
            *reinterpret_cast<ulonglong2 *>(p.gs + dn_at + c * N) = make_ulonglong2(rg[c][0], rg[c][1]);
        }
    __syncthreads();
    if (at.t < kPiece)
#pragma unroll
        for (int i = 0; i < 4; ++i) s_g[0][at.t][at.c + i] = dsum[i];
    __syncthreads();
    if (tid < cs.n) {
        float s = 0.f;
#pragma unroll
        for (int t = 0; t < kPiece; ++t) s += s_g[0][t][tid];
        p.dsum[(long long)slot * p.D + cs.d0 + tid] = s;
    }
}

// ---- 3: the reverse walk --------------------------------------------------------------

template <int L>
struct Smem {  // offsets in floats
    static constexpr int N = kS * L, CH = 2 * kThreads / L;
    static constexpr int kD = 0;                           // [kLen][CH]: delta
    static constexpr int kX = kD + kLen * CH;              // [2][kPiece][CH]: x, two tiles in turn
    static constexpr int kBc = kX + 2 * kPiece * CH;       // [2][2][kPiece][N], two tiles in turn
    static constexpr int kGo = kBc + 4 * kPiece * N;       // [kPiece][CH]
    static constexpr int kRes = kGo + kPiece * CH;         // [3][kPiece][CH]: s, sum q A, C.h
    static constexpr int kStart = kRes + 3 * kPiece * CH;  // [kLen / kPiece][2][kThreads][4]
    static constexpr int kRed = kStart + kLen / kPiece * 2 * kThreads * 4;  // [kWarps][kPiece][2 N]
    static constexpr int kAll = kRed + kWarps * kPiece * 2 * N;
};

template <typename T, int L, bool VEC>
__global__ void __launch_bounds__(kThreads, 3) scan_bwd(ScanParams p, int parts) {
    using M = Smem<L>;
    constexpr int N = M::N, CH = M::CH;
    extern __shared__ __align__(16) float sm[];
    float(*s_d)[CH] = reinterpret_cast<float(*)[CH]>(sm + M::kD);
    float(*s_x)[CH] = reinterpret_cast<float(*)[CH]>(sm + M::kX);
    float(*s_go)[CH] = reinterpret_cast<float(*)[CH]>(sm + M::kGo);
    float(*s_res)[kPiece][CH] = reinterpret_cast<float(*)[kPiece][CH]>(sm + M::kRes);
    ulonglong2 *s_start = reinterpret_cast<ulonglong2 *>(sm + M::kStart);
    float *s_red = sm + M::kRed;

    wait_for_launches();
    const int tid = threadIdx.x, warp = tid >> 5;
    const unsigned split_by = parts * p.G, slot = blockIdx.x / split_by;
    const int gp = blockIdx.x - slot * split_by, g = gp / parts, part = gp - g * parts;
    const int per = (p.D / p.G + CH - 1) / CH;  // channel tiles of a group
    const int first = (int)((long long)per * part / parts), last = (int)((long long)per * (part + 1) / parts);
    const SeqTile seq = seq_tile(p.seq, slot, p.chunk);
    const int ch = tid / L * 2, lane = tid % L;  // the first of this thread's channels
    const int len = seq.ok ? (int)(seq.t1 - seq.t0) : 0;
    const int nt = (len + kPiece - 1) / kPiece;

    // the block's row of sums over channels: token t of the chunk at t * bc_step
    float *bc_out = p.bc + (((long long)part * p.seq.tokens + seq.t0) * p.G + g) * 2 * N;
    const long long bc_step = (long long)p.G * 2 * N;

    for (int ct = g * per + first; ct < g * per + last; ++ct) {
        const Channels cs = channels_of<CH>(p, ct);
        const bool own[2] = {ch < cs.n, ch + 1 < cs.n};
        const long long dn = (long long)(cs.d0 + ch) * N + lane * kS, dn_at = (long long)slot * p.D * N + dn;
        const Place at = place_of<CH>(tid, cs);
        if (nt == 0) {  // a slot without tokens adds nothing
#pragma unroll
            for (int c = 0; c < 2; ++c)
                if (own[c]) *reinterpret_cast<float4 *>(p.gs + dn_at + c * N) = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int i = tid; i < 2 * cs.n; i += kThreads) {
                const int which = i / cs.n, c = i - which * cs.n;
                p.vec[((long long)slot * 2 + which) * p.D + cs.d0 + c] = 0.f;
            }
            continue;
        }
        f2 a2[2][2], h[2][2], carry[2][2], dA[2][2];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            a2[c][0] = a2[c][1] = h[c][0] = h[c][1] = carry[c][0] = carry[c][1] = dA[c][0] = dA[c][1] = 0ull;
            if (own[c]) {
                const float4 r = *reinterpret_cast<const float4 *>(p.A + dn + c * N);
                a2[c][0] = pair(log2_rate(r.x), log2_rate(r.y));
                a2[c][1] = pair(log2_rate(r.z), log2_rate(r.w));
                const ulonglong2 hr = *reinterpret_cast<const ulonglong2 *>(p.hs + dn_at + c * N);
                const ulonglong2 gr = *reinterpret_cast<const ulonglong2 *>(p.gs + dn_at + c * N);
                h[c][0] = hr.x; h[c][1] = hr.y;
                carry[c][0] = gr.x; carry[c][1] = gr.y;
            }
        }
        auto decay = [&](f2 d2, int c, int i) {  // e^{delta A} of pair i of channel c
            float e0, e1;
            split(mul2(d2, a2[c][i]), e0, e1);
            return pair(ex2(e0), ex2(e1));
        };
        float bias[4], skip[4], sD[4] = {0.f, 0.f, 0.f, 0.f}, sb[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            bias[i] = i < at.n && p.dt_bias ? p.dt_bias[cs.d0 + at.c + i] : 0.f;
            skip[i] = i < at.n && p.Dskip ? p.Dskip[cs.d0 + at.c + i] : 0.f;
        }
        // This thread's rows of a tile, loaded one tile ahead.
        BcRows<T, N> bc;
        Four<T, VEC> nx, nd, ng, nz;
        auto fetch = [&](int k, bool back) {
            const long long t0 = seq.t0 + k * kPiece;
            const bool in = t0 + at.t < seq.t1;
            bc.fetch(p, cs.g, t0, seq.t1, back);
            nx.load(p.x, t0 + at.t, p.D, cs.d0 + at.c, at.n, in);
            nd.load(p.dt, t0 + at.t, p.D, cs.d0 + at.c, at.n, in);
            if (back) ng.load(p.dy, t0 + at.t, p.D, cs.d0 + at.c, at.n, in);
            if (back && p.z) nz.load(p.z, t0 + at.t, p.D, cs.d0 + at.c, at.n, in);
        };
        auto bc_of = [&](int k) { return sm + M::kBc + (k & 1) * 2 * kPiece * N; };
        auto x_of = [&](int k) { return s_x + (k & 1) * kPiece; };
        auto put_x = [&](int k, const Four<T, VEC> &v) {  // absent channels: zeros, as they were loaded
            *reinterpret_cast<float4 *>(&x_of(k)[at.t][at.c]) = make_float4(v[0], v[1], v[2], v[3]);
        };
        // forward over the chunk: the state at the start of every piece.  A tile's rows of
        // Bm lie where those of the tile before the last lay, which every thread has left
        // when it is behind the barrier of the last.
        fetch(0, false);
        for (int k = 0; k < nt; ++k) {
            if (at.t < kPiece) {
                const bool in = seq.t0 + k * kPiece + at.t < seq.t1;
#pragma unroll
                for (int i = 0; i < 4; i += 2) {
                    const f2 raw = pair(nd[i] + bias[i], nd[i + 1] + bias[i + 1]);
                    float d0, d1;
                    split(p.softplus ? softplus2(raw) : raw, d0, d1);
                    d0 = in && i < at.n ? d0 : 0.f;
                    d1 = in && i + 1 < at.n ? d1 : 0.f;
                    *reinterpret_cast<float2 *>(&s_d[k * kPiece + at.t][at.c + i]) = make_float2(d0, d1);
                }
                put_x(k, nx);
            }
            float *s_bc = bc_of(k);
            bc.put(s_bc, false);
            __syncthreads();
            if (k + 1 < nt) fetch(k + 1, false);
            else fetch(k, true);
#pragma unroll
            for (int c = 0; c < 2; ++c)
                s_start[(k * 2 + c) * kThreads + tid] = make_ulonglong2(h[c][0], h[c][1]);
            if (k + 1 < nt) {
#pragma unroll
                for (int t = 0; t < kPiece; ++t) {
                    const float2 dd = *reinterpret_cast<const float2 *>(&s_d[k * kPiece + t][ch]);
                    const float2 xx = *reinterpret_cast<const float2 *>(&x_of(k)[t][ch]);
                    const ulonglong2 b = *reinterpret_cast<const ulonglong2 *>(s_bc + t * N + lane * kS);
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        const f2 d2 = both(c ? dd.y : dd.x), x2 = both(c ? dd.y * xx.y : dd.x * xx.x);
                        h[c][0] = fma2(decay(d2, c, 0), h[c][0], mul2(x2, b.x));
                        h[c][1] = fma2(decay(d2, c, 1), h[c][1], mul2(x2, b.y));
                    }
                }
            }
        }
        // back over the chunk
        for (int k = nt - 1; k >= 0; --k) {
            const long long t0 = seq.t0 + k * kPiece;
            const bool in = t0 + at.t < seq.t1 && at.t < kPiece;
            const Four<T, VEC> fx = nx, fd = nd, fg = ng, fz = nz;
            // (the barriers of two tiles lie between the writes of one place of Bm and Cm)
            const int turn = nt - 1 - k + nt;
            float *s_bc = bc_of(turn);
            if (at.t < kPiece) {
                put_x(turn, fx);
                float4 go;
                go.x = p.z ? fg[0] * silu_f(fz[0]) : fg[0];
                go.y = p.z ? fg[1] * silu_f(fz[1]) : fg[1];
                go.z = p.z ? fg[2] * silu_f(fz[2]) : fg[2];
                go.w = p.z ? fg[3] * silu_f(fz[3]) : fg[3];
                *reinterpret_cast<float4 *>(&s_go[at.t][at.c]) = go;
            }
            bc.put(s_bc, true);
            __syncthreads();
            if (k > 0) fetch(k - 1, true);
            // The piece in two halves of four tokens, the second first (its states need the
            // first half's steps once more): half the registers for the states.
#pragma unroll 1
            for (int u = kPiece - 4; u >= 0; u -= 4) {
                f2 hh[5][2][2];
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const ulonglong2 r = s_start[(k * 2 + c) * kThreads + tid];
                    hh[0][c][0] = r.x;
                    hh[0][c][1] = r.y;
                }
                auto step = [&](int t, f2 (&to)[2][2], const f2 (&from)[2][2]) {  // token t of the tile
                    const float2 dd = *reinterpret_cast<const float2 *>(&s_d[k * kPiece + t][ch]);
                    const float2 xx = *reinterpret_cast<const float2 *>(&x_of(turn)[t][ch]);
                    const ulonglong2 b = *reinterpret_cast<const ulonglong2 *>(s_bc + t * N + lane * kS);
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        const f2 d2 = both(c ? dd.y : dd.x), x2 = both(c ? dd.y * xx.y : dd.x * xx.x);
                        to[c][0] = fma2(decay(d2, c, 0), from[c][0], mul2(x2, b.x));
                        to[c][1] = fma2(decay(d2, c, 1), from[c][1], mul2(x2, b.y));
                    }
                };
                if (u > 0)
#pragma unroll
                    for (int t = 0; t < 4; ++t) step(t, hh[0], hh[0]);
                float py[2][4];
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    step(u + w, hh[w + 1], hh[w]);
                    if (p.z) {
                        const ulonglong2 cc = *reinterpret_cast<const ulonglong2 *>(s_bc + (kPiece + u + w) * N + lane * kS);
#pragma unroll
                        for (int c = 0; c < 2; ++c)
                            py[c][w] = sum_of(fma2(cc.x, hh[w + 1][c][0], mul2(cc.y, hh[w + 1][c][1])));
                    }
                }
                if (p.z)
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        const float y = sum4<L>(py[c], lane);
                        if (lane < 4) s_res[2][u + lane][ch + c] = y;
                    }
                float ps[2][4], pq[2][4];
                // Tokens of the half up to the chunk's last.  Those behind it have no step, but the
                // state before them may be infinite, and no step times that is not 0: d_A skips them.
                const int left = len - k * kPiece - u;
#pragma unroll
                for (int w = 3; w >= 0; --w) {
                    const int t = u + w;
                    const float2 dd = *reinterpret_cast<const float2 *>(&s_d[k * kPiece + t][ch]);
                    const float2 xx = *reinterpret_cast<const float2 *>(&x_of(turn)[t][ch]);
                    const float2 go = *reinterpret_cast<const float2 *>(&s_go[t][ch]);
                    const ulonglong2 b = *reinterpret_cast<const ulonglong2 *>(s_bc + t * N + lane * kS);
                    const ulonglong2 cv = *reinterpret_cast<const ulonglong2 *>(s_bc + (kPiece + t) * N + lane * kS);
                    const f2 bb[2] = {b.x, b.y}, cc[2] = {cv.x, cv.y};
                    f2 vb[2] = {0ull, 0ull}, vc[2] = {0ull, 0ull};  // parts of dB and dC
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        const f2 d2 = both(c ? dd.y : dd.x), x2 = both(c ? dd.y * xx.y : dd.x * xx.x), g2 = both(c ? go.y : go.x);
                        f2 s2 = 0ull, q2 = 0ull;
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const f2 gr = fma2(g2, cc[i], carry[c][i]);
                            carry[c][i] = mul2(gr, decay(d2, c, i));
                            const f2 qq = mul2(carry[c][i], hh[w][c][i]);
                            dA[c][i] = fma2(d2, w < left ? qq : 0ull, dA[c][i]);
                            q2 = fma2(qq, a2[c][i], q2);
                            s2 = fma2(gr, bb[i], s2);
                            vb[i] = fma2(gr, x2, vb[i]);
                            vc[i] = fma2(g2, hh[w + 1][c][i], vc[i]);
                        }
                        ps[c][w] = sum_of(s2);
                        pq[c][w] = sum_of(q2);
                    }
                    float v[8];
                    split(vb[0], v[0], v[1]);
                    split(vb[1], v[2], v[3]);
                    split(vc[0], v[4], v[5]);
                    split(vc[1], v[6], v[7]);
                    // sums over the warp's channels: each lane ends with L / 4 of the 8 values
                    int base = 0;
                    if constexpr (L <= 16) {
                        fold<8>(v, 16, tid & 16);
                        base = tid & 16 ? 4 : 0;
                    }
                    if constexpr (L <= 8) {
                        float v4[4] = {v[0], v[1], v[2], v[3]};
                        fold<4>(v4, 8, tid & 8);
                        base += tid & 8 ? 2 : 0;
                        v[0] = v4[0];
                        v[1] = v4[1];
                    }
                    if constexpr (L <= 4) {
                        float v2[2] = {v[0], v[1]};
                        fold<2>(v2, 4, tid & 4);
                        base += tid & 4 ? 1 : 0;
                        v[0] = v2[0];
                    }
#pragma unroll
                    for (int j = 0; j < L / 4; ++j) {
                        const int vi = base + j;
                        s_red[(warp * kPiece + t) * 2 * N + (vi >> 2) * N + lane * kS + (vi & 3)] = v[j];
                    }
                }
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const float s = sum4<L>(ps[c], lane), r = sum4<L>(pq[c], lane);
                    if (lane < 4) {
                        s_res[0][u + lane][ch + c] = s;
                        s_res[1][u + lane][ch + c] = r * 0.6931471806f;  // the rates are in units of log2
                    }
                }
            }
            __syncthreads();
            // what follows reads what lies before this barrier, and ends before the next
            for (int i = tid; i < kPiece * 2 * N; i += kThreads) {
                const int t = k * kPiece + i / (2 * N);
                if (t < len) {
                    float sum = 0.f;
#pragma unroll
                    for (int w = 0; w < kWarps; ++w) sum += s_red[w * kPiece * 2 * N + i];
                    float *o = bc_out + t * bc_step + i % (2 * N);
                    *o = ct > g * per + first ? *o + sum : sum;
                }
            }
            if (in && at.n > 0) {
                float ox[4], od[4], oz[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float s = s_res[0][at.t][at.c + i], r = s_res[1][at.t][at.c + i];
                    const float delta = s_d[k * kPiece + at.t][at.c + i], go = s_go[at.t][at.c + i];
                    ox[i] = p.Dskip ? fmaf(delta, s, skip[i] * go) : delta * s;
                    od[i] = fmaf(fx[i], s, r);
                    if (p.softplus) od[i] *= sigmoid_f(fd[i] + bias[i]);
                    if (p.z) {
                        const float y = s_res[2][at.t][at.c + i];
                        oz[i] = fg[i] * (p.Dskip ? fmaf(skip[i], fx[i], y) : y) * silu_grad_f(fz[i]);
                    }
                    if (i < at.n) {
                        sD[i] = fmaf(go, fx[i], sD[i]);
                        sb[i] += od[i];
                    }
                }
                const long long o = (t0 + at.t) * p.D + cs.d0 + at.c;
                store4<T, VEC>(static_cast<T *>(p.dx) + o, at.n, ox);
                store4<T, VEC>(static_cast<T *>(p.ddt) + o, at.n, od);
                if (p.z) store4<T, VEC>(static_cast<T *>(p.dz) + o, at.n, oz);
            }
        }
#pragma unroll
        for (int c = 0; c < 2; ++c)
            if (own[c]) *reinterpret_cast<ulonglong2 *>(p.gs + dn_at + c * N) = make_ulonglong2(dA[c][0], dA[c][1]);
        __syncthreads();
        if (at.t < kPiece)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                s_res[0][at.t][at.c + i] = sD[i];
                s_res[1][at.t][at.c + i] = sb[i];
            }
        __syncthreads();
        for (int i = tid; i < 2 * cs.n; i += kThreads) {
            const int which = i / cs.n, c = i - which * cs.n;
            float s = 0.f;
#pragma unroll
            for (int t = 0; t < kPiece; ++t) s += s_res[which][t][c];
            p.vec[((long long)slot * 2 + which) * p.D + cs.d0 + c] = s;
        }
        __syncthreads();
    }
}

// ---- 4: the parts' sums ------------------------------------------------------------------

// One vector of four states of a token and group: d_Bm and d_Cm rows lie one
// after the other in every part.
template <typename T>
__global__ void __launch_bounds__(128) scan_bwd_bc(ScanParams p, int parts) {
    wait_for_launches();
    const long long i = (long long)blockIdx.x * 128 + threadIdx.x;
    const int q = p.N / 2;  // vectors of a row of both
    const long long row = i / q;
    const int v = (int)(i - row * q);
    long long tokens = p.seq.tokens;
    if (p.seq.cu) {  // rows behind the last sequence stay as they are
        const long long end = p.seq.cu[p.seq.N];
        tokens = end < 0 ? 0 : end < tokens ? end : tokens;
    }
    if (row >= tokens * p.G) return;
    const float4 *src = reinterpret_cast<const float4 *>(p.bc) + i;
    const long long step = p.seq.tokens * p.G * q;
    float4 s = src[0];
#pragma unroll 8
    for (int k = 1; k < parts; ++k) {
        const float4 o = src[k * step];
        s.x += o.x; s.y += o.y; s.z += o.z; s.w += o.w;
    }
    Vec<T, 4> out;
    out.v[0] = s.x; out.v[1] = s.y; out.v[2] = s.z; out.v[3] = s.w;
    const bool c = v >= q / 2;
    out.store(static_cast<T *>(c ? p.dCm : p.dBm) + row * p.N + (c ? v - q / 2 : v) * 4);
}

// d_A (blockIdx.y = 0: columns of D N), d_Dskip and d_dt_bias (1: columns of 2 D),
// over the slots: 32 columns and 8 slices of the slots per block.
__global__ void __launch_bounds__(256) scan_bwd_sums(ScanParams p, long long slots) {
    __shared__ float red[8][32];
    wait_for_launches();
    const long long cols = blockIdx.y ? 2LL * p.D : (long long)p.D * p.N;
    const long long c = (long long)blockIdx.x * 32 + threadIdx.x;
    if ((long long)blockIdx.x * 32 >= cols) return;
    const float *src = blockIdx.y ? p.vec : p.gs;
    float a = 0.f;
    if (c < cols)
#pragma unroll 8
        for (long long s = threadIdx.y; s < slots; s += 8) a += src[s * cols + c];
    red[threadIdx.y][threadIdx.x] = a;
    __syncthreads();
    if (threadIdx.y || c >= cols) return;
    float v = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) v += red[k][threadIdx.x];
    if (blockIdx.y == 0) p.dA[c] = v;
    else if (c < p.D) {
        if (p.dDskip) p.dDskip[c] = v;
    } else if (p.ddt_bias) {
        p.ddt_bias[c - p.D] = v;
    }
}

int tiles_of_group(int D, int G, int N) {
    const int ch = 2 * kThreads / (N / kS);
    return (D / G + ch - 1) / ch;
}

// Tokens of a chunk: 64, or fewer where that leaves places of the GPU without a block.
int bwd_chunk(int n_seqs, long long tokens, int D, int G, int N) {
    const long long tiles = (long long)G * tiles_of_group(D, G, N);
    int len = n_seqs > 0 ? scan_least_chunk(tokens / n_seqs) : kLen;
    while (len < kLen && (tokens / (2 * len) + n_seqs) * tiles >= kSms * 3) len *= 2;
    return len < kLen ? len : kLen;
}

// Parts that a group's channels are split into: enough blocks to fill the GPU many times,
// at most one per tile of channels.
int channel_parts(int n_seqs, long long tokens, int D, int G, int N) {
    const long long tiles = tiles_of_group(D, G, N);
    const long long rows = (tokens / bwd_chunk(n_seqs, tokens, D, G, N) + n_seqs) * G;
    const long long want = rows > 0 ? (kSms * 32 + rows - 1) / rows : 1;
    return (int)(want < tiles ? want : tiles);
}

template <typename T, int L, bool VEC>
cudaError_t bwd_l(const ScanParams &p, cudaStream_t stream) {
    constexpr int CH = 2 * kThreads / L;
    const long long slots = tile_slots(p.seq, p.chunk);
    const int parts = channel_parts(p.seq.N, p.seq.tokens, p.D, p.G, p.N);
    const long long states = slots * channel_tiles<CH>(p.D, p.G);
    const long long blocks = slots * p.G * parts;
    if (states > 0x7fffffffLL || blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
    cudaError_t err = cudaSuccess;
    if (slots > 0) {
        scan_bwd_state<T, L, VEC><<<(unsigned)states, kThreads, 0, stream>>>(p);
        err = cudaGetLastError();
        if (err == cudaSuccess) err = scan_combine_launch(p, true, stream);
        if (err != cudaSuccess) return err;
        constexpr int bytes = Smem<L>::kAll * sizeof(float);
        err = allow_smem<scan_bwd<T, L, VEC>>(bytes);
        if (err != cudaSuccess) return err;
        err = launch_after(scan_bwd<T, L, VEC>, dim3((unsigned)blocks), dim3(kThreads), bytes, stream, p, parts);
        if (err != cudaSuccess) return err;
    }
    const long long vecs = p.seq.tokens * p.G * (p.N / 2);
    if (vecs > 0 && p.seq.N > 0) {
        const long long grid = (vecs + 127) / 128;
        if (grid > 0x7fffffffLL) return cudaErrorInvalidValue;
        err = launch_after(scan_bwd_bc<T>, dim3((unsigned)grid), dim3(128), 0, stream, p, parts);
        if (err != cudaSuccess) return err;
    }
    const long long cols = ((long long)p.D * p.N + 31) / 32;
    return launch_after(scan_bwd_sums, dim3((unsigned)cols, 2), dim3(32, 8), 0, stream, p, slots);
}

template <typename T>
cudaError_t bwd_t(const ScanParams &p, cudaStream_t stream) {
    const bool vec = (p.D / p.G) % 4 == 0;
    switch (p.N) {
        case 16: return vec ? bwd_l<T, 4, true>(p, stream) : bwd_l<T, 4, false>(p, stream);
        case 32: return vec ? bwd_l<T, 8, true>(p, stream) : bwd_l<T, 8, false>(p, stream);
        case 64: return vec ? bwd_l<T, 16, true>(p, stream) : bwd_l<T, 16, false>(p, stream);
        default: return vec ? bwd_l<T, 32, true>(p, stream) : bwd_l<T, 32, false>(p, stream);
    }
}

// The workspace's parts, in floats, each a multiple of 4.
struct Sizes {
    size_t hs, dsum, gs, vec, bc;
    size_t all() const { return (hs + dsum + gs + vec + bc) * 4; }
};
Sizes sizes(int n_seqs, long long tokens, int D, int G, int N) {
    const size_t slots = (size_t)(tokens / bwd_chunk(n_seqs, tokens, D, G, N) + n_seqs);
    const size_t parts = (size_t)channel_parts(n_seqs, tokens, D, G, N);
    auto up = [](size_t v) { return (v + 3) / 4 * 4; };
    return {slots * D * N, up(slots * D), slots * D * N, up(slots * 2 * D), parts * (size_t)tokens * G * 2 * N};
}

}  // namespace

size_t scan_bwd_workspace(int n_seqs, long long tokens, int D, int G, int N) {
    const size_t b = sizes(n_seqs, tokens, D, G, N).all();
    return b > 16 ? b : 16;
}

void scan_bwd_carve(ScanParams &p, void *workspace) {
    const Sizes s = sizes(p.seq.N, p.seq.tokens, p.D, p.G, p.N);
    p.chunk = bwd_chunk(p.seq.N, p.seq.tokens, p.D, p.G, p.N);
    p.hs = static_cast<float *>(workspace);
    p.dsum = p.hs + s.hs;
    p.gs = p.dsum + s.dsum;
    p.vec = p.gs + s.gs;
    p.bc = p.vec + s.vec;
}

cudaError_t scan_bwd_launch(ScanParams p, bool bf16, cudaStream_t stream, const char **name) {
#define DN_SCAN_BWD "scan_bwd_state+scan_combine+scan_bwd+"
    if (p.seq.N == 0) *name = "scan_bwd_sums";
    else if (p.seq.tokens == 0) *name = bf16 ? DN_SCAN_BWD "scan_bwd_sums<bf16>" : DN_SCAN_BWD "scan_bwd_sums<f32>";
    else *name = bf16 ? DN_SCAN_BWD "scan_bwd_bc+scan_bwd_sums<bf16>" : DN_SCAN_BWD "scan_bwd_bc+scan_bwd_sums<f32>";
#undef DN_SCAN_BWD
    return bf16 ? bwd_t<__nv_bfloat16>(p, stream) : bwd_t<float>(p, stream);
}

}  // namespace dn
