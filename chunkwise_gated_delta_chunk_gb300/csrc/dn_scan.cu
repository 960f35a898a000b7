// Selective state space scan, forward.
//
//     delta = softplus(dt + dt_bias),  h[n] = e^{delta A[n]} h[n] + delta B[n] x,
//     y = (sum_n C[n] h[n] + Dskip x) silu(z)
//
// A thread owns two neighbouring channels and 16 of their states (N / 16 threads share a
// channel pair, a block has 64 channels), and walks the tokens of one sequence or of one
// chunk of it.  So a row of x, dt, z and y is read and written by its own threads
// without any exchange, delta is computed where it is used, and only the rows of Bm and
// Cm, which all channels of a group share, go through shared memory: what a thread loads
// there serves two channels.  (With 4 states of one channel per thread the shared-memory
// pipe, 13 of its cycles per 8 channels and token, and the shuffles of the sum over n took
// most of the time: 252 us at the shape below.)
//
// What bounds it: N exponentials (32 a cycle and SM) and 2 N paired fp32 instructions (64
// pairs a cycle and SM) per channel and token, each 55000 cycles of the shape below (27 us at
// the 2.07 GHz it runs at), against 6 to 8 bytes (20 us).  A cut sequence pays the
// exponentials twice.  The schedulers issue in 0.56 to 0.59 of the cycles: 128 registers a
// thread leave 4 warps for each of them, and more warps spill.
//
// Few channels leave most SMs idle, so sequences are then cut into chunks: one
// launch computes each chunk's state from zero and its sum of delta, a second
// steps the states over the chunks (the state at a chunk's end is
// e^{A sum delta} times the one at its start, plus the chunk's own), and the
// scan itself starts every chunk from its state.  A single token has a kernel of its
// own, one thread per 4 states, so that the states are read and written in whole lines.
//
// Measured (bf16, N = 16, gate): 4 x 2048 tokens of 2048 channels 157 us (states 64,
// their steps 8, scan 85); 64 x 256 tokens of 4096 channels, uncut, 341 us; one token of
// 64 sequences, 2048 channels, 7 us.
#include "dn_scan.cuh"

namespace dn {
namespace {

using namespace scan;

constexpr int kTile = 16;      // tokens whose rows of Bm and Cm are staged at a time
constexpr int kT = 16;         // states of a thread
constexpr int kResident = 16;  // warps of an SM (128 registers a thread)
constexpr int kCh = 64;        // channels of a block: two for each of its threads, N / kT threads sharing two

// Two neighbouring elements; PAIR: their address is a multiple of their size.  (Else
// they stay apart until they are used: joining them would wait for their loads.)
template <typename T, bool PAIR>
struct Two {
    Pack<T, PAIR ? 2 : 1> a, b;
    __device__ __forceinline__ void clear() {
        a.clear();
        b.clear();
    }
    __device__ __forceinline__ void load(const T *src, bool has0, bool has1) {
        if (has0) a.load(src);
        if (!PAIR && has1) b.load(src + 1);
    }
    __device__ __forceinline__ f2 get() const { return PAIR ? pair(a[0], a[PAIR ? 1 : 0]) : pair(a[0], b[0]); }
};
template <typename T, bool PAIR>
__device__ __forceinline__ void store2(T *dst, float a, float b, bool has0, bool has1) {
    if constexpr (PAIR) {
        Vec<T, 2> v;
        v.v[0] = a;
        v.v[1] = b;
        if (has0) v.store(dst);
    } else {
        Vec<T, 1> v;
        v.v[0] = a;
        if (has0) v.store(dst);
        v.v[0] = b;
        if (has1) v.store(dst + 1);
    }
}

// ---- the scan over the tokens of a sequence or a chunk ------------------------------

template <typename T, int L, bool PAIR, bool STATE>
__global__ void __launch_bounds__(32 * L, kResident / L) scan_fwd(ScanParams p) {
    constexpr int NT = 32 * L, N = kT * L, CH = kCh, Q = kT / 4;
    constexpr int kWhich = STATE ? 1 : 2;                // Bm alone, or Cm too
    constexpr int kBc = kTile * N * kWhich / 4 / NT;     // their vectors of a tile per thread
    constexpr int U = 2;                                 // tokens of x, dt, z in flight
    constexpr int S = N <= 64 ? 2 : 1;                   // tiles of Bm and Cm in flight
    using Bcs = Ahead<T, kBc, NT, S>;
    __shared__ __align__(16) char ring[Bcs::kBytes];
    __shared__ __align__(16) float s_bc[kTile][kWhich][N];
    constexpr int kRow = 2 * kT + 4;  // a thread's states in shared memory, rows apart by an odd number of vectors
    __shared__ __align__(16) float s_st[L == 1 ? 32 * kRow : 4];
    auto sync = [] {
        if constexpr (L == 1) __syncwarp();
        else __syncthreads();
    };

    const int tid = threadIdx.x;
    const unsigned tiles = p.G * ((p.D / p.G + CH - 1) / CH);
    const unsigned slot = blockIdx.x / tiles;
    const int ct = blockIdx.x - slot * tiles;
    if (!STATE && p.chunk) wait_for_launches();
    if (blockIdx.x == 0) check_offsets(p.seq, tid, NT);
    const SeqTile seq = p.chunk ? seq_tile(p.seq, slot, p.chunk) : seq_whole(p.seq, (int)slot);
    if (!seq.ok) return;
    if (STATE && seq.t1 >= seq.eos) return;  // nothing starts from the last chunk's end
    const Channels cs = channels_of<CH>(p, ct);
    const int pi = tid / L, lane = tid % L, d = cs.d0 + 2 * pi;
    const bool has0 = 2 * pi < cs.n, has1 = 2 * pi + 1 < cs.n;
    const int len = (int)(seq.t1 - seq.t0);
    const bool gate = !STATE && p.z;

    Bcs bcs;
    auto fetch_bc = [&](int t0, int s) {
#pragma unroll
        for (int k = 0; k < kBc; ++k) {
            const int v = (tid + k * NT) * 4, t = v / (kWhich * N), which = v / N % kWhich, c = v % N;
            bcs.issue(ring, s, k,
                      static_cast<const T *>(which ? p.Cm : p.Bm) + ((seq.t0 + t0 + t) * p.G + cs.g) * N + c,
                      t0 + t < len);
        }
        bcs.commit();
    };
#pragma unroll
    for (int s = 0; s < S; ++s) fetch_bc(s * kTile, s);

    // Rows of x, dt, z and y: a token's offset from the tensors' first element for this
    // thread.  What is fetched lies U tokens ahead of what is computed.
    const long long first = seq.t0 * p.D + d;
    const T *xp = static_cast<const T *>(p.x) + first, *dp = static_cast<const T *>(p.dt) + first;
    const T *zp = gate ? static_cast<const T *>(p.z) + first : xp;
    T *yp = static_cast<T *>(p.y) + first;
    const long long D = p.D;
    Two<T, PAIR> nx[U], nd[U], nz[U];
    // All rows of U tokens at once, and waited for at once when the next U are at hand: a
    // load among those still in flight would make the wait for an older one wait for it too.
    auto fetch = [&](int left) {
#pragma unroll
        for (int k = 0; k < U; ++k)
            if (k < left) {
                nx[k].load(xp + k * D, has0, has1);
                nd[k].load(dp + k * D, has0, has1);
                if (gate) nz[k].load(zp + k * D, has0, has1);
            }
        xp += U * D, dp += U * D, zp += U * D;
    };
#pragma unroll
    for (int k = 0; k < U; ++k) nx[k].clear(), nd[k].clear(), nz[k].clear();
    fetch(len);

    f2 a[2][kT / 2], h[2][kT / 2];  // rates and states of both channels
    const float *from = STATE ? nullptr
                        : p.chunk ? p.hs + (long long)slot * p.D * N
                        : p.h0 ? p.h0 + (long long)seq.n * p.D * N : nullptr;
    // The states of this thread, from or to [channel][N].  L = 1: a block's states lie one
    // after the other in memory; they are read in whole lines and handed to their threads
    // through shared memory (each thread's 32 on their own are 32 lines per access).
    auto exchange = [&](auto *global, f2 (&v)[2][kT / 2], bool out) {
        if constexpr (L > 1) {
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
                for (int i = 0; i < Q; ++i) {
                    const bool has = c ? has1 : has0;
                    auto *at = global + (long long)(2 * pi + c) * N + lane * kT + i * 4;
                    if (out) {
                        if (has) *reinterpret_cast<ulonglong2 *>(const_cast<float *>(at)) = make_ulonglong2(v[c][2 * i], v[c][2 * i + 1]);
                    } else {
                        ulonglong2 r = make_ulonglong2(0ull, 0ull);
                        if (has) r = *reinterpret_cast<const ulonglong2 *>(at);
                        v[c][2 * i] = r.x;
                        v[c][2 * i + 1] = r.y;
                    }
                }
        } else {
            const int block = cs.n * N;  // floats
            if (out) {
#pragma unroll
                for (int c = 0; c < 2; ++c)
#pragma unroll
                    for (int i = 0; i < Q; ++i)
                        *reinterpret_cast<ulonglong2 *>(s_st + tid * kRow + c * kT + i * 4) =
                            make_ulonglong2(v[c][2 * i], v[c][2 * i + 1]);
                __syncwarp();
            }
            for (int f = tid * 4; f < block; f += 128) {
                // float f of the block: channel f / N of thread f / N / 2, state f % N
                float *sp = s_st + f / N / 2 * kRow + f / N % 2 * kT + f % N;
                if (out) *reinterpret_cast<float4 *>(const_cast<float *>(global) + f) = *reinterpret_cast<float4 *>(sp);
                else *reinterpret_cast<float4 *>(sp) = *reinterpret_cast<const float4 *>(global + f);
            }
            __syncwarp();
            if (!out) {
#pragma unroll
                for (int c = 0; c < 2; ++c)
#pragma unroll
                    for (int i = 0; i < Q; ++i) {
                        const ulonglong2 r = *reinterpret_cast<const ulonglong2 *>(s_st + tid * kRow + c * kT + i * 4);
                        const bool has = c ? has1 : has0;
                        v[c][2 * i] = has ? r.x : 0ull;
                        v[c][2 * i + 1] = has ? r.y : 0ull;
                    }
                __syncwarp();
            }
        }
    };
    exchange(p.A + (long long)cs.d0 * N, a, false);
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int i = 0; i < kT / 2; ++i) {
            float lo, hi;
            split(a[c][i], lo, hi);
            a[c][i] = pair(log2_rate(lo), log2_rate(hi));
            h[c][i] = 0ull;
        }
    if (from) exchange(from + (long long)cs.d0 * N, h, false);
    const f2 bias = p.dt_bias ? pair(has0 ? p.dt_bias[d] : 0.f, has1 ? p.dt_bias[d + 1] : 0.f) : 0ull;
    const f2 skip = !STATE && p.Dskip ? pair(has0 ? p.Dskip[d] : 0.f, has1 ? p.Dskip[d + 1] : 0.f) : 0ull;
    // without Dskip x adds nothing, an infinite one neither (its bits masked: a branch takes 2 % longer)
    const f2 keep = !STATE && p.Dskip ? ~0ull : 0ull;
    f2 dsum = 0ull;

    int stage = 0;
    for (int t0 = 0; t0 < len; t0 += kTile) {
        bcs.wait();
        sync();  // the last tile's rows are done with
#pragma unroll
        for (int k = 0; k < kBc; ++k) {
            const Pack<T, 4> r = bcs.get(ring, stage, k);
            const int v = (tid + k * NT) * 4;
            const bool in = t0 + v / (kWhich * N) < len;  // rows behind the last token: zeros
            *reinterpret_cast<float4 *>(&s_bc[0][0][0] + v) =
                in ? make_float4(r[0], r[1], r[2], r[3]) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
        fetch_bc(t0 + S * kTile, stage);
        stage = stage + 1 == S ? 0 : stage + 1;
        sync();
        for (int u = 0; u < kTile && t0 + u < len; u += U) {
            const int left = len - t0 - u;  // tokens from here on
            // the steps of U tokens together: each is a long chain of its own.  A token
            // behind the last has none, and so leaves the states as they are.
            f2 delta[U];
            Two<T, PAIR> fx[U], fz[U];
#pragma unroll
            for (int k = 0; k < U; ++k) {
                fx[k] = nx[k], fz[k] = nz[k];
                delta[k] = add2(nd[k].get(), bias);
            }
            fetch(left - U);
#pragma unroll
            for (int k = 0; k < U; ++k) {
                if (p.softplus) delta[k] = softplus2(delta[k]);
                if (k >= left) delta[k] = 0ull;
            }
#pragma unroll
            for (int k = 0; k < U; ++k) {
                f2 xs = fx[k].get();
                if (k >= left) xs = 0ull;  // not an infinity of two tokens before, times no step
                f2 zs = 0ull;
                if (gate) zs = fz[k].get();
                float e0, e1, x0, x1;
                split(delta[k], e0, e1);
                split(mul2(delta[k], xs), x0, x1);
                const f2 dd[2] = {pair(e0, e0), pair(e1, e1)}, dx[2] = {pair(x0, x0), pair(x1, x1)};
                const float *bc = &s_bc[u + k][0][lane * kT];
                f2 y[2] = {0ull, 0ull};
#pragma unroll
                for (int i = 0; i < Q; ++i) {
                    const ulonglong2 b = *reinterpret_cast<const ulonglong2 *>(bc + i * 4);
                    ulonglong2 cc = make_ulonglong2(0ull, 0ull);
                    if (!STATE) cc = *reinterpret_cast<const ulonglong2 *>(bc + N + i * 4);
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        float w0, w1, w2, w3;
                        split(mul2(dd[c], a[c][2 * i]), w0, w1);
                        split(mul2(dd[c], a[c][2 * i + 1]), w2, w3);
                        f2 &h0 = h[c][2 * i], &h1 = h[c][2 * i + 1];
                        h0 = fma2(pair(ex2(w0), ex2(w1)), h0, mul2(dx[c], b.x));
                        h1 = fma2(pair(ex2(w2), ex2(w3)), h1, mul2(dx[c], b.y));
                        if (!STATE) y[c] = fma2(cc.y, h1, fma2(cc.x, h0, y[c]));
                    }
                }
                if (STATE) {
                    dsum = add2(dsum, delta[k]);
                } else {
                    float o[2];
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        float lo, hi;
                        split(y[c], lo, hi);
                        o[c] = lo + hi;
#pragma unroll
                        for (int bit = 1; bit < L; bit <<= 1) o[c] += __shfl_xor_sync(0xffffffffu, o[c], bit);
                    }
                    f2 out = fma2(skip, xs & keep, pair(o[0], o[1]));
                    if (gate) {
                        float z0, z1;
                        split(zs, z0, z1);
                        out = mul2(out, mul2(zs, pair(sigmoid_f(z0), sigmoid_f(z1))));
                    }
                    split(out, o[0], o[1]);
                    if (lane == 0 && k < left) store2<T, PAIR>(yp, o[0], o[1], has0, has1);
                    yp += D;
                }
            }
        }
    }
    float *to = STATE ? p.hs + (long long)slot * p.D * N
                : p.ht && seq.t1 >= seq.eos ? p.ht + (long long)seq.n * p.D * N : nullptr;
    if (to) exchange(to + (long long)cs.d0 * N, h, true);
    if (STATE && lane == 0) {
        float s0, s1;
        split(dsum, s0, s1);
        if (has0) p.dsum[(long long)slot * p.D + d] = s0;
        if (has1) p.dsum[(long long)slot * p.D + d + 1] = s1;
    }
}

// ---- one token per sequence ----------------------------------------------------------

// One thread per four states (L = N / 4 lanes of a channel) of K sequences, blockIdx.y and
// every gridDim.y-th behind it: the loads of all of them are in flight at once, and the
// rates are read once.
template <typename T, int L, int K>
__global__ void __launch_bounds__(128) scan_step(ScanParams p) {
    constexpr int N = kS * L;
    const unsigned at = blockIdx.x * 128 + threadIdx.x, d = at / L;
    const int lane = at % L;
    const bool in = d < (unsigned)p.D;
    float part[K], x[K], z[K];
    if (in) {
        const unsigned g = d / (unsigned)(p.D / p.G);
        const float4 A = *reinterpret_cast<const float4 *>(p.A + (long long)d * N + lane * kS);
        Vec<T, 4> b[K], c[K];
        Vec<T, 1> fx[K], fd[K], fz[K];
        float4 h[K];
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const long long n = blockIdx.y + k * gridDim.y;
            if (n >= p.seq.N) break;
            const long long row = n * p.D + d, bc = (n * p.G + g) * N + lane * kS;
            h[k] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (p.h0) h[k] = *reinterpret_cast<const float4 *>(p.h0 + row * N + lane * kS);
            fx[k].load(static_cast<const T *>(p.x) + row);
            fd[k].load(static_cast<const T *>(p.dt) + row);
            if (p.z) fz[k].load(static_cast<const T *>(p.z) + row);
            b[k].load(static_cast<const T *>(p.Bm) + bc);
            c[k].load(static_cast<const T *>(p.Cm) + bc);
        }
        const float bias = p.dt_bias ? p.dt_bias[d] : 0.f;
        const float a[4] = {log2_rate(A.x), log2_rate(A.y), log2_rate(A.z), log2_rate(A.w)};
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const long long n = blockIdx.y + k * gridDim.y;
            if (n >= p.seq.N) break;
            const float raw = fd[k].v[0] + bias, delta = p.softplus ? softplus(raw) : raw;
            x[k] = fx[k].v[0];
            if (p.z) z[k] = fz[k].v[0];
            const float dx = delta * x[k];
            h[k].x = fmaf(ex2(delta * a[0]), h[k].x, dx * b[k].v[0]);
            h[k].y = fmaf(ex2(delta * a[1]), h[k].y, dx * b[k].v[1]);
            h[k].z = fmaf(ex2(delta * a[2]), h[k].z, dx * b[k].v[2]);
            h[k].w = fmaf(ex2(delta * a[3]), h[k].w, dx * b[k].v[3]);
            if (p.ht) *reinterpret_cast<float4 *>(p.ht + (n * p.D + d) * N + lane * kS) = h[k];
            part[k] = fmaf(c[k].v[0], h[k].x, fmaf(c[k].v[1], h[k].y, fmaf(c[k].v[2], h[k].z, c[k].v[3] * h[k].w)));
        }
    }
#pragma unroll
    for (int bit = 1; bit < L; bit <<= 1)
#pragma unroll
        for (int k = 0; k < K; ++k) part[k] += __shfl_xor_sync(0xffffffffu, part[k], bit);
    if (!in || lane != 0) return;
    const float skip = p.Dskip ? p.Dskip[d] : 0.f;
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const long long n = blockIdx.y + k * gridDim.y;
        if (n >= p.seq.N) break;
        Vec<T, 1> out;
        out.v[0] = p.Dskip ? fmaf(skip, x[k], part[k]) : part[k];
        if (p.z) out.v[0] *= silu_f(z[k]);
        out.store(static_cast<T *>(p.y) + n * p.D + d);
    }
}

// ---- states over the chunks of a sequence ------------------------------------------

// e^{sum A} s + own over one chunk, `half` being half the rate.  A chunk's decay can lie below
// (or its growth above) what fp32 holds while no token's does, and then one factor of 0 (or
// infinity) would make NaN of an infinite state (or of none).  So it is taken as two equal
// factors, neither of them 0 or infinite: a finite state that the limits change is below
// 2^-124 all the same (or infinite).
__device__ __forceinline__ float step_chunk(float sum, float half, float s, float own) {
    const float f = ex2(fminf(fmaxf(sum * half, -126.f), 127.f));
    return fmaf(f, f * s, own);
}

// (see scan_combine_launch; blockIdx.y = 1: the gradients' walk back).  A thread takes four
// states and loads kAhead chunks at a time: the walk is bound by latency.
template <bool BWD>
__global__ void __launch_bounds__(128) scan_combine(ScanParams p) {
    constexpr int kAhead = 8;
    wait_for_launches();
    const long long i = (long long)blockIdx.x * 128 + threadIdx.x;
    const int q = p.N / 4;  // vectors of a channel's states
    const long long per = (long long)p.D * q;
    const int n = (int)(i / per);
    if (n >= p.seq.N) return;
    const long long at = i - n * per;
    const int d = (int)(at / q);
    long long slot, chunks;
    if (p.seq.cu) {
        const long long bos = p.seq.cu[n], eos = p.seq.cu[n + 1];
        if (bos < 0 || eos < bos || eos > p.seq.tokens) return;
        slot = bos / p.chunk + n;
        chunks = (eos - bos + p.chunk - 1) / p.chunk;
    } else {
        chunks = ((long long)p.seq.T + p.chunk - 1) / p.chunk;
        slot = (chunks > 0 ? chunks : 1) * (long long)n;
    }
    float4 A = *reinterpret_cast<const float4 *>(p.A + at * 4);
    A = make_float4(0.5f * log2_rate(A.x), 0.5f * log2_rate(A.y), 0.5f * log2_rate(A.z), 0.5f * log2_rate(A.w));
    const float4 none = make_float4(0.f, 0.f, 0.f, 0.f);
    const long long mine = (long long)n * per + at;
    const bool back = BWD && blockIdx.y;
    // chunk c of the walk: from the first on, or from the last back
    const long long first = back ? slot + chunks - 1 : slot, step = back ? -1 : 1;
    float4 *vs = reinterpret_cast<float4 *>(back ? p.gs : p.hs) + first * per + at;
    const float *ds = p.dsum + first * p.D + d;
    const float *from = back ? p.dht : p.h0;
    float4 s = from ? reinterpret_cast<const float4 *>(from)[mine] : none;
    if (!back && chunks == 0) vs[0] = s;  // an empty sequence's slot
    for (long long c = 0; c < chunks; c += kAhead) {
        float4 own[kAhead];
        float sum[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
            if (c + k < chunks && (back || c + k < chunks - 1)) {  // the last chunk's own state is not made
                own[k] = vs[(c + k) * step * per];
                sum[k] = ds[(c + k) * step * p.D];
            }
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
            if (c + k < chunks) {
                vs[(c + k) * step * per] = s;
                if (back || c + k < chunks - 1) {
                    s.x = step_chunk(sum[k], A.x, s.x, own[k].x);
                    s.y = step_chunk(sum[k], A.y, s.y, own[k].y);
                    s.z = step_chunk(sum[k], A.z, s.z, own[k].z);
                    s.w = step_chunk(sum[k], A.w, s.w, own[k].w);
                }
            }
    }
    if (back && p.dh0) reinterpret_cast<float4 *>(p.dh0)[mine] = s;
}

template <typename T, int L, bool PAIR>
cudaError_t fwd_l(const ScanParams &p, cudaStream_t stream) {
    const long long slots = p.chunk ? tile_slots(p.seq, p.chunk) : p.seq.N;
    const long long grid = slots * channel_tiles<kCh>(p.D, p.G);
    if (grid > 0x7fffffffLL) return cudaErrorInvalidValue;
    if (p.chunk) {
        scan_fwd<T, L, PAIR, true><<<(unsigned)grid, 32 * L, 0, stream>>>(p);
        cudaError_t err = cudaGetLastError();
        if (err == cudaSuccess) err = scan_combine_launch(p, false, stream);
        if (err != cudaSuccess) return err;
        return launch_after(scan_fwd<T, L, PAIR, false>, dim3((unsigned)grid), dim3(32 * L), 0, stream, p);
    }
    scan_fwd<T, L, PAIR, false><<<(unsigned)grid, 32 * L, 0, stream>>>(p);
    return cudaGetLastError();
}

template <typename T>
cudaError_t fwd_t(const ScanParams &p, cudaStream_t stream) {
    const bool even = (p.D / p.G) % 2 == 0;  // rows and groups begin on a pair
    switch (p.N) {
        case 16: return even ? fwd_l<T, 1, true>(p, stream) : fwd_l<T, 1, false>(p, stream);
        case 32: return even ? fwd_l<T, 2, true>(p, stream) : fwd_l<T, 2, false>(p, stream);
        case 64: return even ? fwd_l<T, 4, true>(p, stream) : fwd_l<T, 4, false>(p, stream);
        default: return even ? fwd_l<T, 8, true>(p, stream) : fwd_l<T, 8, false>(p, stream);
    }
}

// Whether every sequence is one token (and the grid of their kernel can hold them).
bool one_token(const ScanParams &p) {
    return !p.seq.cu && p.seq.T == 1 && p.seq.N <= 4 * 65535 && (long long)p.D * (p.N / kS) < 0x7fffff00LL;
}

// Four sequences a thread where that still makes a block for most places of the GPU.
template <typename T, int L>
cudaError_t step_l(const ScanParams &p, cudaStream_t stream) {
    const long long cols = ((long long)p.D * L + 127) / 128;
    const int rows = (p.seq.N + 3) / 4;
    if (cols * rows >= kSms * 4 || p.seq.N > 65535)
        scan_step<T, L, 4><<<dim3((unsigned)cols, rows), 128, 0, stream>>>(p);
    else
        scan_step<T, L, 1><<<dim3((unsigned)cols, p.seq.N), 128, 0, stream>>>(p);
    return cudaGetLastError();
}

template <typename T>
cudaError_t step_t(const ScanParams &p, cudaStream_t stream) {
    switch (p.N) {
        case 16: return step_l<T, 4>(p, stream);
        case 32: return step_l<T, 8>(p, stream);
        case 64: return step_l<T, 16>(p, stream);
        default: return step_l<T, 32>(p, stream);
    }
}

// Length of the chunks that a forward's sequences are cut into; 0: they are not.  Whole
// sequences where their blocks fill more than half of the GPU's places; else as many
// chunks as fill them once (one block too many would be a second wave: 4 x 2048 tokens of
// 2048 channels in 19 chunks take 156 us, in 15 or 20 chunks 190 to 210).
int fwd_chunk(int n_seqs, long long tokens, int D, int G, int N) {
    const long long blocks = (long long)n_seqs * G * ((D / G + kCh - 1) / kCh);
    const long long parts = (long long)kSms * (kResident / (N / kT)) / blocks;
    const long long mean = tokens / n_seqs;
    const int least = scan_least_chunk(mean);
    if (parts < 2 || mean < 2 * least) return 0;
    const long long len = (mean + parts - 1) / parts;
    return len < least ? least : (int)((len + kTile - 1) / kTile * kTile);
}

}  // namespace

cudaError_t scan_combine_launch(const ScanParams &p, bool bwd, cudaStream_t stream) {
    const long long n = (long long)p.seq.N * p.D * (p.N / 4);  // vectors of all sequences' states
    const long long grid = (n + 127) / 128;
    if (grid > 0x7fffffffLL) return cudaErrorInvalidValue;
    if (grid == 0) return cudaSuccess;
    if (bwd) return launch_after(scan_combine<true>, dim3((unsigned)grid, 2), dim3(128), 0, stream, p);
    return launch_after(scan_combine<false>, dim3((unsigned)grid), dim3(128), 0, stream, p);
}

size_t scan_fwd_workspace(int n_seqs, long long tokens, int D, int G, int N) {
    const int chunk = n_seqs > 0 ? fwd_chunk(n_seqs, tokens, D, G, N) : 0;
    if (chunk == 0) return 0;
    return (size_t)(tokens / chunk + n_seqs) * (size_t)D * (size_t)(N + 1) * 4u;
}

void scan_fwd_carve(ScanParams &p, void *workspace) {
    p.chunk = workspace ? fwd_chunk(p.seq.N, p.seq.tokens, p.D, p.G, p.N) : 0;
    if (p.chunk == 0) return;
    p.nslots = p.seq.tokens / p.chunk + p.seq.N;
    p.hs = static_cast<float *>(workspace);
    p.dsum = p.hs + p.nslots * p.D * p.N;
}

cudaError_t scan_fwd_launch(ScanParams p, bool bf16, cudaStream_t stream, const char **name) {
    if (one_token(p)) {
        *name = bf16 ? "scan_step<bf16>" : "scan_step<f32>";
        return bf16 ? step_t<__nv_bfloat16>(p, stream) : step_t<float>(p, stream);
    }
    *name = p.chunk ? bf16 ? "scan_state+scan_combine+scan_fwd<bf16>" : "scan_state+scan_combine+scan_fwd<f32>"
                    : bf16 ? "scan_fwd<bf16>" : "scan_fwd<f32>";
    return bf16 ? fwd_t<__nv_bfloat16>(p, stream) : fwd_t<float>(p, stream);
}

}  // namespace dn
