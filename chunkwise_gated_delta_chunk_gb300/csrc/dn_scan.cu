// Selective state space scan, forward.
//
//     delta = softplus(dt + dt_bias),  h[n] = e^{delta A[n]} h[n] + delta B[n] x,
//     y = (sum_n C[n] h[n] + Dskip x) silu(z)
//
// A block takes the channels of one tile (128 threads, 4 states of a channel
// each) and walks the tokens of one sequence, or of one chunk of it, in tiles of
// 16.  Per tile the threads first compute delta and delta x of every token and
// channel once, into shared memory, with the rows of Bm and Cm beside them; then
// each thread steps its states through the tokens; then y is finished and stored
// by rows.  The next tile's rows are loaded into registers meanwhile.
//
// What bounds it: N exponentials and 4 N fp32 operations per channel and token
// against 6 to 8 bytes.
//
// Few channels leave most SMs idle, so sequences are then cut into chunks: one
// launch computes each chunk's state from zero and its sum of delta, a second
// steps the states over the chunks (the state at a chunk's end is
// e^{A sum delta} times the one at its start, plus the chunk's own), and the
// scan itself starts every chunk from its state.
#include "dn_scan.cuh"

namespace dn {
namespace {

using namespace scan;

constexpr int kThreads = 128;
constexpr int kTile = 16;    // tokens of a tile
constexpr int kMinChunk = 64;  // the shortest chunk

// ---- the scan over the tokens of a sequence or a chunk ------------------------------

template <typename T, int L, bool VEC, bool STATE>
__global__ void __launch_bounds__(kThreads) scan_fwd(ScanParams p) {
    constexpr int N = kS * L, CH = kThreads / L, CV = CH / 4;
    constexpr int kVecs = (kTile * CV + kThreads - 1) / kThreads;  // vectors of a tile per thread (CH <= 32: one)
    constexpr int kBc = kTile * N / 2 / kThreads;                  // vectors of B and C per thread
    static_assert(kVecs == 1, "a tile is one vector per thread at most");
    __shared__ float2 s_dx[kTile][CH];           // delta, delta x
    __shared__ float s_skip[kTile][CH];          // Dskip x
    __shared__ float s_y[kTile][CH];
    __shared__ __align__(16) float s_bc[2][kTile][N];

    const int tid = threadIdx.x;
    const int tiles = p.G * ((p.D / p.G + CH - 1) / CH);
    const int ct = blockIdx.x % tiles;
    const long long slot = blockIdx.x / tiles;
    if (blockIdx.x == 0) check_offsets(p.seq, tid, kThreads);
    const SeqTile seq = p.chunk ? seq_tile(p.seq, slot, p.chunk) : seq_whole(p.seq, (int)slot);
    if (!seq.ok) return;
    if (STATE && seq.t1 >= seq.eos) return;  // nothing starts from the last chunk's end
    const Channels cs = channels_of<CH>(p, ct);

    // this thread's channel and states
    const int ch = tid / L, lane = tid % L;
    const bool own = ch < cs.n;
    const int d = cs.d0 + ch;
    float a[kS], h[kS];
    const long long dn_at = (long long)d * N + lane * kS;
#pragma unroll
    for (int i = 0; i < kS; ++i) a[i] = h[i] = 0.f;
    if (own) {
        const float4 r = *reinterpret_cast<const float4 *>(p.A + dn_at);
        a[0] = log2_rate(r.x); a[1] = log2_rate(r.y); a[2] = log2_rate(r.z); a[3] = log2_rate(r.w);
        const float *from = STATE ? nullptr
                            : p.chunk ? p.hs + slot * p.D * N
                            : p.h0 ? p.h0 + (long long)seq.n * p.D * N : nullptr;
        if (from) {
            const float4 s = *reinterpret_cast<const float4 *>(from + dn_at);
            h[0] = s.x; h[1] = s.y; h[2] = s.z; h[3] = s.w;
        }
    }
    // this thread's part of a tile: four channels of one token
    const int vt = tid / CV, vc = (tid % CV) * 4;
    const bool loads = vt < kTile;
    const int vn = loads ? cs.n - vc : 0;
    float bias[4], skip[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        bias[i] = i < vn && p.dt_bias ? p.dt_bias[cs.d0 + vc + i] : 0.f;
        skip[i] = i < vn && p.Dskip ? p.Dskip[cs.d0 + vc + i] : 0.f;
    }
    const bool gate = !STATE && p.z;
    float dsum[4] = {0.f, 0.f, 0.f, 0.f};

    float fx[4], fd[4], fz[4] = {0.f, 0.f, 0.f, 0.f}, fb[kBc][4];
    auto fetch = [&](long long t0) {
        const bool in = loads && t0 + vt < seq.t1;
        load4<T, VEC>(p.x, t0 + vt, p.D, cs.d0 + vc, vn, in, fx);
        load4<T, VEC>(p.dt, t0 + vt, p.D, cs.d0 + vc, vn, in, fd);
        if (gate) load4<T, VEC>(p.z, t0 + vt, p.D, cs.d0 + vc, vn, in, fz);
#pragma unroll
        for (int k = 0; k < kBc; ++k) {
            const int v = tid + k * kThreads, which = v / (kTile * N / 4), r = v % (kTile * N / 4);
            const int t = r / (N / 4), c = (r % (N / 4)) * 4;
            if (STATE && which) break;
            load4<T, true>(which ? p.Cm : p.Bm, (t0 + t) * p.G + cs.g, N, c, 4, t0 + t < seq.t1, fb[k]);
        }
    };
    fetch(seq.t0);
    for (long long t0 = seq.t0; t0 < seq.t1; t0 += kTile) {
        float z[4];
        if (loads) {
            const bool in = t0 + vt < seq.t1;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float raw = fd[i] + bias[i];
                const float delta = !in || i >= vn ? 0.f : p.softplus ? softplus(raw) : raw;
                s_dx[vt][vc + i] = make_float2(delta, delta * fx[i]);
                if (!STATE) s_skip[vt][vc + i] = skip[i] * fx[i];
                dsum[i] += delta;
                z[i] = fz[i];
            }
        }
#pragma unroll
        for (int k = 0; k < kBc; ++k) {
            const int v = tid + k * kThreads, which = v / (kTile * N / 4), r = v % (kTile * N / 4);
            if (STATE && which) break;
            *reinterpret_cast<float4 *>(&s_bc[which][0][0] + r * 4) = make_float4(fb[k][0], fb[k][1], fb[k][2], fb[k][3]);
        }
        __syncthreads();
        if (t0 + kTile < seq.t1) fetch(t0 + kTile);
#pragma unroll
        for (int q = 0; q < kTile; q += 4) {
            float part[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float2 dx = s_dx[q + k][ch];
                const float4 b = *reinterpret_cast<const float4 *>(&s_bc[0][q + k][lane * kS]);
                const float bb[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
                for (int i = 0; i < kS; ++i) h[i] = fmaf(ex2(dx.x * a[i]), h[i], dx.y * bb[i]);
                if (!STATE) {
                    const float4 c = *reinterpret_cast<const float4 *>(&s_bc[1][q + k][lane * kS]);
                    part[k] = fmaf(c.x, h[0], fmaf(c.y, h[1], fmaf(c.z, h[2], c.w * h[3])));
                }
            }
            if (!STATE) {
                const float sum = sum4<L>(part, lane);
                if (lane < 4) s_y[q + lane][ch] = sum;
            }
        }
        __syncthreads();
        if (!STATE && loads) {
            float out[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                out[i] = s_y[vt][vc + i] + s_skip[vt][vc + i];
                if (gate) out[i] *= silu_f(z[i]);
            }
            store4<T, VEC>(p.y, t0 + vt, p.D, cs.d0 + vc, vn, t0 + vt < seq.t1, out);
        }
    }
    if (own) {
        float *to = STATE ? p.hs + slot * p.D * N
                    : p.ht && seq.t1 >= seq.eos ? p.ht + (long long)seq.n * p.D * N : nullptr;
        if (to) *reinterpret_cast<float4 *>(to + dn_at) = make_float4(h[0], h[1], h[2], h[3]);
    }
    if (STATE) {  // the chunk's sum of delta, over the threads that share a channel
        __syncthreads();
        if (loads)
#pragma unroll
            for (int i = 0; i < 4; ++i) s_y[vt][vc + i] = dsum[i];
        __syncthreads();
        if (tid < cs.n) {
            float s = 0.f;
#pragma unroll
            for (int t = 0; t < kTile; ++t) s += s_y[t][tid];
            p.dsum[slot * p.D + cs.d0 + tid] = s;
        }
    }
}

// ---- states over the chunks of a sequence ------------------------------------------

// (see scan_combine_launch)
template <bool BWD>
__global__ void __launch_bounds__(128) scan_combine(ScanParams p) {
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
    const float4 A = *reinterpret_cast<const float4 *>(p.A + at * 4);
    const float4 none = make_float4(0.f, 0.f, 0.f, 0.f);
    const long long mine = (long long)n * per + at;
    float4 *hs = reinterpret_cast<float4 *>(p.hs) + slot * per + at;
    const float *ds = p.dsum + slot * p.D + d;
    auto step = [&](float4 &s, float sum, const float4 &own) {
        s.x = fmaf(ex2(sum * log2_rate(A.x)), s.x, own.x);
        s.y = fmaf(ex2(sum * log2_rate(A.y)), s.y, own.y);
        s.z = fmaf(ex2(sum * log2_rate(A.z)), s.z, own.z);
        s.w = fmaf(ex2(sum * log2_rate(A.w)), s.w, own.w);
    };
    constexpr int U = 4;  // chunks loaded ahead
    float4 s = p.h0 ? reinterpret_cast<const float4 *>(p.h0)[mine] : none;
    if (chunks == 0) hs[0] = s;  // an empty sequence's slot
    for (long long c = 0; c < chunks; c += U) {
        float4 own[U];
        float sum[U];
#pragma unroll
        for (int k = 0; k < U; ++k)
            if (c + k < chunks - 1) {
                own[k] = hs[(c + k) * per];
                sum[k] = ds[(c + k) * p.D];
            }
#pragma unroll
        for (int k = 0; k < U; ++k)
            if (c + k < chunks) {
                hs[(c + k) * per] = s;
                if (c + k < chunks - 1) step(s, sum[k], own[k]);
            }
    }
    if (!BWD) return;
    float4 *gs = reinterpret_cast<float4 *>(p.gs) + slot * per + at;
    float4 g = p.dht ? reinterpret_cast<const float4 *>(p.dht)[mine] : none;
    for (long long c = chunks - 1; c >= 0; c -= U) {
        float4 own[U];
        float sum[U];
#pragma unroll
        for (int k = 0; k < U; ++k)
            if (c - k >= 0) {
                own[k] = gs[(c - k) * per];
                sum[k] = ds[(c - k) * p.D];
            }
#pragma unroll
        for (int k = 0; k < U; ++k)
            if (c - k >= 0) {
                gs[(c - k) * per] = g;
                step(g, sum[k], own[k]);
            }
    }
    if (p.dh0) reinterpret_cast<float4 *>(p.dh0)[mine] = g;
}

template <typename T, int L, bool VEC>
cudaError_t fwd_l(const ScanParams &p, cudaStream_t stream) {
    constexpr int CH = kThreads / L;
    const long long slots = p.chunk ? tile_slots(p.seq, p.chunk) : p.seq.N;
    const long long grid = slots * channel_tiles<CH>(p.D, p.G);
    if (grid > 0x7fffffffLL) return cudaErrorInvalidValue;
    if (p.chunk) {
        scan_fwd<T, L, VEC, true><<<(unsigned)grid, kThreads, 0, stream>>>(p);
        const cudaError_t err = scan_combine_launch(p, false, stream);
        if (err != cudaSuccess) return err;
    }
    scan_fwd<T, L, VEC, false><<<(unsigned)grid, kThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

template <typename T>
cudaError_t fwd_t(const ScanParams &p, cudaStream_t stream) {
    const bool vec = (p.D / p.G) % 4 == 0;
    switch (p.N) {
        case 16: return vec ? fwd_l<T, 4, true>(p, stream) : fwd_l<T, 4, false>(p, stream);
        case 32: return vec ? fwd_l<T, 8, true>(p, stream) : fwd_l<T, 8, false>(p, stream);
        case 64: return vec ? fwd_l<T, 16, true>(p, stream) : fwd_l<T, 16, false>(p, stream);
        default: return vec ? fwd_l<T, 32, true>(p, stream) : fwd_l<T, 32, false>(p, stream);
    }
}

// Length of the chunks that a forward's sequences are cut into; 0: they are not.
int fwd_chunk(int n_seqs, long long tokens, int D, int G, int N) {
    const int ch = kThreads / (N / kS);
    const long long blocks = (long long)n_seqs * G * ((D / G + ch - 1) / ch);
    const long long want = kSms * 4;
    if (blocks >= want || tokens / n_seqs < 2 * kMinChunk) return 0;
    const long long parts = (want + blocks - 1) / blocks;
    const long long len = (tokens / n_seqs + parts - 1) / parts;
    return len < kMinChunk ? kMinChunk : (int)((len + kTile - 1) / kTile * kTile);
}

}  // namespace

cudaError_t scan_combine_launch(const ScanParams &p, bool bwd, cudaStream_t stream) {
    const long long n = (long long)p.seq.N * p.D * (p.N / 4);  // vectors of all sequences' states
    const long long grid = (n + 127) / 128;
    if (grid > 0x7fffffffLL) return cudaErrorInvalidValue;
    if (grid == 0) return cudaSuccess;
    if (bwd) scan_combine<true><<<(unsigned)grid, 128, 0, stream>>>(p);
    else scan_combine<false><<<(unsigned)grid, 128, 0, stream>>>(p);
    return cudaGetLastError();
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
    *name = p.chunk ? bf16 ? "scan_state+scan_combine+scan_fwd<bf16>" : "scan_state+scan_combine+scan_fwd<f32>"
                    : bf16 ? "scan_fwd<bf16>" : "scan_fwd<f32>";
    return bf16 ? fwd_t<__nv_bfloat16>(p, stream) : fwd_t<float>(p, stream);
}

}  // namespace dn
