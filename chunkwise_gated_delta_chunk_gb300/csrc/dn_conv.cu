// Short causal convolution (depthwise, W = 2..4 taps), forward and backward.
//
//     u_t[d] = bias[d] + sum_j weight[d, j] x_{t-(W-1)+j}[d],   y = u or silu(u)
//
// Forward.  One thread owns 4 neighbouring channels and walks the tokens of one
// tile, the last W - 1 inputs in registers, so that x is read once but for the
// W - 1 rows before each tile.  Two groups of 8 rows are in flight: with 8 channels
// a thread, or one group of 4 rows, 33 to 60 % of the memory rate instead of 79.
//
// Backward, du = dy act'(u):
//     dx_s = sum_i weight[W-1-i] du_{s+i},  dweight[j] = sum_t du_t x_{t-(W-1)+j},  dbias = sum_t du_t
// One thread owns 4 (bf16) or 2 (fp32) channels and walks a tile and the W - 1
// tokens behind it (whose du reach back into the tile), the last W inputs and du in
// registers.  Its instructions cost it more than its bytes: written plainly it takes 182 for
// 4 channels of a token.  Pairs of channels in the two-wide fp32 instructions, rings of W
// registers that turn whole within an unrolled group, and a path of its own for tokens at
// a tile's edges bring that to 106 (and 221 us to 74).  Now the latency between dependent ones bounds it:
// 12 warps an SM issue in 0.49 of the cycles, and each thread has two chains of W fma2.  Rows come by asynchronous copies
// into the thread's own part of shared memory, so that they hold no registers.  The sums
// over tokens stay in registers over all tiles of a block, are joined over its warps and
// written as one row per block; a second kernel adds the rows in a fixed order.
//
// Both move 2 (forward) and 3 (backward) elements per channel and token for about
// W products and one exponential each.  Measured (bf16, W = 4, silu, 6144 channels):
// forward over 20741 packed tokens 90 us, 5.6 TB/s, bound by memory; backward over
// 4 x 2048 tokens 74 us, 4.1 TB/s.
#include <type_traits>

#include "dn_layer.cuh"

namespace dn {
namespace {

constexpr int kConvThreads = 128;
constexpr int kFwdV = 4;      // channels of a thread where rows allow it
constexpr int kFwdAhead = 8;  // tokens a thread loads before it computes the last such group

// Tokens of a tile: long tiles read fewer rows twice, short ones give a small
// call enough threads.
int conv_fwd_tile(const ConvParams &p, long long cols) {
    for (int len = 64; len > 8; len >>= 1)
        if (tile_slots(p.seq, len) * cols >= (long long)kSms * 1024) return len;
    return 8;
}

// The channels of a thread as pairs: V / 2 of them, or one whose upper half is
// never stored.
template <int V>
struct Pairs {
    static constexpr int P = (V + 1) / 2;
    f2 v[P];
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int i = 0; i < P; ++i) v[i] = 0ull;
    }
    template <typename T>
    __device__ __forceinline__ void from(const Pack<T, V> &a) {
#pragma unroll
        for (int i = 0; i < P; ++i) v[i] = pair(a[2 * i], V > 1 ? a[V > 1 ? 2 * i + 1 : 0] : 0.f);
    }
    __device__ __forceinline__ void to(float (&a)[V]) const {
#pragma unroll
        for (int i = 0; i < P; ++i) {
            float lo, hi;
            split(v[i], lo, hi);
            a[2 * i] = lo;
            if constexpr (V > 1) a[2 * i + 1] = hi;
        }
    }
};

// The taps (V W consecutive floats) and the bias of V channels.
template <int W, int V>
__device__ __forceinline__ void load_taps(const ConvParams &p, int d0, Pairs<V> (&w)[W], Pairs<V> &b) {
    constexpr int P = Pairs<V>::P;
    const float *src = p.weight + (long long)d0 * W;
    float f[V * W];
    if constexpr (V % 4 == 0) {
        Vec<float, V * W> r;
        r.load(src);
#pragma unroll
        for (int i = 0; i < V * W; ++i) f[i] = r.v[i];
    } else {
#pragma unroll
        for (int i = 0; i < V * W; ++i) f[i] = src[i];
    }
#pragma unroll
    for (int i = 0; i < P; ++i) {
#pragma unroll
        for (int j = 0; j < W; ++j) w[j].v[i] = pair(f[2 * i * W + j], V > 1 ? f[V > 1 ? (2 * i + 1) * W + j : 0] : 0.f);
        b.v[i] = p.bias ? pair(p.bias[d0 + 2 * i], V > 1 ? p.bias[d0 + (V > 1 ? 2 * i + 1 : 0)] : 0.f) : 0ull;
    }
}

template <typename T, int W, int V>
__global__ void __launch_bounds__(kConvThreads) conv_fwd(ConvParams p, int len, int cols, unsigned nbx, unsigned slots) {
    if (blockIdx.x == 0) check_offsets(p.seq, threadIdx.y * blockDim.x + threadIdx.x, kConvThreads);
    const unsigned by = blockIdx.x / nbx;
    const int col = (int)(blockIdx.x - by * nbx) * blockDim.x + threadIdx.x;
    const unsigned slot = by * blockDim.y + threadIdx.y;
    if (col >= cols || slot >= slots) return;
    const SeqTile tile = seq_tile(p.seq, slot, len);
    if (!tile.ok) return;
    const int d0 = col * V;
    const T *x = static_cast<const T *>(p.x) + d0;
    T *y = static_cast<T *>(p.y) + d0;
    const T *h0 = p.h0 ? static_cast<const T *>(p.h0) + (long long)tile.n * (W - 1) * p.D + d0 : nullptr;

    Pack<T, V> past[W - 1];  // inputs before the next token, the oldest first
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
        const long long t = tile.t0 - (W - 1) + j;
        past[j].clear();
        if (t >= tile.bos) past[j].load(x + t * p.D);
        else if (h0) past[j].load(h0 + (t - tile.bos + W - 1) * p.D);
    }
    constexpr int U = kFwdAhead, P = Pairs<V>::P;
    const int tokens = (int)(tile.t1 - tile.t0);
    const T *xt = x + tile.t0 * p.D;
    Pack<T, V> next[U];
#pragma unroll
    for (int k = 0; k < U; ++k)
        if (k < tokens) next[k].load(xt + (long long)k * p.D);
    Pairs<V> w[W], b;
    load_taps<W, V>(p, d0, w, b);
    if (tile.c == 0 && p.ht) {
        // the last W - 1 inputs of the sequence; rows of h0 are all read before
        // any is written (ht may be h0), by the one thread that owns them
        T *ht = static_cast<T *>(p.ht) + (long long)tile.n * (W - 1) * p.D + d0;
        const long long n = tile.eos - tile.bos;
#pragma unroll
        for (int j = 0; j < W - 1; ++j) {
            const long long r = n + j;  // row of (h0, x) put together
            Pack<T, V> last;
            last.clear();
            if (r >= W - 1) {
                last.load(x + (tile.bos + r - (W - 1)) * p.D);
            } else {
#pragma unroll
                for (int i = 0; i < W - 1; ++i)  // the tile begins where the sequence does: past is h0
                    if (i == r) last = past[i];
            }
            last.store(ht + (long long)j * p.D);
        }
    }
    T *yt = y + tile.t0 * p.D;
    Pairs<V> before[W - 1];
#pragma unroll
    for (int j = 0; j < W - 1; ++j) before[j].from(past[j]);
    for (int t = 0; t < tokens; t += U) {
        Pack<T, V> in[U];
        const int n = tokens - t;  // tokens from here on
        xt += (long long)U * p.D;
#pragma unroll
        for (int k = 0; k < U; ++k) {
            in[k] = next[k];
            if (U + k < n) next[k].load(xt + (long long)k * p.D);
        }
#pragma unroll
        for (int k = 0; k < U; ++k) {
            if (k >= n) break;
            Pairs<V> now, out;
            now.from(in[k]);
#pragma unroll
            for (int i = 0; i < P; ++i) {
                f2 u = fma2(w[W - 1].v[i], now.v[i], b.v[i]);
#pragma unroll
                for (int j = 0; j < W - 1; ++j) u = fma2(w[j].v[i], before[j].v[i], u);
                if (p.silu) {
                    float u0, u1;
                    split(u, u0, u1);
                    u = mul2(u, pair(sigmoid_f(u0), sigmoid_f(u1)));
                }
                out.v[i] = u;
            }
            Vec<T, V> o;
            out.to(o.v);
            o.store(yt);
            yt += p.D;
#pragma unroll
            for (int j = 0; j + 1 < W - 1; ++j) before[j] = before[j + 1];
            before[W - 2] = now;
        }
    }
}

// One token per sequence: all loads of a thread at once, and few registers, so that the
// whole call is one wave (the kernel above, one token of 64 sequences and 6144 channels:
// 7 us, half of it in a second wave of 8 blocks).
template <typename T, int W, int V>
__global__ void __launch_bounds__(kConvThreads) conv_step(ConvParams p, int cols, unsigned nbx) {
    const unsigned n = blockIdx.x / nbx;
    const int col = (int)(blockIdx.x - n * nbx) * kConvThreads + threadIdx.x;
    if (col >= cols) return;
    const int d0 = col * V;
    const long long state = (long long)n * (W - 1) * p.D + d0;
    Pack<T, V> in[W];  // the last W - 1 inputs, the oldest first, and the token's own
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
        in[j].clear();
        if (p.h0) in[j].load(static_cast<const T *>(p.h0) + state + (long long)j * p.D);
    }
    in[W - 1].load(static_cast<const T *>(p.x) + (long long)n * p.D + d0);
    Pairs<V> w[W], b;
    load_taps<W, V>(p, d0, w, b);
#pragma unroll
    for (int j = 0; j < W; ++j) {
        Pairs<V> v;
        v.from(in[j]);
#pragma unroll
        for (int i = 0; i < Pairs<V>::P; ++i) b.v[i] = fma2(w[j].v[i], v.v[i], b.v[i]);
    }
    Vec<T, V> out;
    b.to(out.v);
#pragma unroll
    for (int i = 0; i < V; ++i) out.v[i] = p.silu ? silu_f(out.v[i]) : out.v[i];
    out.store(static_cast<T *>(p.y) + (long long)n * p.D + d0);
    if (p.ht)
#pragma unroll
        for (int j = 0; j < W - 1; ++j) in[j + 1].store(static_cast<T *>(p.ht) + state + (long long)j * p.D);
}

template <typename T, int W, int V>
cudaError_t conv_fwd_v(const ConvParams &p, cudaStream_t stream, bool &step) {
    const int cols = p.D / V;
    step = false;
    if (!p.seq.cu && p.seq.T == 1) {
        const long long nbx = (cols + kConvThreads - 1) / kConvThreads, grid = nbx * p.seq.N;
        if (grid <= 0x7fffffffLL) {
            step = true;
            conv_step<T, W, V><<<(unsigned)grid, kConvThreads, 0, stream>>>(p, cols, (unsigned)nbx);
            return cudaGetLastError();
        }
    }
    const int len = conv_fwd_tile(p, cols);
    const long long slots = tile_slots(p.seq, len);
    int tx = 8;
    while (tx < kConvThreads && tx < cols) tx <<= 1;
    const int ty = kConvThreads / tx;
    const long long nbx = (cols + tx - 1) / tx, grid = nbx * ((slots + ty - 1) / ty);
    if (grid > 0x7fffffffLL || slots > 0xffffffffLL) return cudaErrorInvalidValue;
    conv_fwd<T, W, V><<<(unsigned)grid, dim3(tx, ty), 0, stream>>>(p, len, cols, (unsigned)nbx, (unsigned)slots);
    return cudaGetLastError();
}

template <typename T, int W>
cudaError_t conv_fwd_w(const ConvParams &p, cudaStream_t stream, bool &step) {
    constexpr int V = kFwdV;
    return p.D % V == 0 ? conv_fwd_v<T, W, V>(p, stream, step) : conv_fwd_v<T, W, 1>(p, stream, step);
}

// `step`: whether the kernel for single tokens was taken
template <typename T>
cudaError_t conv_fwd_t(const ConvParams &p, cudaStream_t stream, bool &step) {
    switch (p.W) {
        case 2: return conv_fwd_w<T, 2>(p, stream, step);
        case 3: return conv_fwd_w<T, 3>(p, stream, step);
        default: return conv_fwd_w<T, 4>(p, stream, step);
    }
}

// ---- backward ------------------------------------------------------------------

constexpr int kBwdWarps = 4;
constexpr int kBwdThreads = kBwdWarps * 32;
constexpr int kGroups = 2;       // groups of tokens in flight (3 and 4 take as long)
constexpr int kBwdResident = 3;  // blocks of an SM (up to 168 registers a thread; 4 take 2 % longer, 5 spill)

// Channels of a thread where rows allow it.
template <typename T>
constexpr int kBwdV = 8 / (int)sizeof(T);

// Tokens of a tile (64, or fewer where these make too few warps to fill the GPU; each
// tile computes W - 1 tokens of the next again) and blocks along the tokens: every block
// writes a row of partial sums, so no more than the GPU holds at once, and each walks the
// same number of tiles.  The tiles are counted from the sizes alone (an upper bound), so
// that the workspace is known without the offsets.
struct BwdGrid {
    int tile, rows;
};
BwdGrid conv_bwd_grid(long long tokens, int n_seqs, int D, int V) {
    const long long cols = (D + 32 * V - 1) / (32 * V);
    BwdGrid g{64, 1};
    while (g.tile > 16 && (tokens / g.tile + n_seqs) * cols < (long long)kSms * 16) g.tile >>= 1;
    const long long most = (tokens / g.tile + n_seqs + kBwdWarps - 1) / kBwdWarps;
    if (most <= 1) return g;
    const long long fill = (kSms * kBwdResident + cols - 1) / cols;
    const long long each = (most + fill - 1) / fill;
    g.rows = (int)((most + each - 1) / each);
    return g;
}

// The rows of x and dy that a thread walks, V elements of each token, fetched
// kGroups groups of K tokens ahead.  The copies go to shared memory
// asynchronously; a thread reads only what it copied itself, so that no barrier
// is needed.  (One 16-bit element is too small for such a copy: it is loaded a
// group ahead into registers.)
template <typename T, typename Tg, int V, int K>
struct Feed {
    static constexpr bool kAsync = sizeof(T) * V >= 4;
    static constexpr int kAhead = kAsync ? kGroups : 1;
    static constexpr int kX = kAsync ? (int)sizeof(T) * V : 0, kG = kAsync ? (int)sizeof(Tg) * V : 0;
    static constexpr int kStage = K * kBwdThreads * (kX + kG);
    static constexpr int kBytes = kAsync ? kAhead * kStage : 16;
    Pack<T, V> now[kAsync ? 1 : K];
    Pack<Tg, V> grad[kAsync ? 1 : K];
    const char *ring;   // this thread's first bytes of x; those of dy lie kBwdThreads kX behind them
    const T *xp;        // the next token to fetch
    const Tg *gp;
    int left;           // tokens not fetched yet (or less than none)

    template <int B>
    static __device__ __forceinline__ void copy(unsigned dst, const void *src) {
        if constexpr (B == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
        else asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(B) : "memory");
    }
    __device__ __forceinline__ int at_g(int s, int k) const {
        return s * kStage + k * kBwdThreads * (kX + kG) + kBwdThreads * kX + threadIdx.x * (kG - kX);
    }
    __device__ __forceinline__ void issue(int s, long long D) {
        const bool full = left >= K;
        if constexpr (kAsync) {
            const unsigned dst = (unsigned)__cvta_generic_to_shared(ring) + s * kStage;
#pragma unroll
            for (int k = 0; k < K; ++k) {
                // what is not fetched keeps what lay there: no result depends on it
                if (!full && k >= left) continue;
                copy<kX>(dst + k * kBwdThreads * (kX + kG), xp + k * D);
                copy<kG>((unsigned)__cvta_generic_to_shared(ring) + at_g(s, k), gp + k * D);
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        } else {
#pragma unroll
            for (int k = 0; k < K; ++k) {
                now[k].clear();
                grad[k].clear();
                if (full || k < left) {
                    now[k].load(xp + k * D);
                    grad[k].load(gp + k * D);
                }
            }
        }
        left -= K;
        xp += K * D;
        gp += K * D;
    }
    __device__ __forceinline__ void start(const char *r, const T *x, const Tg *g, int n, long long D) {
        ring = r + threadIdx.x * kX;
        xp = x;
        gp = g;
        left = n;
#pragma unroll
        for (int s = 0; s < kAhead; ++s) issue(s, D);
    }
    // waits for the oldest of the groups in flight
    __device__ __forceinline__ void wait() {
        if constexpr (kAsync) asm volatile("cp.async.wait_group %0;" ::"n"(kAhead - 1) : "memory");
    }
    __device__ __forceinline__ Pack<T, V> x(int s, int k) const {
        if constexpr (!kAsync) return now[k];
        Pack<T, V> r;
        r.load(reinterpret_cast<const T *>(ring + s * kStage + k * kBwdThreads * (kX + kG)));
        return r;
    }
    __device__ __forceinline__ Pack<Tg, V> g(int s, int k) const {
        if constexpr (!kAsync) return grad[k];
        Pack<Tg, V> r;
        r.load(reinterpret_cast<const Tg *>(ring + at_g(s, k)));
        return r;
    }
};

template <typename T, typename Tg, int W, int V>
__global__ void __launch_bounds__(kBwdThreads, kBwdResident) conv_bwd(ConvParams p, int len, int cols, unsigned slots) {
    if (blockIdx.x == 0 && blockIdx.y == 0) check_offsets(p.seq, threadIdx.x, kBwdThreads);
    constexpr int P = Pairs<V>::P;
    constexpr int K = W == 3 ? 3 : 4;  // tokens of a group: a multiple of W, so that rings of W turn whole
    using F = Feed<T, Tg, V, K>;
    __shared__ __align__(16) char ring[F::kBytes];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int col = blockIdx.x * 32 + lane;
    const int d0 = col * V;
    const bool own = col < cols;
    const long long D = p.D;

    Pairs<V> w[W], b, sw[W], sb;  // sw, sb: sums over this thread's tokens
    b.clear();
    sb.clear();
#pragma unroll
    for (int j = 0; j < W; ++j) w[j].clear(), sw[j].clear();
    if (own) load_taps<W, V>(p, d0, w, b);
    const T *x = static_cast<const T *>(p.x) + d0;
    const Tg *dy = static_cast<const Tg *>(p.dy) + d0;
    T *dx = static_cast<T *>(p.dx) + d0;
    for (unsigned slot = blockIdx.y * kBwdWarps + warp; own && slot < slots; slot += gridDim.y * kBwdWarps) {
        const SeqTile tile = seq_tile(p.seq, slot, len);
        if (!tile.ok) continue;
        const long long state = (long long)tile.n * (W - 1) * D + d0;
        const T *h0 = p.h0 ? static_cast<const T *>(p.h0) + state : nullptr;
        const T *dht = p.dht ? static_cast<const T *>(p.dht) + state : nullptr;
        T *dh0 = p.dh0 && tile.c == 0 ? static_cast<T *>(p.dh0) + state : nullptr;

        // Token t of the tile completes the gradient of input t - (W - 1): a row of the
        // tile, or of h0 in front of a sequence's first tile.  Behind the sequence du is 0.
        const int own_n = (int)(tile.t1 - tile.t0), all_n = own_n + W - 1;
        const long long left = tile.eos - tile.t0;
        const int in_n = left < all_n ? (int)left : all_n;
        const int first = dh0 ? -(W - 1) : 0;  // first row of the tile that is written
        const int tail = !dht ? all_n : left - (W - 1) < all_n ? (int)(left - (W - 1)) : all_n;  // row that ht begins with
        F feed;
        feed.start(ring, x + tile.t0 * D, dy + tile.t0 * D, in_n, D);
        T *op = dx + tile.t0 * D;  // the next row to write
        Pairs<V> xs[W], du[W];     // token t at t % W
#pragma unroll
        for (int j = 0; j < W - 1; ++j) {
            const long long t = tile.t0 - (W - 1) + j;
            Pack<T, V> r;
            r.clear();
            if (t >= tile.bos) r.load(x + t * D);
            else if (h0) r.load(h0 + (t - tile.bos + W - 1) * D);
            xs[j + 1].from(r);
        }
#pragma unroll
        for (int j = 0; j < W; ++j) du[j].clear();

        // one token; EDGE: it may lie behind the tile, and its row in front of it or in ht
        auto token = [&](auto edge, int t, int k, int stage) {
            constexpr bool EDGE = decltype(edge)::value;
            Pairs<V> gs, sum;
            xs[k % W].from(feed.x(stage, k));
            gs.from(feed.g(stage, k));
#pragma unroll
            for (int i = 0; i < P; ++i) {
                f2 d = gs.v[i];
                if (p.silu) {
                    f2 u = fma2(w[W - 1].v[i], xs[k % W].v[i], b.v[i]);
#pragma unroll
                    for (int j = 0; j < W - 1; ++j) u = fma2(w[j].v[i], xs[(k + 1 + j) % W].v[i], u);
                    float u0, u1;
                    split(u, u0, u1);
                    // s (1 + u (1 - s)) with s of both halves
                    const f2 s = pair(sigmoid_f(u0), sigmoid_f(u1));
                    const f2 one = pair(1.f, 1.f), m = fma2(s, pair(-1.f, -1.f), one);
                    d = mul2(d, mul2(s, fma2(u, m, one)));
                }
                if (EDGE && t >= in_n) d = 0ull;
                du[k % W].v[i] = d;
                if (!EDGE || t < own_n) {  // its sums are this tile's
                    sb.v[i] = add2(sb.v[i], d);
#pragma unroll
                    for (int j = 0; j < W; ++j) sw[j].v[i] = fma2(d, xs[(k + 1 + j) % W].v[i], sw[j].v[i]);
                }
                sum.v[i] = mul2(w[W - 1].v[i], du[(k + 1) % W].v[i]);
#pragma unroll
                for (int j = 1; j < W; ++j) sum.v[i] = fma2(w[W - 1 - j].v[i], du[(k + 1 + j) % W].v[i], sum.v[i]);
            }
            const int s = t - (W - 1);
            if (EDGE && s < first) return;
            Vec<T, V> out;
            sum.to(out.v);
            if (EDGE && s >= tail) {
                Pack<T, V> add;
                add.load(dht + (s - (left - (W - 1))) * D);
#pragma unroll
                for (int i = 0; i < V; ++i) out.v[i] += add[i];
            }
            if (EDGE && s < 0) {
                out.store(dh0 + (long long)(s + W - 1) * D);
            } else {
                out.store(op);
                op += D;
            }
        };
        int stage = 0;
        for (int t = 0; t < all_n; t += K) {
            feed.wait();
            if (t >= W - 1 && t + K <= own_n && t + K - (W - 1) <= tail) {
#pragma unroll
                for (int k = 0; k < K; ++k) token(std::false_type{}, t + k, k, stage);
            } else {
#pragma unroll
                for (int k = 0; k < K; ++k)
                    if (t + k < all_n) token(std::true_type{}, t + k, k, stage);
            }
            feed.issue(stage, D);
            stage = stage + 1 == F::kAhead ? 0 : stage + 1;
        }
    }
    // join the warps, tap by tap
    __shared__ float red[kBwdWarps][32 * V];
#pragma unroll
    for (int j = 0; j <= W; ++j) {
        __syncthreads();
        float mine[V];
        (j < W ? sw[j < W ? j : 0] : sb).to(mine);
#pragma unroll
        for (int i = 0; i < V; ++i) red[warp][lane * V + i] = mine[i];
        __syncthreads();
        for (int i = threadIdx.x; i < 32 * V; i += kBwdThreads) {
            const int d = blockIdx.x * 32 * V + i;
            if (d < p.D) {
                float a = 0.f;
#pragma unroll
                for (int k = 0; k < kBwdWarps; ++k) a += red[k][i];
                p.partial[((long long)blockIdx.y * (W + 1) + j) * p.D + d] = a;
            }
        }
    }
}

__global__ void __launch_bounds__(128) conv_bwd_sums(ConvParams p, int rows) {
    wait_for_launches();
    const long long i = (long long)blockIdx.x * 128 + threadIdx.x;
    if (i >= (long long)(p.W + 1) * p.D) return;
    const int j = (int)(i / p.D), d = (int)(i - (long long)j * p.D);
    float a = 0.f;
#pragma unroll 8
    for (int r = 0; r < rows; ++r) a += p.partial[((long long)r * (p.W + 1) + j) * p.D + d];
    if (j < p.W) p.dweight[(long long)d * p.W + j] = a;
    else if (p.dbias) p.dbias[d] = a;
}

template <typename T, typename Tg, int W, int V>
cudaError_t conv_bwd_v(const ConvParams &p, cudaStream_t stream) {
    const int cols = p.D / V;
    const BwdGrid g = conv_bwd_grid(p.seq.tokens, p.seq.N, p.D, kBwdV<T>);
    const dim3 grid((cols + 31) / 32, g.rows);
    const long long slots = tile_slots(p.seq, g.tile);
    if (slots > 0x7fffffffLL) return cudaErrorInvalidValue;
    conv_bwd<T, Tg, W, V><<<grid, kBwdThreads, 0, stream>>>(p, g.tile, cols, (unsigned)slots);
    const long long n = (long long)(W + 1) * p.D;
    const cudaError_t err = cudaGetLastError();
    if (err != cudaSuccess) return err;
    return launch_after(conv_bwd_sums, dim3((unsigned)((n + 127) / 128)), dim3(128), 0, stream, p, g.rows);
}

template <typename T, typename Tg>
cudaError_t conv_bwd_t(const ConvParams &p, cudaStream_t stream) {
    constexpr int V = kBwdV<T>;
    const bool vec = p.D % V == 0;
    switch (p.W) {
        case 2: return vec ? conv_bwd_v<T, Tg, 2, V>(p, stream) : conv_bwd_v<T, Tg, 2, 1>(p, stream);
        case 3: return vec ? conv_bwd_v<T, Tg, 3, V>(p, stream) : conv_bwd_v<T, Tg, 3, 1>(p, stream);
        default: return vec ? conv_bwd_v<T, Tg, 4, V>(p, stream) : conv_bwd_v<T, Tg, 4, 1>(p, stream);
    }
}

}  // namespace

cudaError_t conv_fwd_launch(const ConvParams &p, bool bf16, cudaStream_t stream, const char **name) {
    bool step = false;
    const cudaError_t err = bf16 ? conv_fwd_t<__nv_bfloat16>(p, stream, step) : conv_fwd_t<float>(p, stream, step);
    *name = step ? bf16 ? "conv_step<bf16>" : "conv_step<f32>" : bf16 ? "conv_fwd<bf16>" : "conv_fwd<f32>";
    return err;
}

size_t conv_bwd_workspace(long long tokens, int n_seqs, int D, int W, bool bf16) {
    const int V = bf16 ? kBwdV<__nv_bfloat16> : kBwdV<float>;
    return (size_t)conv_bwd_grid(tokens, n_seqs, D, V).rows * (size_t)(W + 1) * (size_t)D * 4u;
}

cudaError_t conv_bwd_launch(const ConvParams &p, bool bf16, cudaStream_t stream, const char **name) {
    *name = bf16 ? "conv_bwd+conv_bwd_sums<bf16>" : "conv_bwd+conv_bwd_sums<f32>";
    if (!bf16) return conv_bwd_t<float, float>(p, stream);
    return p.dy_f32 ? conv_bwd_t<__nv_bfloat16, float>(p, stream) : conv_bwd_t<__nv_bfloat16, __nv_bfloat16>(p, stream);
}

}  // namespace dn
