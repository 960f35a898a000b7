// Short causal convolution (depthwise, W = 2..4 taps), forward and backward.
//
//     u_t[d] = bias[d] + sum_j weight[d, j] x_{t-(W-1)+j}[d],   y = u or silu(u)
//
// Forward.  One thread owns V neighbouring channels (16 bytes of a row) and
// walks the tokens of one tile, the last W - 1 inputs in registers, so that
// x is read once but for the W - 1 rows before each tile.
//
// Backward, du = dy act'(u):
//     dx_s = sum_i weight[W-1-i] du_{s+i},  dweight[j] = sum_t du_t x_{t-(W-1)+j},  dbias = sum_t du_t
// One thread owns V channels and walks a tile and the W - 1 tokens behind it
// (whose du reach back into the tile), the last W du in registers.  The sums
// over tokens stay in registers over all tiles of a block, are joined over its
// warps in shared memory and written as one row per block; a second kernel adds
// the rows in a fixed order.
//
// Both move 2 (forward) and 3 (backward) elements per channel and token for
// about W products and one exponential each: they are bound by memory.
#include "dn_layer.cuh"

namespace dn {
namespace {

constexpr int kConvThreads = 128;

// Tokens of a tile: long tiles read fewer rows twice, short ones give a small
// call enough threads.
int conv_fwd_tile(const ConvParams &p, long long cols) {
    for (int len = 64; len > 8; len >>= 1)
        if (tile_slots(p.seq, len) * cols >= (long long)kSms * 1024) return len;
    return 8;
}

template <typename T, int W, int V>
__global__ void __launch_bounds__(kConvThreads) conv_fwd(ConvParams p, int len, int cols, long long slots) {
    if (blockIdx.x == 0) check_offsets(p.seq, threadIdx.y * blockDim.x + threadIdx.x, kConvThreads);
    const long long nbx = (cols + blockDim.x - 1) / blockDim.x;
    const long long by = blockIdx.x / nbx;
    const int col = (int)(blockIdx.x - by * nbx) * blockDim.x + threadIdx.x;
    const long long slot = by * blockDim.y + threadIdx.y;
    if (col >= cols || slot >= slots) return;
    const SeqTile tile = seq_tile(p.seq, slot, len);
    if (!tile.ok) return;
    const int d0 = col * V;
    const T *x = static_cast<const T *>(p.x) + d0;
    T *y = static_cast<T *>(p.y) + d0;
    const T *h0 = p.h0 ? static_cast<const T *>(p.h0) + (long long)tile.n * (W - 1) * p.D + d0 : nullptr;

    float w[W][V], b[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
#pragma unroll
        for (int j = 0; j < W; ++j) w[j][i] = p.weight[(long long)(d0 + i) * W + j];
        b[i] = p.bias ? p.bias[d0 + i] : 0.f;
    }
    Vec<T, V> past[W - 1];  // inputs before the next token, the oldest first
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
        const long long t = tile.t0 - (W - 1) + j;
        if (t >= tile.bos) past[j].load(x + t * p.D);
        else if (h0) past[j].load(h0 + (t - tile.bos + W - 1) * p.D);
        else zero(past[j]);
    }
    if (tile.c == 0 && p.ht) {
        // the last W - 1 inputs of the sequence; rows of h0 are all read before
        // any is written (ht may be h0), by the one thread that owns them
        Vec<T, V> last[W - 1];
        const long long n = tile.eos - tile.bos;
#pragma unroll
        for (int j = 0; j < W - 1; ++j) {
            const long long r = n + j;  // row of (h0, x) put together
            if (r >= W - 1) {
                last[j].load(x + (tile.bos + r - (W - 1)) * p.D);
            } else {
                zero(last[j]);
#pragma unroll
                for (int i = 0; i < W - 1; ++i)  // the tile begins where the sequence does: past is h0
                    if (i == r) last[j] = past[i];
            }
        }
        T *ht = static_cast<T *>(p.ht) + (long long)tile.n * (W - 1) * p.D + d0;
#pragma unroll
        for (int j = 0; j < W - 1; ++j) last[j].store(ht + (long long)j * p.D);
    }
    constexpr int U = 4;  // tokens loaded ahead
    for (long long t = tile.t0; t < tile.t1; t += U) {
        Vec<T, V> in[U];
#pragma unroll
        for (int k = 0; k < U; ++k)
            if (t + k < tile.t1) in[k].load(x + (t + k) * p.D);
#pragma unroll
        for (int k = 0; k < U; ++k) {
            if (t + k >= tile.t1) break;
            Vec<T, V> out;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                float u = fmaf(w[W - 1][i], in[k].v[i], b[i]);
#pragma unroll
                for (int j = 0; j < W - 1; ++j) u = fmaf(w[j][i], past[j].v[i], u);
                out.v[i] = p.silu ? silu_f(u) : u;
            }
            out.store(y + (t + k) * p.D);
#pragma unroll
            for (int j = 0; j + 1 < W - 1; ++j) past[j] = past[j + 1];
            past[W - 2] = in[k];
        }
    }
}

template <typename T, int W, int V>
cudaError_t conv_fwd_v(const ConvParams &p, cudaStream_t stream) {
    const int cols = p.D / V;
    const int len = conv_fwd_tile(p, cols);
    const long long slots = tile_slots(p.seq, len);
    int tx = 8;
    while (tx < kConvThreads && tx < cols) tx <<= 1;
    const int ty = kConvThreads / tx;
    const long long grid = ((cols + tx - 1) / tx) * ((slots + ty - 1) / ty);
    if (grid > 0x7fffffffLL) return cudaErrorInvalidValue;
    conv_fwd<T, W, V><<<(unsigned)grid, dim3(tx, ty), 0, stream>>>(p, len, cols, slots);
    return cudaGetLastError();
}

template <typename T, int W>
cudaError_t conv_fwd_w(const ConvParams &p, cudaStream_t stream) {
    constexpr int V = 16 / sizeof(T);
    // a row begins on 16 bytes where D fills whole vectors
    return p.D % V == 0 ? conv_fwd_v<T, W, V>(p, stream) : conv_fwd_v<T, W, 1>(p, stream);
}

template <typename T>
cudaError_t conv_fwd_t(const ConvParams &p, cudaStream_t stream) {
    switch (p.W) {
        case 2: return conv_fwd_w<T, 2>(p, stream);
        case 3: return conv_fwd_w<T, 3>(p, stream);
        default: return conv_fwd_w<T, 4>(p, stream);
    }
}

// ---- backward ------------------------------------------------------------------

constexpr int kBwdWarps = 8;
constexpr int kBwdV = 4;     // channels of a thread where rows allow it
constexpr int kBwdTile = 32;

// Blocks along the tokens: every one writes a row of partial sums, so no more
// than fill the GPU a few times, and no more than there are tiles for their warps.
// `slots` is taken from the sizes alone (an upper bound of the tiles), so that the
// workspace is known without the offsets.
int conv_bwd_rows(long long tokens, int n_seqs, int D) {
    const long long cols = (D + 32 * kBwdV - 1) / (32 * kBwdV);
    const long long slots = tokens / kBwdTile + n_seqs;
    const long long most = (slots + kBwdWarps - 1) / kBwdWarps;
    const long long fill = (kSms * 6 + cols - 1) / cols;
    const long long rows = most < fill ? most : fill;
    return rows < 1 ? 1 : (int)rows;
}

template <typename T, typename Tg, int W, int V>
__global__ void __launch_bounds__(kBwdWarps * 32) conv_bwd(ConvParams p, int cols, long long slots) {
    if (blockIdx.x == 0 && blockIdx.y == 0) check_offsets(p.seq, threadIdx.x, kBwdWarps * 32);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int col = blockIdx.x * 32 + lane;
    const int d0 = col * V;
    const bool own = col < cols;

    float w[W][V], b[V];
    float sw[W][V], sb[V];  // sums over this thread's tokens
#pragma unroll
    for (int i = 0; i < V; ++i) {
#pragma unroll
        for (int j = 0; j < W; ++j) {
            w[j][i] = own ? p.weight[(long long)(d0 + i) * W + j] : 0.f;
            sw[j][i] = 0.f;
        }
        b[i] = own && p.bias ? p.bias[d0 + i] : 0.f;
        sb[i] = 0.f;
    }
    const long long stride = (long long)gridDim.y * kBwdWarps;
    for (long long slot = (long long)blockIdx.y * kBwdWarps + warp; own && slot < slots; slot += stride) {
        const SeqTile tile = seq_tile(p.seq, slot, kBwdTile);
        if (!tile.ok) continue;
        const T *x = static_cast<const T *>(p.x) + d0;
        const Tg *dy = static_cast<const Tg *>(p.dy) + d0;
        T *dx = static_cast<T *>(p.dx) + d0;
        const long long state = (long long)tile.n * (W - 1) * p.D + d0;
        const T *h0 = p.h0 ? static_cast<const T *>(p.h0) + state : nullptr;
        const T *dht = p.dht ? static_cast<const T *>(p.dht) + state : nullptr;

        Vec<T, V> past[W - 1];
#pragma unroll
        for (int j = 0; j < W - 1; ++j) {
            const long long t = tile.t0 - (W - 1) + j;
            if (t >= tile.bos) past[j].load(x + t * p.D);
            else if (h0) past[j].load(h0 + (t - tile.bos + W - 1) * p.D);
            else zero(past[j]);
        }
        float du[W][V];  // du of the last W tokens, the newest last
#pragma unroll
        for (int j = 0; j < W; ++j)
#pragma unroll
            for (int i = 0; i < V; ++i) du[j][i] = 0.f;
        // Token t completes the gradient of input t - (W - 1): a row of the tile, or
        // of h0 in front of a sequence's first tile.  Behind the sequence du is zero.
        for (long long t = tile.t0; t < tile.t1 + (W - 1); ++t) {
            const bool in = t < tile.eos;
            Vec<T, V> now;
            Vec<Tg, V> grad;
            zero(now);
            zero(grad);
            if (in) {
                now.load(x + t * p.D);
                grad.load(dy + t * p.D);
            }
            const bool mine = t < tile.t1;  // its sums are this tile's
#pragma unroll
            for (int i = 0; i < V; ++i) {
#pragma unroll
                for (int j = 0; j + 1 < W; ++j) du[j][i] = du[j + 1][i];
                float u = fmaf(w[W - 1][i], now.v[i], b[i]);
#pragma unroll
                for (int j = 0; j < W - 1; ++j) u = fmaf(w[j][i], past[j].v[i], u);
                const float d = !in ? 0.f : p.silu ? grad.v[i] * silu_grad_f(u) : grad.v[i];
                du[W - 1][i] = d;
                if (mine) {
                    sb[i] += d;
#pragma unroll
                    for (int j = 0; j < W - 1; ++j) sw[j][i] = fmaf(d, past[j].v[i], sw[j][i]);
                    sw[W - 1][i] = fmaf(d, now.v[i], sw[W - 1][i]);
                }
            }
#pragma unroll
            for (int j = 0; j + 1 < W - 1; ++j) past[j] = past[j + 1];
            past[W - 2] = now;

            const long long s = t - (W - 1);
            if (s >= tile.t0 || (tile.c == 0 && p.dh0)) {
                Vec<T, V> out;
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    float a = 0.f;
#pragma unroll
                    for (int j = 0; j < W; ++j) a = fmaf(w[W - 1 - j][i], du[j][i], a);
                    out.v[i] = a;
                }
                const long long r = s - (tile.eos - (W - 1));  // row of ht that holds this input
                if (dht && r >= 0) {
                    Vec<T, V> add;
                    add.load(dht + r * p.D);
#pragma unroll
                    for (int i = 0; i < V; ++i) out.v[i] += add.v[i];
                }
                if (s >= tile.t0) out.store(dx + s * p.D);
                else out.store(static_cast<T *>(p.dh0) + state + (s - tile.bos + W - 1) * p.D);
            }
        }
    }
    // join the warps, tap by tap
    __shared__ float red[kBwdWarps][32 * V];
#pragma unroll
    for (int j = 0; j <= W; ++j) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < V; ++i) red[warp][lane * V + i] = j < W ? sw[j < W ? j : 0][i] : sb[i];
        __syncthreads();
        for (int i = threadIdx.x; i < 32 * V; i += kBwdWarps * 32) {
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
    const long long i = (long long)blockIdx.x * 128 + threadIdx.x;
    if (i >= (long long)(p.W + 1) * p.D) return;
    const int j = (int)(i / p.D), d = (int)(i - (long long)j * p.D);
    float a = 0.f;
    for (int r = 0; r < rows; ++r) a += p.partial[((long long)r * (p.W + 1) + j) * p.D + d];
    if (j < p.W) p.dweight[(long long)d * p.W + j] = a;
    else if (p.dbias) p.dbias[d] = a;
}

template <typename T, typename Tg, int W, int V>
cudaError_t conv_bwd_v(const ConvParams &p, cudaStream_t stream) {
    const int cols = p.D / V;
    const int rows = conv_bwd_rows(p.seq.tokens, p.seq.N, p.D);
    const dim3 grid((cols + 31) / 32, rows);
    conv_bwd<T, Tg, W, V><<<grid, kBwdWarps * 32, 0, stream>>>(p, cols, tile_slots(p.seq, kBwdTile));
    const long long n = (long long)(W + 1) * p.D;
    conv_bwd_sums<<<(unsigned)((n + 127) / 128), 128, 0, stream>>>(p, rows);
    return cudaGetLastError();
}

template <typename T, typename Tg>
cudaError_t conv_bwd_t(const ConvParams &p, cudaStream_t stream) {
    const bool vec = p.D % kBwdV == 0;
    switch (p.W) {
        case 2: return vec ? conv_bwd_v<T, Tg, 2, kBwdV>(p, stream) : conv_bwd_v<T, Tg, 2, 1>(p, stream);
        case 3: return vec ? conv_bwd_v<T, Tg, 3, kBwdV>(p, stream) : conv_bwd_v<T, Tg, 3, 1>(p, stream);
        default: return vec ? conv_bwd_v<T, Tg, 4, kBwdV>(p, stream) : conv_bwd_v<T, Tg, 4, 1>(p, stream);
    }
}

}  // namespace

cudaError_t conv_fwd_launch(const ConvParams &p, bool bf16, cudaStream_t stream, const char **name) {
    *name = bf16 ? "conv_fwd<bf16>" : "conv_fwd<f32>";
    return bf16 ? conv_fwd_t<__nv_bfloat16>(p, stream) : conv_fwd_t<float>(p, stream);
}

size_t conv_bwd_workspace(long long tokens, int n_seqs, int D, int W) {
    return (size_t)conv_bwd_rows(tokens, n_seqs, D) * (size_t)(W + 1) * (size_t)D * 4u;
}

cudaError_t conv_bwd_launch(const ConvParams &p, bool bf16, cudaStream_t stream, const char **name) {
    *name = bf16 ? "conv_bwd<bf16>" : "conv_bwd<f32>";
    if (!bf16) return conv_bwd_t<float, float>(p, stream);
    return p.dy_f32 ? conv_bwd_t<__nv_bfloat16, float>(p, stream) : conv_bwd_t<__nv_bfloat16, __nv_bfloat16>(p, stream);
}

}  // namespace dn
