// Launches of the attention over a sliding window, forward and backward.
#include "dn_window.cuh"

namespace dn {
namespace {

// The sinks' rows of dk and dv: the part of the first key tile's own item and those of the runs of
// query tiles behind its window, in order.  Four columns a thread.
template <typename T>
__global__ void __launch_bounds__(256) sink_sums(WindowParams p, long long slots) {
    wait_for_launches();
    const int hk = blockIdx.x % p.Nk, n = blockIdx.x / p.Nk, D = p.d;
    const SeqTile s = seq_whole(p.seq, n);
    if (!s.ok || s.eos == s.bos) return;
    const int L = (int)(s.eos - s.bos), len = p.part_tiles * kWinTile;
    const QueryTiles qt(0, L < kWinTile ? L : kWinTile, L, kWinTile, Sight{p.window, p.sinks});
    if (qt.end <= qt.last) return;
    const int i = blockIdx.y * 256 + threadIdx.x, per = p.sinks * (D / 4);
    if (i >= 2 * per) return;
    const int w = i / per, row = i % per / (D / 4), col = i % (D / 4) * 4;
    auto at = [&](long long place) {
        return *reinterpret_cast<const float4 *>(p.sink_part + ((place * 2 + w) * p.sinks + row) * D + col);
    };
    const long long base = p.seq.cu ? s.bos / len + n : (long long)n * ((p.seq.T + len - 1) / len);
    float4 v = at(slots * p.part_heads + (long long)n * p.Nk + hk);
    const int group = p.part_heads / p.Nk;
    for (int c = (qt.last + 1) / p.part_tiles; c <= qt.end / p.part_tiles; ++c)
        for (int h = hk * group; h < (hk + 1) * group; ++h) {
            const float4 a = at((base + c) * p.part_heads + h);
            v.x += a.x; v.y += a.y; v.z += a.z; v.w += a.w;
        }
    Vec<T, 4> y;
    y.v[0] = v.x; y.v[1] = v.y; y.v[2] = v.z; y.v[3] = v.w;
    y.store(static_cast<T *>(w == 0 ? p.dv : p.dk) + ((s.bos + row) * p.Nk + hk) * D + col);
    if (isnan(v.x) | isnan(v.y) | isnan(v.z) | isnan(v.w)) {
        // the first key tile's slot, the half that the row lies in
        const long long slot = p.seq.cu ? s.bos / kWinTile + n : (long long)n * ((p.seq.T + kWinTile - 1) / kWinTile);
        atomicOr(p.redo + (slot * 2 + row / 64) * (p.Nq + p.Nk) + p.Nq + hk, 1u);
    }
}

}  // namespace

cudaError_t window_sink_sums(const WindowParams &p, bool bf16, cudaStream_t stream) {
    if (!p.parts) return cudaSuccess;
    const dim3 grid((unsigned)p.seq.N * p.Nk, (2 * p.sinks * (p.d / 4) + 255) / 256);
    const long long slots = tile_slots(p.seq, p.part_tiles * kWinTile);
    return bf16 ? launch_after(sink_sums<__nv_bfloat16>, grid, dim3(256), 0, stream, p, slots)
                : launch_after(sink_sums<float>, grid, dim3(256), 0, stream, p, slots);
}

cudaError_t window_fwd_launch(const WindowParams &p, bool bf16, cudaStream_t stream, const char **name) {
    *name = bf16 ? "window_fwd<bf16>" : "window_fwd<f32>";
    const cudaError_t err = bf16 ? window_tc_fwd(p, stream) : window_simt_fwd(p, stream);
    if (err != cudaSuccess) return err;
    return window_fwd_redo(p, bf16, stream);
}

cudaError_t window_bwd_launch(const WindowParams &p, bool bf16, cudaStream_t stream, const char **name) {
    *name = bf16 ? "window_bwd<bf16>" : "window_bwd<f32>";
    const cudaError_t err = bf16 ? window_tc_bwd(p, stream) : window_simt_bwd(p, stream);
    if (err != cudaSuccess) return err;
    return window_bwd_redo(p, bf16, stream);
}

namespace {

size_t up16(size_t n) { return (n + 15) / 16 * 16; }

// The backward's workspace: D, the marks, the sinks' parts, the query heads' parts.
struct Space {
    size_t redo, sinks, heads, end;
    bool parts, by_head;
    int part_tiles, part_heads;
    Space(const SeqView &s, int Nq, int Nk, int d, int window, int n_sinks, bool bf16) {
        const long long slots = tile_slots(s, kWinTile);
        redo = up16((size_t)s.tokens * Nq * 4);
        sinks = redo + up16((size_t)slots * 2 * (size_t)(Nq + Nk) * 4);
        // fp32: where the key tiles are fewer than two for every SM, an item for each query head
        by_head = !bf16 && Nq > Nk && 2 * slots * Nk < 2 * kSms;
        part_heads = by_head ? Nq : Nk;
        // the queries of a part take about as long as those of a key tile's window; of 16-bit tensors, whose tiles are
        // quick, not fewer than 8 tiles; not more than 32 (the ragged fp32 case: runs of two tiles 235 us, of one 164)
        const int tiles = window / kWinTile + 1, least = bf16 ? 8 : 1;
        part_tiles = tiles < least ? least : tiles > 32 ? 32 : tiles;
        parts = n_sinks > 0 && s.T > window;
        heads = sinks;
        if (parts)
            heads += (size_t)(tile_slots(s, part_tiles * kWinTile) * part_heads + (long long)s.N * Nk) * 2 * (size_t)n_sinks * (size_t)d * 4;
        end = heads + (by_head ? (size_t)s.tokens * Nq * 2 * (size_t)d * 4 : 0);
    }
};

}  // namespace

size_t window_bwd_workspace(long long tokens, int n_seqs, bool packed, int T, int Nq, int Nk, int d, int window, int sinks,
                            bool bf16) {
    const int64_t some = 0;
    const SeqView s{packed ? &some : nullptr, n_seqs, T, tokens, nullptr};
    return Space(s, Nq, Nk, d, window, sinks, bf16).end;
}

void window_bwd_carve(WindowParams &p, void *workspace, bool bf16) {
    const Space s(p.seq, p.Nq, p.Nk, p.d, p.window, p.sinks, bf16);
    char *ws = static_cast<char *>(workspace);
    p.dsum = reinterpret_cast<float *>(ws);
    p.redo = reinterpret_cast<unsigned *>(ws + s.redo);
    p.sink_part = reinterpret_cast<float *>(ws + s.sinks);
    p.head_part = s.by_head ? reinterpret_cast<float *>(ws + s.heads) : nullptr;
    p.parts = s.parts;
    p.part_tiles = s.part_tiles;
    p.part_heads = s.part_heads;
}

}  // namespace dn
