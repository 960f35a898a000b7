// Launches of the attention over a sliding window, forward and backward.
#include "dn_window.h"

namespace dn {

cudaError_t window_fwd_launch(const WindowParams &p, bool bf16, cudaStream_t stream, const char **name) {
    *name = bf16 ? "window_fwd<bf16>" : "window_fwd<f32>";
    const cudaError_t err = bf16 ? window_tc_fwd(p, stream) : window_simt_fwd(p, bf16, false, stream);
    if (err != cudaSuccess) return err;
    return window_simt_fwd(p, bf16, true, stream);
}

cudaError_t window_bwd_launch(const WindowParams &p, bool bf16, cudaStream_t stream, const char **name) {
    *name = bf16 ? "window_bwd<bf16>" : "window_bwd<f32>";
    const cudaError_t err = bf16 ? window_tc_bwd(p, stream) : window_simt_bwd(p, bf16, false, stream);
    if (err != cudaSuccess) return err;
    return window_simt_bwd(p, bf16, true, stream);
}

namespace {

size_t up16(size_t n) { return (n + 15) / 16 * 16; }

// The backward's workspace: D, the marks, the sinks' parts.
struct Space {
    size_t redo, sinks, end;
    bool parts;
    int part_tiles;
    Space(const SeqView &s, int Nq, int Nk, int d, int window, int n_sinks, bool bf16) {
        redo = up16((size_t)s.tokens * Nq * 4);
        sinks = redo + up16((size_t)tile_slots(s, kWinTile) * 2 * (size_t)(Nq + Nk) * 4);
        // the queries of a part take about as long as those of a key tile's window; not fewer
        // than 8 tiles, not more than 32
        const int tiles = window / kWinTile + 1;
        part_tiles = tiles < 8 ? 8 : tiles > 32 ? 32 : tiles;
        parts = bf16 && n_sinks > 0 && s.T > window;
        end = sinks;
        if (parts)
            end += (size_t)(tile_slots(s, part_tiles * kWinTile) + s.N) * (size_t)Nk * 2 * (size_t)n_sinks * (size_t)d * 4;
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
    p.parts = s.parts;
    p.part_tiles = s.part_tiles;
}

}  // namespace dn
