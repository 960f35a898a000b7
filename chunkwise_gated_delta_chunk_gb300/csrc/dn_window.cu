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
    const cudaError_t err = window_simt_bwd(p, bf16, false, stream);
    if (err != cudaSuccess) return err;
    return window_simt_bwd(p, bf16, true, stream);
}

namespace {

size_t up16(size_t n) { return (n + 15) / 16 * 16; }
size_t dsum_bytes(long long tokens, int Nq) { return up16((size_t)tokens * Nq * 4); }

}  // namespace

size_t window_bwd_workspace(long long tokens, int n_seqs, bool packed, int T, int Nq, int Nk, int d, int window, int sinks,
                            bool bf16) {
    const int64_t some = 0;
    SeqView s{packed ? &some : nullptr, n_seqs, T, tokens, nullptr};
    return dsum_bytes(tokens, Nq) + up16((size_t)tile_slots(s, kWinTile) * 2 * (size_t)(Nq + Nk) * 4);
}

void window_bwd_carve(WindowParams &p, void *workspace, bool bf16) {
    p.dsum = static_cast<float *>(workspace);
    p.redo = reinterpret_cast<unsigned *>(static_cast<char *>(workspace) + dsum_bytes(p.seq.tokens, p.Nq));
}

}  // namespace dn
