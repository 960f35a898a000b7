// Internal declarations of the attention over a sliding window and its ring
// cache (public header: dn_window_ops.h).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "dn_layer.h"
#include "dn_window_ops.h"

namespace dn {

constexpr int kWinTile = 128;  // tokens of a tile of the tensor-core kernels
constexpr int kMaxSinks = 128; // sinks lie within a sequence's first tile

struct WindowParams {
    SeqView seq;
    const void *q, *k, *v;  // [tokens, Nq, d], [tokens, Nk, d] twice
    int Nq, Nk, d, window, sinks;
    float scale;
    void *o;     // [tokens, Nq, d]; read by the backward
    float *lse;  // [tokens, Nq]; read by the backward
    // backward
    const void *dout;  // [tokens, Nq, d]
    void *dq, *dk, *dv;
    float *dsum;      // [tokens, Nq] sum over d of dout o
    unsigned *redo;   // [slots of kWinTile tokens][2 halves][Nq + Nk]: marks of dq, and of dk and dv
    // fp32 parts of the sinks' dv and dk, where some query sees the sinks by themselves (parts):
    // [slots of part_tiles tiles][part_heads, Nk or Nq], then [sequences][Nk], of [2][sinks][d]
    float *sink_part;
    bool parts;
    int part_tiles, part_heads;
    float *head_part;  // CUDA-core kernels: [tokens][Nq][2][d] dv and dk of single query heads, or null
};

// A row of o that came out with a NaN may hold what a masked key's value did (0 times
// infinity): the kernels mark its logarithm with this NaN, and such rows are taken again by a
// kernel that skips masked pairs instead of giving them weight 0.
constexpr unsigned kRedoBits = 0x7fc0dea1u;

cudaError_t window_fwd_launch(const WindowParams &p, bool bf16, cudaStream_t stream, const char **name);
cudaError_t window_bwd_launch(const WindowParams &p, bool bf16, cudaStream_t stream, const char **name);
size_t window_bwd_workspace(long long tokens, int n_seqs, bool packed, int T, int Nq, int Nk, int d, int window, int sinks,
                            bool bf16);
void window_bwd_carve(WindowParams &p, void *workspace, bool bf16);

// Tensor-core kernels: bf16 tensors.
cudaError_t window_tc_fwd(const WindowParams &p, cudaStream_t stream);
cudaError_t window_tc_bwd(const WindowParams &p, cudaStream_t stream);

// CUDA-core kernels: fp32 tensors, and (redo) rows that the other kernels marked.
cudaError_t window_simt_fwd(const WindowParams &p, cudaStream_t stream);
cudaError_t window_simt_bwd(const WindowParams &p, cudaStream_t stream);
cudaError_t window_fwd_redo(const WindowParams &p, bool bf16, cudaStream_t stream);  // the marked rows and tiles
cudaError_t window_bwd_redo(const WindowParams &p, bool bf16, cudaStream_t stream);

// The sinks' rows of dk and dv from their parts, where there are any.
cudaError_t window_sink_sums(const WindowParams &p, bool bf16, cudaStream_t stream);

struct CacheParams {
    const void *q, *k, *v;  // step: [N, Nq, d], [N, Nk, d]; fill: k, v [tokens, Nk, d]
    SeqView seq;            // fill
    int N, Nq, Nk, d, window, sinks, ring;
    float scale;
    const int64_t *lengths;
    void *kc, *vc;  // [N, Nk, sinks + ring, d]
    void *o;        // [N, Nq, d]
    unsigned *status;
};
cudaError_t window_fill_launch(const CacheParams &p, bool bf16, cudaStream_t stream, const char **name);
cudaError_t window_step_launch(const CacheParams &p, bool bf16, cudaStream_t stream, const char **name);

}  // namespace dn
