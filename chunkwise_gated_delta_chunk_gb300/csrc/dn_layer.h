// Internal declarations of the operators around the recurrence (public
// header: dn_layer_ops.h): their parameter blocks, launchers and the sizes of
// their workspaces.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "dn_internal.h"
#include "dn_layer_ops.h"

namespace dn {

constexpr int kSms = 152;  // SMs of a GB300: grids and splits are sized for it

// Device address of the status word of the current device (dn_api.cu).
cudaError_t status_ptr(unsigned **out);
// What dn_last_kernel returns on this thread (static storage).
void set_last_kernel(const char *name);

// Sequences of a call: offsets on the device, or N of length T each.
struct SeqView {
    const int64_t *cu;  // [N+1] or null
    int N, T;
    long long tokens;   // B*T
    unsigned *status;
};

// Tiles of `len` tokens that never cross a sequence.  With offsets sequence n
// has its tiles from slot cu[n] / len + n on; without, ceil(T / len) each.
// Either way every sequence has one tile at least, an empty one too.
inline long long tile_slots(const SeqView &s, int len) {
    if (s.N == 0) return 0;
    if (s.cu) return s.tokens / len + s.N;
    const long long per = s.T > 0 ? ((long long)s.T + len - 1) / len : 1;
    return per * s.N;
}

struct ConvParams {
    SeqView seq;
    const void *x, *h0;
    const float *weight, *bias;
    int D, W;
    bool silu;
    void *y, *ht;
    // backward
    const void *dy, *dht;
    bool dy_f32;
    void *dx, *dh0;
    float *dweight, *dbias;
    float *partial;  // [rows of the grid][W + 1][D]
};
cudaError_t conv_fwd_launch(const ConvParams &p, bool bf16, cudaStream_t stream, const char **name);
cudaError_t conv_bwd_launch(const ConvParams &p, bool bf16, cudaStream_t stream, const char **name);
size_t conv_bwd_workspace(long long tokens, int n_seqs, int D, int W, bool bf16);

struct ScanParams {
    SeqView seq;
    const void *x, *dt, *Bm, *Cm, *z;
    const float *A, *Dskip, *dt_bias, *h0;
    int D, G, N;
    bool softplus;
    void *y;
    float *ht;
    // chunk form: per slot of `chunk` tokens
    int chunk;
    long long nslots;
    float *hs;    // [nslots][D][N] state at the chunk's end from zero, then at its start
    float *dsum;  // [nslots][D] sum of delta
    // backward
    const void *dy;
    const float *dht;
    float *gs;    // [nslots][D][N] gradient of the state at the chunk's start from the chunk
                  // alone, then of the state at its end from later, then the chunk's part of d_A
    float *vec;   // [nslots][2][D] the chunk's part of d_Dskip and d_dt_bias
    float *bc;    // [tiles of a group][tokens][G][2 N] parts of d_Bm and d_Cm
    void *dx, *ddt, *dBm, *dCm, *dz;
    float *dA, *dDskip, *ddt_bias, *dh0;
};
cudaError_t scan_fwd_launch(ScanParams p, bool bf16, cudaStream_t stream, const char **name);
cudaError_t scan_bwd_launch(ScanParams p, bool bf16, cudaStream_t stream, const char **name);
size_t scan_fwd_workspace(int n_seqs, long long tokens, int D, int G, int N);
size_t scan_bwd_workspace(int n_seqs, long long tokens, int D, int G, int N);
void scan_fwd_carve(ScanParams &p, void *workspace);
void scan_bwd_carve(ScanParams &p, void *workspace);

struct NormParams {
    const void *x, *z, *dy;
    const float *weight, *bias;
    long long rows;
    int D;
    float eps;
    bool rms;
    void *y, *dx, *dz;
    float *dweight, *dbias;
    float *partial;  // [blocks][2][D]
};
cudaError_t norm_fwd_launch(const NormParams &p, bool bf16, cudaStream_t stream, const char **name);
cudaError_t norm_bwd_launch(const NormParams &p, bool bf16, cudaStream_t stream, const char **name);
size_t norm_bwd_workspace(long long rows, int D, bool bf16);

}  // namespace dn
