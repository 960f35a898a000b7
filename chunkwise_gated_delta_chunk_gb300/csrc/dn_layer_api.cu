// C-ABI front end of the operators around the recurrence: argument checks
// (before any CUDA call) and launches.
#include <math.h>
#include <stdint.h>

#include "dn_layer.h"

#define DN_EXPORT extern "C" __attribute__((visibility("default")))

namespace {

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

template <size_t K>
bool all_aligned(const void *const (&ptrs)[K]) {
    for (const void *p : ptrs)
        if (p && !aligned16(p)) return false;
    return true;
}

bool dtype_ok(dn_dtype d) { return d == DN_BF16 || d == DN_F32; }

bool seqs_ok(const int64_t *cu, int n_seqs, int B, int T) {
    if (n_seqs < 0 || B < 0 || T < 0) return false;
    return cu ? B == 1 : n_seqs == B;
}

// Sequences of a call; the status word is looked up here (the first call on a
// device loads the library's module).
cudaError_t seq_view(dn::SeqView &s, const int64_t *cu, int n_seqs, int B, int T) {
    s.cu = cu;
    s.N = n_seqs;
    s.T = T;
    s.tokens = (long long)B * T;
    return dn::status_ptr(&s.status);
}

// Tokens of a sequence that the kernels count in 32 bits, with room for a tile.
constexpr int kMaxT = 1 << 30;

dn_status done(cudaError_t err, const char *name) {
    if (err != cudaSuccess) return DN_ERR_CUDA;
    dn::set_last_kernel(name);
    return DN_OK;
}

// ---- convolution -----------------------------------------------------------

bool conv_width_ok(int W) { return W >= 2 && W <= 4; }

dn_status conv_check(const void *x, const float *weight, const float *bias, const void *h0, const int64_t *cu,
                     int n_seqs, int B, int T, int D, int W, dn_dtype dtype, unsigned flags) {
    if (!dtype_ok(dtype) || !seqs_ok(cu, n_seqs, B, T) || D <= 0 || W <= 0) return DN_ERR_INVALID_ARG;
    if (flags & ~DN_CONV_SILU) return DN_ERR_INVALID_ARG;
    if (!weight || ((long long)B * T > 0 && !x)) return DN_ERR_INVALID_ARG;
    const void *ptrs[] = {x, weight, bias, h0, cu};
    if (!all_aligned(ptrs)) return DN_ERR_INVALID_ARG;
    return DN_OK;
}

}  // namespace

DN_EXPORT dn_status dn_causal_conv_fwd(const void *x, const float *weight, const float *bias, const void *h0,
                                       const int64_t *cu_seqlens, int n_seqs, int B, int T, int D, int W,
                                       dn_dtype dtype, unsigned flags, void *y, void *ht, dn_stream_t stream) {
    const dn_status st = conv_check(x, weight, bias, h0, cu_seqlens, n_seqs, B, T, D, W, dtype, flags);
    if (st != DN_OK) return st;
    const void *ptrs[] = {y, ht};
    if (!all_aligned(ptrs) || ((long long)B * T > 0 && !y)) return DN_ERR_INVALID_ARG;
    if (!conv_width_ok(W) || T > kMaxT) return DN_ERR_UNSUPPORTED;
    if (n_seqs == 0) return DN_OK;
    dn::ConvParams p{};
    if (seq_view(p.seq, cu_seqlens, n_seqs, B, T) != cudaSuccess) return DN_ERR_CUDA;
    p.x = x; p.weight = weight; p.bias = bias; p.h0 = h0;
    p.D = D; p.W = W; p.silu = flags & DN_CONV_SILU;
    p.y = y; p.ht = ht;
    const char *name = "";
    return done(dn::conv_fwd_launch(p, dtype == DN_BF16, (cudaStream_t)stream, &name), name);
}

DN_EXPORT size_t dn_causal_conv_bwd_workspace_bytes(int n_seqs, int B, int T, int D, int W, dn_dtype dtype) {
    if (n_seqs < 0 || B < 0 || T < 0 || D <= 0 || !conv_width_ok(W) || T > kMaxT || !dtype_ok(dtype)) return 0;
    return dn::conv_bwd_workspace((long long)B * T, n_seqs, D, W, dtype == DN_BF16);
}

DN_EXPORT dn_status dn_causal_conv_bwd(const void *x, const float *weight, const float *bias, const void *h0,
                                       const int64_t *cu_seqlens, int n_seqs, int B, int T, int D, int W,
                                       dn_dtype dtype, unsigned flags, const void *d_y, dn_dtype dy_dtype,
                                       const void *d_ht, void *d_x, float *d_weight, float *d_bias, void *d_h0,
                                       void *workspace, size_t workspace_bytes, dn_stream_t stream) {
    const dn_status st = conv_check(x, weight, bias, h0, cu_seqlens, n_seqs, B, T, D, W, dtype, flags);
    if (st != DN_OK) return st;
    if (dy_dtype != dtype && dy_dtype != DN_F32) return DN_ERR_INVALID_ARG;
    const void *ptrs[] = {d_y, d_ht, d_x, d_weight, d_bias, d_h0};
    if (!all_aligned(ptrs) || !d_weight) return DN_ERR_INVALID_ARG;
    if ((long long)B * T > 0 && (!d_y || !d_x)) return DN_ERR_INVALID_ARG;
    if (!conv_width_ok(W) || T > kMaxT) return DN_ERR_UNSUPPORTED;
    const size_t need = dn::conv_bwd_workspace((long long)B * T, n_seqs, D, W, dtype == DN_BF16);
    if (!workspace || !aligned16(workspace) || workspace_bytes < need) return DN_ERR_INVALID_ARG;
    dn::ConvParams p{};
    if (seq_view(p.seq, cu_seqlens, n_seqs, B, T) != cudaSuccess) return DN_ERR_CUDA;
    p.x = x; p.weight = weight; p.bias = bias; p.h0 = h0;
    p.D = D; p.W = W; p.silu = flags & DN_CONV_SILU;
    p.dy = d_y; p.dy_f32 = dy_dtype == DN_F32; p.dht = d_ht;
    p.dx = d_x; p.dweight = d_weight; p.dbias = d_bias; p.dh0 = d_h0;
    p.partial = static_cast<float *>(workspace);
    const char *name = "";
    return done(dn::conv_bwd_launch(p, dtype == DN_BF16, (cudaStream_t)stream, &name), name);
}

// ---- selective scan ----------------------------------------------------------

namespace {

bool scan_states_ok(int N) { return N == 16 || N == 32 || N == 64 || N == 128; }

bool scan_sizes_ok(int n_seqs, int B, int T, int D, int G, int N, dn_dtype dtype) {
    return n_seqs >= 0 && B >= 0 && T >= 0 && T <= kMaxT && D > 0 && G > 0 && D % G == 0 && scan_states_ok(N) && dtype_ok(dtype);
}

dn_status scan_check(const void *x, const void *dt, const float *A, const void *Bm, const void *Cm,
                     const float *Dskip, const void *z, const float *dt_bias, const float *h0, const int64_t *cu,
                     int n_seqs, int B, int T, int D, int G, int N, dn_dtype dtype, unsigned flags) {
    if (!dtype_ok(dtype) || !seqs_ok(cu, n_seqs, B, T) || D <= 0 || G <= 0 || N <= 0 || D % G != 0)
        return DN_ERR_INVALID_ARG;
    if (flags & ~DN_SCAN_SOFTPLUS) return DN_ERR_INVALID_ARG;
    if (!A || ((long long)B * T > 0 && (!x || !dt || !Bm || !Cm))) return DN_ERR_INVALID_ARG;
    const void *ptrs[] = {x, dt, A, Bm, Cm, Dskip, z, dt_bias, h0, cu};
    if (!all_aligned(ptrs)) return DN_ERR_INVALID_ARG;
    return DN_OK;
}

}  // namespace

DN_EXPORT size_t dn_selective_scan_fwd_workspace_bytes(int n_seqs, int B, int T, int D, int G, int N,
                                                       dn_dtype dtype) {
    if (!scan_sizes_ok(n_seqs, B, T, D, G, N, dtype) || n_seqs == 0) return 0;
    return dn::scan_fwd_workspace(n_seqs, (long long)B * T, D, G, N);
}

DN_EXPORT dn_status dn_selective_scan_fwd(const void *x, const void *dt, const float *A, const void *Bm,
                                          const void *Cm, const float *Dskip, const void *z, const float *dt_bias,
                                          const float *h0, const int64_t *cu_seqlens, int n_seqs, int B, int T,
                                          int D, int G, int N, dn_dtype dtype, unsigned flags, void *y, float *ht,
                                          void *workspace, size_t workspace_bytes, dn_stream_t stream) {
    const dn_status st = scan_check(x, dt, A, Bm, Cm, Dskip, z, dt_bias, h0, cu_seqlens, n_seqs, B, T, D, G, N,
                                    dtype, flags);
    if (st != DN_OK) return st;
    const void *ptrs[] = {y, ht};
    if (!all_aligned(ptrs) || ((long long)B * T > 0 && !y)) return DN_ERR_INVALID_ARG;
    if (!scan_states_ok(N) || T > kMaxT) return DN_ERR_UNSUPPORTED;
    if (n_seqs == 0) return DN_OK;
    const size_t need = dn::scan_fwd_workspace(n_seqs, (long long)B * T, D, G, N);
    if (need > 0 && (!workspace || !aligned16(workspace) || workspace_bytes < need)) return DN_ERR_INVALID_ARG;
    dn::ScanParams p{};
    if (seq_view(p.seq, cu_seqlens, n_seqs, B, T) != cudaSuccess) return DN_ERR_CUDA;
    p.x = x; p.dt = dt; p.Bm = Bm; p.Cm = Cm; p.z = z;
    p.A = A; p.Dskip = Dskip; p.dt_bias = dt_bias; p.h0 = h0;
    p.D = D; p.G = G; p.N = N; p.softplus = flags & DN_SCAN_SOFTPLUS;
    p.y = y; p.ht = ht;
    dn::scan_fwd_carve(p, need > 0 ? workspace : nullptr);
    const char *name = "";
    return done(dn::scan_fwd_launch(p, dtype == DN_BF16, (cudaStream_t)stream, &name), name);
}

DN_EXPORT size_t dn_selective_scan_bwd_workspace_bytes(int n_seqs, int B, int T, int D, int G, int N,
                                                       dn_dtype dtype) {
    if (!scan_sizes_ok(n_seqs, B, T, D, G, N, dtype)) return 0;
    return dn::scan_bwd_workspace(n_seqs, (long long)B * T, D, G, N);
}

DN_EXPORT dn_status dn_selective_scan_bwd(const void *x, const void *dt, const float *A, const void *Bm,
                                          const void *Cm, const float *Dskip, const void *z, const float *dt_bias,
                                          const float *h0, const int64_t *cu_seqlens, int n_seqs, int B, int T,
                                          int D, int G, int N, dn_dtype dtype, unsigned flags, const void *d_y,
                                          const float *d_ht, void *d_x, void *d_dt, float *d_A, void *d_Bm,
                                          void *d_Cm, float *d_Dskip, void *d_z, float *d_dt_bias, float *d_h0,
                                          void *workspace, size_t workspace_bytes, dn_stream_t stream) {
    const dn_status st = scan_check(x, dt, A, Bm, Cm, Dskip, z, dt_bias, h0, cu_seqlens, n_seqs, B, T, D, G, N,
                                    dtype, flags);
    if (st != DN_OK) return st;
    const void *ptrs[] = {d_y, d_ht, d_x, d_dt, d_A, d_Bm, d_Cm, d_Dskip, d_z, d_dt_bias, d_h0};
    if (!all_aligned(ptrs) || !d_A) return DN_ERR_INVALID_ARG;
    if ((long long)B * T > 0 && (!d_y || !d_x || !d_dt || !d_Bm || !d_Cm || (z != nullptr) != (d_z != nullptr)))
        return DN_ERR_INVALID_ARG;
    if (!scan_states_ok(N) || T > kMaxT) return DN_ERR_UNSUPPORTED;
    const size_t need = dn::scan_bwd_workspace(n_seqs, (long long)B * T, D, G, N);
    if (!workspace || !aligned16(workspace) || workspace_bytes < need) return DN_ERR_INVALID_ARG;
    dn::ScanParams p{};
    if (seq_view(p.seq, cu_seqlens, n_seqs, B, T) != cudaSuccess) return DN_ERR_CUDA;
    p.x = x; p.dt = dt; p.Bm = Bm; p.Cm = Cm; p.z = z;
    p.A = A; p.Dskip = Dskip; p.dt_bias = dt_bias; p.h0 = h0;
    p.D = D; p.G = G; p.N = N; p.softplus = flags & DN_SCAN_SOFTPLUS;
    p.dy = d_y; p.dht = d_ht;
    p.dx = d_x; p.ddt = d_dt; p.dBm = d_Bm; p.dCm = d_Cm; p.dz = d_z;
    p.dA = d_A; p.dDskip = d_Dskip; p.ddt_bias = d_dt_bias; p.dh0 = d_h0;
    dn::scan_bwd_carve(p, workspace);
    const char *name = "";
    return done(dn::scan_bwd_launch(p, dtype == DN_BF16, (cudaStream_t)stream, &name), name);
}

// ---- layer norm ----------------------------------------------------------------

namespace {

constexpr int kNormMaxD = 16384;

dn_status norm_check(const void *x, const float *weight, const float *bias, const void *z, int64_t rows, int D,
                     dn_dtype dtype, float eps, unsigned flags) {
    if (!dtype_ok(dtype) || rows < 0 || D <= 0) return DN_ERR_INVALID_ARG;
    if (!(eps >= 0.f) || isinf(eps)) return DN_ERR_INVALID_ARG;
    if (flags & ~DN_NORM_RMS) return DN_ERR_INVALID_ARG;
    if (rows > 0 && !x) return DN_ERR_INVALID_ARG;
    const void *ptrs[] = {x, weight, bias, z};
    if (!all_aligned(ptrs)) return DN_ERR_INVALID_ARG;
    return DN_OK;
}

}  // namespace

DN_EXPORT dn_status dn_layer_norm_fwd(const void *x, const float *weight, const float *bias, const void *z,
                                      int64_t rows, int D, dn_dtype dtype, float eps, unsigned flags, void *y,
                                      dn_stream_t stream) {
    const dn_status st = norm_check(x, weight, bias, z, rows, D, dtype, eps, flags);
    if (st != DN_OK) return st;
    if (!aligned16(y) || (rows > 0 && !y)) return DN_ERR_INVALID_ARG;
    if (D > kNormMaxD) return DN_ERR_UNSUPPORTED;
    if (rows == 0) return DN_OK;
    dn::NormParams p{};
    p.x = x; p.z = z; p.weight = weight; p.bias = bias;
    p.rows = rows; p.D = D; p.eps = eps; p.rms = flags & DN_NORM_RMS;
    p.y = y;
    const char *name = "";
    return done(dn::norm_fwd_launch(p, dtype == DN_BF16, (cudaStream_t)stream, &name), name);
}

DN_EXPORT size_t dn_layer_norm_bwd_workspace_bytes(int64_t rows, int D, dn_dtype dtype) {
    if (rows < 0 || D <= 0 || D > kNormMaxD || !dtype_ok(dtype)) return 0;
    return dn::norm_bwd_workspace(rows, D, dtype == DN_BF16);
}

DN_EXPORT dn_status dn_layer_norm_bwd(const void *x, const float *weight, const float *bias, const void *z,
                                      int64_t rows, int D, dn_dtype dtype, float eps, unsigned flags,
                                      const void *d_y, void *d_x, float *d_weight, float *d_bias, void *d_z,
                                      void *workspace, size_t workspace_bytes, dn_stream_t stream) {
    const dn_status st = norm_check(x, weight, bias, z, rows, D, dtype, eps, flags);
    if (st != DN_OK) return st;
    const void *ptrs[] = {d_y, d_x, d_weight, d_bias, d_z};
    if (!all_aligned(ptrs)) return DN_ERR_INVALID_ARG;
    if (rows > 0 && (!d_y || !d_x || (z != nullptr) != (d_z != nullptr))) return DN_ERR_INVALID_ARG;
    if (D > kNormMaxD) return DN_ERR_UNSUPPORTED;
    const bool sums = d_weight || d_bias;
    if (sums && (!workspace || !aligned16(workspace) ||
                 workspace_bytes < dn::norm_bwd_workspace(rows, D, dtype == DN_BF16)))
        return DN_ERR_INVALID_ARG;
    if (rows == 0 && !sums) return DN_OK;
    dn::NormParams p{};
    p.x = x; p.z = z; p.weight = weight; p.bias = bias;
    p.rows = rows; p.D = D; p.eps = eps; p.rms = flags & DN_NORM_RMS;
    p.dy = d_y; p.dx = d_x; p.dweight = d_weight; p.dbias = d_bias; p.dz = d_z;
    p.partial = sums ? static_cast<float *>(workspace) : nullptr;
    const char *name = "";
    return done(dn::norm_bwd_launch(p, dtype == DN_BF16, (cudaStream_t)stream, &name), name);
}

// ---- norms around a block --------------------------------------------------------

namespace {

dn_status block_check(dn::BlockParams &p, const void *x, const void *residual, const void *z, const float *scale,
                      const float *post_weight, const float *post_bias, const float *weight, const float *bias,
                      int64_t rows, int D, dn_dtype dtype, dn_dtype residual_dtype, float eps, unsigned flags) {
    if (!dtype_ok(dtype) || rows < 0 || D <= 0) return DN_ERR_INVALID_ARG;
    if (residual_dtype != dtype && residual_dtype != DN_F32) return DN_ERR_INVALID_ARG;
    if (!(eps >= 0.f) || isinf(eps)) return DN_ERR_INVALID_ARG;
    if (flags & ~(DN_NORM_RMS | DN_NORM_POST)) return DN_ERR_INVALID_ARG;
    if (rows > 0 && (!x || !residual)) return DN_ERR_INVALID_ARG;
    const void *ptrs[] = {x, residual, z, scale, post_weight, post_bias, weight, bias};
    if (!all_aligned(ptrs)) return DN_ERR_INVALID_ARG;
    p.x = x; p.residual = residual; p.z = z;
    p.scale = scale; p.post_weight = post_weight; p.post_bias = post_bias; p.weight = weight; p.bias = bias;
    p.rows = rows; p.D = D;
    p.bf16 = dtype == DN_BF16; p.res_f32 = residual_dtype == DN_F32;
    p.eps = eps; p.rms = flags & DN_NORM_RMS; p.post = flags & DN_NORM_POST;
    return DN_OK;
}

}  // namespace

DN_EXPORT dn_status dn_block_norm_fwd(const void *x, const void *residual, const void *z, const float *scale,
                                      const float *post_weight, const float *post_bias, const float *weight,
                                      const float *bias, int64_t rows, int D, dn_dtype dtype, dn_dtype residual_dtype,
                                      float eps, unsigned flags, void *y, void *residual_out, dn_stream_t stream) {
    dn::BlockParams p{};
    const dn_status st = block_check(p, x, residual, z, scale, post_weight, post_bias, weight, bias, rows, D, dtype,
                                     residual_dtype, eps, flags);
    if (st != DN_OK) return st;
    const void *ptrs[] = {y, residual_out};
    if (!all_aligned(ptrs) || (rows > 0 && (!y || !residual_out))) return DN_ERR_INVALID_ARG;
    if (D > kNormMaxD) return DN_ERR_UNSUPPORTED;
    if (rows == 0) return DN_OK;
    p.y = y; p.residual_out = residual_out;
    const char *name = "";
    return done(dn::block_fwd_launch(p, (cudaStream_t)stream, &name), name);
}

DN_EXPORT size_t dn_block_norm_bwd_workspace_bytes(int64_t rows, int D, dn_dtype dtype, dn_dtype residual_dtype) {
    if (rows < 0 || D <= 0 || D > kNormMaxD || !dtype_ok(dtype)) return 0;
    if (residual_dtype != dtype && residual_dtype != DN_F32) return 0;
    return dn::block_bwd_workspace(rows, D, dtype == DN_BF16, residual_dtype == DN_F32);
}

DN_EXPORT dn_status dn_block_norm_bwd(const void *x, const void *residual, const void *z, const float *scale,
                                      const float *post_weight, const float *post_bias, const float *weight,
                                      const float *bias, int64_t rows, int D, dn_dtype dtype, dn_dtype residual_dtype,
                                      float eps, unsigned flags, const void *d_y, const void *d_residual_out, void *d_x,
                                      void *d_residual, void *d_z, float *d_scale, float *d_post_weight,
                                      float *d_post_bias, float *d_weight, float *d_bias, void *workspace,
                                      size_t workspace_bytes, dn_stream_t stream) {
    dn::BlockParams p{};
    const dn_status st = block_check(p, x, residual, z, scale, post_weight, post_bias, weight, bias, rows, D, dtype,
                                     residual_dtype, eps, flags);
    if (st != DN_OK) return st;
    const void *ptrs[] = {d_y, d_residual_out, d_x, d_residual, d_z, d_scale, d_post_weight, d_post_bias, d_weight, d_bias};
    if (!all_aligned(ptrs)) return DN_ERR_INVALID_ARG;
    if (rows > 0 && (!d_y || !d_x || !d_residual || (z != nullptr) != (d_z != nullptr))) return DN_ERR_INVALID_ARG;
    if (D > kNormMaxD) return DN_ERR_UNSUPPORTED;
    const bool sums = d_scale || d_post_weight || d_post_bias || d_weight || d_bias;
    if (sums && (!workspace || !aligned16(workspace) ||
                 workspace_bytes < dn::block_bwd_workspace(rows, D, p.bf16, p.res_f32)))
        return DN_ERR_INVALID_ARG;
    if (rows == 0 && !sums) return DN_OK;
    p.dy = d_y; p.dresidual_out = d_residual_out;
    p.dx = d_x; p.dresidual = d_residual; p.dz = d_z;
    p.dscale = d_scale; p.dpost_weight = d_post_weight; p.dpost_bias = d_post_bias; p.dweight = d_weight; p.dbias = d_bias;
    p.partial = sums ? static_cast<float *>(workspace) : nullptr;
    const char *name = "";
    return done(dn::block_bwd_launch(p, (cudaStream_t)stream, &name), name);
}
