// C-ABI front end of the attention over a sliding window and its ring cache:
// argument checks (before any CUDA call) and launches.
#include <math.h>
#include <stdint.h>

#include "dn_window.h"

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
bool head_ok(int d) { return d == 64 || d == 128; }
// Tokens and rows that the kernels count in 32 bits, with room for a tile.
constexpr int kMaxT = 1 << 30;
constexpr long long kMaxTokens = (1ll << 31) - 256;

bool seqs_ok(const int64_t *cu, int n_seqs, int B, int T) {
    if (n_seqs < 0 || B < 0 || T < 0) return false;
    return cu ? B == 1 : n_seqs == B;
}

cudaError_t seq_view(dn::SeqView &s, const int64_t *cu, int n_seqs, int B, int T) {
    s.cu = cu;
    s.N = n_seqs;
    s.T = T;
    s.tokens = (long long)B * T;
    return dn::status_ptr(&s.status);
}

dn_status done(cudaError_t err, const char *name) {
    if (err != cudaSuccess) return DN_ERR_CUDA;
    dn::set_last_kernel(name);
    return DN_OK;
}

float scale_of(float scale, int d) { return scale > 0.f ? scale : 1.f / sqrtf((float)d); }

dn_status attn_check(const void *q, const void *k, const void *v, const void *o, const float *lse, const int64_t *cu,
                     int n_seqs, int B, int T, int Nq, int Nk, int d, int window, int sinks, dn_dtype dtype, float scale) {
    if (!dtype_ok(dtype) || !seqs_ok(cu, n_seqs, B, T) || Nq <= 0 || Nk <= 0 || Nq % Nk != 0 || d <= 0)
        return DN_ERR_INVALID_ARG;
    if (window < 1 || sinks < 0 || isnan(scale) || isinf(scale)) return DN_ERR_INVALID_ARG;
    if ((long long)B * T > 0 && (!q || !k || !v || !o || !lse)) return DN_ERR_INVALID_ARG;
    const void *ptrs[] = {q, k, v, o, lse, cu};
    if (!all_aligned(ptrs)) return DN_ERR_INVALID_ARG;
    if (!head_ok(d) || sinks > dn::kMaxSinks || T > kMaxT || (long long)B * T > kMaxTokens) return DN_ERR_UNSUPPORTED;
    return DN_OK;
}

dn::WindowParams attn_params(const void *q, const void *k, const void *v, int T, int Nq, int Nk, int d, int window,
                             int sinks, float scale, void *o, float *lse) {
    dn::WindowParams p{};
    p.q = q; p.k = k; p.v = v;
    p.Nq = Nq; p.Nk = Nk; p.d = d;
    p.window = window < T ? window : T > 0 ? T : 1;  // no token sees further back than the sequence is long
    p.sinks = sinks;
    p.scale = scale_of(scale, d);
    p.o = o; p.lse = lse;
    return p;
}

}  // namespace

DN_EXPORT dn_status dn_window_attn_fwd(const void *q, const void *k, const void *v, const int64_t *cu_seqlens, int n_seqs,
                                       int B, int T, int Nq, int Nk, int d, int window, int sinks, dn_dtype dtype,
                                       float scale, void *o, float *lse, dn_stream_t stream) {
    const dn_status st = attn_check(q, k, v, o, lse, cu_seqlens, n_seqs, B, T, Nq, Nk, d, window, sinks, dtype, scale);
    if (st != DN_OK) return st;
    if (n_seqs == 0 || (long long)B * T == 0) return DN_OK;
    dn::WindowParams p = attn_params(q, k, v, T, Nq, Nk, d, window, sinks, scale, o, lse);
    if (seq_view(p.seq, cu_seqlens, n_seqs, B, T) != cudaSuccess) return DN_ERR_CUDA;
    const char *name = "";
    return done(dn::window_fwd_launch(p, dtype == DN_BF16, (cudaStream_t)stream, &name), name);
}

DN_EXPORT size_t dn_window_attn_bwd_workspace_bytes(int packed, int n_seqs, int B, int T, int Nq, int Nk, int d, int window,
                                                    int sinks, dn_dtype dtype) {
    if (!dtype_ok(dtype) || n_seqs < 0 || B < 0 || T < 0 || Nq <= 0 || Nk <= 0 || Nq % Nk != 0 || !head_ok(d)) return 0;
    if (window < 1 || sinks < 0 || sinks > dn::kMaxSinks || T > kMaxT || (long long)B * T > kMaxTokens) return 0;
    return dn::window_bwd_workspace((long long)B * T, n_seqs, packed != 0, T, Nq, Nk, d, window, sinks, dtype == DN_BF16);
}

DN_EXPORT dn_status dn_window_attn_bwd(const void *q, const void *k, const void *v, const void *o, const float *lse,
                                       const int64_t *cu_seqlens, int n_seqs, int B, int T, int Nq, int Nk, int d,
                                       int window, int sinks, dn_dtype dtype, float scale, const void *d_o, void *d_q,
                                       void *d_k, void *d_v, void *workspace, size_t workspace_bytes, dn_stream_t stream) {
    const dn_status st = attn_check(q, k, v, o, lse, cu_seqlens, n_seqs, B, T, Nq, Nk, d, window, sinks, dtype, scale);
    if (st != DN_OK) return st;
    const void *ptrs[] = {d_o, d_q, d_k, d_v, workspace};
    if (!all_aligned(ptrs)) return DN_ERR_INVALID_ARG;
    if (n_seqs == 0 || (long long)B * T == 0) return DN_OK;
    if (!d_o || !d_q || !d_k || !d_v) return DN_ERR_INVALID_ARG;
    const bool bf16 = dtype == DN_BF16;
    const size_t need = dn::window_bwd_workspace((long long)B * T, n_seqs, cu_seqlens != nullptr, T, Nq, Nk, d, window,
                                                 sinks, bf16);
    if (!workspace || workspace_bytes < need) return DN_ERR_INVALID_ARG;
    dn::WindowParams p = attn_params(q, k, v, T, Nq, Nk, d, window, sinks, scale, const_cast<void *>(o),
                                     const_cast<float *>(lse));
    if (seq_view(p.seq, cu_seqlens, n_seqs, B, T) != cudaSuccess) return DN_ERR_CUDA;
    p.dout = d_o; p.dq = d_q; p.dk = d_k; p.dv = d_v;
    dn::window_bwd_carve(p, workspace, bf16);
    const char *name = "";
    return done(dn::window_bwd_launch(p, bf16, (cudaStream_t)stream, &name), name);
}

DN_EXPORT dn_status dn_window_cache_fill(const void *k, const void *v, const int64_t *cu_seqlens, int n_seqs, int B, int T,
                                         int Nk, int d, int sinks, int ring, dn_dtype dtype, const int64_t *lengths,
                                         void *k_cache, void *v_cache, dn_stream_t stream) {
    if (!dtype_ok(dtype) || !seqs_ok(cu_seqlens, n_seqs, B, T) || Nk <= 0 || d <= 0 || sinks < 0 || ring < 1)
        return DN_ERR_INVALID_ARG;
    const void *ptrs[] = {k, v, cu_seqlens, lengths, k_cache, v_cache};
    if (!all_aligned(ptrs)) return DN_ERR_INVALID_ARG;
    const bool any = n_seqs > 0 && (long long)B * T > 0;
    if (any && (!k || !v || !k_cache || !v_cache)) return DN_ERR_INVALID_ARG;
    if (!head_ok(d) || (long long)sinks + ring > kMaxT || T > kMaxT || (long long)B * T > kMaxTokens || Nk > 65536)
        return DN_ERR_UNSUPPORTED;
    if (!any) return DN_OK;
    dn::CacheParams p{};
    if (seq_view(p.seq, cu_seqlens, n_seqs, B, T) != cudaSuccess) return DN_ERR_CUDA;
    p.k = k; p.v = v;
    p.N = n_seqs; p.Nk = Nk; p.d = d; p.sinks = sinks; p.ring = ring;
    p.lengths = lengths;
    p.kc = k_cache; p.vc = v_cache;
    p.status = p.seq.status;
    const char *name = "";
    return done(dn::window_fill_launch(p, dtype == DN_BF16, (cudaStream_t)stream, &name), name);
}

DN_EXPORT dn_status dn_window_attn_step(const void *q, const void *k, const void *v, int n_seqs, int Nq, int Nk, int d,
                                        int window, int sinks, int ring, dn_dtype dtype, float scale,
                                        const int64_t *lengths, void *k_cache, void *v_cache, void *o, dn_stream_t stream) {
    if (!dtype_ok(dtype) || n_seqs < 0 || Nq <= 0 || Nk <= 0 || Nq % Nk != 0 || d <= 0) return DN_ERR_INVALID_ARG;
    if (window < 1 || sinks < 0 || ring < window || isnan(scale) || isinf(scale)) return DN_ERR_INVALID_ARG;
    const void *ptrs[] = {q, k, v, lengths, k_cache, v_cache, o};
    if (!all_aligned(ptrs)) return DN_ERR_INVALID_ARG;
    if (n_seqs > 0 && (!q || !k || !v || !lengths || !k_cache || !v_cache || !o)) return DN_ERR_INVALID_ARG;
    if (!head_ok(d) || (long long)sinks + ring > kMaxT || (long long)n_seqs * Nq > kMaxTokens / 16) return DN_ERR_UNSUPPORTED;
    if (n_seqs == 0) return DN_OK;
    dn::CacheParams p{};
    if (dn::status_ptr(&p.status) != cudaSuccess) return DN_ERR_CUDA;
    p.q = q; p.k = k; p.v = v;
    p.N = n_seqs; p.Nq = Nq; p.Nk = Nk; p.d = d; p.window = window; p.sinks = sinks; p.ring = ring;
    p.scale = scale_of(scale, d);
    p.lengths = lengths;
    p.kc = k_cache; p.vc = v_cache; p.o = o;
    const char *name = "";
    return done(dn::window_step_launch(p, dtype == DN_BF16, (cudaStream_t)stream, &name), name);
}
