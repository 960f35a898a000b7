"""GB300 chunkwise gated delta rule forward -- Python binding of the C ABI.

The binding only marshals arguments: every step of the forward runs in the
CUDA kernels of ``libdnchunk.so`` (declared in ``include/dn_chunk_fwd.h``).
There is no CPU path: if the library is missing, :func:`load` raises.
PyTorch supplies device memory and streams.

Names follow the C ABI: :func:`dn_chunk_fwd`,
:func:`dn_chunk_fwd_workspace_bytes`, :func:`dn_chunk_fwd_noalloc`,
:func:`dn_recurrent_fwd`, :func:`dn_chunk_bwd`,
:func:`dn_chunk_bwd_workspace_bytes`, :func:`dn_check`,
:func:`dn_status_str`, :func:`dn_last_kernel`.  :func:`recurrent_fwd` and
:func:`chunk_bwd` are conveniences for the token-serial entry point and the
backward.  :func:`chunk_fwd` is a convenience that allocates
``o``, ``ht`` and the workspace with torch and calls :func:`dn_chunk_fwd`.

The operators around the recurrence (``include/dn_layer_ops.h``) are
:func:`causal_conv_fwd` and :func:`causal_conv_bwd`, :func:`selective_scan_fwd`
and :func:`selective_scan_bwd`, :func:`layer_norm_fwd` and
:func:`layer_norm_bwd`, :func:`block_norm_fwd` and :func:`block_norm_bwd`; they check
their tensors and allocate what is not given.  So do those of the attention over a sliding
window that stands between such layers (``include/dn_window_ops.h``):
:func:`window_attn_fwd`, :func:`window_attn_bwd`, :func:`window_cache_fill`,
:func:`window_attn_step`.

These and the conveniences above, given a ``stream``, work as under
``torch.cuda.stream(stream)``: what they allocate is that stream's memory, and what they
read has to be ready there.
"""
from __future__ import annotations

import ctypes
import functools
import os
import threading

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libdnchunk.so")

DN_OK = 0
DN_ERR_INVALID_ARG = 1
DN_ERR_UNSUPPORTED = 2
DN_ERR_CUDA = 3
DN_ERR_TIMEOUT = 4
DN_ERR_DEVICE_ARG = 5

DN_BF16 = 0
DN_F32 = 1

# Option bits of the ``flags`` argument.
DN_QK_L2NORM = 1
DN_CONV_SILU = 1
DN_SCAN_SOFTPLUS = 1
DN_NORM_RMS = 1
DN_NORM_POST = 2

# Every symbol the public headers declare.
ABI_SYMBOLS = ("dn_chunk_fwd", "dn_chunk_fwd_workspace_bytes", "dn_chunk_fwd_noalloc",
               "dn_recurrent_fwd", "dn_chunk_bwd", "dn_chunk_bwd_workspace_bytes", "dn_check",
               "dn_status_str", "dn_last_kernel",
               "dn_causal_conv_fwd", "dn_causal_conv_bwd", "dn_causal_conv_bwd_workspace_bytes",
               "dn_selective_scan_fwd", "dn_selective_scan_fwd_workspace_bytes",
               "dn_selective_scan_bwd", "dn_selective_scan_bwd_workspace_bytes",
               "dn_layer_norm_fwd", "dn_layer_norm_bwd", "dn_layer_norm_bwd_workspace_bytes",
               "dn_block_norm_fwd", "dn_block_norm_bwd", "dn_block_norm_bwd_workspace_bytes",
               "dn_window_attn_fwd", "dn_window_attn_bwd", "dn_window_attn_bwd_workspace_bytes",
               "dn_window_cache_fill", "dn_window_attn_step")

# Size of the library's fixed scratch array used by dn_chunk_fwd_noalloc.
DN_NOALLOC_SCRATCH_BYTES = 64 * 1024 * 1024

_lib = None
_lock = threading.Lock()


class DnError(RuntimeError):
    def __init__(self, status: int, what: str = "dn_chunk_fwd"):
        self.status = status
        super().__init__("%s failed: %s" % (what, dn_status_str(status)))


def load(path: str | None = None):
    """Load ``libdnchunk.so`` (raises if it has not been built)."""
    global _lib
    if path is None and _lib is not None:  # set once, complete
        return _lib
    with _lock:
        if _lib is not None and path is None:
            return _lib
        p = path or LIB_PATH
        if not os.path.exists(p):
            raise RuntimeError(
                "libdnchunk.so is not built (%s); run `python -c \"import __graft_entry__ as g; "
                "g.build()\"` -- there is no fallback path" % p)
        lib = ctypes.CDLL(p)
        P, I, F = ctypes.c_void_p, ctypes.c_int, ctypes.c_float
        Z, U = ctypes.c_size_t, ctypes.c_uint
        lib.dn_chunk_fwd.argtypes = [P, P, P, P, P, P, P, I, I, I, I, I, I, I, I, F, U, I, P, P, P, Z,
                                     P]
        lib.dn_chunk_fwd.restype = I
        lib.dn_chunk_fwd_workspace_bytes.argtypes = [I, I, I, I, I, I, I, I, I]
        lib.dn_chunk_fwd_workspace_bytes.restype = Z
        lib.dn_chunk_fwd_noalloc.argtypes = [P, P, P, P, P, P, P, I, I, I, I, I, I, I, I, F, U, I, P,
                                             P, P]
        lib.dn_chunk_fwd_noalloc.restype = I
        lib.dn_recurrent_fwd.argtypes = [P, P, P, P, P, P, P, I, I, I, I, I, I, I, I, F, U, P, P, P]
        lib.dn_recurrent_fwd.restype = I
        lib.dn_chunk_bwd.argtypes = [P, P, P, P, P, P, P, I, I, I, I, I, I, I, I, F, U, P, P, P, P,
                                     P, P, P, P, P, Z, P]
        lib.dn_chunk_bwd.restype = I
        lib.dn_chunk_bwd_workspace_bytes.argtypes = [I, I, I, I, I, I, I, I]
        lib.dn_chunk_bwd_workspace_bytes.restype = Z
        L = ctypes.c_longlong
        lib.dn_causal_conv_fwd.argtypes = [P] * 5 + [I] * 6 + [U, P, P, P]
        lib.dn_causal_conv_bwd.argtypes = [P] * 5 + [I] * 6 + [U, P, I] + [P] * 6 + [Z, P]
        lib.dn_causal_conv_bwd_workspace_bytes.argtypes = [I] * 6
        lib.dn_selective_scan_fwd.argtypes = [P] * 10 + [I] * 7 + [U, P, P, P, Z, P]
        lib.dn_selective_scan_fwd_workspace_bytes.argtypes = [I] * 7
        lib.dn_selective_scan_bwd.argtypes = [P] * 10 + [I] * 7 + [U] + [P] * 12 + [Z, P]
        lib.dn_selective_scan_bwd_workspace_bytes.argtypes = [I] * 7
        lib.dn_layer_norm_fwd.argtypes = [P] * 4 + [L, I, I, F, U, P, P]
        lib.dn_layer_norm_bwd.argtypes = [P] * 4 + [L, I, I, F, U] + [P] * 6 + [Z, P]
        lib.dn_layer_norm_bwd_workspace_bytes.argtypes = [L, I, I]
        lib.dn_block_norm_fwd.argtypes = [P] * 8 + [L, I, I, I, F, U, P, P, P]
        lib.dn_block_norm_bwd.argtypes = [P] * 8 + [L, I, I, I, F, U] + [P] * 11 + [Z, P]
        lib.dn_block_norm_bwd_workspace_bytes.argtypes = [L, I, I, I]
        lib.dn_window_attn_fwd.argtypes = [P] * 4 + [I] * 9 + [F, P, P, P]
        lib.dn_window_attn_bwd.argtypes = [P] * 6 + [I] * 9 + [F] + [P] * 5 + [Z, P]
        lib.dn_window_attn_bwd_workspace_bytes.argtypes = [I] * 10
        lib.dn_window_cache_fill.argtypes = [P] * 3 + [I] * 8 + [P] * 4
        lib.dn_window_cache_fill.restype = I
        lib.dn_window_attn_step.argtypes = [P] * 3 + [I] * 8 + [F] + [P] * 5
        lib.dn_window_attn_step.restype = I
        for op in ("causal_conv", "selective_scan", "layer_norm", "block_norm", "window_attn"):
            getattr(lib, "dn_%s_fwd" % op).restype = I
            getattr(lib, "dn_%s_bwd" % op).restype = I
            getattr(lib, "dn_%s_bwd_workspace_bytes" % op).restype = Z
        lib.dn_selective_scan_fwd_workspace_bytes.restype = Z
        lib.dn_check.argtypes = [P]
        lib.dn_check.restype = I
        lib.dn_status_str.argtypes = [I]
        lib.dn_status_str.restype = ctypes.c_char_p
        lib.dn_last_kernel.argtypes = []
        lib.dn_last_kernel.restype = ctypes.c_char_p
        if path is None:
            _lib = lib
        return lib


def _ptr(x):
    """Device pointer of a tensor (or an int address, or None -> NULL)."""
    if x is None:
        return None
    if isinstance(x, int):
        return x or None
    if not x.is_contiguous():
        raise ValueError("tensors passed to dn_chunk_fwd must be contiguous")
    return x.data_ptr()


def _stream(stream):
    if stream is None:
        import torch
        # the handle alone: making a Stream object takes 3 us, half a small call
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _under(stream, device, torch):
    """The context of a given stream (an object or a raw handle), for a call that was given one.

    The whole call is made in it, so that what it allocates comes from that stream's memory.
    A tensor of another stream's could still be in use there when the call writes it, and
    could be handed on there before the call is done with it.
    """
    if not isinstance(stream, torch.cuda.Stream):
        handle = stream if isinstance(stream, int) else stream.cuda_stream
        # 0 and 1 name the default stream (torch makes a new stream of a handle of 0)
        stream = (torch.cuda.default_stream(device) if handle in (0, 1)
                  else torch.cuda.ExternalStream(handle, device=device))
    return torch.cuda.stream(stream)


def dn_chunk_fwd(q, k, v, beta, g, h0, cu_seqlens, n_seqs, B, T, Nk, Nv, dk, dv, dtype,
                 scale, chunk, o, ht, workspace=None, workspace_bytes=None, stream=None,
                 flags=0) -> int:
    """Call the C entry point as is; returns its status code.

    ``workspace`` is a device tensor (its byte size is passed unless
    ``workspace_bytes`` is given), an int address, or None.  ``flags`` is the
    C argument of that name (0 or :data:`DN_QK_L2NORM`).
    """
    lib = load()
    if workspace_bytes is None:
        workspace_bytes = 0
        if workspace is not None and not isinstance(workspace, int):
            workspace_bytes = workspace.numel() * workspace.element_size()
    return lib.dn_chunk_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(beta), _ptr(g), _ptr(h0),
                            _ptr(cu_seqlens), int(n_seqs), int(B), int(T), int(Nk), int(Nv),
                            int(dk), int(dv), int(dtype), float(scale), int(flags), int(chunk),
                            _ptr(o), _ptr(ht), _ptr(workspace), int(workspace_bytes),
                            _stream(stream))


def dn_chunk_fwd_noalloc(q, k, v, beta, g, h0, cu_seqlens, n_seqs, B, T, Nk, Nv, dk, dv, dtype,
                         scale, chunk, o, ht, stream=None, flags=0) -> int:
    """Call the C entry point that takes no workspace (it uses the library's
    fixed scratch array and allocates nothing); returns its status code."""
    lib = load()
    return lib.dn_chunk_fwd_noalloc(_ptr(q), _ptr(k), _ptr(v), _ptr(beta), _ptr(g), _ptr(h0),
                                    _ptr(cu_seqlens), int(n_seqs), int(B), int(T), int(Nk),
                                    int(Nv), int(dk), int(dv), int(dtype), float(scale), int(flags),
                                    int(chunk), _ptr(o), _ptr(ht), _stream(stream))


def dn_recurrent_fwd(q, k, v, beta, g, h0, cu_seqlens, n_seqs, B, T, Nk, Nv, dk, dv, dtype,
                     scale, o, ht, stream=None, flags=0) -> int:
    """Call the token-serial C entry point as is; returns its status code."""
    lib = load()
    return lib.dn_recurrent_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(beta), _ptr(g), _ptr(h0),
                                _ptr(cu_seqlens), int(n_seqs), int(B), int(T), int(Nk), int(Nv),
                                int(dk), int(dv), int(dtype), float(scale), int(flags), _ptr(o),
                                _ptr(ht), _stream(stream))


def recurrent_fwd(q, k, v, beta, g=None, h0=None, cu_seqlens=None, scale=None,
                  output_final_state=True, stream=None, o=None, ht=None,
                  use_qk_l2norm_in_kernel=False):
    """Allocate ``o`` (and ``ht``) and run :func:`dn_recurrent_fwd` (shapes
    and options as for :func:`chunk_fwd`)."""
    import torch
    if stream is not None:
        with _under(stream, q.device, torch):
            return recurrent_fwd(q, k, v, beta, g, h0, cu_seqlens, scale, output_final_state, None,
                                 o, ht, use_qk_l2norm_in_kernel)
    B, T, Nk, dk = q.shape
    Nv, dv = v.shape[2], v.shape[3]
    N = (cu_seqlens.numel() - 1) if cu_seqlens is not None else B
    if o is None:
        o = torch.empty(B, T, Nv, dv, dtype=q.dtype, device=q.device)
    if ht is None and output_final_state:
        ht = torch.empty(N, Nv, dk, dv, dtype=torch.float32, device=q.device)
    st = dn_recurrent_fwd(q, k, v, beta, g, h0, cu_seqlens, N, B, T, Nk, Nv, dk, dv,
                          dtype_code(q.dtype), 0.0 if scale is None else scale, o,
                          ht if output_final_state else None, stream,
                          flags=DN_QK_L2NORM if use_qk_l2norm_in_kernel else 0)
    if st != DN_OK:
        raise DnError(st, "dn_recurrent_fwd")
    return o, (ht if output_final_state else None)


def dn_chunk_fwd_workspace_bytes(n_seqs, B, T, Nk, Nv, dk, dv, dtype, chunk=64) -> int:
    return int(load().dn_chunk_fwd_workspace_bytes(int(n_seqs), int(B), int(T), int(Nk), int(Nv),
                                                   int(dk), int(dv), int(dtype), int(chunk)))


def workspace_for(q, v, n_seqs, chunk=64):
    """A uint8 device tensor of the workspace size for these inputs (or None)."""
    import torch
    B, T, Nk, dk = q.shape
    Nv, dv = v.shape[2], v.shape[3]
    nbytes = dn_chunk_fwd_workspace_bytes(n_seqs, B, T, Nk, Nv, dk, dv, dtype_code(q.dtype), chunk)
    if nbytes == 0:
        return None
    return torch.empty(nbytes, dtype=torch.uint8, device=q.device)


def dn_check(stream=None) -> int:
    return load().dn_check(_stream(stream))


def dn_status_str(status: int) -> str:
    try:
        return load().dn_status_str(int(status)).decode()
    except RuntimeError:
        return "status %d" % status


def dn_last_kernel() -> str:
    return load().dn_last_kernel().decode()


def dtype_code(dtype) -> int:
    import torch
    if dtype is torch.bfloat16:
        return DN_BF16
    if dtype is torch.float32:
        return DN_F32
    raise ValueError("unsupported dtype %s (bf16 or fp32)" % dtype)


def chunk_fwd(q, k, v, beta, g=None, h0=None, cu_seqlens=None, scale=None,
              output_final_state=True, chunk=64, stream=None, o=None, ht=None, workspace=None,
              use_qk_l2norm_in_kernel=False):
    """Allocate ``o`` (and ``ht``, and the workspace) and run :func:`dn_chunk_fwd`.

    q, k ``[B, T, Nk, dk]``; v ``[B, T, Nv, dv]``; beta, g ``[B, T, Nv]`` fp32;
    h0 ``[N, Nv, dk, dv]`` fp32; cu_seqlens int64 ``[N+1]`` on the device.
    ``use_qk_l2norm_in_kernel`` sets :data:`DN_QK_L2NORM` (the kernels
    normalise every q and k row).  Returns ``(o, ht)`` (``ht`` is None unless
    ``output_final_state``).
    """
    import torch
    if stream is not None:
        with _under(stream, q.device, torch):
            return chunk_fwd(q, k, v, beta, g, h0, cu_seqlens, scale, output_final_state, chunk,
                             None, o, ht, workspace, use_qk_l2norm_in_kernel)
    B, T, Nk, dk = q.shape
    Nv, dv = v.shape[2], v.shape[3]
    N = (cu_seqlens.numel() - 1) if cu_seqlens is not None else B
    if o is None:
        o = torch.empty(B, T, Nv, dv, dtype=q.dtype, device=q.device)
    if ht is None and output_final_state:
        ht = torch.empty(N, Nv, dk, dv, dtype=torch.float32, device=q.device)
    if workspace is None:
        workspace = workspace_for(q, v, N, chunk)
    st = dn_chunk_fwd(q, k, v, beta, g, h0, cu_seqlens, N, B, T, Nk, Nv, dk, dv,
                      dtype_code(q.dtype), 0.0 if scale is None else scale, chunk, o,
                      ht if output_final_state else None, workspace, stream=stream,
                      flags=DN_QK_L2NORM if use_qk_l2norm_in_kernel else 0)
    if st != DN_OK:
        raise DnError(st)
    return o, (ht if output_final_state else None)


def dn_chunk_bwd(q, k, v, beta, g, h0, cu_seqlens, n_seqs, B, T, Nk, Nv, dk, dv, dtype, scale,
                 flags, d_o, d_ht, d_q, d_k, d_v, d_beta, d_g, d_h0, workspace,
                 workspace_bytes=None, stream=None) -> int:
    """Call the backward C entry point as is; returns its status code."""
    lib = load()
    if workspace_bytes is None:
        workspace_bytes = 0
        if workspace is not None and not isinstance(workspace, int):
            workspace_bytes = workspace.numel() * workspace.element_size()
    return lib.dn_chunk_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(beta), _ptr(g), _ptr(h0),
                            _ptr(cu_seqlens), int(n_seqs), int(B), int(T), int(Nk), int(Nv),
                            int(dk), int(dv), int(dtype), float(scale), int(flags), _ptr(d_o),
                            _ptr(d_ht), _ptr(d_q), _ptr(d_k), _ptr(d_v), _ptr(d_beta), _ptr(d_g),
                            _ptr(d_h0), _ptr(workspace), int(workspace_bytes), _stream(stream))


def dn_chunk_bwd_workspace_bytes(n_seqs, B, T, Nk, Nv, dk, dv, dtype) -> int:
    return int(load().dn_chunk_bwd_workspace_bytes(int(n_seqs), int(B), int(T), int(Nk),
                                                   int(Nv), int(dk), int(dv), int(dtype)))


def chunk_bwd(q, k, v, beta, g=None, h0=None, cu_seqlens=None, scale=None, do=None, dht=None,
              stream=None, workspace=None, use_qk_l2norm_in_kernel=False):
    """Gradients of :func:`chunk_fwd`'s loss ``sum(do * o) + sum(dht * ht)``
    (with the same ``use_qk_l2norm_in_kernel``).

    Allocates the fp32 gradients and the workspace with torch and runs
    :func:`dn_chunk_bwd`.  Returns a dict with ``dq``, ``dk``, ``dv``,
    ``dbeta``, ``dg`` (None when g is None) and ``dh0`` (None when h0 is None).
    """
    import torch
    if stream is not None:
        with _under(stream, q.device, torch):
            return chunk_bwd(q, k, v, beta, g, h0, cu_seqlens, scale, do, dht, None, workspace,
                             use_qk_l2norm_in_kernel)
    B, T, Nk, dk = q.shape
    Nv, dv = v.shape[2], v.shape[3]
    N = (cu_seqlens.numel() - 1) if cu_seqlens is not None else B
    f32 = dict(dtype=torch.float32, device=q.device)
    out = dict(dq=torch.empty(q.shape, **f32), dk=torch.empty(k.shape, **f32),
               dv=torch.empty(v.shape, **f32), dbeta=torch.empty(beta.shape, **f32),
               dg=None if g is None else torch.empty(beta.shape, **f32),
               dh0=None if h0 is None else torch.empty(N, Nv, dk, dv, **f32))
    if workspace is None:
        nbytes = dn_chunk_bwd_workspace_bytes(N, B, T, Nk, Nv, dk, dv, dtype_code(q.dtype))
        workspace = torch.empty(max(nbytes, 16), dtype=torch.uint8, device=q.device)
    st = dn_chunk_bwd(q, k, v, beta, g, h0, cu_seqlens, N, B, T, Nk, Nv, dk, dv,
                      dtype_code(q.dtype), 0.0 if scale is None else scale,
                      DN_QK_L2NORM if use_qk_l2norm_in_kernel else 0, do, dht,
                      out["dq"], out["dk"], out["dv"], out["dbeta"], out["dg"], out["dh0"],
                      workspace, stream=stream)
    if st != DN_OK:
        raise DnError(st, "dn_chunk_bwd")
    return out


# ---- operators around the recurrence (include/dn_layer_ops.h) -------------


def _operand(name, t, shape, dtype, device, optional=True):
    """Address of a tensor that is what the C entry point takes it for (else ValueError)."""
    if t is None:
        if optional:
            return None
        raise ValueError("%s is required" % name)
    if t.dtype is dtype and t.shape == shape and t.device == device and t.is_contiguous():
        return t.data_ptr()
    raise ValueError("%s must be a contiguous %s tensor of shape %s on %s, not %s of shape %s on %s%s"
                     % (name, dtype, tuple(shape), device, t.dtype, tuple(t.shape), t.device,
                        "" if t.is_contiguous() else ", not contiguous"))


def _device_of(x, torch):
    """The device of a call's first tensor, which has to be the current one."""
    device = x.device
    if device.type != "cuda":
        raise ValueError("tensors must be on a CUDA device, not on %s" % device)
    if device.index != torch._C._cuda_getDevice():
        raise ValueError("tensors are on %s, which is not the current device" % device)
    return device


def _fit(what, sizes):
    """Refuses sizes (or'ed together) that an int of the C arguments would cut short."""
    if sizes >> 31:
        raise DnError(DN_ERR_UNSUPPORTED, what)


def _sequences(B, cu_seqlens, device):
    """Number of sequences and the offsets' address."""
    import torch
    if cu_seqlens is None:
        return B, None
    if B != 1:
        raise ValueError("cu_seqlens needs B = 1, not %d" % B)
    if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 1:
        raise ValueError("cu_seqlens must have one dimension of N + 1 offsets")
    return cu_seqlens.numel() - 1, _operand("cu_seqlens", cu_seqlens, cu_seqlens.shape, torch.int64,
                                            device)


@functools.lru_cache(maxsize=4096)
def _workspace_bytes(entry, *sizes):
    """What a *_workspace_bytes entry point gives for these sizes (they alone decide)."""
    return getattr(load(), entry)(*sizes)


def _space(nbytes, workspace, device):
    """The caller's workspace, or a new one; and its address and bytes."""
    import torch
    if workspace is None:
        if nbytes == 0:
            return None, None, 0
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=device)
    elif workspace.device != device or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on %s" % device)
    return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()


def causal_conv_fwd(x, weight, bias=None, h0=None, cu_seqlens=None, silu=True,
                    output_final_state=True, stream=None, y=None, ht=None):
    """Short depthwise causal convolution (``dn_causal_conv_fwd``).

    x ``[B, T, D]``; weight ``[D, W]`` and bias ``[D]`` fp32, W = 2..4; h0
    ``[N, W-1, D]`` the inputs before each sequence, of x's type; cu_seqlens
    int64 ``[N+1]`` on the device.  ``silu`` applies silu to the result.  One
    decoding step is T = 1 with h0 given; ``ht`` may then be ``h0`` itself.
    Returns ``(y, ht)`` (``ht`` is None unless ``output_final_state``).
    """
    import torch
    device = _device_of(x, torch)
    if stream is not None:
        with _under(stream, device, torch):
            return causal_conv_fwd(x, weight, bias, h0, cu_seqlens, silu, output_final_state, None,
                                   y, ht)
    B, T, D = x.shape
    W = weight.shape[-1]
    f32, dt = torch.float32, x.dtype
    code = dtype_code(dt)
    N, cu = _sequences(B, cu_seqlens, device)
    _fit("dn_causal_conv_fwd", N | B | T | D | W)
    state = (N, W - 1, D)
    if y is None:
        y = torch.empty_like(x, memory_format=torch.contiguous_format)
    if not output_final_state:
        ht = None
    elif ht is None:
        ht = torch.empty(state, dtype=dt, device=device)
    st = load().dn_causal_conv_fwd(
        _operand("x", x, x.shape, dt, device), _operand("weight", weight, (D, W), f32, device, False),
        _operand("bias", bias, (D,), f32, device), _operand("h0", h0, state, dt, device), cu, N, B, T,
        D, W, code, DN_CONV_SILU if silu else 0, _operand("y", y, x.shape, dt, device),
        _operand("ht", ht, state, dt, device), torch._C._cuda_getCurrentRawStream(device.index))
    if st != DN_OK:
        raise DnError(st, "dn_causal_conv_fwd")
    return y, ht


def causal_conv_bwd(x, weight, bias=None, h0=None, cu_seqlens=None, silu=True, dy=None, dht=None,
                    stream=None, workspace=None):
    """Gradients of :func:`causal_conv_fwd`'s loss ``sum(dy * y) + sum(dht * ht)``.

    ``dy`` has x's type or fp32 (what :func:`chunk_bwd` returns).  Returns a
    dict with ``dx`` and ``dh0`` (None when h0 is None) of x's type, and
    ``dweight`` and ``dbias`` (None when bias is None) in fp32.
    """
    import torch
    device = _device_of(x, torch)
    if stream is not None:
        with _under(stream, device, torch):
            return causal_conv_bwd(x, weight, bias, h0, cu_seqlens, silu, dy, dht, None, workspace)
    B, T, D = x.shape
    W = weight.shape[-1]
    f32, dt = torch.float32, x.dtype
    code = dtype_code(dt)
    N, cu = _sequences(B, cu_seqlens, device)
    _fit("dn_causal_conv_bwd", N | B | T | D | W)
    state = (N, W - 1, D)
    if dy is None:
        raise ValueError("dy is required")
    gt = dy.dtype if dy.dtype == f32 else dt
    lib = load()
    out = dict(dx=torch.empty_like(x, memory_format=torch.contiguous_format),
               dweight=torch.empty((D, W), dtype=f32, device=device),
               dbias=None if bias is None else torch.empty(D, dtype=f32, device=device),
               dh0=None if h0 is None else torch.empty(state, dtype=dt, device=device))
    need = _workspace_bytes("dn_causal_conv_bwd_workspace_bytes", N, B, T, D, W, code)
    workspace, ws, wsb = _space(need, workspace, device)
    st = lib.dn_causal_conv_bwd(
        _operand("x", x, x.shape, dt, device), _operand("weight", weight, (D, W), f32, device, False),
        _operand("bias", bias, (D,), f32, device), _operand("h0", h0, state, dt, device), cu, N, B, T,
        D, W, code, DN_CONV_SILU if silu else 0, _operand("dy", dy, x.shape, gt, device),
        dtype_code(gt), _operand("dht", dht, state, dt, device), out["dx"].data_ptr(),
        out["dweight"].data_ptr(), _ptr(out["dbias"]), _ptr(out["dh0"]), ws, wsb,
        torch._C._cuda_getCurrentRawStream(device.index))
    if st != DN_OK:
        raise DnError(st, "dn_causal_conv_bwd")
    return out


def _scan_inputs(what, x, dt, A, B, C, D, z, dt_bias, h0, cu_seqlens, dt_softplus):
    """Checked addresses and sizes of a scan, in the order of the C arguments."""
    import torch
    device = _device_of(x, torch)
    Bt, T, Di = x.shape
    G, Ns = B.shape[-2:]
    f32, ty = torch.float32, x.dtype
    code = dtype_code(ty)
    N, cu = _sequences(Bt, cu_seqlens, device)
    _fit(what, N | Bt | T | Di | G | Ns)
    rows, bc, state = x.shape, (Bt, T, G, Ns), (N, Di, Ns)
    ptrs = (_operand("x", x, rows, ty, device), _operand("dt", dt, rows, ty, device, False),
            _operand("A", A, (Di, Ns), f32, device, False), _operand("B", B, bc, ty, device, False),
            _operand("C", C, bc, ty, device, False), _operand("D", D, (Di,), f32, device),
            _operand("z", z, rows, ty, device), _operand("dt_bias", dt_bias, (Di,), f32, device),
            _operand("h0", h0, state, f32, device), cu)
    sizes = (N, Bt, T, Di, G, Ns, code)
    return device, ty, bc, state, ptrs, sizes, DN_SCAN_SOFTPLUS if dt_softplus else 0


def selective_scan_fwd(x, dt, A, B, C, D=None, z=None, dt_bias=None, h0=None, cu_seqlens=None,
                       dt_softplus=True, output_final_state=True, stream=None, y=None, ht=None,
                       workspace=None):
    """Selective state space scan (``dn_selective_scan_fwd``).

    x, dt, z ``[B, T, D]`` and B, C ``[B, T, G, N]`` of one type; A ``[D, N]``,
    D and dt_bias ``[D]``, h0 ``[n_seqs, D, N]`` fp32; N = 16, 32, 64 or 128;
    cu_seqlens int64 ``[n_seqs+1]`` on the device.  ``dt_softplus`` passes
    dt + dt_bias through log(1 + e^.).  One decoding step is T = 1 with h0
    given; ``ht`` may then be ``h0`` itself.  Returns ``(y, ht)`` (``ht`` is
    None unless ``output_final_state``).
    """
    import torch
    if stream is not None:
        with _under(stream, _device_of(x, torch), torch):
            return selective_scan_fwd(x, dt, A, B, C, D, z, dt_bias, h0, cu_seqlens, dt_softplus,
                                      output_final_state, None, y, ht, workspace)
    device, ty, bc, state, ptrs, sizes, flags = _scan_inputs(
        "dn_selective_scan_fwd", x, dt, A, B, C, D, z, dt_bias, h0, cu_seqlens, dt_softplus)
    if y is None:
        y = torch.empty_like(x, memory_format=torch.contiguous_format)
    if not output_final_state:
        ht = None
    elif ht is None:
        ht = torch.empty(state, dtype=torch.float32, device=device)
    lib = load()
    need = _workspace_bytes("dn_selective_scan_fwd_workspace_bytes", *sizes)
    workspace, ws, wsb = _space(need, workspace, device)
    st = lib.dn_selective_scan_fwd(*ptrs, *sizes, flags, _operand("y", y, x.shape, ty, device),
                                   _operand("ht", ht, state, torch.float32, device), ws, wsb,
                                   torch._C._cuda_getCurrentRawStream(device.index))
    if st != DN_OK:
        raise DnError(st, "dn_selective_scan_fwd")
    return y, ht


def selective_scan_bwd(x, dt, A, B, C, D=None, z=None, dt_bias=None, h0=None, cu_seqlens=None,
                       dt_softplus=True, dy=None, dht=None, stream=None, workspace=None):
    """Gradients of :func:`selective_scan_fwd`'s loss ``sum(dy * y) + sum(dht * ht)``.

    Returns a dict with ``dx``, ``ddt``, ``dz``, ``dB``, ``dC`` of x's type and
    ``dA``, ``dD``, ``ddt_bias``, ``dh0`` in fp32; those of absent inputs are None.
    """
    import torch
    if stream is not None:
        with _under(stream, _device_of(x, torch), torch):
            return selective_scan_bwd(x, dt, A, B, C, D, z, dt_bias, h0, cu_seqlens, dt_softplus,
                                      dy, dht, None, workspace)
    device, ty, bc, state, ptrs, sizes, flags = _scan_inputs(
        "dn_selective_scan_bwd", x, dt, A, B, C, D, z, dt_bias, h0, cu_seqlens, dt_softplus)
    f32 = torch.float32

    def like(t, shape, dtype):
        return None if t is None else torch.empty(shape, dtype=dtype, device=device)

    out = dict(dx=like(x, x.shape, ty), ddt=like(x, x.shape, ty), dA=like(A, A.shape, f32),
               dB=like(B, bc, ty), dC=like(C, bc, ty), dD=like(D, (x.shape[2],), f32),
               dz=like(z, x.shape, ty), ddt_bias=like(dt_bias, (x.shape[2],), f32),
               dh0=like(h0, state, f32))
    lib = load()
    need = _workspace_bytes("dn_selective_scan_bwd_workspace_bytes", *sizes)
    workspace, ws, wsb = _space(need, workspace, device)
    st = lib.dn_selective_scan_bwd(
        *ptrs, *sizes, flags, _operand("dy", dy, x.shape, ty, device, False),
        _operand("dht", dht, state, f32, device), _ptr(out["dx"]), _ptr(out["ddt"]), _ptr(out["dA"]),
        _ptr(out["dB"]), _ptr(out["dC"]), _ptr(out["dD"]), _ptr(out["dz"]), _ptr(out["ddt_bias"]),
        _ptr(out["dh0"]), ws, wsb, torch._C._cuda_getCurrentRawStream(device.index))
    if st != DN_OK:
        raise DnError(st, "dn_selective_scan_bwd")
    return out


def layer_norm_fwd(x, weight=None, bias=None, z=None, eps=1e-5, rms=False, stream=None, y=None):
    """Layer norm over the last dimension of x (``dn_layer_norm_fwd``).

    weight and bias ``[D]`` fp32; ``z`` of x's shape and type multiplies the
    result by silu(z); ``rms`` takes no mean (root mean square norm).  ``y``
    may be x or z.  Returns y.
    """
    import torch
    device = _device_of(x, torch)
    if stream is not None:
        with _under(stream, device, torch):
            return layer_norm_fwd(x, weight, bias, z, eps, rms, None, y)
    D = x.shape[-1]
    _fit("dn_layer_norm_fwd", D)
    f32, dt = torch.float32, x.dtype
    if y is None:
        y = torch.empty_like(x, memory_format=torch.contiguous_format)
    st = load().dn_layer_norm_fwd(
        _operand("x", x, x.shape, dt, device), _operand("weight", weight, (D,), f32, device),
        _operand("bias", bias, (D,), f32, device), _operand("z", z, x.shape, dt, device),
        x.numel() // D if D else 0, D, dtype_code(dt), eps, DN_NORM_RMS if rms else 0,
        _operand("y", y, x.shape, dt, device), torch._C._cuda_getCurrentRawStream(device.index))
    if st != DN_OK:
        raise DnError(st, "dn_layer_norm_fwd")
    return y


def layer_norm_bwd(x, weight=None, bias=None, z=None, eps=1e-5, rms=False, dy=None, stream=None,
                   workspace=None):
    """Gradients of :func:`layer_norm_fwd`'s loss ``sum(dy * y)``.

    Returns a dict with ``dx`` and ``dz`` of x's type and ``dweight`` and
    ``dbias`` in fp32; those of absent inputs are None.
    """
    import torch
    device = _device_of(x, torch)
    if stream is not None:
        with _under(stream, device, torch):
            return layer_norm_bwd(x, weight, bias, z, eps, rms, dy, None, workspace)
    D = x.shape[-1]
    _fit("dn_layer_norm_bwd", D)
    rows = x.numel() // D if D else 0
    f32, dt = torch.float32, x.dtype
    code = dtype_code(dt)
    lib = load()
    out = dict(dx=torch.empty_like(x, memory_format=torch.contiguous_format),
               dweight=None if weight is None else torch.empty_like(weight),
               dbias=None if bias is None else torch.empty_like(bias),
               dz=None if z is None else torch.empty_like(x, memory_format=torch.contiguous_format))
    need = 0
    if weight is not None or bias is not None:
        need = _workspace_bytes("dn_layer_norm_bwd_workspace_bytes", rows, D, code)
    workspace, ws, wsb = _space(need, workspace, device)
    st = lib.dn_layer_norm_bwd(
        _operand("x", x, x.shape, dt, device), _operand("weight", weight, (D,), f32, device),
        _operand("bias", bias, (D,), f32, device), _operand("z", z, x.shape, dt, device), rows, D,
        code, eps, DN_NORM_RMS if rms else 0, _operand("dy", dy, x.shape, dt, device, False),
        out["dx"].data_ptr(), _ptr(out["dweight"]), _ptr(out["dbias"]), _ptr(out["dz"]), ws, wsb,
        torch._C._cuda_getCurrentRawStream(device.index))
    if st != DN_OK:
        raise DnError(st, "dn_layer_norm_bwd")
    return out


def _vector(name, t, D, device, f32):
    """Address of an optional fp32 vector of D elements (else ValueError)."""
    if t is None:
        return None
    if t.dtype is f32 and t.dim() == 1 and t.numel() == D and t.device == device and t.is_contiguous():
        return t.data_ptr()
    return _operand(name, t, (D,), f32, device)


def _block_inputs(what, x, residual, z, scale, post_weight, post_bias, weight, bias, eps, rms, post):
    """Checked addresses and sizes of a block's norms, in the order of the C arguments."""
    import torch
    device = _device_of(x, torch)
    shape, f32, dt = x.shape, torch.float32, x.dtype
    D = shape[-1]
    _fit(what, D)
    code = dtype_code(dt)
    if residual is None:
        raise ValueError("residual is required")
    rt = f32 if residual.dtype is f32 else dt
    return device, rt, (_operand("x", x, shape, dt, device), _operand("residual", residual, shape, rt, device),
                        None if z is None else _operand("z", z, shape, dt, device),
                        _vector("scale", scale, D, device, f32), _vector("post_weight", post_weight, D, device, f32),
                        _vector("post_bias", post_bias, D, device, f32), _vector("weight", weight, D, device, f32),
                        _vector("bias", bias, D, device, f32),
                        x.numel() // D if D else 0, D, code, code if rt is dt else DN_F32), (
        eps, (DN_NORM_RMS if rms else 0) | (DN_NORM_POST if post else 0))


def block_norm_fwd(x, residual, z=None, scale=None, post_weight=None, post_bias=None, weight=None,
                   bias=None, eps=1e-5, rms=False, post=True, stream=None, y=None,
                   residual_out=None):
    """The norm after a block, its gate and residual scale, and the norm before the next block
    (``dn_block_norm_fwd``)::

        h = residual + scale sigmoid(z) (norm(x) post_weight + post_bias)
        y = norm(h) weight + bias

    x is the block's output, z (of x's shape and type) its gate; residual is of x's type or
    fp32; the five vectors are fp32 ``[D]``.  ``post=False`` leaves the norm of x out, ``rms``
    takes no mean in either norm.  ``y`` may be x or z, ``residual_out`` may be residual.
    Returns ``(y, residual_out)``, the latter being h.
    """
    import torch
    if stream is not None:
        with _under(stream, _device_of(x, torch), torch):
            return block_norm_fwd(x, residual, z, scale, post_weight, post_bias, weight, bias, eps,
                                  rms, post, None, y, residual_out)
    device, rt, args, kind = _block_inputs("dn_block_norm_fwd", x, residual, z, scale, post_weight,
                                           post_bias, weight, bias, eps, rms, post)
    if y is None:
        y = torch.empty_like(x, memory_format=torch.contiguous_format)
    if residual_out is None:
        residual_out = torch.empty_like(residual, memory_format=torch.contiguous_format)
    st = load().dn_block_norm_fwd(*args, *kind, _operand("y", y, x.shape, x.dtype, device),
                                  _operand("residual_out", residual_out, x.shape, rt, device),
                                  torch._C._cuda_getCurrentRawStream(device.index))
    if st != DN_OK:
        raise DnError(st, "dn_block_norm_fwd")
    return y, residual_out


def block_norm_bwd(x, residual, z=None, scale=None, post_weight=None, post_bias=None, weight=None,
                   bias=None, eps=1e-5, rms=False, post=True, dy=None, dresidual_out=None,
                   stream=None, workspace=None):
    """Gradients of :func:`block_norm_fwd`'s loss ``sum(dy * y) + sum(dresidual_out * residual_out)``.

    ``dresidual_out`` has residual's type (None: zero).  Returns a dict with ``dx``, ``dz`` of x's
    type, ``dresidual`` of residual's and ``dscale``, ``dpost_weight``, ``dpost_bias``, ``dweight``,
    ``dbias`` in fp32; those of absent inputs are None.
    """
    import torch
    if stream is not None:
        with _under(stream, _device_of(x, torch), torch):
            return block_norm_bwd(x, residual, z, scale, post_weight, post_bias, weight, bias, eps, rms,
                                  post, dy, dresidual_out, None, workspace)
    device, rt, args, kind = _block_inputs("dn_block_norm_bwd", x, residual, z, scale, post_weight,
                                           post_bias, weight, bias, eps, rms, post)
    lib = load()

    def like(t):
        return None if t is None else torch.empty_like(t, memory_format=torch.contiguous_format)

    out = dict(dx=like(x), dresidual=like(residual), dz=like(z), dscale=like(scale),
               dpost_weight=like(post_weight), dpost_bias=like(post_bias), dweight=like(weight),
               dbias=like(bias))
    need = 0
    if not (scale is None and post_weight is None and post_bias is None and weight is None and bias is None):
        need = _workspace_bytes("dn_block_norm_bwd_workspace_bytes", *args[-4:])
    workspace, ws, wsb = _space(need, workspace, device)
    st = lib.dn_block_norm_bwd(*args, *kind, _operand("dy", dy, x.shape, x.dtype, device, False),
                               _operand("dresidual_out", dresidual_out, x.shape, rt, device),
                               *(_ptr(t) for t in out.values()), ws, wsb,
                               torch._C._cuda_getCurrentRawStream(device.index))
    if st != DN_OK:
        raise DnError(st, "dn_block_norm_bwd")
    return out


# ---- attention over a sliding window (include/dn_window_ops.h) ------------


def _window_inputs(what, q, k, v, window, sinks, cu_seqlens, scale):
    """Checked addresses and sizes of a windowed attention, in the order of the C arguments."""
    import torch
    device = _device_of(q, torch)
    B, T, Nq, d = q.shape
    Nk = k.shape[-2]
    dt = q.dtype
    code = dtype_code(dt)
    N, cu = _sequences(B, cu_seqlens, device)
    if window < 1 or sinks < 0:
        raise ValueError("window must be 1 or more and sinks 0 or more, not %s and %s" % (window, sinks))
    _fit(what, N | B | T | Nq | Nk | d | sinks)
    kv = (B, T, Nk, d)
    ptrs = (_operand("q", q, q.shape, dt, device), _operand("k", k, kv, dt, device, False),
            _operand("v", v, kv, dt, device, False))
    # a window beyond the sequence's length is that length: what an int holds is enough
    sizes = (N, B, T, Nq, Nk, d, min(window, 2**31 - 1), sinks, code)
    return device, dt, ptrs, cu, sizes, 0.0 if scale is None else scale


def window_attn_fwd(q, k, v, window, sinks=0, cu_seqlens=None, scale=None, stream=None, o=None,
                    lse=None):
    """Causal attention over the last ``window`` tokens, the own one among them, and the first
    ``sinks`` ones (``dn_window_attn_fwd``).

    q ``[B, T, Nq, d]``; k, v ``[B, T, Nk, d]``, Nq a multiple of Nk; d = 64 or 128; bf16 or
    fp32; sinks up to 128; cu_seqlens int64 ``[N+1]`` on the device; ``scale`` None, or 0 and
    less: 1 / sqrt(d).
    Returns ``(o, lse)``, the latter ``[B, T, Nq]`` fp32: the logarithms of the softmax's sums,
    which :func:`window_attn_bwd` takes.
    """
    import torch
    if stream is not None:
        with _under(stream, _device_of(q, torch), torch):
            return window_attn_fwd(q, k, v, window, sinks, cu_seqlens, scale, None, o, lse)
    device, dt, ptrs, cu, sizes, scale = _window_inputs("dn_window_attn_fwd", q, k, v, window, sinks,
                                                        cu_seqlens, scale)
    if o is None:
        o = torch.empty_like(q, memory_format=torch.contiguous_format)
    if lse is None:
        lse = torch.empty(q.shape[:3], dtype=torch.float32, device=device)
    st = load().dn_window_attn_fwd(*ptrs, cu, *sizes, scale, _operand("o", o, q.shape, dt, device),
                                   _operand("lse", lse, q.shape[:3], torch.float32, device),
                                   torch._C._cuda_getCurrentRawStream(device.index))
    if st != DN_OK:
        raise DnError(st, "dn_window_attn_fwd")
    return o, lse


def window_attn_bwd(q, k, v, o, lse, window, sinks=0, cu_seqlens=None, scale=None, do=None,
                    stream=None, workspace=None):
    """Gradients of :func:`window_attn_fwd`'s loss ``sum(do * o)``; o and lse are its results.

    Returns a dict with ``dq``, ``dk`` and ``dv`` of q's type.
    """
    import torch
    if stream is not None:
        with _under(stream, _device_of(q, torch), torch):
            return window_attn_bwd(q, k, v, o, lse, window, sinks, cu_seqlens, scale, do, None,
                                   workspace)
    device, dt, ptrs, cu, sizes, scale = _window_inputs("dn_window_attn_bwd", q, k, v, window, sinks,
                                                        cu_seqlens, scale)
    lib = load()
    rest = (_operand("o", o, q.shape, dt, device, False),
            _operand("lse", lse, q.shape[:3], torch.float32, device, False))
    out = dict(dq=torch.empty_like(q, memory_format=torch.contiguous_format),
               dk=torch.empty_like(k, memory_format=torch.contiguous_format),
               dv=torch.empty_like(v, memory_format=torch.contiguous_format))
    need = _workspace_bytes("dn_window_attn_bwd_workspace_bytes", 0 if cu is None else 1, *sizes)
    workspace, ws, wsb = _space(need, workspace, device)
    st = lib.dn_window_attn_bwd(*ptrs, *rest, cu, *sizes, scale, _operand("do", do, q.shape, dt, device, False),
                                *(t.data_ptr() for t in out.values()), ws, wsb,
                                torch._C._cuda_getCurrentRawStream(device.index))
    if st != DN_OK:
        raise DnError(st, "dn_window_attn_bwd")
    return out


def _cache(k_cache, v_cache, N, Nk, d, sinks, dt, device):
    """Checked addresses of a ring cache, and its ring."""
    slots = k_cache.shape[2] if k_cache.dim() == 4 else 0
    shape = (N, Nk, slots, d)
    if slots <= sinks:
        raise ValueError("the cache must be [N, Nk, sinks + ring, d] with a ring of one slot at least")
    return (_operand("k_cache", k_cache, shape, dt, device, False),
            _operand("v_cache", v_cache, shape, dt, device, False)), slots - sinks


def window_cache_fill(k, v, k_cache, v_cache, lengths=None, sinks=0, cu_seqlens=None, stream=None):
    """Puts the tokens of k and v ``[B, T, Nk, d]`` into the ring caches
    ``[N, Nk, sinks + ring, d]`` (``dn_window_cache_fill``).

    The token at position p of its sequence goes to slot p (p < sinks), else to
    ``sinks + (p - sinks) % ring``.  ``lengths`` int64 ``[N]`` on the device are the tokens that
    each sequence had before these (None: none).  Returns ``(k_cache, v_cache)``.
    """
    import torch
    device = _device_of(k, torch)
    if stream is not None:
        with _under(stream, device, torch):
            return window_cache_fill(k, v, k_cache, v_cache, lengths, sinks, cu_seqlens)
    B, T, Nk, d = k.shape
    dt = k.dtype
    code = dtype_code(dt)
    N, cu = _sequences(B, cu_seqlens, device)
    if sinks < 0:
        raise ValueError("sinks must be 0 or more, not %s" % sinks)
    _fit("dn_window_cache_fill", N | B | T | Nk | d | sinks)
    caches, ring = _cache(k_cache, v_cache, N, Nk, d, sinks, dt, device)
    _fit("dn_window_cache_fill", ring)
    st = load().dn_window_cache_fill(
        _operand("k", k, k.shape, dt, device), _operand("v", v, k.shape, dt, device, False), cu, N, B, T, Nk, d,
        sinks, ring, code, _operand("lengths", lengths, (N,), torch.int64, device), *caches,
        torch._C._cuda_getCurrentRawStream(device.index))
    if st != DN_OK:
        raise DnError(st, "dn_window_cache_fill")
    return k_cache, v_cache


def window_attn_step(q, k, v, k_cache, v_cache, lengths, window, sinks=0, scale=None, stream=None,
                     o=None):
    """One decoding step of :func:`window_attn_fwd` over the ring caches (``dn_window_attn_step``).

    q ``[N, 1, Nq, d]``, k, v ``[N, 1, Nk, d]``: the new token of every sequence; its key and value
    are put into the caches.  ``lengths`` int64 ``[N]`` on the device: the tokens that each
    sequence had before (the caller adds one when all layers have run).  The ring has ``window``
    slots at least.  Returns o.
    """
    import torch
    device = _device_of(q, torch)
    if stream is not None:
        with _under(stream, device, torch):
            return window_attn_step(q, k, v, k_cache, v_cache, lengths, window, sinks, scale, None, o)
    N, T, Nq, d = q.shape
    if T != 1:
        raise ValueError("a step takes one token of every sequence, not %d" % T)
    Nk = k.shape[-2]
    dt = q.dtype
    code = dtype_code(dt)
    if window < 1 or sinks < 0:
        raise ValueError("window must be 1 or more and sinks 0 or more, not %s and %s" % (window, sinks))
    _fit("dn_window_attn_step", N | Nq | Nk | d | window | sinks)
    caches, ring = _cache(k_cache, v_cache, N, Nk, d, sinks, dt, device)
    _fit("dn_window_attn_step", ring)
    if o is None:
        o = torch.empty_like(q, memory_format=torch.contiguous_format)
    kv = (N, 1, Nk, d)
    st = load().dn_window_attn_step(
        _operand("q", q, q.shape, dt, device), _operand("k", k, kv, dt, device, False),
        _operand("v", v, kv, dt, device, False), N, Nq, Nk, d, window, sinks, ring, code,
        0.0 if scale is None else scale, _operand("lengths", lengths, (N,), torch.int64, device, False),
        *caches, _operand("o", o, q.shape, dt, device), torch._C._cuda_getCurrentRawStream(device.index))
    if st != DN_OK:
        raise DnError(st, "dn_window_attn_step")
    return o
