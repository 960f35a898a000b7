"""The attention over a sliding window, its cache and the norms around a block refuse bad arguments on the
host, before anything reaches the device (no GPU needed)."""
import ctypes

import pytest
import torch

import chunkwise_gated_delta_chunk_gb300 as dn
from test_layer_abi import A, BAD, NO, call

OK = dn.DN_OK


@pytest.fixture(scope="module")
def clib():
    from chunkwise_gated_delta_chunk_gb300 import _build
    _build.build()
    return dn.load()


FWD = dict(q=A, k=A, v=A, cu=None, n=2, B=2, T=8, Nq=4, Nk=2, d=64, w=5, sinks=1, dtype=dn.DN_BF16, scale=0.0, o=A, lse=A, s=None)
BWD = dict(FWD, do=A, dq=A, dk=A, dv=A, ws=A, wsb=1 << 30)
COMMON = [(dict(q=None), BAD), (dict(k=None), BAD), (dict(v=None), BAD), (dict(o=None), BAD), (dict(lse=None), BAD), (dict(q=A + 2), BAD),
          (dict(lse=A + 4), BAD), (dict(n=3), BAD), (dict(cu=A), BAD), (dict(cu=A + 8, B=1), BAD), (dict(T=-1), BAD), (dict(Nq=0), BAD),
          (dict(Nk=0), BAD), (dict(Nk=3), BAD), (dict(d=0), BAD), (dict(w=0), BAD), (dict(w=-5), BAD), (dict(sinks=-1), BAD),
          (dict(dtype=2), BAD), (dict(scale=float("nan")), BAD), (dict(scale=float("inf")), BAD), (dict(d=32), NO), (dict(d=256), NO),
          (dict(sinks=129), NO), (dict(T=(1 << 30) + 1), NO), (dict(T=1 << 30), NO), (dict(n=0, B=0), OK), (dict(T=0), OK)]


@pytest.mark.parametrize("over,code", COMMON)
def test_window_attn_fwd(clib, over, code):
    assert call(clib.dn_window_attn_fwd, "q k v cu n B T Nq Nk d w sinks dtype scale o lse s", FWD, over) == code


@pytest.mark.parametrize("over,code", COMMON + [(dict(do=None), BAD), (dict(dq=None), BAD), (dict(dk=A + 8), BAD), (dict(dv=None), BAD),
                                                (dict(ws=None), BAD), (dict(ws=A + 4), BAD), (dict(wsb=16), BAD)])
def test_window_attn_bwd(clib, over, code):
    order = "q k v o lse cu n B T Nq Nk d w sinks dtype scale do dq dk dv ws wsb s"
    assert call(clib.dn_window_attn_bwd, order, BWD, over) == code


def test_window_attn_bwd_workspace(clib):
    f = clib.dn_window_attn_bwd_workspace_bytes
    good = (0, 4, 4, 2048, 16, 8, 128, 512, 4, dn.DN_BF16)
    assert f(*good) >= 4 * 2048 * 16 * 4 and f(*good) % 16 == 0
    for at, bad in ((1, -1), (3, -1), (4, 7), (5, 0), (6, 32), (7, 0), (8, 129), (9, 3)):
        assert f(*good[:at], bad, *good[at + 1:]) == 0


FILL = dict(k=A, v=A, cu=None, n=2, B=2, T=8, Nk=2, d=64, sinks=1, ring=7, dtype=dn.DN_BF16, len=A, kc=A, vc=A, s=None)


@pytest.mark.parametrize("over,code", [
    (dict(k=None), BAD), (dict(v=None), BAD), (dict(kc=None), BAD), (dict(vc=A + 8), BAD), (dict(len=A + 8), BAD), (dict(n=1), BAD),
    (dict(ring=0), BAD), (dict(sinks=-1), BAD), (dict(dtype=5), BAD), (dict(Nk=0), BAD), (dict(d=48), NO),
    (dict(ring=1 << 30), NO), (dict(T=0), OK), (dict(n=0, B=0), OK),
])
def test_window_cache_fill(clib, over, code):
    assert call(clib.dn_window_cache_fill, "k v cu n B T Nk d sinks ring dtype len kc vc s", FILL, over) == code


STEP = dict(q=A, k=A, v=A, n=2, Nq=4, Nk=2, d=64, w=5, sinks=1, ring=7, dtype=dn.DN_BF16, scale=0.0, len=A, kc=A, vc=A, o=A, s=None)


@pytest.mark.parametrize("over,code", [
    (dict(q=None), BAD), (dict(k=None), BAD), (dict(len=None), BAD), (dict(kc=None), BAD), (dict(o=None), BAD), (dict(o=A + 2), BAD),
    (dict(n=-1), BAD), (dict(Nk=3), BAD), (dict(w=0), BAD), (dict(w=8), BAD), (dict(sinks=-2), BAD), (dict(dtype=9), BAD),
    (dict(scale=float("nan")), BAD), (dict(d=256), NO), (dict(ring=1 << 30), NO), (dict(n=0), OK),
])
def test_window_attn_step(clib, over, code):
    assert call(clib.dn_window_attn_step, "q k v n Nq Nk d w sinks ring dtype scale len kc vc o s", STEP, over) == code


BLOCK = dict(x=A, r=A, z=A, scale=A, pw=A, pb=A, w=A, b=A, rows=4, D=8, dtype=dn.DN_BF16, rt=dn.DN_F32, eps=1e-5, flags=3, y=A, ro=A, s=None)
BLOCK_BWD = dict(BLOCK, dy=A, dro=A, dx=A, dr=A, dz=A, ds=A, dpw=A, dpb=A, dw=A, db=A, ws=A, wsb=1 << 30)
BLOCK_COMMON = [(dict(x=None), BAD), (dict(r=None), BAD), (dict(x=A + 2), BAD), (dict(scale=A + 4), BAD), (dict(pb=A + 8), BAD),
                (dict(rows=-1), BAD), (dict(D=0), BAD), (dict(dtype=2), BAD), (dict(rt=7), BAD), (dict(dtype=dn.DN_F32, rt=dn.DN_BF16), BAD),
                (dict(eps=-1.0), BAD), (dict(eps=float("nan")), BAD), (dict(eps=float("inf")), BAD), (dict(flags=4), BAD), (dict(D=16385), NO)]


@pytest.mark.parametrize("over,code", BLOCK_COMMON + [(dict(y=None), BAD), (dict(ro=None), BAD), (dict(ro=A + 8), BAD), (dict(rows=0), OK)])
def test_block_norm_fwd(clib, over, code):
    assert call(clib.dn_block_norm_fwd, "x r z scale pw pb w b rows D dtype rt eps flags y ro s", BLOCK, over) == code


@pytest.mark.parametrize("over,code", BLOCK_COMMON + [(dict(dy=None), BAD), (dict(dx=None), BAD), (dict(dr=None), BAD), (dict(dz=None), BAD),
                                                      (dict(z=None), BAD), (dict(dw=A + 4), BAD), (dict(ws=None), BAD), (dict(wsb=16), BAD),
                                                      (dict(rows=0, ds=None, dpw=None, dpb=None, dw=None, db=None), OK)])
def test_block_norm_bwd(clib, over, code):
    order = "x r z scale pw pb w b rows D dtype rt eps flags dy dro dx dr dz ds dpw dpb dw db ws wsb s"
    assert call(clib.dn_block_norm_bwd, order, BLOCK_BWD, over) == code


def test_binding_refuses_what_the_library_would_misread(monkeypatch):
    """Shapes, types, devices: on CPU tensors taken for the current device's."""
    monkeypatch.setattr(dn, "_device_of", lambda x, torch: x.device)
    q = torch.zeros(2, 5, 4, 64, dtype=torch.bfloat16)
    k = torch.zeros(2, 5, 2, 64, dtype=torch.bfloat16)
    for bad in (k[:, :4].contiguous(), k.float(), k.transpose(1, 2), torch.zeros(2, 5, 2, 128, dtype=torch.bfloat16), None):
        with pytest.raises(ValueError):
            dn.window_attn_fwd(q, k, bad, 4)
    for window, sinks in ((0, 0), (-1, 0), (4, -1)):
        with pytest.raises(ValueError):
            dn.window_attn_fwd(q, k, k, window, sinks)
        with pytest.raises(ValueError):
            dn.window_attn_bwd(q, k, k, q, torch.zeros(2, 5, 4), window, sinks, do=q)
    with pytest.raises(ValueError):
        dn.window_attn_fwd(q.half(), k.half(), k.half(), 4)
    with pytest.raises(ValueError):
        dn.window_attn_fwd(q, k, k, 4, cu_seqlens=torch.zeros(3, dtype=torch.int64))  # B = 2
    with pytest.raises(ValueError):
        dn.window_attn_bwd(q, k, k, q, torch.zeros(2, 4, 5), 4, do=q)
    with pytest.raises(ValueError):
        dn.window_attn_bwd(q, k, k, q, torch.zeros(2, 5, 4), 4)
    one = q[:, :1].contiguous(), k[:, :1].contiguous()
    cache = torch.zeros(2, 2, 9, 64, dtype=torch.bfloat16)
    n = torch.zeros(2, dtype=torch.int64)
    with pytest.raises(ValueError):
        dn.window_attn_step(q, k, k, cache, cache, n, 4)
    for kc, vc, ln, sinks in ((cache[:1], cache, n, 1), (cache, cache.float(), n, 1), (cache, cache, n[:1], 1), (cache, cache, n.int(), 1),
                              (cache, cache, None, 1), (cache, cache, n, 9), (cache[0], cache[0], n, 1)):
        with pytest.raises(ValueError):
            dn.window_attn_step(one[0], one[1], one[1], kc, vc, ln, 4, sinks)
        if ln is not None:
            with pytest.raises(ValueError):
                dn.window_cache_fill(k, k, kc, vc, ln, sinks)
    x = torch.zeros(3, 8)
    for bad in (x.double(), x[:2], None):
        with pytest.raises(ValueError):
            dn.block_norm_fwd(x, bad)
    with pytest.raises(ValueError):
        dn.block_norm_fwd(x, x, scale=torch.zeros(3))
    with pytest.raises(ValueError):
        dn.block_norm_bwd(x, x)


@pytest.mark.parametrize("N,T,Nq", [(1, 2**32 + 3, 1), (2**32 + 2, 1, 1), (1, 1, 2**32 + 8)])
def test_sizes_above_an_int_are_refused(monkeypatch, N, T, Nq):
    """Cut to 32 bits these would be other sizes."""
    monkeypatch.setattr(dn, "_device_of", lambda x, torch: x.device)
    q = torch.zeros(1, dtype=torch.bfloat16).expand(N, T, Nq, 64)
    k = torch.zeros(1, dtype=torch.bfloat16).expand(N, T, 1, 64)
    with pytest.raises(dn.DnError) as e:
        dn.window_attn_fwd(q, k, k, 4)
    assert e.value.status == NO
    with pytest.raises(dn.DnError):
        dn.window_attn_bwd(q, k, k, q, q, 4, do=q)
    if T == 1:
        with pytest.raises(dn.DnError):
            dn.window_attn_step(q, k, k, k, k, k, 4)
    if Nq == 1:
        with pytest.raises(dn.DnError):
            dn.window_cache_fill(q, q, q, q)
    with pytest.raises(dn.DnError):
        dn.block_norm_fwd(torch.zeros(1).expand(2, 2**32 + 1), torch.zeros(1).expand(2, 2**32 + 1))
