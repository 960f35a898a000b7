"""The operators around the recurrence refuse bad arguments on the host, before
anything reaches the device (no GPU needed)."""
import pytest
import torch

import chunkwise_gated_delta_chunk_gb300 as dn

A = 1 << 20  # fake, 16-byte aligned device address: rejected before any use
BAD, NO = dn.DN_ERR_INVALID_ARG, dn.DN_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def clib():
    from chunkwise_gated_delta_chunk_gb300 import _build
    _build.build()
    return dn.load()


def call(f, order, defaults, over):
    args = dict(defaults)
    for k in over:
        assert k in args, k
    args.update(over)
    return f(*[args[k] for k in order.split()])


SEQ = dict(cu=None, n=2, B=2, T=8)
CONV = dict(SEQ, x=A, w=A, bias=None, h0=None, D=8, W=4, dtype=dn.DN_BF16, flags=1, y=A, ht=None, s=None)
CONV_BWD = dict(CONV, dy=A, gt=dn.DN_BF16, dht=None, dx=A, dw=A, db=None, dh0=None, ws=A, wsb=1 << 30)


@pytest.mark.parametrize("over,code", [
    (dict(x=None), BAD), (dict(w=None), BAD), (dict(y=None), BAD), (dict(x=A + 2), BAD), (dict(ht=A + 8), BAD),
    (dict(n=3), BAD), (dict(cu=A), BAD), (dict(cu=A + 4, B=1), BAD), (dict(T=-1), BAD), (dict(D=0), BAD),
    (dict(W=0), BAD), (dict(dtype=2), BAD), (dict(flags=2), BAD), (dict(W=1), NO), (dict(W=5), NO),
    (dict(n=0, B=0), dn.DN_OK), (dict(n=0, B=1, cu=A), dn.DN_OK),
])
def test_conv_fwd(clib, over, code):
    assert call(clib.dn_causal_conv_fwd, "x w bias h0 cu n B T D W dtype flags y ht s", CONV, over) == code


@pytest.mark.parametrize("over,code", [
    (dict(dy=None), BAD), (dict(dx=None), BAD), (dict(dw=None), BAD), (dict(db=A + 4), BAD), (dict(ws=None), BAD),
    (dict(wsb=16), BAD), (dict(ws=A + 8), BAD), (dict(gt=3), BAD), (dict(dtype=dn.DN_F32), BAD),  # bf16 d_y of fp32 x
    (dict(flags=8), BAD), (dict(W=7), NO),
])
def test_conv_bwd(clib, over, code):
    order = "x w bias h0 cu n B T D W dtype flags dy gt dht dx dw db dh0 ws wsb s"
    assert call(clib.dn_causal_conv_bwd, order, CONV_BWD, over) == code


SCAN = dict(SEQ, x=A, dt=A, A=A, Bm=A, Cm=A, Ds=None, z=None, db=None, h0=None, D=8, G=2, N=16, dtype=dn.DN_BF16,
            flags=1, y=A, ht=None, ws=None, wsb=0, s=None)
SCAN_BWD = dict(SCAN, dy=A, dht=None, dx=A, ddt=A, dA=A, dBm=A, dCm=A, dDs=None, dz=None, ddb=None, dh0=None, ws=A,
                wsb=1 << 40)


@pytest.mark.parametrize("over,code", [
    (dict(x=None), BAD), (dict(dt=None), BAD), (dict(A=None), BAD), (dict(Cm=None), BAD), (dict(y=None), BAD),
    (dict(z=A + 4), BAD), (dict(G=3), BAD), (dict(G=0), BAD), (dict(N=0), BAD), (dict(flags=4), BAD),
    (dict(n=1), BAD), (dict(dtype=9), BAD), (dict(N=8), NO), (dict(N=24), NO), (dict(N=256), NO),
    (dict(T=4096), BAD),  # cut into chunks: needs its workspace
    (dict(T=4096, ws=A, wsb=64), BAD), (dict(T=4096, ws=A + 8, wsb=1 << 30), BAD), (dict(n=0, B=0), dn.DN_OK),
])
def test_scan_fwd(clib, over, code):
    order = "x dt A Bm Cm Ds z db h0 cu n B T D G N dtype flags y ht ws wsb s"
    assert call(clib.dn_selective_scan_fwd, order, SCAN, over) == code


@pytest.mark.parametrize("over,code", [
    (dict(dy=None), BAD), (dict(dx=None), BAD), (dict(dA=None), BAD), (dict(dCm=None), BAD), (dict(z=A), BAD),
    (dict(dz=A), BAD), (dict(ddb=A + 4), BAD), (dict(ws=None), BAD), (dict(wsb=64), BAD), (dict(N=20), NO),
])
def test_scan_bwd(clib, over, code):
    order = "x dt A Bm Cm Ds z db h0 cu n B T D G N dtype flags dy dht dx ddt dA dBm dCm dDs dz ddb dh0 ws wsb s"
    assert call(clib.dn_selective_scan_bwd, order, SCAN_BWD, over) == code


NORM = dict(x=A, w=None, b=None, z=None, rows=4, D=64, dtype=dn.DN_F32, eps=1e-5, flags=0, y=A, s=None)
NORM_BWD = dict(NORM, dy=A, dx=A, dw=A, db=None, dz=None, ws=A, wsb=1 << 30)


@pytest.mark.parametrize("over,code", [
    (dict(x=None), BAD), (dict(y=None), BAD), (dict(w=A + 4), BAD), (dict(rows=-1), BAD), (dict(D=0), BAD),
    (dict(eps=-1.0), BAD), (dict(eps=float("nan")), BAD), (dict(eps=float("inf")), BAD), (dict(flags=2), BAD),
    (dict(dtype=5), BAD), (dict(D=16385), NO), (dict(rows=0), dn.DN_OK),
])
def test_norm_fwd(clib, over, code):
    assert call(clib.dn_layer_norm_fwd, "x w b z rows D dtype eps flags y s", NORM, over) == code


@pytest.mark.parametrize("over,code", [
    (dict(dy=None), BAD), (dict(dx=None), BAD), (dict(z=A), BAD), (dict(dz=A), BAD), (dict(ws=None), BAD),
    (dict(wsb=64), BAD), (dict(D=20000), NO), (dict(rows=0, dw=None, ws=None), dn.DN_OK),
])
def test_norm_bwd(clib, over, code):
    order = "x w b z rows D dtype eps flags dy dx dw db dz ws wsb s"
    assert call(clib.dn_layer_norm_bwd, order, NORM_BWD, over) == code


def test_workspace_sizes(clib):
    """Zero for sizes that are refused and for single tokens; chunks of the scan grow with the tokens."""
    f, b = clib.dn_selective_scan_fwd_workspace_bytes, clib.dn_selective_scan_bwd_workspace_bytes
    assert f(64, 64, 1, 2048, 1, 16, dn.DN_BF16) == 0
    assert f(1, 1, 4096, 64, 1, 16, dn.DN_BF16) > 0
    assert f(1, 1, 4096, 64, 1, 20, dn.DN_BF16) == f(1, 1, 4096, 64, 3, 16, dn.DN_BF16) == 0
    states = (4096 // 64 + 1) * 64 * 16 * 4  # one fp32 state per chunk and sequence
    assert b(1, 1, 4096, 64, 1, 16, dn.DN_BF16) >= 2 * states
    assert b(1, 1, 4096, 64, 1, 16, 7) == 0
    assert clib.dn_causal_conv_bwd_workspace_bytes(2, 2, 64, 128, 4, dn.DN_BF16) >= 5 * 128 * 4
    assert clib.dn_causal_conv_bwd_workspace_bytes(2, 2, 64, 128, 9, dn.DN_BF16) == 0
    assert clib.dn_layer_norm_bwd_workspace_bytes(100, 64, dn.DN_F32) >= 2 * 64 * 4
    assert clib.dn_layer_norm_bwd_workspace_bytes(100, 16385, dn.DN_F32) == 0


def test_binding_refuses_host_tensors():
    """The Python functions refuse tensors that are not on a CUDA device."""
    x = torch.zeros(1, 4, 8)
    with pytest.raises(ValueError, match="CUDA"):
        dn.causal_conv_fwd(x, torch.zeros(8, 4))
    with pytest.raises(ValueError, match="CUDA"):
        dn.layer_norm_bwd(x, dy=x)
    with pytest.raises(ValueError, match="CUDA"):
        dn.selective_scan_fwd(x, x, torch.zeros(8, 16), torch.zeros(1, 4, 1, 16), torch.zeros(1, 4, 1, 16))
