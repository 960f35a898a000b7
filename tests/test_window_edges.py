"""GPU: attention over a window, its cache and the norms around a block at the edges of what their headers allow:
tensors that begin on 16 bytes and on no more; scores that rise steeply along the keys, and to the end of fp32."""
import pytest
import torch

import window_reference as wref
from conftest import cuda_ok
from test_block_norm import args
from test_block_norm import inputs as block_inputs
from test_window_attn import DEV, DTYPES, check, half_of, inputs, normal, ok, wide

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not cuda_ok(), reason="needs a CUDA GPU")]


# ---- tensors that begin on 16 bytes ------------------------------------------------------------


class Behind:
    """Tensors 16 bytes behind an aligned address, each with 16 bytes in front of it and behind it that hold 7."""

    def __init__(self):
        self.all = []

    def __call__(self, x, keep=True):
        if x is None:
            return None
        pad = 16 // x.element_size()
        space = torch.full((x.numel() + 2 * pad,), 7, dtype=x.dtype, device=x.device)
        view = space[pad:pad + x.numel()].view(x.shape)
        if keep:
            view.copy_(x)
        assert view.data_ptr() % 32 == 16
        self.all.append((space, pad, x.numel()))
        return view

    def untouched(self):
        return all((s[:p] == 7).all() and (s[p + n:] == 7).all() for s, p, n in self.all)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Nq,Nk,T,window,sinks", [(4, 2, 150, 70, 4), (3, 1, 520, 100, 40), (2, 2, 1, 1, 0)])
def test_attention_on_16_bytes(lib, dtype, d, Nq, Nk, T, window, sinks):
    """The same bits as with tensors on 256 bytes, and nothing beside the tensors is written."""
    t = inputs(dtype, B=2, T=T, Nq=Nq, Nk=Nk, d=d, seed=d + T)
    o, lse = lib.window_attn_fwd(t["q"], t["k"], t["v"], window, sinks)
    want = lib.window_attn_bwd(t["q"], t["k"], t["v"], o, lse, window, sinks, do=t["do"])
    ok(lib)
    off = Behind()
    u = {n: off(x) for n, x in t.items()}
    o2, lse2 = off(o, False), off(lse, False)
    lib.window_attn_fwd(u["q"], u["k"], u["v"], window, sinks, o=o2, lse=lse2)
    ok(lib)
    assert torch.equal(o2, o) and torch.equal(lse2, lse)
    got = {n: off(x, False) for n, x in want.items()}
    code = lib.dtype_code(dtype)
    need = lib.load().dn_window_attn_bwd_workspace_bytes(0, 2, 2, T, Nq, Nk, d, window, sinks, code)
    space = off(torch.empty(need, dtype=torch.uint8, device=DEV), False)
    at = lambda x: x.data_ptr()
    assert lib.load().dn_window_attn_bwd(at(u["q"]), at(u["k"]), at(u["v"]), at(o2), at(lse2), None, 2, 2, T, Nq, Nk, d, window,
                                         sinks, code, 0.0, at(u["do"]), at(got["dq"]), at(got["dk"]), at(got["dv"]), at(space),
                                         need, torch.cuda.current_stream().cuda_stream) == lib.DN_OK
    ok(lib)
    assert all(torch.equal(got[n], want[n]) for n in want)
    assert off.untouched()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("d", [64, 128])
def test_cache_on_16_bytes(lib, dtype, d):
    N, Nq, Nk, window, sinks, ring = 2, 6, 2, 50, 3, 60
    t = inputs(dtype, B=N, T=41, Nq=Nq, Nk=Nk, d=d, seed=d)
    new = {n: t[n][:, :1].contiguous() for n in "qkv"}
    g = torch.Generator().manual_seed(1)
    cache = [normal(g, N, Nk, sinks + ring, d, dtype=dtype) for _ in range(2)]
    had = torch.tensor([5, 777], device=DEV)

    def calls(place, o):
        k, v, kc, vc, ln = (place(x) for x in (t["k"], t["v"], *cache, had))
        lib.window_cache_fill(k, v, kc, vc, ln, sinks)
        lib.window_attn_step(*(place(new[n]) for n in "qkv"), kc, vc, place(ln + 41), window, sinks, o=o)
        return kc, vc

    o = torch.empty_like(new["q"])
    want = calls(lambda x: x.clone(), o)
    off = Behind()
    o2 = off(o, False)
    got = calls(off, o2)
    ok(lib)
    assert torch.equal(o2, o) and all(torch.equal(a, b) for a, b in zip(got, want))
    assert off.untouched()


@pytest.mark.parametrize("types", [(torch.bfloat16, torch.float32), (torch.bfloat16, torch.bfloat16), (torch.float32, torch.float32)])
@pytest.mark.parametrize("D", [1024, 520, 33])
def test_block_on_16_bytes(lib, types, D):
    rows = 37
    t, g = block_inputs(types, rows, D, seed=D)
    y, h = lib.block_norm_fwd(*args(t))
    want = lib.block_norm_bwd(*args(t), **g)
    off = Behind()
    u, ug = ({n: off(x) for n, x in m.items()} for m in (t, g))
    y2, h2 = off(y, False), off(h, False)
    lib.block_norm_fwd(*args(u), y=y2, residual_out=h2)
    ok(lib)
    assert torch.equal(y2, y) and torch.equal(h2, h)
    got = {n: off(x, False) for n, x in want.items()}
    code = [lib.dtype_code(x) for x in types]
    need = lib.load().dn_block_norm_bwd_workspace_bytes(rows, D, *code)
    space = off(torch.empty(need, dtype=torch.uint8, device=DEV), False)
    at = lambda x: None if x is None else x.data_ptr()
    assert lib.load().dn_block_norm_bwd(*(at(x) for x in args(u)), rows, D, *code, 1e-5, lib.DN_NORM_POST, at(ug["dy"]),
                                        at(ug["dresidual_out"]), *(at(x) for x in got.values()), at(space), need,
                                        torch.cuda.current_stream().cuda_stream) == lib.DN_OK
    ok(lib)
    assert all(want[n] is None or torch.equal(got[n], want[n]) for n in want)
    assert off.untouched()


# ---- references of the weights that move ---------------------------------------------------------


def steep(Nq, Nk, d, T, seed):
    """bf16 operands whose scores (scale 1) rise by 13 from one half of a key tile to the next, so that the reference
    that a row's weights are relative to moves in every tile, for one half's sake or the other's."""
    t = inputs(torch.bfloat16, B=1, T=T, Nq=Nq, Nk=Nk, d=d, seed=seed)
    t["q"] *= 0.125
    t["q"][..., 0] = 1
    t["k"][..., 0] = 13 * (torch.arange(T, device=DEV)[None, :, None] // 64)  # whole numbers that bf16 holds
    return t


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Nq,Nk,window,sinks", [(4, 2, 5000, 0), (3, 1, 700, 40)])
def test_references_that_move_in_every_tile(lib, d, Nq, Nk, window, sinks):
    """Both threads of a row move on in the same tile: results within their bounds, and the same bits every time."""
    t = steep(Nq, Nk, d, 1250, d)
    o, lse, out = check(lib, t, window, sinks, scale=1.0, label="steep")
    for _ in range(50):
        again = lib.window_attn_fwd(t["q"], t["k"], t["v"], window, sinks, scale=1.0)
        assert torch.equal(again[0], o) and torch.equal(again[1], lse)
    ok(lib)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Nq,Nk", [(2, 1), (3, 1)])
@pytest.mark.parametrize("rise,at", [(80, [300]), (85.5, [300]), (86, [300]), (86.5, [300]), (87, [300]), (87.5, [300]), (88, [300]),
                                     (88.5, [300]), (89, [300]), (100, [300]), (86.5, [320, 321, 322, 323]), (87, [300, 330]),
                                     (86.5, [300, 331, 400, 470, 590]), (85.5, list(range(300, 316)))])
def test_scores_that_rise_to_the_end_of_fp32(lib, d, Nq, Nk, rise, at):
    """Keys whose scores lie `rise` above those of all others (e^87.3 is 2^126, e^88.7 2^128): in the last tile that a
    row sees, and in one before it.  Values of 1 at most, so that no product passes fp32."""
    t = inputs(torch.bfloat16, B=1, T=600, Nq=Nq, Nk=Nk, d=d, seed=3)
    t["q"].zero_()
    t["q"][..., 0] = 8
    t["k"][..., 0] = 0
    t["k"][:, at, :, 0] = rise / 8  # bf16 holds it
    t["v"].clamp_(-1, 1)
    assert float(t["k"][0, at[0], 0, 0]) * 8 == rise
    check(lib, t, 5000, 0, scale=1.0, label="rise %g" % rise)
    check(lib, t, 290, 4, scale=1.0, label="rise %g, window" % rise)


# ---- rows that do see what is not finite ------------------------------------------------------------


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_rows_that_see_a_bad_value(lib, dtype, d, bad):
    """Every row that sees it has it in its column, and in all others what it has without it; lse and dv, which
    do not depend on values, are as without it everywhere; dq, through D, is NaN."""
    T, window, sinks, at = 600, 150, 4, 290
    t = inputs(dtype, B=1, T=T, Nq=2, Nk=1, d=d, seed=6)
    w = wide(t)
    want = wref.attention(w["q"], w["k"], w["v"], window, sinks, None, None, w["do"], half_of(dtype))
    seeing = torch.tensor([at <= i < at + window for i in range(T)])
    others = torch.arange(d) != 5
    t["v"][0, at, 0, 5] = bad
    o, lse = lib.window_attn_fwd(t["q"], t["k"], t["v"], window, sinks)
    out = lib.window_attn_bwd(t["q"], t["k"], t["v"], o, lse, window, sinks, do=t["do"])
    ok(lib)
    column = o[0, seeing][:, :, 5].float()
    assert torch.isnan(column).all() if bad != bad else (column == bad).all()
    wref.close(o[..., others], (want["o"][0][..., others], want["o"][1][..., others]), "other columns")
    wref.close(o[:, ~seeing], (want["o"][0][:, ~seeing], want["o"][1][:, ~seeing]), "other rows")
    wref.close(lse, want["lse"], "lse")
    wref.close(out["dv"], want["dv"], "dv")
    assert torch.isnan(out["dq"][0, seeing]).all()
    wref.close(out["dq"][:, ~seeing], (want["dq"][0][:, ~seeing], want["dq"][1][:, ~seeing]), "dq")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_rows_that_see_a_bad_key(lib, dtype, d, bad):
    """A key's infinity times a query's sign: a score of -infinity is a weight of 0, one of +infinity or NaN a row
    of NaN."""
    T, window, sinks, at = 600, 150, 4, 290
    t = inputs(dtype, B=1, T=T, Nq=2, Nk=1, d=d, seed=6)
    t["q"][..., 5] = t["q"][..., 5].sign() + (t["q"][..., 5] == 0)
    # for the reference: a score 40 below its others' sizes on the rows whose weight is 0 (e^-40 of theirs)
    finite = 0.0 if bad != bad else 40.0 * d ** 0.5 * (1 if bad > 0 else -1)
    w = wide(t)
    w["k"][0, at, 0, 5] = finite
    want = wref.attention(w["q"], w["k"], w["v"], window, sinks, half=half_of(dtype))
    t["k"][0, at, 0, 5] = bad
    o, lse = lib.window_attn_fwd(t["q"], t["k"], t["v"], window, sinks)
    ok(lib)
    seeing = torch.tensor([at <= i < at + window for i in range(T)])[:, None]
    gone = seeing & ~(t["q"][0, :, :, 5].cpu() * bad < 0)  # NaN: all that see it
    assert gone.any() and (bad != bad or (seeing & ~gone).any())
    assert torch.isnan(o[0].cpu()[gone]).all() and torch.isnan(lse[0].cpu()[gone]).all()
    for n, x in (("o", o), ("lse", lse)):
        wref.close(x[0].cpu()[~gone], (want[n][0][0][~gone], want[n][1][0][~gone]), n)
