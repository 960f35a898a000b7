"""The operators around the recurrence on the paths that small calls do not take: sequences cut into
chunks at every N, chunks of 64 tokens in the gradient, several channel tiles a block, blocks that walk
many rows or tiles, operands in place.  Every output against 64 bits; which path a call takes is read
from its workspace's size."""
import random

import pytest
import torch

import layer_bounds as bounds
import layer_reference as ref
from conftest import cuda_ok
from test_layer_ops import (DEV, DTYPES, NAMES, conv_inputs, norm_check, norm_inputs, ok, same, scan_args,
                            scan_inputs)

on_gpu = pytest.mark.skipif(not cuda_ok(), reason="needs a CUDA GPU")


# ---- the bounds themselves (no GPU) --------------------------------------------------------


@pytest.mark.parametrize("lengths,softplus,gate,N,G", [([0, 1, 2, 33, 40, 0, 17], True, True, 16, 2),
                                                       ([40, 50], False, False, 32, 1)])
def test_bounded_scan_is_the_scan(monkeypatch, lengths, softplus, gate, N, G):
    """The two walks give what differentiation of the definition gives; plain fp32 arithmetic stays within
    the bounds, an input of 11 bits does not."""
    monkeypatch.setattr("test_layer_ops.DEV", "cpu")
    t, grads = scan_inputs(torch.float32, D=6 * G, G=G, N=N, lengths=lengths, gate=gate, seed=3)
    if not softplus:
        t["dt"], t["dt_bias"] = t["dt"].abs() * 0.3, None
    want = bounds.scan(ref.in_64_bits(t), ref.in_64_bits(grads), lengths, softplus, 16, 16)
    leaves = ref.in_64_bits(t, grad=True)
    y, ht = ref.scan(leaves, lengths, softplus)
    by_diff = ref.gradients([y, ht], [grads["dy"], grads["dht"]], leaves)
    for name, v in [("y", y), ("ht", ht)] + [("d" + k, v) for k, v in by_diff.items()]:
        torch.testing.assert_close(want[name][0], v.detach(), rtol=1e-10, atol=1e-10)
    y32, ht32 = ref.scan(t, lengths, softplus)
    bounds.within(y32, want["y"], "y")
    bounds.within(ht32, want["ht"], "ht")
    with pytest.raises(AssertionError, match="times the bound"):
        bounds.within(ref.scan(dict(t, B=t["B"].half().float()), lengths, softplus)[0], want["y"], "y")


# ---- selective scan ------------------------------------------------------------------------


def up4(n):
    return (n + 3) // 4 * 4


def fwd_chunk(lib, n, B, T, D, G, N, code):
    """Tokens of a chunk, from the slots that the workspace holds; 0 where sequences are whole."""
    size = lib.load().dn_selective_scan_fwd_workspace_bytes(n, B, T, D, G, N, code)
    if size == 0:
        return 0
    slots = size // (4 * D * (N + 1))
    return max(c for c in range(16, B * T + 16, 16) if B * T // c + n == slots)


def bwd_chunk(lib, n, B, T, D, G, N, code):
    """(tokens of a chunk, parts that a group's channels are split into)."""
    size = lib.load().dn_selective_scan_bwd_workspace_bytes(n, B, T, D, G, N, code)
    found = []
    for chunk in (16, 32, 48, 64):
        slots = B * T // chunk + n
        rest = size // 4 - (2 * slots * D * N + up4(slots * D) + up4(2 * slots * D))
        row = B * T * G * 2 * N
        if rest > 0 and rest % row == 0 and rest // row <= D:
            found.append((chunk, rest // row))
    assert len(found) == 1, found
    return found[0]


def path_check(lib, t, grads, lengths, label, softplus=True, cut=None, chunk=None, shared=None):
    """All outputs within their bounds, and the path taken: cut (forward in chunks), chunk (tokens of the
    gradient's), shared (whether a block takes several channel tiles)."""
    B, T, D = t["x"].shape
    G, N = t["B"].shape[2:]
    n = B if lengths is None else len(lengths)
    sizes = (n, B, T, D, G, N, lib.dtype_code(t["x"].dtype))
    fc, (bc, parts) = fwd_chunk(lib, *sizes), bwd_chunk(lib, *sizes)
    tiles = -(-(D // G) // (1024 // N))  # a block of 128 threads holds 4 states of two channels each
    assert (cut is None or bool(fc) == cut) and (chunk is None or bc == chunk), (label, fc, bc)
    assert shared is None or (parts < tiles) == shared, (label, parts, tiles)
    cu = None if lengths is None else ref.offsets(lengths, DEV)
    want = bounds.scan(ref.in_64_bits(t), ref.in_64_bits(grads), lengths, softplus, max(fc, bc), B * T // bc + n)
    used = T if lengths is None else sum(lengths)
    y, ht = lib.selective_scan_fwd(*scan_args(t), cu, dt_softplus=softplus)
    ok(lib)
    bounds.within(y[:, :used], [v[:, :used] for v in want["y"]], label + " y")
    bounds.within(ht, want["ht"], label + " ht")
    out = lib.selective_scan_bwd(*scan_args(t), cu, dt_softplus=softplus, dy=grads["dy"], dht=grads["dht"])
    ok(lib)
    for name in NAMES:
        if t[name] is None:
            continue
        got, w = out["d" + name], want["d" + name]
        if name in ("x", "dt", "B", "C", "z"):
            got, w = got[:, :used], [v[:, :used] for v in w]
        bounds.within(got, w, label + " d" + name)


MIXED = [0, 1, 2, 64, 65, 0, 300, 17, 200, 0, 33]


@pytest.mark.gpu
@on_gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("N", [16, 32, 64, 128])
@pytest.mark.parametrize("D,G,gate", [(70, 1, True), (66, 2, False)])
def test_scan_packed_in_chunks(lib, dtype, N, D, G, gate):
    """Empty, short and long sequences in one call, the long ones cut, at every N."""
    t, grads = scan_inputs(dtype, D=D, G=G, N=N, lengths=MIXED, gate=gate, seed=N + G, pad=3)
    path_check(lib, t, grads, MIXED, "N=%d" % N, cut=True)


@pytest.mark.gpu
@on_gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("N", [16, 32, 64, 128])
def test_scan_rows_in_chunks(lib, dtype, N):
    """Rows of one length, cut, no state before them, delta without softplus."""
    t, grads = scan_inputs(dtype, B=3, T=157, D=45, N=N, h0=False, gate=N < 64, extras=False, seed=N)
    t["dt"] = t["dt"].abs() * 0.3
    path_check(lib, t, grads, None, "N=%d" % N, softplus=False, cut=True)


@pytest.mark.gpu
@on_gpu
@pytest.mark.parametrize("B,T,D,N,tokens", [(8, 100, 512, 128, 32), (16, 150, 512, 64, 48)])
def test_scan_in_longer_chunks(lib, B, T, D, N, tokens):
    """Chunks that fill the GPU once, longer than the shortest."""
    t, grads = scan_inputs(torch.float32, B=B, T=T, D=D, N=N, seed=N)
    assert fwd_chunk(lib, B, B, T, D, 1, N, lib.DN_F32) == tokens
    path_check(lib, t, grads, None, "N=%d" % N)


@pytest.mark.gpu
@on_gpu
@pytest.mark.parametrize("N,D,G,gate,lengths", [
    (16, 1290, 2, True, MIXED), (32, 450, 2, True, MIXED * 2), (64, 258, 2, False, MIXED * 2),
    (128, 258, 2, True, MIXED), (128, 201, 1, False, MIXED)])
def test_scan_gradient_chunks_of_64(lib, N, D, G, gate, lengths):
    """The gradient's longest chunks, channels of a group beyond a tile and odd, gated and not."""
    for dtype in DTYPES:
        t, grads = scan_inputs(dtype, D=D, G=G, N=N, lengths=lengths, gate=gate, seed=N + D)
        path_check(lib, t, grads, lengths, "N=%d" % N, chunk=64)


@pytest.mark.gpu
@on_gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("N,D,gate", [(128, 137, True), (16, 1150, False)])
def test_scan_gradient_several_tiles_a_block(lib, dtype, N, D, gate):
    """So many sequences that a block takes several tiles of a group's channels, one after the other."""
    rng = random.Random(5)
    lengths = [rng.randint(0, 5) for _ in range(300)] + [150]
    t, grads = scan_inputs(dtype, D=D, N=N, lengths=lengths, gate=gate, seed=N)
    path_check(lib, t, grads, lengths, "N=%d" % N, shared=True)


@pytest.mark.gpu
@on_gpu
def test_scan_small_calls_are_as_exact(lib):
    """Whole sequences and single tokens within the same bounds."""
    for dtype in DTYPES:
        t, grads = scan_inputs(dtype, B=5, T=21, D=36, G=2, N=32, seed=1)
        path_check(lib, t, grads, None, "T=21", cut=False)
        t, grads = scan_inputs(dtype, B=65, T=1, D=36, G=2, N=128, seed=2)
        path_check(lib, t, grads, None, "T=1", cut=False)


@pytest.mark.gpu
@on_gpu
@pytest.mark.parametrize("T", [40, 200])
def test_scan_total_forgetting_and_no_step(lib, T):
    """A = -inf forgets everything at a token with a step; a token without one keeps the state."""
    t, _ = scan_inputs(torch.float32, B=1, T=T, D=8, gate=False, extras=False, h0=True, seed=13)
    t["dt"] = t["dt"].abs() + 0.1
    still = torch.zeros(T, dtype=torch.bool)
    still[5:9] = still[T - 12:] = still[T // 2] = True
    t["dt"][:, still] = 0
    t["A"][:] = float("-inf")
    y, ht = lib.selective_scan_fwd(*scan_args(t), dt_softplus=False)
    ok(lib)
    rows = ref.in_64_bits(t)
    h, want = rows["h0"][0], []
    for s in range(T):
        if not still[s]:
            h = (rows["dt"][0, s] * rows["x"][0, s])[:, None] * rows["B"][0, s]
        want.append((h * rows["C"][0, s]).sum(-1))
    ref.close(y[0], torch.stack(want), 64, "y")
    ref.close(ht[0], h, 64, "ht")
    t["dt"][:] = 0  # no step anywhere
    _, ht = lib.selective_scan_fwd(*scan_args(t), dt_softplus=False)
    assert torch.equal(ht, t["h0"])


# ---- convolution -----------------------------------------------------------------------------


def conv64(t, lengths, silu):
    """The convolution over whole sequences at once."""
    x, w = t["x"], t["weight"]
    W = w.shape[1]
    ys, hts = [], []
    for n, (b, lo, hi) in enumerate(ref.spans(x.shape[0], x.shape[1], lengths)):
        row = torch.cat([t["h0"][n], x[b, lo:hi]])
        u = sum(row[j:j + hi - lo] * w[:, j] for j in range(W)) + t["bias"]
        ys.append(u * torch.sigmoid(u) if silu else u)
        hts.append(row[hi - lo:])
    return torch.cat(ys), torch.stack(hts)


@pytest.mark.gpu
@on_gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("D,W,lengths", [(6144, 4, [1500, 0, 3, 1203, 294]), (4097, 3, None), (6150, 2, [2, 2900, 33])])
def test_conv_gradient_many_tiles_a_warp(lib, dtype, D, W, lengths):
    """Each warp walks several tiles: the feed starts again at each, the sums over tokens go on."""
    t, grads = conv_inputs(dtype, B=2, T=2011, D=D, W=W, lengths=lengths, seed=D)
    n, (B, T, _) = 2 if lengths is None else len(lengths), t["x"].shape
    rows = lib.load().dn_causal_conv_bwd_workspace_bytes(n, B, T, D, W, lib.dtype_code(dtype)) // (4 * D * (W + 1))
    cu = None if lengths is None else ref.offsets(lengths, DEV)
    tiles = sum(-(-m // 64) for m in (lengths or [T] * B))  # at least
    assert tiles > 4 * rows, (tiles, rows)  # four warps a row
    leaves = ref.in_64_bits(t, grad=True)
    y64, ht64 = conv64(leaves, lengths, True)
    want = ref.gradients([y64, ht64], [grads["dy"].reshape(-1, D), grads["dht"]], leaves)
    y, ht = lib.causal_conv_fwd(t["x"], t["weight"], t["bias"], t["h0"], cu)
    out = lib.causal_conv_bwd(t["x"], t["weight"], t["bias"], t["h0"], cu, dy=grads["dy"], dht=grads["dht"])
    ok(lib)
    terms = float(t["x"].abs().max()) * float(t["weight"].abs().sum(1).max()) + 1
    ref.close(y.reshape(-1, D), y64, 4 * W + 32, "y", scale=terms)
    assert torch.equal(ht.double().cpu(), ht64.detach())
    for name in ("x", "h0"):
        ref.close(out["d" + name], want[name], 4 * W + 32, "d" + name, scale=max(terms, float(want[name].abs().max())))
    # A sum over tokens: T / (4 rows) of a thread's own, then the warps and the rows; each term is du x with
    # du within 4 W + 32 roundings of at most |dy| (1 + |u|).  Terms of either sign: their absolute sum.
    steps = B * T / (4 * rows) + 4 + rows + 4 * W + 32
    top = float((grads["dy"].double().abs().sum((0, 1)) * (1 + terms)).max())
    ref.close(out["dbias"], want["bias"], steps, "dbias", scale=top)
    ref.close(out["dweight"], want["weight"], steps, "dweight", scale=top * float(t["x"].abs().max()))
    # and, far below those bounds' size, no term lost or counted twice: one token's is about 1
    for name in ("weight", "bias"):
        assert (out["d" + name].double().cpu() - want[name]).abs().max() < 0.01, name


# ---- layer norm --------------------------------------------------------------------------------


@pytest.mark.gpu
@on_gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,D,rms,gate", [(rows, D, both, both) for both in (True, False) for rows, D in (
    (6203, 1024), (3203, 2048), (1603, 4096), (603, 8192), (1003, 1031), (1003, 2500), (703, 4095))] + [
        (3203, 2048, True, False), (3203, 2048, False, True), (1003, 1031, True, False), (1003, 1031, False, True)])
def test_norm_many_rows_a_block(lib, dtype, rows, D, rms, gate):
    """Rows of many threads, several a block: the copies ahead come round, sums through shared memory follow
    one another, and the gradients of weight and bias add up."""
    t, dy = norm_inputs(dtype, rows, D, gate=gate, seed=D)
    blocks = lib.load().dn_layer_norm_bwd_workspace_bytes(rows, D, lib.dtype_code(dtype)) // (8 * D)
    assert rows > 2 * blocks, (rows, blocks)
    norm_check(lib, t, dy, rms, "norm %d x %d" % (rows, D))


# ---- operands in place -------------------------------------------------------------------------


@pytest.mark.gpu
@on_gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,D", [(700, 128), (19, 33), (1300, 1024), (700, 1031)])
def test_norm_in_place_forms(lib, dtype, rows, D):
    """y over x or z; d_x over d_y or x, d_z over z: the same bits as in tensors of their own."""
    t, dy = norm_inputs(dtype, rows, D, gate=True, seed=D)
    x, w, b, z = (t[k] for k in ("x", "weight", "bias", "z"))
    want = lib.layer_norm_fwd(x, w, b, z)
    for name in ("x", "z"):
        c = dict(x=x.clone(), z=z.clone())
        assert torch.equal(lib.layer_norm_fwd(c["x"], w, b, c["z"], y=c[name]), want)
    grads = lib.layer_norm_bwd(x, w, b, z, dy=dy)
    raw, code = lib.load(), lib.dtype_code(dtype)
    n = raw.dn_layer_norm_bwd_workspace_bytes(rows, D, code)
    stream = torch.cuda.current_stream().cuda_stream
    for over in ("dy", "x"):
        c = dict(x=x.clone(), z=z.clone(), dy=dy.clone())
        dw, db, space = torch.empty_like(w), torch.empty_like(b), torch.empty(n, dtype=torch.uint8, device=DEV)
        assert raw.dn_layer_norm_bwd(c["x"].data_ptr(), w.data_ptr(), b.data_ptr(), c["z"].data_ptr(), rows, D, code,
                                     1e-5, 0, c["dy"].data_ptr(), c[over].data_ptr(), dw.data_ptr(), db.data_ptr(),
                                     c["z"].data_ptr(), space.data_ptr(), n, stream) == lib.DN_OK
        assert same([c[over], c["z"], dw, db], [grads[k] for k in ("dx", "dz", "dweight", "dbias")])


@pytest.mark.gpu
@on_gpu
@pytest.mark.parametrize("lengths", [[40], MIXED])
def test_scan_state_gradient_in_place(lib, lengths):
    """d_h0 over d_ht."""
    D, N = 20, 16
    t, grads = scan_inputs(torch.float32, D=D, N=N, lengths=lengths, seed=4)
    cu, n, T = ref.offsets(lengths, DEV), len(lengths), sum(lengths)
    want = lib.selective_scan_bwd(*scan_args(t), cu, dy=grads["dy"], dht=grads["dht"])
    raw, code = lib.load(), lib.DN_F32
    size = raw.dn_selective_scan_bwd_workspace_bytes(n, 1, T, D, 1, N, code)
    space = torch.empty(size, dtype=torch.uint8, device=DEV)
    out = {k: torch.empty_like(t[k]) for k in NAMES}
    state = grads["dht"].clone()
    p = {k: v.data_ptr() for k, v in out.items()}
    assert raw.dn_selective_scan_bwd(
        *[t[k].data_ptr() for k in NAMES], cu.data_ptr(), n, 1, T, D, 1, N, code, 1, grads["dy"].data_ptr(),
        state.data_ptr(), p["x"], p["dt"], p["A"], p["B"], p["C"], p["D"], p["z"], p["dt_bias"], state.data_ptr(),
        space.data_ptr(), size, torch.cuda.current_stream().cuda_stream) == lib.DN_OK
    assert torch.equal(state, want["dh0"])
    assert same([out[k] for k in NAMES[:-1]], [want["d" + k] for k in NAMES[:-1]])
