"""GPU: attention over a window and the norms around a block where calls go wrong or take other paths:
many tiles a block, the sinks' queries in several runs, streams and graphs, workspaces that calls share,
tensors whose offsets pass 32 bits; and all of them together, as a model's layers use them."""
import pytest
import torch

import layer_reference as ref
import window_reference as wref
import workloads
from conftest import cuda_ok
from test_block_norm import NAMES, args, block64
from test_block_norm import inputs as block_inputs
from test_layer_edges import stream_of
from test_layer_ops import same
from test_window_attn import DEV, DTYPES, check, half_of, inputs, normal, ok, wide

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not cuda_ok(), reason="needs a CUDA GPU")]


# ---- paths of larger calls ------------------------------------------------------------


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("Nq,Nk", [(16, 2), (15, 5)])
def test_many_tiles_a_block(lib, dtype, Nq, Nk):
    """More tiles than blocks, several times over: pairs of heads, and pairs of tiles."""
    check(lib, inputs(dtype, B=8, T=1100, Nq=Nq, Nk=Nk, seed=Nq), 130, 7, label="many")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("lengths", [None, [2300, 50, 0, 1500]])
@pytest.mark.parametrize("Nq,Nk,sinks", [(4, 2, 4), (3, 1, 100)])
def test_sinks_seen_by_many_tiles(lib, dtype, lengths, Nq, Nk, sinks):
    """The queries that see the sinks alone come in several runs, whose sums are joined."""
    check(lib, inputs(dtype, B=1, T=3400, Nq=Nq, Nk=Nk, lengths=lengths, pad=9 if lengths else 0, seed=Nq), 100, sinks,
          lengths, label="runs", pad=9 if lengths else 0)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("Nq,Nk", [(3, 1), (2, 1)])
def test_many_short_sequences(lib, dtype, Nq, Nk):
    """Tiles that are mostly empty: a pair of tiles of tokens has one alone, many times in a row."""
    lengths = [(7 * i) % 6 for i in range(1000)] + [200]
    check(lib, inputs(dtype, lengths=lengths, Nq=Nq, Nk=Nk, seed=1), 4, 1, lengths, label="short")


@pytest.mark.parametrize("dtype", DTYPES)
def test_long_window(lib, dtype):
    """A window of more tiles than a run of the sinks' queries may have."""
    check(lib, inputs(dtype, B=1, T=5700, Nq=1, Nk=1, seed=2), 4200, 4, label="long window")


@pytest.mark.parametrize("dtype", DTYPES)
def test_bad_sinks(lib, dtype):
    """A bad sink reaches every row of its heads, and none of the others."""
    t = inputs(dtype, B=1, T=1500, Nq=4, Nk=2, seed=3)
    w = wide(t)
    want = wref.attention(w["q"][:, :, 2:], w["k"][:, :, 1:], w["v"][:, :, 1:], 100, 4, None, None, w["do"][:, :, 2:], half_of(dtype))
    t["v"][0, 2, 0, 7] = float("nan")
    o, lse = lib.window_attn_fwd(t["q"], t["k"], t["v"], 100, 4)
    out = lib.window_attn_bwd(t["q"], t["k"], t["v"], o, lse, 100, 4, do=t["do"])
    ok(lib)
    assert torch.isnan(o[0, 2:, :2, 7]).all() and torch.isfinite(o[0, :2]).all()
    assert torch.isnan(out["dq"][0, 2:, :2]).all() and torch.isfinite(out["dv"]).all()
    wref.close(o[:, :, 2:], want["o"], "o")
    for n, x in (("dq", out["dq"][:, :, 2:]), ("dk", out["dk"][:, :, 1:]), ("dv", out["dv"][:, :, 1:])):
        wref.close(x, want[n], n)


@pytest.mark.parametrize("D,biases", [(1024, True), (1024, False), (2048, False), (2056, False), (4096, False), (4096, True), (33, True),
                                      (2049, False), (8192, False)])
@pytest.mark.parametrize("rows", [1801, 4000])
def test_block_many_rows(lib, D, biases, rows):
    """Every block takes several rows, odd numbers of them too, one and two at a time: the gradients of its rows as those
    of calls of a few rows, and its sums over the rows within their bound."""
    types = (torch.bfloat16, torch.float32)
    t, g = block_inputs(types, rows, D, biases=biases, seed=D)
    out = lib.block_norm_bwd(*args(t), **g)
    y, h = lib.block_norm_fwd(*args(t))
    total = {k: 0 for k in NAMES[3:]}
    for lo in range(0, rows, 500):
        part = {k: (v[lo:lo + 500].clone() if k in ("x", "residual", "z") else v) for k, v in t.items()}
        pg = {k: v[lo:lo + 500].clone() for k, v in g.items()}
        o2 = lib.block_norm_bwd(*args(part), **pg)
        y2, h2 = lib.block_norm_fwd(*args(part))
        assert torch.equal(y[lo:lo + 500], y2) and torch.equal(h[lo:lo + 500], h2)
        for n in ("dx", "dz", "dresidual"):
            assert torch.equal(out[n][lo:lo + 500], o2[n]), n
        for n in total:
            if t[n] is not None:
                total[n] = total[n] + o2["d" + n].double()
    for n, want in total.items():
        if t[n] is None:
            continue
        # each side's sum of `rows` terms is off by at most rows 2^-24 of the terms' sizes; these add up at random
        # to sqrt(rows) of them, and the largest is some 6 deviations
        assert (out["d" + n].double() - want).abs().max() <= 2 * rows * 2.0 ** -24 * 6 * max(1.0, float(want.abs().max())), n


def test_lengths_at_the_end_of_64_bits(lib):
    """Positions that 64 bits hold are kept by the ring; a length that they would pass is reported, and nothing is
    written for its sequence."""
    top = 2 ** 63 - 1
    t = inputs(torch.float32, B=2, T=3, Nq=1, Nk=1, seed=1)
    kc, vc = (torch.full((2, 1, 9, 64), 7.0, device=DEV) for _ in range(2))
    lib.dn_check()
    lib.window_cache_fill(t["k"], t["v"], kc, vc, torch.tensor([top - 2, top - 3], device=DEV), 2)
    assert lib.dn_check() == lib.DN_ERR_DEVICE_ARG
    assert (kc[0] == 7).all() and (vc[0] == 7).all()
    want = wref.cache_of(t["k"][1], top - 3, 2, 7, torch.full((1, 9, 64), 7.0, device=DEV))
    assert torch.equal(kc[1], want)
    ok(lib)


# ---- streams, graphs, workspaces ---------------------------------------------------------


def calls(lib, seed=1):
    """Every entry point as a function of its stream that returns the tensors it made."""
    lengths = [700, 1, 0, 300]
    t = inputs(torch.bfloat16, lengths=lengths, Nq=4, Nk=2, d=128, seed=seed)
    f = inputs(torch.float32, B=2, T=330, Nq=4, Nk=2, d=64, seed=seed)
    cu = ref.offsets(lengths, DEV)
    b, bg = block_inputs((torch.bfloat16, torch.float32), 1003, 512, seed=seed)
    g = torch.Generator().manual_seed(seed)
    cache = [normal(g, 4, 2, 304, 128, dtype=torch.bfloat16) for _ in range(2)]
    step = {n: t[n][0, :4, None].contiguous() for n in "qkv"}
    had = torch.tensor([0, 5, 290, 5000], device=DEV)
    kept = dict()
    for name, x, c in (("t", t, cu), ("f", f, None)):
        kept[name] = lib.window_attn_fwd(x["q"], x["k"], x["v"], 200, 4, c)
    torch.cuda.synchronize()

    def copies(st):
        stream = None if st is None else st if isinstance(st, torch.cuda.Stream) else torch.cuda.ExternalStream(st)
        with torch.cuda.stream(stream):
            return [c.clone() for c in cache]

    def fill(st):
        kc, vc = copies(st)
        lib.window_cache_fill(t["k"], t["v"], kc, vc, had, 4, cu, stream=st)
        return [kc, vc]

    def steps(st):
        kc, vc = copies(st)
        return [lib.window_attn_step(step["q"], step["k"], step["v"], kc, vc, had, 200, 4, stream=st), kc, vc]

    every = dict(
        attn=lambda st: lib.window_attn_fwd(t["q"], t["k"], t["v"], 200, 4, cu, stream=st),
        attn_bwd=lambda st: lib.window_attn_bwd(t["q"], t["k"], t["v"], *kept["t"], 200, 4, cu, do=t["do"], stream=st),
        attn_f32=lambda st: lib.window_attn_fwd(f["q"], f["k"], f["v"], 200, 4, stream=st),
        attn_f32_bwd=lambda st: lib.window_attn_bwd(f["q"], f["k"], f["v"], *kept["f"], 200, 4, do=f["do"], stream=st),
        fill=fill, step=steps,
        block=lambda st: lib.block_norm_fwd(*args(b), stream=st),
        block_bwd=lambda st: lib.block_norm_bwd(*args(b), **bg, stream=st))
    return every


NAMED = ("attn", "attn_bwd", "attn_f32", "attn_f32_bwd", "fill", "step", "block", "block_bwd")


def tensors(out):
    return list(out.values()) if isinstance(out, dict) else list(out)


def go(call, stream=None):
    return tensors(call(stream))


@pytest.mark.parametrize("name", NAMED)
def test_given_a_stream(lib, name):
    """Outputs and workspace are of the stream that was given, by object or handle, and a busy stream's results
    are those of an idle one."""
    call = calls(lib)[name]
    want = go(call)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream):
        with torch.cuda.stream(side):
            torch.cuda._sleep(10_000_000)
        got = go(call, stream)
        junk = [torch.full((1 << 20,), 7, dtype=torch.uint8, device=DEV) for _ in range(20)]  # the caller's own stream goes on
        torch.cuda.synchronize()
        assert [stream_of(o) for o in got] == [side.cuda_stream] * len(got)
        assert same(got, want)
        del junk
    ok(lib)


@pytest.mark.parametrize("name", NAMED)
def test_captured_and_replayed(lib, name):
    call = calls(lib)[name]
    want = go(call)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.stream(side):
            with torch.cuda.graph(graph, stream=side):
                held = go(call, stream)
        for _ in range(2):
            for h in held:
                h.fill_(7)
            graph.replay()
            torch.cuda.synchronize()
            assert same(held, want)
    ok(lib)


def test_two_streams_at_once(lib):
    one, two = (calls(lib, s) for s in (1, 2))
    want = [[go(c[n]) for n in NAMED] for c in (one, two)]
    torch.cuda.synchronize()
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(3):
        got = []
        for c, s in zip((one, two), streams):
            with torch.cuda.stream(s):
                got.append([go(c[n]) for n in NAMED])
        torch.cuda.synchronize()
        assert all(same(a, b) for g, w in zip(got, want) for a, b in zip(g, w))
    ok(lib)


@pytest.mark.parametrize("dtype", DTYPES)
def test_graphs_that_share_a_workspace(lib, dtype):
    """Nothing in a workspace is read before the call writes it: two captured backwards of other inputs take turns
    on one, which holds ones and NaN at first."""
    pairs = []
    for seed in (1, 2):
        t = inputs(dtype, B=2, T=700, Nq=4, Nk=2, seed=seed)
        if seed == 2:
            t["k"][0, 300, 0, 3] = float("inf")
        o, lse = lib.window_attn_fwd(t["q"], t["k"], t["v"], 150, 4)
        pairs.append((t, o, lse, lib.window_attn_bwd(t["q"], t["k"], t["v"], o, lse, 150, 4, do=t["do"])))
    need = lib.load().dn_window_attn_bwd_workspace_bytes(0, 2, 2, 700, 4, 2, 64, 150, 4, lib.dtype_code(dtype))
    space = torch.full((need,), 255, dtype=torch.uint8, device=DEV)
    torch.cuda.synchronize()
    side, graphs = torch.cuda.Stream(), []
    for t, o, lse, _ in pairs:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.stream(side):
            with torch.cuda.graph(graph, stream=side):
                held = lib.window_attn_bwd(t["q"], t["k"], t["v"], o, lse, 150, 4, do=t["do"], workspace=space)
        graphs.append((graph, held))
    for n in (0, 1, 1, 0, 1):
        graph, held = graphs[n]
        for h in held.values():
            h.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        for k, h in held.items():
            assert torch.equal(h.isnan(), pairs[n][3][k].isnan()) and torch.equal(h.nan_to_num(), pairs[n][3][k].nan_to_num())
    ok(lib)


def test_block_workspace_is_not_read(lib):
    t, g = block_inputs((torch.bfloat16, torch.bfloat16), 2000, 1032, seed=4)
    want = lib.block_norm_bwd(*args(t), **g)
    need = lib.load().dn_block_norm_bwd_workspace_bytes(2000, 1032, lib.DN_BF16, lib.DN_BF16)
    got = lib.block_norm_bwd(*args(t), **g, workspace=torch.full((need,), 255, dtype=torch.uint8, device=DEV))
    assert all(torch.equal(got[k], want[k]) for k in want)


# ---- offsets beyond 32 bits ------------------------------------------------------------------


def test_cache_of_more_than_32_bits(lib):
    """A ring of 2^24 slots and more: keys and values lie behind 2^31 elements, the last ones and those before the ring
    begins anew."""
    ring, window, d, Nq = (1 << 24) + 77, 300, 128, 4
    kc, vc = (torch.zeros(1, 1, ring, d, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    T, had = 500, ring - 350
    t = inputs(torch.bfloat16, B=1, T=T, Nq=Nq, Nk=1, d=d, seed=9)
    lib.window_cache_fill(t["k"][:, :T - 1].contiguous(), t["v"][:, :T - 1].contiguous(), kc, vc, torch.tensor([had], device=DEV))
    rows = {n: t[n][:, T - 1:].contiguous() for n in "qkv"}
    o = lib.window_attn_step(rows["q"], rows["k"], rows["v"], kc, vc, torch.tensor([had + T - 1], device=DEV), window)
    ok(lib)
    at = [(had + i) % ring for i in range(T)]
    assert torch.equal(kc[0, 0, at], t["k"][0, :, 0]) and torch.equal(vc[0, 0, at], t["v"][0, :, 0])
    w = wide(t)
    want = wref.attention(w["q"], w["k"], w["v"], window, 0, half=half_of(torch.bfloat16))["o"]
    wref.close(o[0, 0], (want[0][0, -1], want[1][0, -1]), "last step")
    # the whole ring as the window: all of it zeros but for the tokens above
    o = lib.window_attn_step(rows["q"], rows["k"], rows["v"], kc, vc, torch.tensor([had + T - 1], device=DEV), ring)
    ok(lib)
    q, k, v = (rows["q"][0, 0].double().cpu(), w["k"][0, :, 0], w["v"][0, :, 0])
    p = torch.exp(d ** -0.5 * (q @ k.T))  # a zero key's weight is 1
    want = p @ v / (p.sum(-1, keepdim=True) + (ring - T))
    # a weight is off by half a step of bf16 and by 2^-10 of itself for sums over 2^24 keys, the result by half a step
    bound = (p @ v.abs() / (p.sum(-1, keepdim=True) + (ring - T))) * (2.0 ** -8 + 2.0 ** -10) + want.abs() * 2.0 ** -8
    wref.close(o[0, 0], (want, bound + 1e-12), "the whole ring")


def test_attention_of_more_than_32_bits(lib):
    """2^31 elements and more of queries: the last rows as in a sequence of their own."""
    T, Nq, d, window, tail = 530_000, 32, 128, 64, 700
    assert T * Nq * d > 2 ** 31
    make = lambda h: torch.empty(1, T, h, d, dtype=torch.bfloat16, device=DEV).normal_()
    torch.manual_seed(5)
    q, do, k, v = make(Nq), make(Nq), make(1), make(1)
    o, lse = lib.window_attn_fwd(q, k, v, window)
    out = lib.window_attn_bwd(q, k, v, o, lse, window, do=do)
    ok(lib)
    last = {n: x[:, T - tail:].contiguous() for n, x in dict(q=q, k=k, v=v, do=do).items()}
    del q, do, k, v
    w = wide(last)
    want = wref.attention(w["q"], w["k"], w["v"], window, 0, None, None, w["do"], half_of(torch.bfloat16))
    inner = slice(window, tail)  # rows that see no token before these
    for n, x in (("o", o), ("lse", lse), ("dq", out["dq"]), ("dk", out["dk"]), ("dv", out["dv"])):
        wref.close(x[:, T - tail:][:, inner], (want[n][0][:, inner], want[n][1][:, inner]), n)


def test_block_of_more_than_32_bits(lib):
    rows, D = 1_050_000, 2056
    assert rows * D > 2 ** 31
    torch.manual_seed(6)
    make = lambda: torch.empty(rows, D, dtype=torch.bfloat16, device=DEV).normal_()
    x, residual, z, dy = make(), make(), make(), make()
    weight = torch.rand(D, device=DEV) + 0.5
    y, h = lib.block_norm_fwd(x, residual, z, weight=weight)
    out = lib.block_norm_bwd(x, residual, z, weight=weight, dy=dy)
    ok(lib)
    s = slice(rows - 301, rows)
    few = [u[s].clone() for u in (x, residual, z, dy)]
    y2, h2 = lib.block_norm_fwd(*few[:3], weight=weight)
    o2 = lib.block_norm_bwd(*few[:3], weight=weight, dy=few[3])
    assert torch.equal(y[s], y2) and torch.equal(h[s], h2)
    assert all(torch.equal(out[n][s], o2[n]) for n in ("dx", "dz", "dresidual"))


# ---- all of it together ------------------------------------------------------------------


def layers64(x, p, window, sinks):
    """A block's attention between the norms, in 64 bits: x [T, D] and the residual; returns y, residual."""
    Nq, Nk, d = 4, 2, 64
    x2, h = block64(dict(x=x, residual=p["residual"], z=p["z"], scale=None, post_weight=p["w0"], post_bias=None, weight=p["w1"],
                         bias=None), 1e-5, True, True)
    T = x.shape[0]
    q, k, v = x2.split((Nq * d, Nk * d, Nk * d), -1)
    q, k, v = q.view(T, Nq, d), k.view(T, Nk, d), v.view(T, Nk, d)
    seen = wref.seen_mask(T, window, sinks)
    rows = []
    for i in range(Nq):
        s = (d ** -0.5 * q[:, i] @ k[:, i // 2].T).masked_fill(~seen, -torch.inf)
        rows.append(torch.softmax(s, -1) @ v[:, i // 2])
    o = torch.cat(rows, -1)
    o = torch.cat((o, o), -1)
    return block64(dict(x=o, residual=h, z=None, scale=p["s"], post_weight=p["w2"], post_bias=None, weight=p["w3"], bias=None),
                   1e-5, True, True)


@pytest.mark.parametrize("dtype", DTYPES)
def test_a_block_trained(lib, dtype):
    """Norm, attention, norm and their gradients, each from the one before, against automatic differentiation
    in 64 bits.  Every stage is off by its own bound and passes on what it gets: the norms at most twice its share of a row, the
    attention through the weights, whose logarithms are off by 16 of it (queries and keys of length 8, both).  The two norms and the
    attention, forward and backward: (2 + 17 + 2) roundings each way of bf16's 2^-8 / sqrt(3) in the mean, or
    2^-24 sqrt(512) of fp32."""
    T, D, Nq, Nk, d, window, sinks = 300, 512, 4, 2, 64, 90, 3
    g = torch.Generator().manual_seed(21)
    x, z, residual = (normal(g, T, D, dtype=dtype) for _ in range(3))
    p = dict(residual=residual, z=z, s=normal(g, D), **{"w%d" % i: normal(g, D, scale=0.2) + 1 for i in range(4)})
    dy, dh = normal(g, T, D, dtype=dtype), normal(g, T, D, dtype=dtype)
    kind = dict(rms=True, post=True)

    first = (x, residual, z, None, p["w0"], None, p["w1"], None)
    y, h = lib.block_norm_fwd(*first, **kind)
    q, k, v = (u.contiguous().view(1, T, -1, d) for u in y.split((Nq * d, Nk * d, Nk * d), -1))
    o, lse = lib.window_attn_fwd(q, k, v, window, sinks)
    o2 = torch.cat((o.view(T, -1),) * 2, -1)
    second = (o2, h, None, p["s"], p["w2"], None, p["w3"], None)
    y2, h2 = lib.block_norm_fwd(*second, **kind)
    b2 = lib.block_norm_bwd(*second, **kind, dy=dy, dresidual_out=dh)
    do = (b2["dx"][:, :Nq * d] + b2["dx"][:, Nq * d:]).view(1, T, Nq, d)
    a = lib.window_attn_bwd(q, k, v, o, lse, window, sinks, do=do)
    dyy = torch.cat([a[n].view(T, -1) for n in ("dq", "dk", "dv")], -1)
    b1 = lib.block_norm_bwd(*first, **kind, dy=dyy, dresidual_out=b2["dresidual"])
    ok(lib)

    u = {n: t.double().cpu().requires_grad_() for n, t in dict(p, x=x).items()}
    want = layers64(u["x"], u, window, sinks)
    (want[0] * dy.double().cpu() + want[1] * dh.double().cpu()).sum().backward()
    tol = 2 * 21 * (2.0 ** -8 / 3 ** 0.5 if dtype == torch.bfloat16 else 2.0 ** -24 * 512 ** 0.5)
    got = dict(x=b1["dx"], residual=b1["dresidual"], z=b1["dz"], w0=b1["dpost_weight"], w1=b1["dweight"], s=b2["dscale"],
               w2=b2["dpost_weight"], w3=b2["dweight"])
    for n, t in got.items():
        assert (t.double().cpu() - u[n].grad).norm() <= tol * u[n].grad.norm(), n
    for t, w in ((y2, want[0]), (h2, want[1])):
        assert (t.double().cpu() - w).norm() <= tol / 2 * w.norm()


def test_a_prompt_and_its_tokens(lib):
    """A layer of the gated delta rule and one of attention, with the norms around them, in fp32: prompts of several
    lengths through the forms for whole sequences, then token by token through those for steps; every token's row as
    the whole sequences give it.  The rule's two forms agree within 1e-4 of the norm; a norm passes on twice that
    at most, the attention 17 times (a block trained, above)."""
    Nq, Nk, d, D, window, sinks, ring = 4, 2, 64, 512, 50, 3, 64
    full, had, N = 150, [0, 33, 120], 3
    r = workloads.to_device(workloads.make_inputs(N, full, 2, 4, 128, 128, dtype=torch.float32, gate_mu=3.0, seed=77), DEV)
    g = torch.Generator().manual_seed(78)
    residual, z = normal(g, N, full, D), normal(g, N, full, D)
    w = [normal(g, D, scale=0.2) + 1 for _ in range(4)]
    scale = r.get("scale")

    def before(o, res, z):
        y, h = lib.block_norm_fwd(o, res, z, None, w[0], None, w[1], None, rms=True, post=True)
        return [u.contiguous().unflatten(-1, (-1, d)) for u in y.split((Nq * d, Nk * d, Nk * d), -1)], h

    def after(o, h):
        o = o.flatten(-2)
        return lib.block_norm_fwd(torch.cat((o, o), -1), h, None, None, w[2], None, w[3], None, rms=True, post=True)

    # the whole sequences
    o, _ = lib.chunk_fwd(*(r[n] for n in ("q", "k", "v", "beta", "g")), scale=scale)
    (q, k, v), h = before(o.flatten(-2), residual, z)
    whole = after(lib.window_attn_fwd(q, k, v, window, sinks)[0], h)

    # prompts, packed
    cu = ref.offsets(had, DEV)
    pack = lambda x: torch.cat([x[b, :had[b]] for b in range(N)])[None].contiguous()
    o, state = lib.chunk_fwd(*(pack(r[n]) for n in ("q", "k", "v", "beta", "g")), cu_seqlens=cu, scale=scale)
    (q, k, v), h = before(o.flatten(-2), pack(residual), pack(z))
    rows = after(lib.window_attn_fwd(q, k, v, window, sinks, cu)[0], h)
    kc, vc = (torch.full((N, Nk, sinks + ring, d), float("nan"), device=DEV) for _ in range(2))
    lib.window_cache_fill(k, v, kc, vc, sinks=sinks, cu_seqlens=cu)
    lengths = torch.tensor(had, device=DEV)
    got = [[rows[i][0, cu[b]:cu[b + 1]] for b in range(N)] for i in range(2)]
    # tokens
    for i in range(full - max(had)):
        one = lambda x: torch.stack([x[b, had[b] + i] for b in range(N)])[:, None].contiguous()
        o, state = lib.recurrent_fwd(*(one(r[n]) for n in ("q", "k", "v", "beta", "g")), h0=state, scale=scale)
        (q, k, v), h = before(o.flatten(-2), one(residual), one(z))
        rows = after(lib.window_attn_step(q, k, v, kc, vc, lengths, window, sinks), h)
        for n in range(2):
            for b in range(N):
                got[n][b] = torch.cat((got[n][b], rows[n][b]))
        lengths += 1
    ok(lib)
    for n in range(2):
        for b in range(N):
            want = whole[n][b, :had[b] + full - max(had)]
            assert got[n][b].shape == want.shape
            assert (got[n][b] - want).norm() <= 2 * 17 * 2 * 1e-4 * want.norm(), (n, b)
