"""GPU: attention over a sliding window with sinks and its ring cache through the C ABI, against the
definitions in 64 bits within the bounds that window_reference derives."""
import pytest
import torch

import layer_reference as ref
import window_reference as wref
from conftest import cuda_ok

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not cuda_ok(), reason="needs a CUDA GPU")]

DTYPES = [torch.bfloat16, torch.float32]
DEV = "cuda"
INF, NAN = float("inf"), float("nan")


def half_of(dtype):
    return torch.finfo(dtype).eps / 2 if dtype == torch.bfloat16 else 0.0


def normal(g, *shape, dtype=torch.float32, scale=1.0):
    return (scale * torch.randn(*shape, generator=g)).to(dtype).to(DEV)


def inputs(dtype, B=2, T=100, Nq=2, Nk=1, d=64, lengths=None, pad=0, seed=0):
    g = torch.Generator().manual_seed(seed)
    if lengths is not None:
        B, T = 1, sum(lengths) + pad
    return dict(q=normal(g, B, T, Nq, d, dtype=dtype), k=normal(g, B, T, Nk, d, dtype=dtype),
                v=normal(g, B, T, Nk, d, dtype=dtype), do=normal(g, B, T, Nq, d, dtype=dtype))


def wide(t):
    return {k: v.double().cpu() for k, v in t.items()}


def ok(lib):
    assert lib.dn_check() == lib.DN_OK


def check(lib, t, window, sinks, lengths=None, scale=None, label="", pad=0):
    cu = None if lengths is None else ref.offsets(lengths, DEV)
    used = t["q"].shape[1] - pad
    o = torch.full_like(t["q"], 7.0)
    lse = torch.full(t["q"].shape[:3], 7.0, device=DEV)
    lib.window_attn_fwd(t["q"], t["k"], t["v"], window, sinks, cu, scale=scale, o=o, lse=lse)
    ok(lib)
    assert (o[:, used:] == 7).all() and (lse[:, used:] == 7).all(), label  # rows behind the last sequence
    w = {k: v[:, :used] for k, v in wide(t).items()}
    want = wref.attention(w["q"], w["k"], w["v"], window, sinks, lengths, scale, w["do"], half_of(t["q"].dtype))
    wref.close(o[:, :used], want["o"], label + " o")
    wref.close(lse[:, :used], want["lse"], label + " lse")
    out = lib.window_attn_bwd(t["q"], t["k"], t["v"], o, lse, window, sinks, cu, scale=scale, do=t["do"])
    ok(lib)
    for name in ("dq", "dk", "dv"):
        wref.close(out[name][:, :used], want[name], label + " " + name)
    return o, lse, out


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("T", [1, 2, 63, 64, 65, 127, 128, 129, 191, 257, 400])
def test_lengths(lib, dtype, d, T):
    check(lib, inputs(dtype, T=T, d=d, seed=T + d), 70, 4, label="T=%d d=%d" % (T, d))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("window", [1, 2, 63, 64, 65, 127, 128, 129, 130, 255, 299, 300, 5000, 2**31 + 5])
def test_windows(lib, dtype, window):
    for sinks in (0, 3):
        check(lib, inputs(dtype, B=1, T=300, seed=window % 1000), window, sinks, label="w=%d s=%d" % (window, sinks))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("sinks", [1, 16, 31, 32, 33, 63, 64, 65, 127, 128])
def test_sinks(lib, dtype, sinks):
    for window in (9, 140):
        check(lib, inputs(dtype, B=1, T=520, d=128, seed=sinks), window, sinks, label="s=%d w=%d" % (sinks, window))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("Nq,Nk", [(1, 1), (3, 3), (6, 2), (8, 1), (5, 1), (16, 8), (20, 4)])
def test_heads(lib, dtype, Nq, Nk):
    check(lib, inputs(dtype, B=2, T=210, Nq=Nq, Nk=Nk, seed=Nq), 90, 5, label="heads %d %d" % (Nq, Nk))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("lengths,pad", [([0, 1, 2, 33, 128, 0, 129, 300, 5, 0], 3), ([7], 0), ([0, 0], 4), ([513, 1, 260], 130)])
@pytest.mark.parametrize("d", [64, 128])
def test_packed(lib, dtype, lengths, pad, d):
    t = inputs(dtype, lengths=lengths, pad=pad, Nq=4, Nk=2, d=d, seed=9)
    for name in t:  # what lies behind the last sequence is not looked at
        t[name][:, t[name].shape[1] - pad:] = NAN
    check(lib, t, 100, 6, lengths, label="packed", pad=pad)


@pytest.mark.parametrize("dtype", DTYPES)
def test_scale(lib, dtype):
    for scale in (0.01, 1.5):
        check(lib, inputs(dtype, T=150, seed=4), 60, 2, scale=scale, label="scale %g" % scale)


@pytest.mark.parametrize("dtype", DTYPES)
def test_maxima_that_grow_and_fall(lib, dtype):
    """Scores of hundreds, rising and falling along the keys: the running maximum moves by more than any
    threshold, and early keys weigh nothing later on."""
    t = inputs(dtype, B=1, T=700, Nq=2, Nk=1, d=128, seed=5)
    ramp = torch.linspace(-1, 1, 700, device=DEV)[None, :, None, None]
    for sign in (1, -1):
        u = dict(t, q=(t["q"].abs() * 2).to(dtype), k=(t["k"].abs() * 4 * sign * ramp).to(dtype))
        check(lib, u, 400, 8, label="ramp %d" % sign)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("bad", [NAN, INF, -INF])
@pytest.mark.parametrize("d", [64, 128])
def test_masked_values_reach_nothing(lib, dtype, bad, d):
    """A bad key and value at one token: rows that do not see it come out as without it, its gradient too."""
    T, window, sinks, at = 600, 150, 4, 290
    t = inputs(dtype, B=1, T=T, Nq=2, Nk=1, d=d, seed=6)
    w = wide(t)
    want = wref.attention(w["q"], w["k"], w["v"], window, sinks, None, None, w["do"], half_of(dtype))
    blind = torch.tensor([i < at or i >= at + window for i in range(T)])
    for names in (("v",), ("k",), ("k", "v")):
        u = {n: x.clone() for n, x in t.items()}
        for n in names:
            u[n][0, at, 0, 5] = bad
        o, lse = lib.window_attn_fwd(u["q"], u["k"], u["v"], window, sinks)
        ok(lib)
        pick = lambda pair: (pair[0][:, blind], pair[1][:, blind])
        wref.close(o[:, blind], pick(want["o"]), "o %s" % (names,))
        wref.close(lse[:, blind], pick(want["lse"]), "lse %s" % (names,))
        seeing = o[0, ~blind][:, :, 5].float()
        assert not torch.isfinite(seeing).all()
        out = lib.window_attn_bwd(u["q"], u["k"], u["v"], o, lse, window, sinks, do=t["do"])
        ok(lib)
        wref.close(out["dq"][:, blind], pick(want["dq"]), "dq %s" % (names,))
        # keys that no query shares with the bad one: none that sees the bad token sees them
        far = torch.tensor([sinks <= j <= at - window or j >= at + window for j in range(T)])
        for name in ("dk", "dv"):
            wref.close(out[name][:, far], (want[name][0][:, far], want[name][1][:, far]), "%s %s" % (name, names))


@pytest.mark.parametrize("dtype", DTYPES)
def test_bad_queries_stay_in_their_rows(lib, dtype):
    T, window, at = 400, 100, 250
    t = inputs(dtype, B=1, T=T, Nq=2, Nk=2, d=64, seed=7)
    w = wide(t)
    want = wref.attention(w["q"], w["k"], w["v"], window, 0, None, None, w["do"], half_of(dtype))
    for name in ("q", "do"):
        u = {n: x.clone() for n, x in t.items()}
        u[name][0, at, 1] = NAN
        o, lse = lib.window_attn_fwd(u["q"], u["k"], u["v"], window)
        out = lib.window_attn_bwd(u["q"], u["k"], u["v"], o, lse, window, do=u["do"])
        ok(lib)
        other = torch.arange(T) != at
        wref.close(o[:, other], (want["o"][0][:, other], want["o"][1][:, other]), "o")
        assert torch.isnan(o[0, at, 1]).all() == (name == "q")
        wref.close(out["dq"][:, other], (want["dq"][0][:, other], want["dq"][1][:, other]), "dq")
        assert torch.isnan(out["dq"][0, at, 1]).all()
        far = torch.tensor([j <= at - window or j > at for j in range(T)])
        for n in ("dk", "dv"):
            wref.close(out[n][:, far], (want[n][0][:, far], want[n][1][:, far]), n)
            assert torch.isnan(out[n][0, at, 1]).all()


@pytest.mark.parametrize("dtype", DTYPES)
def test_gradient_by_differences(lib, dtype):
    """The gradient along a direction against the loss's difference, both from the entry points (fp32), and the
    bf16 gradient against the fp32 one."""
    t = inputs(torch.float32, B=1, T=150, Nq=2, Nk=1, d=64, seed=8)
    if dtype == torch.bfloat16:
        t = {k: v.to(dtype).float() for k, v in t.items()}
    window, sinks = 40, 3
    args = lambda u: (u["q"], u["k"], u["v"], window, sinks)
    o, lse = lib.window_attn_fwd(*args(t))
    out = lib.window_attn_bwd(t["q"], t["k"], t["v"], o, lse, window, sinks, do=t["do"])
    if dtype == torch.bfloat16:
        b = {k: v.to(dtype) for k, v in t.items()}
        ob, lb = lib.window_attn_fwd(*args(b))
        low = lib.window_attn_bwd(b["q"], b["k"], b["v"], ob, lb, window, sinks, do=b["do"])
        for n in out:  # roundings of p, dS, o and the result: independent, each half a step at most
            assert (low[n].float() - out[n]).norm() <= 4 * 2.0 ** -8 * out[n].norm()
        return
    for name in ("q", "k", "v"):
        g = torch.Generator().manual_seed(1)
        way = normal(g, *t[name].shape)
        eps = 1e-2
        loss = []
        for s in (1, -1):
            u = dict(t)
            u[name] = t[name] + s * eps * way
            loss.append((lib.window_attn_fwd(*args(u))[0].double() * t["do"].double()).sum())
        diff = float(loss[0] - loss[1]) / (2 * eps)
        along = float((out["d" + name].double() * way.double()).sum())
        # central differences: an error of the order eps^2 times the third derivative along `way`
        assert abs(diff - along) <= 1e-2 * float(out["d" + name].norm() * way.norm()), name


@pytest.mark.parametrize("dtype", DTYPES)
def test_same_bits_every_time(lib, dtype):
    t = inputs(dtype, lengths=[700, 1, 300], Nq=8, Nk=2, d=128, seed=11)
    cu = ref.offsets([700, 1, 300], DEV)

    def call():
        o, lse = lib.window_attn_fwd(t["q"], t["k"], t["v"], 200, 4, cu)
        out = lib.window_attn_bwd(t["q"], t["k"], t["v"], o, lse, 200, 4, cu, do=t["do"])
        return [o, lse, out["dq"], out["dk"], out["dv"]]

    first = call()
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(first, call()))


def test_malformed_offsets_are_reported(lib):
    t = inputs(torch.bfloat16, lengths=[50, 50], Nq=2, Nk=1, seed=12)
    lib.dn_check()
    for cu in ([0, 60, 50], [0, 50, 101], [1, 50, 100], [0, -5, 100]):
        cu = torch.tensor(cu, dtype=torch.int64, device=DEV)
        o, lse = lib.window_attn_fwd(t["q"], t["k"], t["v"], 20, 2, cu)
        assert lib.dn_check() == lib.DN_ERR_DEVICE_ARG
        lib.window_attn_bwd(t["q"], t["k"], t["v"], o, lse, 20, 2, cu, do=t["do"])
        assert lib.dn_check() == lib.DN_ERR_DEVICE_ARG
        kc = torch.zeros(2, 1, 22, 64, dtype=torch.bfloat16, device=DEV)
        lib.window_cache_fill(t["k"], t["v"], kc, kc.clone(), sinks=2, cu_seqlens=cu)
        assert lib.dn_check() == lib.DN_ERR_DEVICE_ARG


# ---- the ring cache ---------------------------------------------------------------------------


def caches(dtype, N, Nk, slots, d, seed):
    g = torch.Generator().manual_seed(seed)
    return [normal(g, N, Nk, slots, d, dtype=dtype) for _ in range(2)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("sinks,ring", [(0, 1), (0, 50), (4, 16), (7, 64), (3, 400), (128, 9)])
def test_fill(lib, dtype, sinks, ring):
    lengths = [0, 1, 5, 130, 33, 0, 64]
    for had in (None, [0, 3, 2, 900, 4, 11, 2**40]):
        t = inputs(dtype, lengths=lengths, pad=2, Nq=3, Nk=3, seed=ring)
        kc, vc = caches(dtype, len(lengths), 3, sinks + ring, 64, 1)
        want = [c.clone() for c in (kc, vc)]
        at = 0
        for n, length in enumerate(lengths):
            for name, w in zip("kv", want):
                w[n] = wref.cache_of(t[name][0, at:at + length], had[n] if had else 0, sinks, ring, w[n])
            at += length
        given = None if had is None else torch.tensor(had, device=DEV)
        lib.window_cache_fill(t["k"], t["v"], kc, vc, given, sinks, ref.offsets(lengths, DEV))
        ok(lib)
        assert torch.equal(kc, want[0]) and torch.equal(vc, want[1])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("Nq,Nk,d", [(2, 1, 64), (3, 3, 128), (16, 2, 128), (40, 2, 64), (5, 1, 128), (24, 3, 64), (64, 2, 128)])
def test_steps_continue_a_prompt(lib, dtype, Nq, Nk, d):
    """A prompt into the cache, then token by token: each step is the row that the whole sequence has there."""
    window, sinks, ring = 37, 4, 45
    T, prompt = 140, 90
    t = inputs(dtype, B=3, T=T, Nq=Nq, Nk=Nk, d=d, seed=Nq)
    kc, vc = caches(dtype, 3, Nk, sinks + ring, d, 2)
    kc[:], vc[:] = NAN, NAN  # slots that nothing was written to are not looked at
    # the three sequences start at other places: each has had its own number of tokens
    had = [0, 20, prompt]
    lengths = torch.tensor(had, device=DEV)
    cu = ref.offsets(had, DEV)
    packed = {n: torch.cat([t[n][b, :had[b]] for b in range(3)])[None].contiguous() for n in "kv"}
    lib.window_cache_fill(packed["k"], packed["v"], kc, vc, None, sinks, cu)
    w = wide(t)
    want = wref.attention(w["q"], w["k"], w["v"], window, sinks, half=half_of(dtype))["o"]
    for i in range(T - prompt):
        rows = {n: torch.stack([t[n][b, had[b] + i] for b in range(3)])[:, None].contiguous() for n in "qkv"}
        o = lib.window_attn_step(rows["q"], rows["k"], rows["v"], kc, vc, lengths, window, sinks)
        for b in range(3):
            wref.close(o[b, 0], (want[0][b, had[b] + i], want[1][b, had[b] + i]), "step %d of %d" % (i, b))
        lengths += 1
    ok(lib)
    assert lengths.tolist() == [h + T - prompt for h in had]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("N,window,ring,sinks", [(1, 1, 1, 0), (2, 1, 1, 3), (1, 700, 700, 4), (2, 2000, 2100, 128), (5, 333, 400, 1),
                                                 (1, 5000, 5000, 0), (40, 257, 257, 16)])
def test_step_sizes(lib, dtype, N, window, ring, sinks):
    Nq, Nk, d = 8, 2, 128
    g = torch.Generator().manual_seed(N + window)
    t = {n: normal(g, N, 1, h, d, dtype=dtype) for n, h in (("q", Nq), ("k", Nk), ("v", Nk))}
    kc, vc = caches(dtype, N, Nk, sinks + ring, d, 3)
    had = [[0, 1, sinks, sinks + 1, ring, sinks + ring - 1, sinks + ring, 3 * ring + 17, 2**33 + 5][(i * 5 + 8) % 9] for i in range(N)]
    before = [kc.clone(), vc.clone()]
    o = lib.window_attn_step(t["q"], t["k"], t["v"], kc, vc, torch.tensor(had, device=DEV), window, sinks)
    ok(lib)
    for n in range(N):
        p = had[n]
        for c, b, name in ((kc, before[0], "k"), (vc, before[1], "v")):
            b[n, :, wref.slot(p, sinks, ring)] = t[name][n, 0]
        at = [j for j in range(min(sinks, p + 1))] + [j for j in range(max(sinks, p + 1 - window), p + 1)]
        at = [wref.slot(j, sinks, ring) for j in at]
        # as a sequence of its own whose last token sees everything
        k, v = (b[n][:, at].transpose(0, 1).double().cpu()[None] for b in before)
        q = t["q"][n].double().cpu().expand(1, len(at), Nq, d).clone()
        q[:, :-1] = 0
        want = wref.attention(q, k, v, len(at), 0, half=half_of(dtype))["o"]
        wref.close(o[n, 0], (want[0][0, -1], want[1][0, -1]), "sequence %d at %d" % (n, p))
    assert torch.equal(kc, before[0]) and torch.equal(vc, before[1])


@pytest.mark.parametrize("dtype", DTYPES)
def test_step_bad_values_outside_the_window(lib, dtype):
    window, ring, sinks, Nk, d = 100, 160, 4, 2, 64
    g = torch.Generator().manual_seed(3)
    t = {n: normal(g, 1, 1, h, d, dtype=dtype) for n, h in (("q", 4), ("k", Nk), ("v", Nk))}
    kc, vc = caches(dtype, 1, Nk, sinks + ring, d, 4)
    had = torch.tensor([1000], device=DEV)
    clean = lib.window_attn_step(t["q"], t["k"], t["v"], kc.clone(), vc.clone(), had, window, sinks)
    for p in list(range(1000 - ring, 1001 - window)):
        kc[:, :, wref.slot(p, sinks, ring)] = NAN
        vc[:, :, wref.slot(p, sinks, ring)] = INF
    got = lib.window_attn_step(t["q"], t["k"], t["v"], kc, vc, had, window, sinks)
    assert torch.equal(got, clean)


def test_negative_lengths_are_reported(lib):
    t = inputs(torch.bfloat16, B=2, T=1, Nq=2, Nk=1, seed=1)
    kc, vc = caches(torch.bfloat16, 2, 1, 10, 64, 1)
    lib.dn_check()
    lib.window_attn_step(t["q"], t["k"], t["v"], kc, vc, torch.tensor([3, -1], device=DEV), 8, 2)
    assert lib.dn_check() == lib.DN_ERR_DEVICE_ARG
    lib.window_cache_fill(t["k"], t["v"], kc, vc, torch.tensor([-7, 0], device=DEV), 2)
    assert lib.dn_check() == lib.DN_ERR_DEVICE_ARG
    ok(lib)
