"""GPU: the operators around the recurrence (short causal convolution, selective
scan, layer norm) through the C ABI, against their definitions in 64 bits.

Tolerances (layer_reference.close): half a step of a 16-bit output, and a number
of fp32 roundings counted from the formulas:

* convolution: W products and sums, then silu (an exponential, a sum, a quotient:
  at most 8 units each in 2^-24) -- 4 W + 32, and as many for a gradient, whose sums
  over T tokens add one each: 4 W + 32 + T;
* scan: per token the exponential (4 units), its argument (delta within 8 units, the
  product 2: together at most 10 |delta A| e^-|delta A| < 4) and two sums -- 10 per
  token of the sequence, 64 for the rest; the gradient takes two such walks: 30 per token;
* norm: D terms per sum, added in fewer than 64 steps, the root and quotient -- 128;
  a gradient over the rows adds one per row.
"""
import pytest
import torch

import layer_reference as ref
from conftest import cuda_ok

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not cuda_ok(), reason="needs a CUDA GPU")]

DTYPES = [torch.bfloat16, torch.float32]
RAGGED = [0, 1, 2, 3, 33, 64, 0, 70, 5, 0]
DEV = "cuda"


def gen(seed):
    return torch.Generator().manual_seed(seed)


def normal(g, *shape, dtype=torch.float32, scale=1.0):
    return (scale * torch.randn(*shape, generator=g)).to(dtype).to(DEV)


def ok(lib):
    assert lib.dn_check() == lib.DN_OK


# ---- convolution -------------------------------------------------------------


def conv_inputs(dtype, B=2, T=37, D=64, W=4, lengths=None, bias=True, h0=True, seed=0, pad=0):
    g = gen(seed)
    n = B if lengths is None else len(lengths)
    if lengths is not None:
        B, T = 1, sum(lengths) + pad
    t = dict(x=normal(g, B, T, D, dtype=dtype), weight=normal(g, D, W, scale=0.6),
             bias=normal(g, D, scale=0.3) if bias else None,
             h0=normal(g, n, W - 1, D, dtype=dtype) if h0 else None)
    grads = dict(dy=normal(g, B, T, D, dtype=dtype), dht=normal(g, n, W - 1, D, dtype=dtype))
    return t, grads


def conv_check(lib, t, grads, lengths, silu, label, dy_f32=False, dht=True):
    W = t["weight"].shape[1]
    T = t["x"].shape[1]
    cu = None if lengths is None else ref.offsets(lengths, DEV)
    y, ht = lib.causal_conv_fwd(t["x"], t["weight"], t["bias"], t["h0"], cu, silu=silu)
    ok(lib)
    leaves = ref.in_64_bits(t, grad=True)
    y64, ht64 = ref.conv(leaves, lengths, silu)
    used = T if lengths is None else sum(lengths)
    terms = float(t["x"].abs().max()) * float(t["weight"].abs().sum(1).max()) + 1 if used else 1.0
    ref.close(y[:, :used], y64[:, :used], 4 * W + 32, label + " y", scale=terms)
    assert torch.equal(ht.double().cpu(), ht64.detach()), label
    dy = grads["dy"].float() if dy_f32 else grads["dy"]
    out = lib.causal_conv_bwd(t["x"], t["weight"], t["bias"], t["h0"], cu, silu=silu, dy=dy,
                              dht=grads["dht"] if dht else None)
    ok(lib)
    mask = torch.zeros_like(grads["dy"])
    mask[:, :used] = 1
    want = ref.gradients([y64, ht64], [grads["dy"] * mask, grads["dht"] if dht else None], leaves)
    for name in ("x", "weight", "bias", "h0"):
        if t[name] is None:
            assert out["d" + name] is None
            continue
        got, w = out["d" + name], want[name]
        if name == "x":
            got, w = got[:, :used], w[:, :used]
        ref.close(got, w, 4 * W + 32 + (0 if name in ("x", "h0") else y.shape[0] * used), label + " d" + name,
                  scale=max(terms, float(w.abs().max()) if w.numel() else 0.0))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("D", [1, 7, 64, 132, 257])
def test_conv_sizes(lib, dtype, W, D):
    t, grads = conv_inputs(dtype, D=D, W=W, seed=W * 1000 + D)
    conv_check(lib, t, grads, None, True, "conv %d %d" % (W, D))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("D", [24, 33])
@pytest.mark.parametrize("h0", [True, False])
def test_conv_packed(lib, dtype, D, h0):
    t, grads = conv_inputs(dtype, D=D, lengths=RAGGED, h0=h0, seed=10 + D, pad=3)
    conv_check(lib, t, grads, RAGGED, True, "conv packed", dy_f32=dtype == torch.bfloat16)


@pytest.mark.parametrize("T", [1, 2, 8, 31, 32, 33, 64, 65, 200])
def test_conv_lengths(lib, T):
    t, grads = conv_inputs(torch.bfloat16, B=3, T=T, D=40, seed=T)
    conv_check(lib, t, grads, None, True, "conv T=%d" % T)


def test_conv_options(lib):
    for silu, bias, dht in ((False, True, True), (True, False, True), (False, False, False)):
        t, grads = conv_inputs(torch.float32, bias=bias, h0=dht, seed=5)
        conv_check(lib, t, grads, None, silu, "conv options", dht=dht)


def test_conv_steps_in_place_equal_the_prompt(lib):
    """Single tokens, each from the state the last one left in the same buffer."""
    t, _ = conv_inputs(torch.bfloat16, B=5, T=9, D=72, seed=6)
    y, ht = lib.causal_conv_fwd(t["x"], t["weight"], t["bias"], t["h0"])
    state = t["h0"].clone()
    for s in range(9):
        step, same = lib.causal_conv_fwd(t["x"][:, s:s + 1].contiguous(), t["weight"], t["bias"], state, ht=state)
        assert same is state
        assert torch.equal(step, y[:, s:s + 1])
    assert torch.equal(state, ht)


def test_conv_bad_token_stays_in_its_window(lib):
    """An infinite input reaches the W tokens that read it and no gradient before them."""
    t, grads = conv_inputs(torch.float32, B=1, T=40, D=8, h0=False, seed=7)
    t["x"][0, 39] = float("inf")
    y, _ = lib.causal_conv_fwd(t["x"], t["weight"], t["bias"])
    assert torch.isfinite(y[0, :39]).all()
    out = lib.causal_conv_bwd(t["x"], t["weight"], t["bias"], dy=grads["dy"])
    assert torch.isfinite(out["dx"][0, :36]).all()
    lengths = [20, 20]
    t["x"][0, 39] = 0.0
    t["x"][0, 19] = float("inf")  # the last token of the first sequence
    out = lib.causal_conv_bwd(t["x"], t["weight"], t["bias"], cu_seqlens=ref.offsets(lengths, DEV), dy=grads["dy"])
    assert torch.isfinite(out["dx"][0, 20:]).all()


# ---- selective scan --------------------------------------------------------------


def scan_inputs(dtype, B=2, T=37, D=20, G=1, N=16, lengths=None, gate=True, h0=True, extras=True, seed=0, pad=0):
    g = gen(seed)
    n = B if lengths is None else len(lengths)
    if lengths is not None:
        B, T = 1, sum(lengths) + pad
    t = dict(x=normal(g, B, T, D, dtype=dtype), dt=normal(g, B, T, D, dtype=dtype),
             A=-torch.rand(D, N, generator=g).mul(3).add(0.1).to(DEV), B=normal(g, B, T, G, N, dtype=dtype),
             C=normal(g, B, T, G, N, dtype=dtype), D=normal(g, D) if extras else None,
             z=normal(g, B, T, D, dtype=dtype) if gate else None,
             dt_bias=normal(g, D).sub(1.5) if extras else None, h0=normal(g, n, D, N) if h0 else None)
    grads = dict(dy=normal(g, B, T, D, dtype=dtype), dht=normal(g, n, D, N))
    return t, grads


NAMES = ("x", "dt", "A", "B", "C", "D", "z", "dt_bias", "h0")


def scan_args(t):
    return [t[k] for k in NAMES]


def scan_check(lib, t, grads, lengths, label, softplus=True, dht=True):
    B, T, D = t["x"].shape
    used = T if lengths is None else sum(lengths)
    longest = T if lengths is None else max(lengths)
    cu = None if lengths is None else ref.offsets(lengths, DEV)
    y, ht = lib.selective_scan_fwd(*scan_args(t), cu, dt_softplus=softplus)
    ok(lib)
    leaves = ref.in_64_bits(t, grad=True)
    y64, ht64 = ref.scan(leaves, lengths, softplus)
    ref.close(y[:, :used], y64[:, :used], 10 * longest + 64, label + " y")
    ref.close(ht, ht64, 10 * longest + 64, label + " ht")
    out = lib.selective_scan_bwd(*scan_args(t), cu, dt_softplus=softplus, dy=grads["dy"],
                                 dht=grads["dht"] if dht else None)
    ok(lib)
    mask = torch.zeros_like(grads["dy"])
    mask[:, :used] = 1
    want = ref.gradients([y64, ht64], [grads["dy"] * mask, grads["dht"] if dht else None], leaves)
    for name in NAMES:
        if t[name] is None:
            assert out["d" + name] is None
            continue
        got, w = out["d" + name], want[name]
        if name in ("x", "dt", "B", "C", "z"):
            got, w = got[:, :used], w[:, :used]
        extra = B * used if name in ("A", "D", "dt_bias") else D if name in ("B", "C") else 0
        ref.close(got, w, 30 * longest + 64 + extra, label + " d" + name)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("N", [16, 32, 64, 128])
@pytest.mark.parametrize("D,G", [(36, 1), (22, 2), (1, 1), (72, 2)])
def test_scan_sizes(lib, dtype, N, D, G):
    t, grads = scan_inputs(dtype, T=21, D=D, G=G, N=N, seed=N + D)
    scan_check(lib, t, grads, None, "scan N=%d D=%d" % (N, D))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("h0,gate", [(True, False), (False, True)])
def test_scan_packed(lib, dtype, h0, gate):
    lengths = [0, 1, 2, 64, 65, 0, 130, 17, 0]
    t, grads = scan_inputs(dtype, D=34, lengths=lengths, h0=h0, gate=gate, seed=3, pad=5)
    scan_check(lib, t, grads, lengths, "scan packed", dht=h0)


@pytest.mark.parametrize("T", [1, 7, 8, 16, 17, 63, 64, 65, 129, 300])
def test_scan_lengths(lib, T):
    t, grads = scan_inputs(torch.bfloat16, B=2, T=T, D=40, seed=T)
    scan_check(lib, t, grads, None, "scan T=%d" % T)


def test_scan_options(lib):
    for softplus, gate, extras, h0 in ((False, True, True, True), (True, False, False, False)):
        t, grads = scan_inputs(torch.float32, T=90, gate=gate, extras=extras, h0=h0, seed=9)
        if not softplus:
            t["dt"] = t["dt"].abs() * 0.3
            t["dt_bias"] = None
        scan_check(lib, t, grads, None, "scan options", softplus=softplus, dht=h0)


def test_scan_steps_in_place_continue_a_prompt(lib):
    """A prompt, then single tokens from the state in one buffer, against one walk in 64 bits."""
    t, _ = scan_inputs(torch.float32, B=3, T=150, D=48, seed=11)
    y64, ht64 = ref.scan(ref.in_64_bits(t))

    def part(lo, hi):
        return [t[k][:, lo:hi].contiguous() if k in ("x", "dt", "B", "C", "z") else t[k] for k in NAMES]

    head = part(0, 140)
    y, state = lib.selective_scan_fwd(*head)
    ys = [y]
    for s in range(140, 150):
        args = part(s, s + 1)
        args[-1] = state
        step, same = lib.selective_scan_fwd(*args, ht=state)
        assert same is state
        ys.append(step)
    ref.close(torch.cat(ys, 1), y64, 10 * 150 + 64, "steps y")
    ref.close(state, ht64, 10 * 150 + 64, "steps ht")


@pytest.mark.parametrize("n", [1, 3, 64, 613])
@pytest.mark.parametrize("dtype", DTYPES)
def test_single_tokens(lib, dtype, n):
    """One token of n sequences, with and without a state before it."""
    for h0 in (True, False):
        t, grads = scan_inputs(dtype, B=n, T=1, D=36, G=2, h0=h0, seed=n)
        scan_check(lib, t, grads, None, "scan one token", dht=h0)
        t, grads = conv_inputs(dtype, B=n, T=1, D=36, h0=h0, seed=n)
        conv_check(lib, t, grads, None, True, "conv one token", dht=h0)
    t, grads = conv_inputs(dtype, B=n, T=1, D=7, W=3, seed=n)
    conv_check(lib, t, grads, None, False, "conv one token", dht=True)


def test_many_single_tokens(lib):
    """More sequences than a grid has rows of blocks."""
    n, D = 300_000, 8
    g = torch.Generator(device=DEV).manual_seed(64)
    rnd = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    x, dt, B, C, A = rnd(n, 1, D), rnd(n, 1, D), rnd(n, 1, 1, 16), rnd(n, 1, 1, 16), -rnd(D, 16).abs()
    for m in (300_000, 262_000, 66_000):
        y, ht = lib.selective_scan_fwd(x[:m], dt[:m], A, B[:m], C[:m])
        tail = dict(x=x[m - 3:m], dt=dt[m - 3:m], A=A, B=B[m - 3:m], C=C[m - 3:m])
        y64, ht64 = ref.scan(ref.in_64_bits(tail))
        ref.close(y[-3:], y64, 74, "many y")
        ref.close(ht[-3:], ht64, 74, "many ht")
    w = rnd(D, 4)
    y, ht = lib.causal_conv_fwd(x, w)
    y64, ht64 = ref.conv(ref.in_64_bits(dict(x=x[-3:], weight=w)))
    ref.close(y[-3:], y64, 48, "many conv")
    assert torch.equal(ht[-3:].double().cpu(), ht64)


def test_scan_long_prompt_in_place(lib):
    """A single sequence long enough to be cut into chunks, its state given back in the buffer it came in."""
    t, _ = scan_inputs(torch.float32, B=1, T=1000, D=12, seed=12)
    y64, ht64 = ref.scan(ref.in_64_bits(t))
    state = t["h0"].clone()
    args = scan_args(t)
    args[-1] = state
    y, _ = lib.selective_scan_fwd(*args, ht=state)
    ok(lib)
    ref.close(y, y64, 10 * 1000 + 64, "long y")
    ref.close(state, ht64, 10 * 1000 + 64, "long ht")


def test_scan_total_forgetting(lib):
    """A = -inf forgets everything at each step, and keeps the state where delta is 0."""
    t, _ = scan_inputs(torch.float32, B=1, T=40, D=8, gate=False, h0=True, seed=13)
    t["A"][:] = float("-inf")
    y, ht = lib.selective_scan_fwd(*scan_args(t))
    t["A"][:] = -1e30
    y2, ht2 = lib.selective_scan_fwd(*scan_args(t))
    assert torch.isfinite(y).all() and torch.equal(y, y2) and torch.equal(ht, ht2)


@pytest.mark.parametrize("T", [2, 3, 15, 31, 33])
@pytest.mark.parametrize("D", [6, 7])
def test_scan_infinite_state_stays_infinite(lib, T, D):
    """An input that overflows leaves an infinity in its channel, whatever the length; the others stay finite."""
    t, _ = scan_inputs(torch.float32, B=1, T=T, D=D, gate=False, seed=14)
    t["x"][0, (T // 2) * 2 - 1, 3] = float("inf")  # the second token of the last whole pair
    y64, ht64 = ref.scan(ref.in_64_bits(t))
    y, ht = lib.selective_scan_fwd(*scan_args(t))
    ok(lib)
    assert torch.isinf(ht64[0, 3]).all()
    assert torch.equal(ht[0, 3].double().cpu(), ht64[0, 3])
    keep = [d for d in range(D) if d != 3]
    ref.close(y[:, :, keep], y64[:, :, keep], 10 * T + 64, "y of the others")
    ref.close(ht[:, keep], ht64[:, keep], 10 * T + 64, "ht of the others")


# ---- layer norm ------------------------------------------------------------------


def norm_inputs(dtype, rows, D, weight=True, bias=True, gate=False, seed=0):
    g = gen(seed)
    t = dict(x=normal(g, rows, D, dtype=dtype, scale=2.0) + 0.5, weight=normal(g, D) if weight else None,
             bias=normal(g, D) if bias else None, z=normal(g, rows, D, dtype=dtype, scale=2.0) if gate else None)
    return t, normal(g, rows, D, dtype=dtype)


def norm_check(lib, t, dy, rms, label):
    y = lib.layer_norm_fwd(t["x"], t["weight"], t["bias"], t["z"], rms=rms)
    leaves = ref.in_64_bits(t, grad=True)
    y64 = ref.norm(leaves, rms=rms)
    # a row of few columns can have a deviation far below its values: their ratio counts
    x = leaves["x"].detach()
    dev = torch.sqrt(((x if rms else x - x.mean(-1, keepdim=True)) ** 2).mean(-1) + 1e-5)
    ratio = float((x.abs().amax(-1) / dev).max()) if x.numel() else 1.0
    ref.close(y, y64, 128 * max(1.0, ratio), label + " y")
    out = lib.layer_norm_bwd(t["x"], t["weight"], t["bias"], t["z"], rms=rms, dy=dy)
    want = ref.gradients([y64], [dy], leaves)
    for name in ("x", "weight", "bias", "z"):
        if t[name] is None:
            assert out["d" + name] is None
            continue
        steps = (128 + (y.shape[0] if name in ("weight", "bias") else 0)) * max(1.0, ratio)
        w = want[name]
        # d_x is a difference of terms of the size of d r
        scale = float(w.abs().max()) if w.numel() else 1.0
        if name == "x" and w.numel():
            scale = max(scale, float((dy.double().cpu() / dev[:, None]).abs().max() * 4))
        ref.close(out["d" + name], w, steps, label + " d" + name, scale=scale)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("D", [1, 2, 3, 8, 31, 32, 33, 64, 100, 128, 129, 256, 257, 512, 520, 513, 1024, 2048, 2049,
                               4096, 5000, 8192, 8193, 16383, 16384])
def test_norm_sizes(lib, dtype, D):
    for rms, gate in ((False, True), (True, False)):
        t, dy = norm_inputs(dtype, 5, D, gate=gate, seed=D)
        if D == 1 and not rms:
            t["x"] = t["x"] * 0 + 1.0  # one column is its own mean
        norm_check(lib, t, dy, rms, "norm D=%d rms=%s" % (D, rms))


@pytest.mark.parametrize("rows", [1, 2, 7, 8, 9, 609, 5000])
def test_norm_rows(lib, rows):
    for D in (128, 40, 272):
        t, dy = norm_inputs(torch.bfloat16, rows, D, gate=True, seed=rows)
        norm_check(lib, t, dy, True, "norm rows=%d" % rows)


@pytest.mark.parametrize("weight,bias,gate,rms", [(False, False, False, False), (True, False, True, False),
                                                  (False, True, True, True), (False, False, True, True)])
def test_norm_options(lib, weight, bias, gate, rms):
    t, dy = norm_inputs(torch.float32, 33, 96, weight, bias, gate, seed=4)
    norm_check(lib, t, dy, rms, "norm options")


def test_norm_in_place(lib):
    t, dy = norm_inputs(torch.bfloat16, 19, 128, gate=True, seed=8)
    want = lib.layer_norm_fwd(t["x"], t["weight"], t["bias"], t["z"])
    x = t["x"].clone()
    assert lib.layer_norm_fwd(x, t["weight"], t["bias"], t["z"], y=x) is x
    assert torch.equal(x, want)


def test_norm_bad_row_stays_alone(lib):
    t, dy = norm_inputs(torch.float32, 6, 64, seed=2)
    clean = lib.layer_norm_fwd(t["x"], t["weight"], t["bias"])
    t["x"][2, 5] = float("nan")
    y = lib.layer_norm_fwd(t["x"], t["weight"], t["bias"])
    keep = [0, 1, 3, 4, 5]
    assert torch.equal(y[keep], clean[keep]) and torch.isnan(y[2]).all()


def test_norm_large_mean(lib):
    """The variance is taken about the mean: a mean of 1000 deviations costs no more than its own rounding."""
    t, dy = norm_inputs(torch.float32, 16, 512, seed=3)
    t["x"] = t["x"] + 2000.0
    norm_check(lib, t, dy, False, "norm mean")


# ---- empty calls, rows behind the last sequence, bad offsets -----------------------


def test_no_tokens(lib):
    """Without tokens the final state is the initial one and the parameters' gradients are zero."""
    for lengths in (None, [0, 0, 0]):
        t, grads = conv_inputs(torch.bfloat16, B=3, T=0, D=16, lengths=lengths, seed=1)
        cu = None if lengths is None else ref.offsets(lengths, DEV)
        y, ht = lib.causal_conv_fwd(t["x"], t["weight"], t["bias"], t["h0"], cu)
        assert y.numel() == 0 and torch.equal(ht, t["h0"])
        out = lib.causal_conv_bwd(t["x"], t["weight"], t["bias"], t["h0"], cu, dy=grads["dy"], dht=grads["dht"])
        assert not out["dweight"].any() and not out["dbias"].any() and torch.equal(out["dh0"], grads["dht"])
        t, grads = scan_inputs(torch.bfloat16, B=3, T=0, D=16, lengths=lengths, seed=1)
        y, ht = lib.selective_scan_fwd(*scan_args(t), cu)
        assert y.numel() == 0 and torch.equal(ht, t["h0"])
        out = lib.selective_scan_bwd(*scan_args(t), cu, dy=grads["dy"], dht=grads["dht"])
        assert not out["dA"].any() and not out["dD"].any() and torch.equal(out["dh0"], grads["dht"])
    t, dy = norm_inputs(torch.float32, 0, 24, gate=True)
    assert lib.layer_norm_fwd(t["x"], t["weight"], t["bias"], t["z"]).numel() == 0
    out = lib.layer_norm_bwd(t["x"], t["weight"], t["bias"], t["z"], dy=dy)
    assert not out["dweight"].any() and not out["dbias"].any()
    ok(lib)


def test_no_sequences(lib):
    cu = torch.zeros(1, dtype=torch.int64, device=DEV)
    t, grads = conv_inputs(torch.float32, D=8, lengths=[], pad=4, seed=1)
    y, ht = lib.causal_conv_fwd(t["x"], t["weight"], t["bias"], None, cu)
    assert ht.shape == (0, 3, 8)
    out = lib.causal_conv_bwd(t["x"], t["weight"], t["bias"], None, cu, dy=grads["dy"])
    assert not out["dweight"].any()
    t, grads = scan_inputs(torch.float32, D=8, lengths=[], h0=False, pad=4, seed=1)
    lib.selective_scan_fwd(*scan_args(t), cu)
    out = lib.selective_scan_bwd(*scan_args(t), cu, dy=grads["dy"])
    assert not out["dA"].any() and not out["ddt_bias"].any()
    ok(lib)


def test_rows_behind_the_last_sequence_are_left(lib):
    lengths, pad, D = [3, 70], 9, 40
    cu = ref.offsets(lengths, DEV)
    t, grads = conv_inputs(torch.bfloat16, D=D, lengths=lengths, pad=pad, seed=1)
    y = torch.full_like(t["x"], 7.0)
    lib.causal_conv_fwd(t["x"], t["weight"], t["bias"], t["h0"], cu, y=y)
    assert (y[:, 73:] == 7).all() and not (y[:, :73] == 7).all()
    t, grads = scan_inputs(torch.bfloat16, D=D, lengths=lengths, pad=pad, seed=1)
    y = torch.full_like(t["x"], 7.0)
    lib.selective_scan_fwd(*scan_args(t), cu, y=y)
    assert (y[:, 73:] == 7).all()
    ok(lib)


@pytest.mark.parametrize("dtype", DTYPES)
def test_gradients_behind_the_last_sequence_are_left(lib, dtype):
    """The gradients' rows there keep what they held, and no value of x or dy there counts."""
    lengths, pad, D, W, N = [3, 0, 70], 9, 40, 4, 16
    used, T = sum(lengths), sum(lengths) + pad
    cu = ref.offsets(lengths, DEV)
    c, code, raw = len(lengths), lib.dtype_code(dtype), lib.load()

    def ptr(x):
        return x.data_ptr()

    def left(*outs):
        for o in outs:
            assert (o[:, used:] == 7).all() and torch.isfinite(o[:, :used]).all() and not (o[:, :used] == 7).all()

    stream = torch.cuda.current_stream().cuda_stream
    t, grads = conv_inputs(dtype, D=D, lengths=lengths, pad=pad, seed=2)
    t["x"][:, used:] = float("nan")
    grads["dy"][:, used:] = float("inf")
    dx = torch.full_like(t["x"], 7.0)
    dw, db, dh0 = torch.empty_like(t["weight"]), torch.empty_like(t["bias"]), torch.empty_like(t["h0"])
    n = raw.dn_causal_conv_bwd_workspace_bytes(c, 1, T, D, W, code)
    space = torch.empty(n, dtype=torch.uint8, device=DEV)
    assert raw.dn_causal_conv_bwd(
        ptr(t["x"]), ptr(t["weight"]), ptr(t["bias"]), ptr(t["h0"]), ptr(cu), c, 1, T, D, W, code, 1,
        ptr(grads["dy"]), code, ptr(grads["dht"]), ptr(dx), ptr(dw), ptr(db), ptr(dh0), ptr(space), n,
        stream) == lib.DN_OK
    left(dx)
    assert all(torch.isfinite(v).all() for v in (dw, db, dh0))
    t, grads = scan_inputs(dtype, D=D, N=N, lengths=lengths, pad=pad, seed=2)
    for name in ("x", "dt", "B", "C", "z"):
        t[name][:, used:] = float("nan")
    grads["dy"][:, used:] = float("inf")
    rows = {k: torch.full_like(t[k], 7.0) for k in ("x", "dt", "B", "C", "z")}
    sums = {k: torch.empty_like(t[k]) for k in ("A", "D", "dt_bias", "h0")}
    n = raw.dn_selective_scan_bwd_workspace_bytes(c, 1, T, D, 1, N, code)
    space = torch.empty(n, dtype=torch.uint8, device=DEV)
    assert raw.dn_selective_scan_bwd(
        *[ptr(t[k]) for k in NAMES], ptr(cu), c, 1, T, D, 1, N, code, 1, ptr(grads["dy"]), ptr(grads["dht"]),
        ptr(rows["x"]), ptr(rows["dt"]), ptr(sums["A"]), ptr(rows["B"]), ptr(rows["C"]), ptr(sums["D"]),
        ptr(rows["z"]), ptr(sums["dt_bias"]), ptr(sums["h0"]), ptr(space), n, stream) == lib.DN_OK
    left(*rows.values())
    assert all(torch.isfinite(v).all() for v in sums.values())
    ok(lib)


@pytest.mark.parametrize("bad", [[0, 5, 3, 20], [1, 5, 9, 20], [0, 5, 9, 21], [0, 30, 31, 20], [-4, 5, 9, 20]])
def test_malformed_offsets_are_reported(lib, bad):
    """Offsets that decrease, do not begin at 0 or pass the tensor: no access leaves the tensors."""
    cu = torch.tensor(bad, dtype=torch.int64, device=DEV)
    t, grads = conv_inputs(torch.float32, D=8, lengths=[10, 5, 5], seed=1)
    lib.causal_conv_fwd(t["x"], t["weight"], t["bias"], t["h0"], cu)
    assert lib.dn_check() == lib.DN_ERR_DEVICE_ARG
    lib.causal_conv_bwd(t["x"], t["weight"], t["bias"], t["h0"], cu, dy=grads["dy"])
    assert lib.dn_check() == lib.DN_ERR_DEVICE_ARG
    t, grads = scan_inputs(torch.float32, D=8, lengths=[10, 5, 5], seed=1)
    lib.selective_scan_fwd(*scan_args(t), cu)
    assert lib.dn_check() == lib.DN_ERR_DEVICE_ARG
    lib.selective_scan_bwd(*scan_args(t), cu, dy=grads["dy"])
    assert lib.dn_check() == lib.DN_ERR_DEVICE_ARG
    assert lib.dn_check() == lib.DN_OK


# ---- differences, streams, graphs, repeated bits -------------------------------------


def directional(f, leaves, grads, eps):
    """(f(x + eps v) - f(x - eps v)) / 2 eps and <grad, v> for one direction v over all leaves."""
    v = {k: torch.randn(t.shape, generator=gen(77)).to(t) for k, t in leaves.items()}
    up = f({k: t + eps * v[k] for k, t in leaves.items()})
    down = f({k: t - eps * v[k] for k, t in leaves.items()})
    return (up - down) / (2 * eps), sum((grads["d" + k].double() * v[k].double()).sum().item() for k in leaves)


def test_gradients_against_differences(lib):
    """Central differences of the fp32 forwards.  With steps of 2^-8 the quotient is off by the third
    derivative (2^-16 of it, of the order of the gradient's own size) and by the forwards' rounding
    (each of the n outputs within 2^-20, added at random: 2^-20 sqrt(n) / 2^-8 = 2^-12 sqrt(n) against
    a quotient of the order of sqrt(n)): 1 % of the larger of the quotient and sqrt(n) covers both."""
    eps = 2.0 ** -8

    def check(num, ana, n):
        assert abs(num - ana) <= 0.01 * max(abs(num), n ** 0.5), (num, ana)

    t, g = conv_inputs(torch.float32, B=1, T=33, D=12, seed=21)
    out = lib.causal_conv_bwd(t["x"], t["weight"], t["bias"], t["h0"], dy=g["dy"], dht=g["dht"])

    def f(l):
        y, ht = lib.causal_conv_fwd(l["x"], l["weight"], l["bias"], l["h0"])
        return ((y.double() * g["dy"]).sum() + (ht.double() * g["dht"]).sum()).item()

    check(*directional(f, t, out, eps), t["x"].numel())

    t, g = scan_inputs(torch.float32, B=1, T=80, D=12, seed=22)
    t["z"] = t["z"] * 0.5
    out = lib.selective_scan_bwd(*scan_args(t), dy=g["dy"], dht=g["dht"])

    def f(l):
        y, ht = lib.selective_scan_fwd(*scan_args(l))
        return ((y.double() * g["dy"]).sum() + (ht.double() * g["dht"]).sum()).item()

    small = 2.0 ** -10  # the scan bends more strongly
    check(*directional(f, t, out, small), t["x"].numel() * 16)

    t, dy = norm_inputs(torch.float32, 9, 48, gate=True, seed=23)
    out = lib.layer_norm_bwd(t["x"], t["weight"], t["bias"], t["z"], dy=dy)
    check(*directional(lambda l: (lib.layer_norm_fwd(l["x"], l["weight"], l["bias"], l["z"]).double() * dy).sum().item(),
                       t, out, eps), t["x"].numel())


def all_calls(lib, seed):
    """One call of every entry point on inputs of this seed: a function that makes them and returns the outputs."""
    lengths = [70, 0, 33, 200]
    cu = ref.offsets(lengths, DEV)
    c, cg = conv_inputs(torch.bfloat16, D=48, lengths=lengths, seed=seed)
    s, sg = scan_inputs(torch.bfloat16, D=48, lengths=lengths, seed=seed)
    n, ndy = norm_inputs(torch.bfloat16, 303, 128, gate=True, seed=seed)

    def go():
        outs = list(lib.causal_conv_fwd(c["x"], c["weight"], c["bias"], c["h0"], cu))
        outs += lib.causal_conv_bwd(c["x"], c["weight"], c["bias"], c["h0"], cu, dy=cg["dy"], dht=cg["dht"]).values()
        outs += lib.selective_scan_fwd(*scan_args(s), cu)
        outs += lib.selective_scan_bwd(*scan_args(s), cu, dy=sg["dy"], dht=sg["dht"]).values()
        outs.append(lib.layer_norm_fwd(n["x"], n["weight"], n["bias"], n["z"]))
        outs += lib.layer_norm_bwd(n["x"], n["weight"], n["bias"], n["z"], dy=ndy).values()
        return outs

    return go, (c, s, n)


def same(a, b):
    assert len(a) == len(b)
    return all(torch.equal(x, y) for x, y in zip(a, b))


def test_calls_repeat_bit_for_bit(lib):
    go, _ = all_calls(lib, 31)
    assert same(go(), go())


def test_calls_on_two_streams_at_once(lib):
    go1, _ = all_calls(lib, 32)
    go2, _ = all_calls(lib, 33)
    want1, want2 = go1(), go2()
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(3):
        with torch.cuda.stream(s1):
            got1 = go1()
        with torch.cuda.stream(s2):
            got2 = go2()
        torch.cuda.synchronize()
        assert same(got1, want1) and same(got2, want2)


def test_calls_given_a_stream(lib):
    """The stream is an argument; the workspace that a call makes for itself outlives the call there."""
    lengths = [70, 0, 33, 200]
    cu = ref.offsets(lengths, DEV)
    s, sg = scan_inputs(torch.bfloat16, D=48, lengths=lengths, seed=35)
    n, ndy = norm_inputs(torch.bfloat16, 303, 128, seed=35)

    def go(stream):
        outs = list(lib.selective_scan_fwd(*scan_args(s), cu, stream=stream))
        outs += lib.selective_scan_bwd(*scan_args(s), cu, dy=sg["dy"], stream=stream).values()
        outs += lib.layer_norm_bwd(n["x"], n["weight"], n["bias"], dy=ndy, stream=stream).values()
        return [o for o in outs if o is not None]

    want = go(None)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream):
        got = go(stream)
        junk = [torch.full((1 << 20,), 7, dtype=torch.uint8, device=DEV) for _ in range(20)]  # the caller's own stream goes on
        torch.cuda.synchronize()
        assert same(got, want)
        del junk


def test_calls_captured_and_replayed(lib):
    go, (c, s, n) = all_calls(lib, 34)
    go()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        with torch.cuda.graph(graph, stream=stream):
            held = go()
    torch.cuda.current_stream().wait_stream(stream)
    for t in (c, s, n):
        t["x"].mul_(0.5)
    graph.replay()
    torch.cuda.synchronize()
    want = go()
    torch.cuda.synchronize()
    assert same(held, want)
    ok(lib)


# ---- used together -------------------------------------------------------------------


@pytest.mark.parametrize("lengths", [None, [100, 0, 29, 71]])
def test_gated_delta_layer(lib, lengths):
    """q, k and v through the convolution, the gated delta rule, the gated norm of its heads; and back.

    The recurrence between them is held to its own bound (bf16: 5e-3 of the norm of its outputs), so the
    chain is compared stage by stage on the stages' own inputs, and end to end at three such bounds."""
    from oracle import recurrent
    H, d, D = 2, 64, 128
    t, _ = conv_inputs(torch.bfloat16, B=2, T=100, D=3 * D, lengths=lengths, seed=41)
    B, T, _ = t["x"].shape
    cu = None if lengths is None else ref.offsets(lengths, DEV)
    mixed, _ = lib.causal_conv_fwd(t["x"], t["weight"], t["bias"], t["h0"], cu)
    q, k, v = (mixed[..., i * D:(i + 1) * D].reshape(B, T, H, d).contiguous() for i in range(3))
    g = gen(42)
    beta = torch.sigmoid(torch.randn(B, T, H, generator=g)).to(DEV)
    decay = torch.nn.functional.logsigmoid(3 + torch.randn(B, T, H, generator=g)).to(DEV)
    o, _ = lib.chunk_fwd(q, k, v, beta, decay, None, cu, use_qk_l2norm_in_kernel=True)
    z = normal(g, B, T, H, d, dtype=torch.bfloat16)
    weight = 1 + normal(g, d, scale=0.1)
    y = lib.layer_norm_fwd(o, weight, None, z, rms=True)
    ok(lib)

    c64, _ = ref.conv(ref.in_64_bits(t), lengths)
    qkv = [c64[..., i * D:(i + 1) * D].reshape(B, T, H, d) for i in range(3)]
    cu_cpu = None if cu is None else cu.cpu()
    o64, _ = recurrent(*qkv, beta.cpu(), decay.cpu(), None, cu_cpu, d ** -0.5, use_qk_l2norm_in_kernel=True)
    y64 = ref.norm(dict(x=torch.from_numpy(o64), weight=weight.double().cpu(), z=z.double().cpu()), rms=True)
    rel = float((y.double().cpu() - y64).norm() / y64.norm())
    assert rel <= 3 * 5e-3, rel

    dy = normal(g, B, T, H, d, dtype=torch.bfloat16)
    back = lib.layer_norm_bwd(o, weight, None, z, rms=True, dy=dy)
    grads = lib.chunk_bwd(q, k, v, beta, decay, None, cu, do=back["dx"], use_qk_l2norm_in_kernel=True)
    dmixed = torch.cat([grads[n].reshape(B, T, D) for n in ("dq", "dk", "dv")], -1)  # fp32
    out = lib.causal_conv_bwd(t["x"], t["weight"], t["bias"], t["h0"], cu, dy=dmixed)
    ok(lib)
    assert all(torch.isfinite(x.float()).all() for x in out.values())
    leaves = ref.in_64_bits(t, grad=True)
    want = ref.gradients(ref.conv(leaves, lengths), [dmixed, None], leaves)
    for name in ("x", "weight", "bias", "h0"):
        ref.close(out["d" + name], want[name], 4 * 4 + 32 + B * T, "layer d" + name,
                  scale=max(float(want[name].abs().max()), float(dmixed.abs().max()) * 4))


def test_scan_layer_prompt_then_tokens(lib):
    """Convolution, scan and norm over a prompt and then token by token, states carried in place, against
    the same layer over all tokens at once in 64 bits."""
    B, T, P, D, N = 2, 50, 40, 32, 16
    c, _ = conv_inputs(torch.float32, B=B, T=T, D=D, seed=51)
    s, _ = scan_inputs(torch.float32, B=B, T=T, D=D, N=N, seed=52)
    weight = normal(gen(53), D)
    conv_state, scan_state = c["h0"].clone(), s["h0"].clone()
    ys = []
    for lo, hi in [(0, P)] + [(i, i + 1) for i in range(P, T)]:
        u, _ = lib.causal_conv_fwd(c["x"][:, lo:hi].contiguous(), c["weight"], c["bias"], conv_state, ht=conv_state)
        cut = {k: s[k][:, lo:hi].contiguous() for k in ("dt", "B", "C", "z")}
        y, _ = lib.selective_scan_fwd(u, cut["dt"], s["A"], cut["B"], cut["C"], s["D"], cut["z"], s["dt_bias"],
                                      scan_state, ht=scan_state)
        ys.append(lib.layer_norm_fwd(y, weight))
    ok(lib)
    u64, cs64 = ref.conv(ref.in_64_bits(c))
    y64, ss64 = ref.scan(dict(ref.in_64_bits(s), x=u64))
    dev = y64.std(-1, unbiased=False).min().item()
    want = ref.norm(dict(x=y64, weight=weight.double().cpu()))
    ratio = max(1.0, float(y64.abs().max()) / dev)
    ref.close(scan_state, ss64, 10 * T + 128, "layer state")
    assert torch.equal(conv_state.double().cpu(), cs64)
    ref.close(torch.cat(ys, 1), want, (10 * T + 256) * ratio, "layer y")


# ---- more than 2^31 elements ------------------------------------------------------------


def test_conv_beyond_32_bits(lib):
    """The last tokens of 600000 x 4096 elements."""
    T, D, n = 600_000, 4096, 40
    g = torch.Generator(device=DEV).manual_seed(61)
    x = torch.randn(1, T, D, generator=g, device=DEV, dtype=torch.bfloat16)
    dy = torch.randn(1, T, D, generator=g, device=DEV, dtype=torch.bfloat16)
    w = torch.randn(D, 4, generator=g, device=DEV)
    y, ht = lib.causal_conv_fwd(x, w)
    assert torch.equal(ht, x[:, -3:])
    out = lib.causal_conv_bwd(x, w, dy=dy)
    leaves = ref.in_64_bits(dict(x=x[:, -n - 3:], weight=w), grad=True)
    y64, _ = ref.conv(leaves)
    terms = float(x[:, -n:].abs().max()) * float(w.abs().sum(1).max())
    ref.close(y[:, -n:], y64[:, 3:], 48, "long conv y", scale=terms)
    grad = ref.gradients([y64], [torch.cat([torch.zeros_like(dy[:, :3]), dy[:, -n:]], 1)], leaves)["x"]
    ref.close(out["dx"][:, -n:], grad[:, 3:], 48, "long conv dx", scale=max(terms, float(grad.abs().max())))
    ok(lib)


def test_norm_beyond_32_bits(lib):
    """The last rows of 1100000 x 2048 elements."""
    rows, D, n = 1_100_000, 2048, 5
    g = torch.Generator(device=DEV).manual_seed(62)
    x = torch.randn(rows, D, generator=g, device=DEV, dtype=torch.bfloat16)
    w = torch.randn(D, generator=g, device=DEV)
    y = lib.layer_norm_fwd(x, w)
    leaves = ref.in_64_bits(dict(x=x[-n:], weight=w), grad=True)
    y64 = ref.norm(leaves)
    ref.close(y[-n:], y64, 128 * 6, "long norm y")
    out = lib.layer_norm_bwd(x, w, dy=y)
    grad = ref.gradients([y64], [y[-n:]], leaves)["x"]
    ref.close(out["dx"][-n:], grad, 128 * 6, "long norm dx", scale=float((y[-n:].abs().max() * w.abs().max()) * 4))


def test_scan_beyond_32_bits(lib):
    """The last tokens of 1100000 x 2048 elements, whose states forget within a few of them: the decay of a
    token is at most e^-4, that of the 24 tokens before those compared below e^-96."""
    T, D, N, n = 1_100_000, 2048, 16, 48
    g = torch.Generator(device=DEV).manual_seed(63)
    x = torch.randn(1, T, D, generator=g, device=DEV, dtype=torch.bfloat16)
    dt = (1 + torch.rand(1, T, D, generator=g, device=DEV)).bfloat16()
    A = -4 - torch.rand(D, N, generator=g, device=DEV)
    B = torch.randn(1, T, 1, N, generator=g, device=DEV, dtype=torch.bfloat16)
    C = torch.randn(1, T, 1, N, generator=g, device=DEV, dtype=torch.bfloat16)
    y, ht = lib.selective_scan_fwd(x, dt, A, B, C, dt_softplus=False)
    tail = dict(x=x[:, -n:], dt=dt[:, -n:], A=A, B=B[:, -n:], C=C[:, -n:])
    leaves = ref.in_64_bits(tail, grad=True)
    y64, ht64 = ref.scan(leaves, softplus=False)
    keep = n - 24
    ref.close(y[:, -keep:], y64[:, -keep:], 10 * n + 64, "long scan y")
    ref.close(ht, ht64, 10 * n + 64, "long scan ht")
    dy = y
    out = lib.selective_scan_bwd(x, dt, A, B, C, dt_softplus=False, dy=dy)
    grads = ref.gradients([y64], [dy[:, -n:]], leaves)
    for name in ("x", "dt", "B", "C"):
        ref.close(out["d" + name][:, -keep:], grads[name][:, -keep:], 30 * n + 64 + D, "long scan d" + name)
    ok(lib)
