"""Cases of the operators that stand around the gated delta rule in a layer.

Three operators, each forward and backward:

* the short causal convolution that q, k and v (or x) pass before a recurrence;
* the selective state space scan, for prompts and for single tokens;
* layer norm, with its root-mean-square form and its output gate.

A case is a dict of plain values.  ``prepare`` draws its inputs on the GPU,
``run`` makes one pass, ``exact`` evaluates the definition in 64 bits.
"""
import math
import random

import torch

# False: the plain form below, in torch; True: the framework's entry points.
own = False

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def listed():
    return [
        # one decoding step of 64 sequences: q, k and v of 16 heads of 128 side by side, tap state in and out
        dict(name="conv decode b64", op="conv_fwd", dtype="bf16", B=64, T=1, packed=0, D=6144, W=4, silu=True, h0=True),
        # the prompts of 8 requests packed: q, k of 8 heads and v of 32, ragged lengths up to 4096
        dict(name="conv packed prompts", op="conv_fwd", dtype="bf16", B=1, T=4096, packed=8, D=6144, W=4, silu=True, h0=False),
        # a training step's backward of that convolution at the headline's batch
        dict(name="conv training", op="conv_bwd", dtype="bf16", B=4, T=2048, packed=0, D=6144, W=4, silu=True, h0=False),
        # an fp32 fine-tuning step over packed samples, odd channel count
        dict(name="conv training odd fp32", op="conv_bwd", dtype="fp32", B=1, T=700, packed=9, D=1001, W=3, silu=True, h0=True),
        # one decoding step of 64 sequences
        dict(name="scan decode b64", op="scan_fwd", dtype="bf16", B=64, T=1, packed=0, D=2048, N=16, G=1, gate=True, h0=True),
        # prompts at the headline's batch and length
        dict(name="scan prompts", op="scan_fwd", dtype="bf16", B=4, T=2048, packed=0, D=2048, N=16, G=1, gate=True, h0=False),
        # a training step at the headline's batch and length
        dict(name="scan training", op="scan_bwd", dtype="bf16", B=4, T=2048, packed=0, D=2048, N=16, G=1, gate=True, h0=False),
        # packed samples in fp32: two groups, wider states, carried states, no gate
        dict(name="scan training ragged fp32", op="scan_bwd", dtype="fp32", B=1, T=600, packed=7, D=1010, N=32, G=2, gate=False, h0=True),
        # the gated root-mean-square norm of every head's output, at the headline's batch
        dict(name="norm heads gated", op="norm_fwd", dtype="bf16", rows=131072, D=128, rms=True, gate=True, bias=False),
        # layer norm of a few rows of the model's width, as in decoding
        dict(name="norm decode", op="norm_fwd", dtype="bf16", rows=64, D=2048, rms=False, gate=False, bias=True),
        # backward of the gated norm of the heads
        dict(name="norm heads training", op="norm_bwd", dtype="bf16", rows=131072, D=128, rms=True, gate=True, bias=False),
        # backward of a wide layer norm, odd rows
        dict(name="norm wide training", op="norm_bwd", dtype="bf16", rows=16383, D=4096, rms=False, gate=False, bias=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """One more case: any operator, sizes spread over their logarithm, odd ones among them."""
    op = rng.choice(["conv_fwd", "conv_bwd", "scan_fwd", "scan_bwd", "norm_fwd", "norm_bwd"])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    if op.startswith("norm"):
        D = rng.choice([_log(rng, 1, 16384), 64 * rng.randint(1, 128), 1 << rng.randint(4, 13)])
        rows = _log(rng, 1, max(2, min(200000, (1 << (25 if dtype == "bf16" else 24)) // D)))
        return dict(op=op, dtype=dtype, rows=rows, D=D, rms=rng.random() < 0.5, gate=rng.random() < 0.5, bias=rng.random() < 0.5)
    packed = rng.choice([0, rng.randint(1, 24)])
    if op.startswith("conv"):
        D = rng.choice([_log(rng, 1, 8192), 64 * rng.randint(1, 128)])
        most = 1 << (25 if dtype == "bf16" else 24)
    else:
        N = rng.choice([16, 16, 16, 32, 64, 128])
        G = rng.choice([1, 1, 2, 4])
        D = G * rng.choice([_log(rng, 1, 4096 // G), 32 * rng.randint(1, 128 // G)])
        most = (1 << (24 if dtype == "bf16" else 23)) * 16 // N
    seqs = packed or rng.choice([1, 2, 4, rng.randint(1, 64)])
    T = rng.choice([1, _log(rng, 1, 4096), _log(rng, 16, 4096)])
    T = max(1, min(T, most // (D * seqs)))
    case = dict(op=op, dtype=dtype, B=1 if packed else seqs, T=T, packed=packed, D=D)
    if op.startswith("conv"):
        return dict(case, W=rng.choice([2, 3, 4, 4]), silu=rng.random() < 0.8, h0=rng.random() < 0.5)
    return dict(case, N=N, G=G, gate=rng.random() < 0.6, h0=rng.random() < 0.5)


def lengths(case):
    """Tokens of each sequence: B of T each, or `packed` ones of 1 to T drawn from the case's own sizes."""
    if not case["packed"]:
        return [case["T"]] * case["B"]
    rng = random.Random("%d %d %d" % (case["packed"], case["T"], case["D"]))
    return [rng.randint(1, case["T"]) for _ in range(case["packed"])]


# ---- inputs ---------------------------------------------------------------------------------------------------------


def inputs(case, seed):
    """The tensors of a case, by the names of the entry points' arguments."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def normal(*shape, dtype=dt, scale=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)

    f32 = torch.float32
    D = case["D"]
    if case["op"].startswith("norm"):
        rows = case["rows"]
        t = dict(x=normal(rows, D, scale=1.5) + 0.25, weight=1 + normal(D, dtype=f32, scale=0.1),
                 bias=normal(D, dtype=f32, scale=0.1) if case["bias"] else None,
                 z=normal(rows, D) if case["gate"] else None)
        if case["op"] == "norm_bwd":
            t["dy"] = normal(rows, D)
        return t
    lens = lengths(case)
    n, tokens = len(lens), sum(lens)
    B, T = (1, tokens) if case["packed"] else (case["B"], case["T"])
    cu = None
    if case["packed"]:
        cu = torch.tensor([0] + lens, dtype=torch.int64, device="cuda").cumsum(0)
    if case["op"].startswith("conv"):
        W = case["W"]
        t = dict(x=normal(B, T, D), weight=normal(D, W, dtype=f32, scale=W ** -0.5), bias=normal(D, dtype=f32, scale=0.1),
                 h0=normal(n, W - 1, D) if case["h0"] else None, cu_seqlens=cu)
        if case["op"] == "conv_bwd":
            t.update(dy=normal(B, T, D), dht=normal(n, W - 1, D) if case["h0"] else None)
        return t
    N, G = case["N"], case["G"]
    step = torch.exp(torch.empty(D, device="cuda").uniform_(math.log(1e-3), math.log(0.1), generator=g))
    t = dict(x=normal(B, T, D), dt=normal(B, T, D, scale=0.5),
             A=-torch.arange(1, N + 1, device="cuda", dtype=f32).repeat(D, 1) * (1 + 0.05 * normal(D, N, dtype=f32)),
             B=normal(B, T, G, N), C=normal(B, T, G, N), D=1 + normal(D, dtype=f32, scale=0.1),
             z=normal(B, T, D) if case["gate"] else None,
             dt_bias=step + torch.log(-torch.expm1(-step)),  # softplus of it is the step
             h0=normal(n, D, N, dtype=f32, scale=0.1) if case["h0"] else None, cu_seqlens=cu)
    if case["op"] == "scan_bwd":
        t.update(dy=normal(B, T, D), dht=normal(n, D, N, dtype=f32, scale=0.1) if case["h0"] else None)
    return t


def prepare(case, seed):
    t = inputs(case, seed)
    x = t["x"]
    state = dict(case=case, t=t)
    # the outputs of a step belong to the program: it gives the same buffers to each call
    if case["op"].endswith("fwd"):
        state["y"] = torch.empty_like(x)
        if case["op"] == "conv_fwd":
            state["ht"] = torch.empty(len(lengths(case)), case["W"] - 1, case["D"], dtype=x.dtype, device="cuda")
        if case["op"] == "scan_fwd":
            state["ht"] = torch.empty(len(lengths(case)), case["D"], case["N"], dtype=torch.float32, device="cuda")
    if not case["op"].startswith("norm"):
        # where the plain form finds each sequence: offsets, and the sequence of each token
        lens = torch.tensor(lengths(case), device="cuda")
        state["offsets"] = torch.cat([torch.zeros(1, dtype=torch.int64, device="cuda"), lens.cumsum(0)])
        state["of"] = torch.repeat_interleave(torch.arange(lens.numel(), device="cuda"), lens)
        state["longest"] = max(lengths(case))
    return state


# ---- one pass -------------------------------------------------------------------------------------------------------


def run(state):
    case, t = state["case"], state["t"]
    if own:
        return _run_own(case, t, state)
    return {"conv_fwd": _conv_fwd, "conv_bwd": _conv_bwd, "scan_fwd": _scan_fwd, "scan_bwd": _scan_bwd,
            "norm_fwd": _norm_fwd, "norm_bwd": _norm_bwd}[case["op"]](case, t, state)


def _run_own(case, t, state):
    import chunkwise_gated_delta_chunk_gb300 as dn

    op = case["op"]
    if op == "conv_fwd":
        return dn.causal_conv_fwd(t["x"], t["weight"], t["bias"], t["h0"], t["cu_seqlens"], silu=case["silu"],
                                  y=state["y"], ht=state["ht"])
    if op == "conv_bwd":
        return dn.causal_conv_bwd(t["x"], t["weight"], t["bias"], t["h0"], t["cu_seqlens"], silu=case["silu"],
                                  dy=t["dy"], dht=t["dht"])
    if op == "scan_fwd":
        return dn.selective_scan_fwd(t["x"], t["dt"], t["A"], t["B"], t["C"], t["D"], t["z"], t["dt_bias"], t["h0"],
                                     t["cu_seqlens"], dt_softplus=True, y=state["y"], ht=state["ht"])
    if op == "scan_bwd":
        return dn.selective_scan_bwd(t["x"], t["dt"], t["A"], t["B"], t["C"], t["D"], t["z"], t["dt_bias"], t["h0"],
                                     t["cu_seqlens"], dt_softplus=True, dy=t["dy"], dht=t["dht"])
    if op == "norm_fwd":
        return dn.layer_norm_fwd(t["x"], t["weight"], t["bias"], t["z"], eps=1e-5, rms=case["rms"], y=state["y"])
    return dn.layer_norm_bwd(t["x"], t["weight"], t["bias"], t["z"], eps=1e-5, rms=case["rms"], dy=t["dy"])


# ---- the plain forms: elementary torch in 32 bits ------------------------------------------------------------------------


def _silu(u):
    return u / (1 + torch.exp(-u))


def _silu_grad(u):
    s = 1 / (1 + torch.exp(-u))
    return s * (1 + u * (1 - s))


def _extended(case, x, h0, state):
    """Each sequence's W - 1 earlier inputs and then its tokens, one sequence after the other; and the row of each token."""
    W, D = case["W"], case["D"]
    n = state["offsets"].numel() - 1
    at = torch.arange(x.shape[0], device=x.device) + (state["of"] + 1) * (W - 1)
    ext = torch.zeros(x.shape[0] + n * (W - 1), D, device=x.device)
    ext[at] = x
    first = state["offsets"][:-1] + torch.arange(n, device=x.device) * (W - 1)
    early = first[:, None] + torch.arange(W - 1, device=x.device)
    if h0 is not None:
        ext[early] = h0
    return ext, at, early


def _conv_pre(case, t, state):
    x = t["x"].float().reshape(-1, case["D"])
    ext, at, early = _extended(case, x, None if t["h0"] is None else t["h0"].float(), state)
    taps = ext.unfold(0, case["W"], 1)[at - (case["W"] - 1)]  # [tokens, D, W]
    return ext, at, early, taps, (taps * t["weight"]).sum(-1) + t["bias"]


def _conv_fwd(case, t, state):
    ext, at, early, _, u = _conv_pre(case, t, state)
    y = _silu(u) if case["silu"] else u
    last = early + (state["offsets"][1:] - state["offsets"][:-1])[:, None]
    return y.to(t["x"].dtype).reshape(t["x"].shape), ext[last].to(t["x"].dtype)


def _conv_bwd(case, t, state):
    ext, at, early, taps, u = _conv_pre(case, t, state)
    dy = t["dy"].float().reshape(-1, case["D"])
    du = dy * _silu_grad(u) if case["silu"] else dy
    dpad = torch.zeros(ext.shape[0] + case["W"] - 1, case["D"], device=ext.device)
    dpad[at] = du
    dext = (dpad.unfold(0, case["W"], 1) * t["weight"].flip(1)).sum(-1)
    if t["dht"] is not None:
        last = early + (state["offsets"][1:] - state["offsets"][:-1])[:, None]
        dext[last] += t["dht"].float()
    out = dict(dx=dext[at].to(t["x"].dtype).reshape(t["x"].shape),
               dweight=(taps * du[:, :, None]).double().sum(0).float(), dbias=du.double().sum(0).float(), dh0=None)
    if t["h0"] is not None:
        out["dh0"] = dext[early].to(t["x"].dtype)
    return out


def _softplus(v):
    return torch.clamp(v, min=0) + torch.log1p(torch.exp(-torch.abs(v)))


def _scanned(a, b, longest):
    """h[t] = a[t] h[t-1] + b[t] along dimension 0, in doubling steps; a is 0 where a sequence begins."""
    k = 1
    while k < longest:  # log2(longest) steps
        b = torch.cat([b[:k], b[k:] + a[k:] * b[:-k]])
        if 2 * k < longest:
            a = torch.cat([a[:k], a[k:] * a[:-k]])
        k *= 2
    return b


def _scan_states(case, t, state):
    """The scan's terms and its states [tokens, D, N]."""
    D, N, G = case["D"], case["N"], case["G"]
    x = t["x"].float().reshape(-1, D)
    raw = t["dt"].float().reshape(-1, D) + t["dt_bias"]
    delta = _softplus(raw)
    Bm = t["B"].float().reshape(-1, G, N).repeat_interleave(D // G, 1)
    Cm = t["C"].float().reshape(-1, G, N).repeat_interleave(D // G, 1)
    decay = torch.exp(delta[:, :, None] * t["A"])
    add = (delta * x)[:, :, None] * Bm
    first = state["offsets"][:-1]
    seen = decay.clone()
    if t["h0"] is not None:
        add[first] += decay[first] * t["h0"]
    seen[first] = 0
    return x, raw, delta, Bm, Cm, decay, _scanned(seen, add, state["longest"])


def _scan_fwd(case, t, state):
    x, _, _, _, Cm, _, h = _scan_states(case, t, state)
    y = (h * Cm).sum(-1) + t["D"] * x
    if t["z"] is not None:
        y = y * _silu(t["z"].float().reshape(y.shape))
    return y.to(t["x"].dtype).reshape(t["x"].shape), h[state["offsets"][1:] - 1]


def _scan_bwd(case, t, state):
    D, N, G = case["D"], case["N"], case["G"]
    x, raw, delta, Bm, Cm, decay, h = _scan_states(case, t, state)
    dy = t["dy"].float().reshape(-1, D)
    dtype, shape = t["x"].dtype, t["x"].shape
    out = dict(dz=None, dh0=None)
    if t["z"] is not None:
        z = t["z"].float().reshape(-1, D)
        out["dz"] = (dy * ((h * Cm).sum(-1) + t["D"] * x) * _silu_grad(z)).to(dtype).reshape(shape)
        dy = dy * _silu(z)
    first, last = state["offsets"][:-1], state["offsets"][1:] - 1
    add = dy[:, :, None] * Cm
    if t["dht"] is not None:
        add[last] += t["dht"]
    later = torch.cat([decay[1:], decay[:1]])
    later[last] = 0
    g = _scanned(later.flip(0), add.flip(0), state["longest"]).flip(0)
    del add, later
    before = torch.cat([h[:1], h[:-1]])
    before[first] = 0 if t["h0"] is None else t["h0"]
    q = g * decay * before
    del before
    s = (g * Bm).sum(-1)
    ddelta = (q * t["A"]).sum(-1) + s * x
    ddt = ddelta / (1 + torch.exp(-raw))
    out.update(dx=(s * delta + t["D"] * dy).to(dtype).reshape(shape), ddt=ddt.to(dtype).reshape(shape),
               ddt_bias=ddt.double().sum(0).float(), dD=(dy * x).double().sum(0).float(),
               dA=(q * delta[:, :, None]).double().sum(0).float(),
               dB=(g * (delta * x)[:, :, None]).reshape(-1, G, D // G, N).sum(2).to(dtype).reshape(t["B"].shape),
               dC=(h * dy[:, :, None]).reshape(-1, G, D // G, N).sum(2).to(dtype).reshape(t["C"].shape))
    if t["h0"] is not None:
        out["dh0"] = (g * decay)[first]
    return out


def _norm_parts(case, t):
    x = t["x"].float()
    c = x if case["rms"] else x - x.mean(-1, keepdim=True)
    r = 1 / torch.sqrt((c * c).mean(-1, keepdim=True) + 1e-5)
    n = c * r * t["weight"]
    return c * r, r, n if t["bias"] is None else n + t["bias"]


def _norm_fwd(case, t, state):
    _, _, n = _norm_parts(case, t)
    return (n if t["z"] is None else n * _silu(t["z"].float())).to(t["x"].dtype)


def _norm_bwd(case, t, state):
    xhat, r, n = _norm_parts(case, t)
    dy, dtype = t["dy"].float(), t["x"].dtype
    out = dict(dz=None, dbias=None)
    if t["z"] is not None:
        z = t["z"].float()
        out["dz"] = (dy * n * _silu_grad(z)).to(dtype)
        dy = dy * _silu(z)
    if t["bias"] is not None:
        out["dbias"] = dy.double().sum(0).float()
    d = dy * t["weight"]
    inner = d - xhat * (d * xhat).mean(-1, keepdim=True)
    if not case["rms"]:
        inner = inner - d.mean(-1, keepdim=True)
    out.update(dx=(r * inner).to(dtype), dweight=(dy * xhat).double().sum(0).float())
    return out


# ---- what a pass cannot do without ----------------------------------------------------------------------------------------


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    D = case["D"]
    bwd = case["op"].endswith("bwd")
    if case["op"].startswith("norm"):
        whole = case["rows"] * D
        vectors = 4 * D * (1 + (1 if case["bias"] else 0))
        moved = (4 if case["gate"] else 2) + 1 if bwd else 2 + (1 if case["gate"] else 0)
        return dict(bytes=whole * e * moved + vectors * (2 if bwd else 1), flops=whole * (20 if bwd else 8))
    lens = lengths(case)
    whole = sum(lens) * D
    if case["op"].startswith("conv"):
        W = case["W"]
        state = len(lens) * (W - 1) * D * e
        vectors = 4 * D * (W + 1)
        if bwd:  # x, dy in, dx out; the state and its final gradient in, its gradient out
            return dict(bytes=3 * whole * e + (3 * state if case["h0"] else 0) + 2 * vectors, flops=whole * (6 * W + 12))
        return dict(bytes=2 * whole * e + state * (2 if case["h0"] else 1) + vectors, flops=whole * (2 * W + 4))
    N = case["N"]
    bc = 2 * sum(lens) * case["G"] * N * e
    state = len(lens) * D * N * 4
    vectors = 4 * D * (N + 2)
    gate = 1 if case["gate"] else 0
    if bwd:  # x, dt, dy (and z) in, dx, ddt (and dz) out; B, C in, dB, dC out
        return dict(bytes=(5 + 2 * gate) * whole * e + 2 * bc + (3 * state if case["h0"] else 0) + 2 * vectors,
                    flops=whole * (20 * N + 20))
    return dict(bytes=(3 + gate) * whole * e + bc + state * (2 if case["h0"] else 1) + vectors, flops=whole * (7 * N + 10))


# ---- the definitions in 64 bits --------------------------------------------------------------------------------------------


def exact(case, seed):
    t = inputs(case, seed)
    bwd = case["op"].endswith("bwd")
    if case["op"].startswith("scan") and (case["T"] > 8192 or sum(lengths(case)) * case["D"] * case["N"] > 300_000_000):
        return None
    leaves = {k: v.double().requires_grad_(bwd) for k, v in t.items() if v is not None and k not in ("cu_seqlens", "dy", "dht")}
    with torch.set_grad_enabled(bwd):
        outs = {"conv": _exact_conv, "scan": _exact_scan, "norm": _exact_norm}[case["op"][:4]](case, leaves)
    if not bwd:
        return outs
    y, ht = outs if isinstance(outs, tuple) else (outs, None)
    loss = (y * t["dy"].double()).sum()
    if ht is not None and t["dht"] is not None:
        loss = loss + (ht * t["dht"].double()).sum()
    grads = dict(zip(leaves, torch.autograd.grad(loss, list(leaves.values()))))
    named = {"conv": ["x", "weight", "bias", "h0"], "scan": ["x", "dt", "A", "B", "C", "D", "z", "dt_bias", "h0"],
             "norm": ["x", "weight", "bias", "z"]}[case["op"][:4]]
    return {"d" + k: grads.get(k) for k in named}


def _exact_conv(case, t):
    W = case["W"]
    x = t["x"].reshape(-1, case["D"])
    ys, hts, at = [], [], 0
    for n, length in enumerate(lengths(case)):
        early = t["h0"][n] if "h0" in t else x.new_zeros(W - 1, case["D"])
        row = torch.cat([early, x[at:at + length]])
        u = t["bias"] + 0 * row[W - 1:]
        for j in range(W):
            u = u + t["weight"][:, j] * row[j:j + length]
        ys.append(u * torch.sigmoid(u) if case["silu"] else u)
        hts.append(row[length:])
        at += length
    return torch.cat(ys).reshape(t["x"].shape), torch.stack(hts)


def _exact_scan(case, t):
    """Token by token, all sequences side by side; a sequence that has ended keeps its state."""
    D, N, G = case["D"], case["N"], case["G"]
    lens = lengths(case)
    begin = [sum(lens[:i]) for i in range(len(lens))]
    x, raw = t["x"].reshape(-1, D), t["dt"].reshape(-1, D) + t["dt_bias"]
    delta = torch.logaddexp(raw, torch.zeros_like(raw))
    Bm, Cm = t["B"].reshape(-1, G, 1, N), t["C"].reshape(-1, G, 1, N)
    h = t["h0"] if "h0" in t else x.new_zeros(len(lens), D, N)
    order = sorted(range(len(lens)), key=lambda i: -lens[i])  # the longest first: those still running are in front
    h = h[torch.tensor(order, device=x.device)]
    starts = torch.tensor([begin[i] for i in order], device=x.device)
    ys, rows, done = [], [], []
    for k in range(max(lens)):
        m = sum(1 for i in order if lens[i] > k)
        if m < h.shape[0]:
            done.append(h[m:])
            h = h[:m]
        at = starts[:m] + k
        d, u = delta[at], x[at]
        h = torch.exp(d[:, :, None] * t["A"]) * h + ((d * u).reshape(m, G, -1, 1) * Bm[at]).reshape(m, D, N)
        ys.append((h.reshape(m, G, -1, N) * Cm[at]).sum(-1).reshape(m, D) + t["D"] * u)
        rows.append(at)
    done.append(h)
    ends = torch.cat(done[::-1])
    back = torch.tensor([order.index(i) for i in range(len(lens))], device=x.device)
    y = torch.cat(ys)[torch.argsort(torch.cat(rows))].reshape(t["x"].shape)
    if "z" in t:
        y = y * t["z"] * torch.sigmoid(t["z"])
    return y, ends[back]


def _exact_norm(case, t):
    x = t["x"]
    if case["rms"]:
        n = x * torch.rsqrt(x.pow(2).mean(-1, keepdim=True) + 1e-5)
    else:
        n = (x - x.mean(-1, keepdim=True)) * torch.rsqrt(x.var(-1, unbiased=False, keepdim=True) + 1e-5)
    n = n * t["weight"]
    if "bias" in t:
        n = n + t["bias"]
    return n * t["z"] * torch.sigmoid(t["z"]) if "z" in t else n
