"""Cases of the operators that a layer of attention puts beside the gated delta rule.

* Attention over a sliding window with a few first tokens that stay visible
  (sinks): prompts, training steps, single tokens over a ring cache, and the
  cache's filling.  With ``w = window`` and ``s = sinks`` token t sees the
  tokens j with ``t - w < j <= t`` or ``j < s, j <= t``.
* The norms after a block and before the next one, with the block's gate and
  residual scale, in one pass: ``h = residual + scale sigmoid(z) norm(x)`` and
  ``y = norm(h)``; forward and backward.

A case is a dict of plain values.  ``prepare`` draws its inputs on the GPU,
``run`` makes one pass, ``exact`` evaluates the definition in 64 bits.
"""
import math
import random

import torch

# False: the plain form below, in torch; True: the framework's entry points.
own = False

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
EPS = 1e-5


def listed():
    return [
        # prompts of 8 requests packed, ragged lengths up to 4096, 32 query heads on 8 key heads
        dict(name="attn packed prompts", op="attn_fwd", dtype="bf16", B=1, T=4096, packed=8, Nq=32, Nk=8, d=128, window=1024, sinks=4),
        # one long document, a wide window
        dict(name="attn long prompt", op="attn_fwd", dtype="bf16", B=1, T=32768, packed=0, Nq=32, Nk=8, d=128, window=4096, sinks=128),
        # a training step, forward and backward, at the headline's batch, heads and length
        dict(name="attn training", op="attn_train", dtype="bf16", B=4, T=2048, packed=0, Nq=16, Nk=16, d=128, window=512, sinks=4),
        # an fp32 fine-tuning step over packed samples, odd window, three query heads on each key head
        dict(name="attn training ragged fp32", op="attn_train", dtype="fp32", B=1, T=600, packed=7, Nq=6, Nk=2, d=64, window=101, sinks=3),
        # one decoding step of 64 sequences of all ages
        dict(name="attn step b64", op="attn_step", dtype="bf16", N=64, Nq=32, Nk=4, d=128, window=2048, sinks=4, ring=2048),
        # one decoding step of one sequence: latency
        dict(name="attn step b1", op="attn_step", dtype="bf16", N=1, Nq=16, Nk=4, d=128, window=4096, sinks=4, ring=4096),
        # the packed prompts' keys and values go into the caches that their decoding reads
        dict(name="cache fill prompts", op="fill", dtype="bf16", B=1, T=4096, packed=8, Nk=8, d=128, sinks=4, ring=1024, started=False),
        # a further piece of every sequence, fp32, odd ring
        dict(name="cache fill pieces fp32", op="fill", dtype="fp32", B=6, T=130, packed=0, Nk=3, d=64, sinks=5, ring=333, started=True),
        # between two blocks, the headline's tokens, gated, residual stream in fp32
        dict(name="block norm", op="block_fwd", dtype="bf16", res="fp32", rows=8192, D=2048, rms=True, post=True, gate=True, scale=True, bias=False),
        # the same for a few rows, as in decoding: the residual sum and the next norm alone
        dict(name="block norm decode", op="block_fwd", dtype="bf16", res="bf16", rows=64, D=2048, rms=True, post=False, gate=False, scale=False, bias=False),
        # backward between two blocks in training
        dict(name="block norm training", op="block_bwd", dtype="bf16", res="fp32", rows=8192, D=2048, rms=True, post=True, gate=True, scale=True, bias=False),
        # backward with layer norms and biases, wide rows, an odd number of them
        dict(name="block norm wide training", op="block_bwd", dtype="bf16", res="bf16", rows=16383, D=4096, rms=False, post=True, gate=False, scale=True, bias=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """One more case: any operator, sizes spread over their logarithm, odd ones among them."""
    op = rng.choice(["attn_fwd", "attn_fwd", "attn_train", "attn_train", "attn_step", "attn_step", "fill", "block_fwd", "block_bwd"])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    if op.startswith("block"):
        D = rng.choice([_log(rng, 16, 16384), 64 * rng.randint(1, 128), 1 << rng.randint(4, 13)])
        rows = _log(rng, 1, max(2, min(200000, (1 << (25 if dtype == "bf16" else 24)) // D)))
        return dict(op=op, dtype=dtype, res=rng.choice([dtype, "fp32"]), rows=rows, D=D, rms=rng.random() < 0.6, post=rng.random() < 0.6,
                    gate=rng.random() < 0.5, scale=rng.random() < 0.5, bias=rng.random() < 0.4)
    d = rng.choice([64, 128])
    Nk = rng.choice([1, 2, 4, 8, rng.randint(1, 12)])
    Nq = Nk * rng.choice([1, 2, 4, 8, rng.randint(1, 8)])
    sinks = rng.choice([0, 4, _log(rng, 1, 128)])
    if op == "attn_step":
        window = _log(rng, 1, 8192)
        ring = window + rng.choice([0, 0, rng.randint(1, 64)])
        N = _log(rng, 1, max(1, min(256, (1 << (27 if dtype == "bf16" else 26)) // (2 * Nk * d * (sinks + ring)))))
        return dict(op=op, dtype=dtype, N=N, Nq=Nq, Nk=Nk, d=d, window=window, sinks=sinks, ring=ring)
    packed = rng.choice([0, rng.randint(1, 24)])
    seqs = packed or rng.choice([1, 2, 4, rng.randint(1, 16)])
    T = rng.choice([_log(rng, 1, 8192), _log(rng, 64, 8192)])
    if op == "fill":
        T = max(1, min(T, (1 << 24) // (seqs * Nk * d)))
        return dict(op=op, dtype=dtype, B=1 if packed else seqs, T=T, packed=packed, Nk=Nk, d=d, sinks=sinks, ring=_log(rng, 1, 4096),
                    started=rng.random() < 0.5)
    window = _log(rng, 2, 8192)
    most = 1 << (36 if dtype == "bf16" else 33)  # elements of all products of queries and keys
    T = max(16 if op == "attn_train" else 1, min(T, (1 << 27) // (seqs * Nq * d), most // (seqs * Nq * d * min(T, window + sinks))))
    return dict(op=op, dtype=dtype, B=1 if packed else seqs, T=T, packed=packed, Nq=Nq, Nk=Nk, d=d, window=window, sinks=sinks)


def lengths(case):
    """Tokens of each sequence: B of T each, or `packed` ones of 1 to T drawn from the case's own sizes."""
    if not case["packed"]:
        return [case["T"]] * case["B"]
    rng = random.Random("%d %d %d" % (case["packed"], case["T"], case["Nk"]))
    return [rng.randint(1, case["T"]) for _ in range(case["packed"])]


def ages(case):
    """Tokens that each sequence of a cache has had: none, fewer than the ring holds, many times as many."""
    if case["op"] == "fill":
        n = len(lengths(case))
        if not case["started"]:
            return [0] * n
    else:
        n = case["N"]
    rng = random.Random("%d %d %d" % (n, case["ring"], case["Nk"]))
    ring = case["sinks"] + case["ring"]
    old = [ring + rng.randint(0, 9 * ring) for _ in range(n)]
    for i in range(1, n, 3):
        old[i] = rng.randint(0, ring)
    return old


# ---- inputs ---------------------------------------------------------------------------------------------------------


def inputs(case, seed):
    """The tensors of a case, by the names of the entry points' arguments."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt, f32 = DTYPES[case["dtype"]], torch.float32

    def normal(*shape, dtype=dt, scale=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)

    if case["op"].startswith("block"):
        rows, D, bias = case["rows"], case["D"], case["bias"]
        rt = DTYPES[case["res"]]
        t = dict(x=normal(rows, D, scale=1.5) + 0.25, residual=normal(rows, D, dtype=rt, scale=2.0),
                 z=normal(rows, D) if case["gate"] else None,
                 scale=0.5 + normal(D, dtype=f32, scale=0.1) if case["scale"] else None,
                 post_weight=1 + normal(D, dtype=f32, scale=0.1) if case["post"] else None,
                 post_bias=normal(D, dtype=f32, scale=0.1) if case["post"] and bias else None,
                 weight=1 + normal(D, dtype=f32, scale=0.1), bias=normal(D, dtype=f32, scale=0.1) if bias else None)
        if case["op"] == "block_bwd":
            t.update(dy=normal(rows, D), dresidual_out=normal(rows, D, dtype=rt))
        return t
    Nk, d = case["Nk"], case["d"]
    if case["op"] == "attn_step":
        n, B, T = case["N"], case["N"], 1
        cu = None
    else:
        lens = lengths(case)
        n = len(lens)
        B, T = (1, sum(lens)) if case["packed"] else (case["B"], case["T"])
        cu = torch.tensor([0] + lens, dtype=torch.int64, device="cuda").cumsum(0) if case["packed"] else None
    t = dict(k=normal(B, T, Nk, d), v=normal(B, T, Nk, d))
    if case["op"] != "fill":
        t["q"] = normal(B, T, case["Nq"], d)
    if case["op"].startswith("attn_") and case["op"] != "attn_step":
        t["cu_seqlens"] = cu
        if case["op"] == "attn_train":
            t["do"] = normal(B, T, case["Nq"], d)
        return t
    # caches: what the sequences have left in them so far, zeros where nothing was written
    slots = case["sinks"] + case["ring"]
    had = torch.tensor(ages(case), device="cuda")
    written = (torch.arange(slots, device="cuda") < had[:, None])[:, None, :, None]
    t.update(k_cache=normal(n, Nk, slots, d) * written, v_cache=normal(n, Nk, slots, d) * written, lengths=had)
    if case["op"] == "fill":
        t["cu_seqlens"] = cu
    return t


def prepare(case, seed):
    t = inputs(case, seed)
    state = dict(case=case, t=t)
    # the outputs of a step belong to the program: it gives the same buffers to each call
    if case["op"] in ("attn_fwd", "attn_step"):
        state["o"] = torch.empty_like(t["q"])
    if case["op"] == "attn_fwd":
        state["lse"] = torch.empty(t["q"].shape[:3], dtype=torch.float32, device="cuda")
    if case["op"] == "block_fwd":
        state["y"], state["residual_out"] = torch.empty_like(t["x"]), torch.empty_like(t["residual"])
    return state


# ---- one pass -------------------------------------------------------------------------------------------------------


def run(state):
    case, t = state["case"], state["t"]
    if own:
        return _run_own(case, t, state)
    return {"attn_fwd": _attn_fwd, "attn_train": _attn_train, "attn_step": _attn_step, "fill": _fill, "block_fwd": _block_fwd,
            "block_bwd": _block_bwd}[case["op"]](case, t)


def _run_own(case, t, state):
    import chunkwise_gated_delta_chunk_gb300 as dn

    op = case["op"]
    if op == "attn_fwd":
        return dn.window_attn_fwd(t["q"], t["k"], t["v"], case["window"], case["sinks"], t["cu_seqlens"], o=state["o"], lse=state["lse"])
    if op == "attn_train":
        o, lse = dn.window_attn_fwd(t["q"], t["k"], t["v"], case["window"], case["sinks"], t["cu_seqlens"])
        grads = dn.window_attn_bwd(t["q"], t["k"], t["v"], o, lse, case["window"], case["sinks"], t["cu_seqlens"], do=t["do"])
        return dict(o=o, lse=lse, **grads)
    if op == "attn_step":
        o = dn.window_attn_step(t["q"], t["k"], t["v"], t["k_cache"], t["v_cache"], t["lengths"], case["window"], case["sinks"],
                                o=state["o"])
        return o, t["k_cache"], t["v_cache"]
    if op == "fill":
        return dn.window_cache_fill(t["k"], t["v"], t["k_cache"], t["v_cache"], t["lengths"], case["sinks"], t["cu_seqlens"])
    kinds = dict(eps=EPS, rms=case["rms"], post=case["post"])
    args = [t[k] for k in ("x", "residual", "z", "scale", "post_weight", "post_bias", "weight", "bias")]
    if op == "block_fwd":
        return dn.block_norm_fwd(*args, **kinds, y=state["y"], residual_out=state["residual_out"])
    return dn.block_norm_bwd(*args, **kinds, dy=t["dy"], dresidual_out=t["dresidual_out"])


# ---- the plain forms: elementary torch in 32 bits ------------------------------------------------------------------------


def _pieces(case):
    """Runs of query tokens and the tokens they may see: (first, last + 1, row of tokens, sinks before, first key)."""
    at = 0
    for length in lengths(case):
        for q0 in range(0, length, 512):
            q1 = min(length, q0 + 512)
            lo = max(0, q0 - case["window"] + 1)
            yield at, q0, q1, min(case["sinks"], lo), lo
        at += length


def _heads(rows, Nk):
    """[tokens, heads, d] to [Nk, heads of a key head x tokens, d]."""
    m, H, d = rows.shape
    return rows.reshape(m, Nk, H // Nk, d).permute(1, 2, 0, 3).reshape(Nk, H // Nk * m, d)


def _tokens(rows, m):
    """And back."""
    Nk, r, d = rows.shape
    return rows.reshape(Nk, r // m, m, d).permute(2, 0, 1, 3).reshape(m, r // m * Nk, d)


def _piece(case, t, piece, tensors):
    at, q0, q1, s, lo = piece
    device = t["q"].device
    keys = torch.cat([torch.arange(s, device=device), torch.arange(lo, q1, device=device)])
    queries = torch.arange(q0, q1, device=device)[:, None]
    seen = (keys <= queries) & ((keys > queries - case["window"]) | (keys < case["sinks"]))
    q, k, v = tensors
    Q = _heads(q[at + q0:at + q1].float(), case["Nk"])
    K, V = (x[at + keys].float().transpose(0, 1) for x in (k, v))
    scores = (Q @ K.transpose(1, 2)) * case["d"] ** -0.5
    scores = scores.reshape(case["Nk"], -1, q1 - q0, keys.numel()).masked_fill(~seen, -math.inf)
    top = scores.amax(-1, keepdim=True)
    P = torch.exp(scores - top)
    total = P.sum(-1, keepdim=True)
    P = (P / total).reshape(case["Nk"], -1, keys.numel())
    lse = (top + torch.log(total)).reshape(case["Nq"], q1 - q0).transpose(0, 1)
    return at + keys, Q, K, V, P, lse


def _flat(t, *names):
    return [t[n].reshape(-1, *t[n].shape[2:]) for n in names]


def _attn_fwd(case, t):
    tensors = _flat(t, "q", "k", "v")
    o = torch.empty_like(tensors[0])
    lse = torch.empty(o.shape[:2], device=o.device)
    for piece in _pieces(case):
        at, q0, q1 = piece[:3]
        _, _, _, V, P, l = _piece(case, t, piece, tensors)
        o[at + q0:at + q1] = _tokens(P @ V, q1 - q0).to(o.dtype)
        lse[at + q0:at + q1] = l
    return o.reshape(t["q"].shape), lse.reshape(t["q"].shape[:3])


def _attn_train(case, t):
    tensors = _flat(t, "q", "k", "v")
    do, = _flat(t, "do")
    o, dq = torch.empty_like(tensors[0]), torch.empty_like(tensors[0])
    lse = torch.empty(o.shape[:2], device=o.device)
    dk, dv = (torch.zeros(x.shape, device=o.device) for x in tensors[1:])
    c = case["d"] ** -0.5
    for piece in _pieces(case):
        at, q0, q1 = piece[:3]
        rows = slice(at + q0, at + q1)
        keys, Q, K, V, P, lse[rows] = _piece(case, t, piece, tensors)
        O = P @ V
        G = _heads(do[rows].float(), case["Nk"])
        S = P * (G @ V.transpose(1, 2) - (G * O).sum(-1, keepdim=True)) * c
        o[rows] = _tokens(O, q1 - q0).to(o.dtype)
        dq[rows] = _tokens(S @ K, q1 - q0).to(o.dtype)
        dk[keys] += (S.transpose(1, 2) @ Q).transpose(0, 1)
        dv[keys] += (P.transpose(1, 2) @ G).transpose(0, 1)
    out = dict(o=o, lse=lse, dq=dq, dk=dk.to(o.dtype), dv=dv.to(o.dtype))
    return {k: v.reshape(t["q"].shape[:2] + v.shape[1:]) for k, v in out.items()}


def _slot(position, sinks, ring):
    return torch.where(position < sinks, position, sinks + (position - sinks) % ring)


def _attn_step(case, t):
    N, Nk, sinks, ring = case["N"], case["Nk"], case["sinks"], case["ring"]
    had = t["lengths"][:, None]
    each = torch.arange(N, device=had.device)
    where = _slot(t["lengths"], sinks, ring)
    t["k_cache"][each, :, where] = t["k"][:, 0]
    t["v_cache"][each, :, where] = t["v"][:, 0]
    # the newest position that each slot holds
    slot = torch.arange(sinks + ring, device=had.device)
    holds = torch.where(slot < sinks, slot, had - (had - slot) % ring)
    seen = (holds <= had) & ((holds < sinks) | (holds >= sinks) & (holds > had - case["window"]))
    seen &= (slot < sinks) | (holds >= sinks)
    q = t["q"].float().reshape(N, Nk, -1, case["d"])
    scores = (q @ t["k_cache"].float().transpose(2, 3)) * case["d"] ** -0.5
    scores = scores.masked_fill(~seen[:, None, None], -math.inf)
    P = torch.exp(scores - scores.amax(-1, keepdim=True))
    o = (P @ t["v_cache"].float()) / P.sum(-1, keepdim=True)
    return o.reshape(t["q"].shape).to(t["q"].dtype), t["k_cache"], t["v_cache"]


def _fill(case, t):
    sinks, ring = case["sinks"], case["ring"]
    k, v = _flat(t, "k", "v")
    at = 0
    for n, (had, length) in enumerate(zip(ages(case), lengths(case))):
        i = torch.arange(length, device=k.device)
        last = max(sinks - had, length - ring, 0)  # the ring keeps the tokens from here on
        for part in (i[:max(0, min(sinks - had, length))], i[last:]):
            where = _slot(had + part, sinks, ring)
            t["k_cache"][n, :, where] = k[at + part].transpose(0, 1)
            t["v_cache"][n, :, where] = v[at + part].transpose(0, 1)
        at += length
    return t["k_cache"], t["v_cache"]


def _normed(x, rms):
    """The row's deviations over their root mean square, and the factor."""
    c = x if rms else x - x.mean(-1, keepdim=True)
    r = 1 / torch.sqrt((c * c).mean(-1, keepdim=True) + EPS)
    return c * r, r


def _block(case, t):
    x = t["x"].float()
    xhat, r = _normed(x, case["rms"]) if case["post"] else (x, None)
    p = xhat
    if t["post_weight"] is not None:
        p = p * t["post_weight"]
    if t["post_bias"] is not None:
        p = p + t["post_bias"]
    gate = 1 / (1 + torch.exp(-t["z"].float())) if case["gate"] else None
    f = gate if t["scale"] is None else t["scale"] if gate is None else gate * t["scale"]
    h = t["residual"].float() + (p if f is None else p * f)
    hhat, rh = _normed(h, case["rms"])
    return xhat, r, p, gate, f, h, hhat, rh


def _block_fwd(case, t):
    h, hhat = _block(case, t)[5:7]
    y = hhat * t["weight"]
    if t["bias"] is not None:
        y = y + t["bias"]
    return y.to(t["x"].dtype), h.to(t["residual"].dtype)


def _unnormed(d, hat, r, rms):
    """The gradient of the row whose deviations are `hat`, from theirs."""
    inner = d - hat * (d * hat).mean(-1, keepdim=True)
    if not rms:
        inner = inner - d.mean(-1, keepdim=True)
    return r * inner


def _rows_sum(x):
    return x.double().sum(0).float()


def _block_bwd(case, t):
    xhat, r, p, gate, f, h, hhat, rh = _block(case, t)
    dtype = t["x"].dtype
    dy = t["dy"].float()
    out = dict(dz=None, dscale=None, dpost_weight=None, dpost_bias=None, dbias=None, dweight=_rows_sum(dy * hhat))
    if t["bias"] is not None:
        out["dbias"] = _rows_sum(dy)
    dh = t["dresidual_out"].float() + _unnormed(dy * t["weight"], hhat, rh, case["rms"])
    out["dresidual"] = dh.to(t["residual"].dtype)
    if t["scale"] is not None:
        out["dscale"] = _rows_sum(dh * p if gate is None else dh * p * gate)
    if gate is not None:
        dg = dh * p if t["scale"] is None else dh * p * t["scale"]
        out["dz"] = (dg * gate * (1 - gate)).to(dtype)
    dp = dh if f is None else dh * f
    if t["post_weight"] is not None:
        out["dpost_weight"] = _rows_sum(dp * xhat)
    if t["post_bias"] is not None:
        out["dpost_bias"] = _rows_sum(dp)
    if case["post"]:
        dp = _unnormed(dp * t["post_weight"], xhat, r, case["rms"])
    out["dx"] = dp.to(dtype)
    return out


# ---- what a pass cannot do without ----------------------------------------------------------------------------------------


def _pairs(length, window, sinks):
    """Visible (query, key) pairs of a sequence."""
    def inside(n, w):  # sum over t < n of min(t + 1, w)
        w = min(n, w)
        return w * (w + 1) // 2 + (n - w) * w

    # beyond the window: min(sinks, t + 1 - window) more
    return inside(length, window) + inside(max(0, length - window), sinks)


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    if case["op"].startswith("block"):
        whole, D = case["rows"] * case["D"], case["D"]
        er = 4 if case["res"] == "fp32" else 2
        vectors = 4 * D * (1 + case["scale"] + case["post"] + case["bias"] + (case["post"] and case["bias"]))
        if case["op"] == "block_fwd":  # x, residual (and z) in, y and the residual stream out
            return dict(bytes=whole * ((2 + case["gate"]) * e + 2 * er) + vectors, flops=whole * (8 + 6 * case["post"] + 6 * case["gate"]))
        # x, dy (and z), residual and its gradient in; dx (and dz) and the residual's gradient out
        return dict(bytes=whole * ((3 + 2 * case["gate"]) * e + 3 * er) + 2 * vectors,
                    flops=whole * (20 + 14 * case["post"] + 12 * case["gate"]))
    Nk, d = case["Nk"], case["d"]
    if case["op"] == "attn_step":
        seen = sum(min(n, case["sinks"]) + min(max(0, n - case["sinks"]), case["window"] - 1) for n in ages(case))
        # old keys and values in; the new ones in and out; q in, o out
        return dict(bytes=2 * seen * Nk * d * e + case["N"] * d * e * (4 * Nk + 2 * case["Nq"]) + 8 * case["N"],
                    flops=4 * (seen + case["N"]) * case["Nq"] * d)
    lens = lengths(case)
    if case["op"] == "fill":
        sinks, ring = case["sinks"], case["ring"]
        kept = 0
        for had, n in zip(ages(case), lens):
            first = max(0, min(sinks - had, n))
            kept += first + n - max(sinks - had, n - ring, 0) if n > sinks - had else first
        return dict(bytes=4 * kept * Nk * d * e, flops=0)
    pairs = sum(_pairs(n, case["window"], case["sinks"]) for n in lens) * case["Nq"]
    q, kv = (sum(lens) * h * d * e for h in (case["Nq"], Nk))
    lse = 4 * sum(lens) * case["Nq"]
    if case["op"] == "attn_fwd":
        return dict(bytes=2 * q + 2 * kv + lse, flops=4 * pairs * d)
    # q, k, v, do in; o, dq, dk, dv out; two products forward, five backward
    return dict(bytes=4 * q + 4 * kv + lse, flops=14 * pairs * d)


# ---- the definitions in 64 bits --------------------------------------------------------------------------------------------


def exact(case, seed):
    t = inputs(case, seed)
    if case["op"].startswith("block"):
        return _exact_block(case, t)
    if case["op"] == "fill":
        return _exact_fill(case, t)
    if case["op"] == "attn_step":
        return _exact_step(case, t)
    if work(case)["flops"] > 1 << 43:
        return None
    return _exact_attn(case, t)


def _softmax_rows(q, k, v, seen):
    """Outputs [m, d] and logarithms of the sums [m] of queries q [m, d] over the keys that `seen` leaves."""
    scores = (q * q.shape[-1] ** -0.5) @ k.T
    scores = torch.where(seen, scores, scores.new_tensor(-math.inf))
    lse = torch.logsumexp(scores, -1)
    return torch.exp(scores - lse[:, None]) @ v, lse


def _exact_attn(case, t):
    train = case["op"] == "attn_train"
    G = case["Nq"] // case["Nk"]
    q, k, v = (x.reshape(-1, *x.shape[2:]) for x in (t["q"], t["k"], t["v"]))
    o = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    lse = torch.zeros(q.shape[:2], dtype=torch.float64, device=q.device)
    dq, dk, dv = torch.zeros_like(o), *(torch.zeros(k.shape, dtype=torch.float64, device=q.device) for _ in range(2))
    begin = 0
    for length in lengths(case):
        for a in range(0, length, 4096):
            b = min(a + 4096, length)
            lo = max(0, a + 1 - case["window"])
            first = min(lo, case["sinks"])
            pos = torch.tensor(list(range(first)) + list(range(lo, b)), device=q.device)
            dist = torch.arange(a, b, device=q.device)[:, None] - pos
            seen = (dist >= 0) & ((dist < case["window"]) | (pos < case["sinks"]))
            rows = slice(begin + a, begin + b)
            for h in range(case["Nq"]):
                leaves = [q[rows, h].double(), k[begin + pos, h // G].double(), v[begin + pos, h // G].double()]
                with torch.set_grad_enabled(train):
                    leaves = [x.requires_grad_(train) for x in leaves]
                    oh, lh = _softmax_rows(*leaves, seen)
                o[rows, h], lse[rows, h] = oh.detach(), lh.detach()
                if train:
                    gq, gk, gv = torch.autograd.grad((oh * t["do"].reshape(q.shape)[rows, h].double()).sum(), leaves)
                    dq[rows, h] = gq
                    dk[:, h // G].index_add_(0, begin + pos, gk)
                    dv[:, h // G].index_add_(0, begin + pos, gv)
        begin += length
    lead = t["q"].shape[:2]
    if train:
        return {name: x.reshape(lead + x.shape[1:]) for name, x in dict(o=o, lse=lse, dq=dq, dk=dk, dv=dv).items()}
    return o.reshape(t["q"].shape), lse.reshape(t["q"].shape[:3])


def _exact_step(case, t):
    sinks, ring, G = case["sinks"], case["ring"], case["Nq"] // case["Nk"]
    o = torch.zeros(t["q"].shape, dtype=torch.float64, device="cuda")
    for n, had in enumerate(ages(case)):
        place = had if had < sinks else sinks + (had - sinks) % ring
        t["k_cache"][n, :, place], t["v_cache"][n, :, place] = t["k"][n, 0], t["v"][n, 0]
        seen = [p for p in range(min(sinks, had + 1))] + [p for p in range(max(sinks, had + 1 - case["window"]), had + 1)]
        at = torch.tensor([p if p < sinks else sinks + (p - sinks) % ring for p in seen], device="cuda")
        whole = torch.ones(G, len(seen), dtype=torch.bool, device="cuda")
        for h in range(case["Nk"]):
            of = slice(h * G, (h + 1) * G)
            o[n, 0, of] = _softmax_rows(t["q"][n, 0, of].double(), t["k_cache"][n, h, at].double(), t["v_cache"][n, h, at].double(), whole)[0]
    return o, t["k_cache"], t["v_cache"]


def _exact_fill(case, t):
    """Which token each slot holds at last: later ones overwrite earlier ones."""
    sinks, ring = case["sinks"], case["ring"]
    at = 0
    for n, (had, length) in enumerate(zip(ages(case), lengths(case))):
        holds = {}
        for p in range(had, had + length):
            holds[p if p < sinks else sinks + (p - sinks) % ring] = p - had
        slots = torch.tensor(list(holds), device="cuda")
        rows = torch.tensor(list(holds.values()), device="cuda") + at
        for name in ("k", "v"):
            flat = t[name].reshape(-1, case["Nk"], case["d"])
            t[name + "_cache"][n].index_copy_(1, slots, flat[rows].transpose(0, 1).contiguous())
        at += length
    return t["k_cache"], t["v_cache"]


def _exact_norm(x, weight, bias, rms):
    if rms:
        n = x * torch.rsqrt(x.pow(2).mean(-1, keepdim=True) + EPS)
    else:
        n = (x - x.mean(-1, keepdim=True)) * torch.rsqrt(x.var(-1, unbiased=False, keepdim=True) + EPS)
    n = n if weight is None else n * weight
    return n if bias is None else n + bias


def _exact_block(case, t):
    bwd = case["op"] == "block_bwd"
    names = ("x", "residual", "z", "scale", "post_weight", "post_bias", "weight", "bias")
    u = {k: None if t[k] is None else t[k].double().requires_grad_(bwd) for k in names}
    with torch.set_grad_enabled(bwd):
        branch = _exact_norm(u["x"], u["post_weight"], u["post_bias"], case["rms"]) if case["post"] else u["x"]
        if u["z"] is not None:
            branch = branch * torch.sigmoid(u["z"])
        if u["scale"] is not None:
            branch = branch * u["scale"]
        h = u["residual"] + branch
        y = _exact_norm(h, u["weight"], u["bias"], case["rms"])
        if not bwd:
            return y, h
        loss = (y * t["dy"].double()).sum() + (h * t["dresidual_out"].double()).sum()
    given = [k for k in names if u[k] is not None]
    grads = dict(zip(given, torch.autograd.grad(loss, [u[k] for k in given])))
    return {"d" + k: grads.get(k) for k in names}
