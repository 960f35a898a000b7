"""The operators around the recurrence in 64 bits, token by token from their
definitions, and the comparison of a kernel's outputs with them.  Gradients
come from automatic differentiation of these definitions."""
from __future__ import annotations

import torch


def spans(B, T, lengths):
    """(batch row, first, last + 1) of each sequence."""
    if lengths is None:
        return [(b, 0, T) for b in range(B)]
    out, at = [], 0
    for n in lengths:
        out.append((0, at, at + n))
        at += n
    return out


def offsets(lengths, device):
    return torch.tensor([0] + list(lengths), dtype=torch.int64, device=device).cumsum(0)


def conv(t, lengths=None, silu=True):
    x, w = t["x"], t["weight"]
    B, T, D = x.shape
    W = w.shape[1]
    y = torch.zeros_like(x)
    hts = []
    for n, (b, lo, hi) in enumerate(spans(B, T, lengths)):
        early = t["h0"][n] if t.get("h0") is not None else x.new_zeros(W - 1, D)
        row = torch.cat([early, x[b, lo:hi]])
        u = torch.stack([(row[s:s + W] * w.T).sum(0) for s in range(hi - lo)]) if hi > lo else x.new_zeros(0, D)
        if t.get("bias") is not None:
            u = u + t["bias"]
        if silu:
            u = u / (1 + torch.exp(-u))
        y = torch.cat([y[:b], torch.cat([y[b, :lo], u, y[b, hi:]])[None], y[b + 1:]])
        hts.append(row[hi - lo:])
    return y, torch.stack(hts) if hts else x.new_zeros(0, W - 1, D)


def scan(t, lengths=None, softplus=True):
    x, A, Bm, Cm = t["x"], t["A"], t["B"], t["C"]
    B, T, D = x.shape
    G, N = Bm.shape[2:]
    y = torch.zeros_like(x)
    hts = []
    for n, (b, lo, hi) in enumerate(spans(B, T, lengths)):
        h = t["h0"][n] if t.get("h0") is not None else x.new_zeros(D, N)
        rows = []
        for s in range(lo, hi):
            d = t["dt"][b, s]
            if t.get("dt_bias") is not None:
                d = d + t["dt_bias"]
            if softplus:
                d = torch.logaddexp(d, torch.zeros_like(d))
            bb = Bm[b, s].repeat_interleave(D // G, 0)
            cc = Cm[b, s].repeat_interleave(D // G, 0)
            h = torch.exp(d[:, None] * A) * h + (d * x[b, s])[:, None] * bb
            out = (h * cc).sum(1)
            if t.get("D") is not None:
                out = out + t["D"] * x[b, s]
            rows.append(out)
        if rows:
            y = torch.cat([y[:b], torch.cat([y[b, :lo], torch.stack(rows), y[b, hi:]])[None], y[b + 1:]])
        hts.append(h)
    if t.get("z") is not None:
        y = y * t["z"] / (1 + torch.exp(-t["z"]))
    return y, torch.stack(hts) if hts else x.new_zeros(0, D, N)


def norm(t, eps=1e-5, rms=False):
    x = t["x"]
    c = x if rms else x - x.mean(-1, keepdim=True)
    y = c / torch.sqrt((c * c).mean(-1, keepdim=True) + eps)
    if t.get("weight") is not None:
        y = y * t["weight"]
    if t.get("bias") is not None:
        y = y + t["bias"]
    if t.get("z") is not None:
        y = y * t["z"] / (1 + torch.exp(-t["z"]))
    return y


def in_64_bits(t, grad=False):
    return {k: None if v is None else v.detach().double().cpu().requires_grad_(grad) for k, v in t.items()}


def gradients(outs, cotangents, leaves):
    """Gradients of sum(cotangent * output) with respect to the leaves (a dict)."""
    loss = sum((o * c.double().cpu()).sum() for o, c in zip(outs, cotangents) if c is not None)
    names = [k for k, v in leaves.items() if v is not None]
    got = torch.autograd.grad(loss, [leaves[k] for k in names], allow_unused=True)
    return {k: torch.zeros_like(leaves[k]) if g is None else g for k, g in zip(names, got)}


def close(got, want, steps, label="", scale=None):
    """A kernel's output against the one in 64 bits.

    The one rounding to a 16-bit type is off by at most half a step of the value
    (finfo.eps / 2).  Before it the kernel computes in fp32: `steps` roundings of
    at most 2^-24 each of the largest value of the output (or of `scale`, where
    the terms are larger than what they sum to)."""
    if want.numel() == 0:
        assert got.shape == want.shape, label
        return
    g, w = got.detach().double().cpu(), want.detach()
    assert g.shape == w.shape, (label, g.shape, w.shape)
    assert torch.isfinite(g).all(), label
    half = torch.finfo(got.dtype).eps / 2 if got.dtype != torch.float32 else 0.0
    top = float(w.abs().max()) if scale is None else scale
    fine = steps * 2.0 ** -24
    off = (g - w).abs()
    # fp32's error is rounded along with the value: (1 + half)
    limit = half * w.abs() + (1 + half) * fine * top
    worst = float((off - limit).max())
    assert worst <= 0, (label, "over by", worst, "largest error", float(off.max()), "of", top)
