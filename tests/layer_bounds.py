"""The selective scan and its gradients in 64 bits, written out as two walks, each value with a
bound on what fp32 arithmetic may be off.

The bounds follow the values through the recurrence: an error of h decays with h, one of a decay
counts with the state that it multiplies.  So they are tight where the state forgets, other than a
count of roundings times the largest value.  With u = 2^-24, half a step of fp32:

* delta: a sum (u), softplus within 8 u of its value; below 2^-126 it may be 0;
* the decay e^{delta A}: its exponent is off by delta's error and 3 products, the exponential by
  4 u; where a sequence is cut into chunks of L tokens, the sum of delta over one is off by up to L u
  of it, which counts as L u |delta A| for each of its tokens;
* a gate: silu and its derivative within (2 |z| + 9) u;
* sums over N states: 14 additions; over channels: 16 and one for every tile of 8; over tokens: the
  tokens of a chunk, the slots, and 20;
* the gradient that a chunk sends to its start is a sum of up to L terms, each off by u of the sum.

Terms of second order are covered by 5 % on all of it."""
from __future__ import annotations

import torch

U = 2.0 ** -24


def scan(t, grads, lengths, softplus, chunk, slots, dht=True):
    """{name: (value, bound)} of y, ht and the gradients; t and grads in 64 bits on the CPU."""
    x, dt, A, Bm, Cm = (t[k] for k in ("x", "dt", "A", "B", "C"))
    skip, z, bias = t["D"], t["z"], t["dt_bias"]
    Bt, T, D = x.shape
    G, N = Bm.shape[2:]
    aA = A.abs()
    zero = x.new_zeros
    out = {k: [zero(v.shape), zero(v.shape)] for k, v in
           dict(y=x, dx=x, ddt=x, dz=x, dB=Bm, dC=Cm, dA=A).items()}
    n_seqs = Bt if lengths is None else len(lengths)
    for k, shape in dict(ht=(n_seqs, D, N), dh0=(n_seqs, D, N), dD=(D,), ddt_bias=(D,)).items():
        out[k] = [zero(shape), zero(shape)]
    terms = {k: zero(v[0].shape) for k, v in out.items()}  # sums of absolute values, for the sums over tokens
    spans = [(b, 0, T) for b in range(Bt)]
    if lengths is not None:
        ends = torch.tensor([0] + list(lengths)).cumsum(0).tolist()
        spans = [(0, a, b) for a, b in zip(ends[:-1], ends[1:])]

    def wide(rows):  # [G, N] of a token to every channel
        return rows.repeat_interleave(D // G, 0)

    def joined(v):  # and back, summed over a group's channels
        return v.reshape(G, D // G, N).sum(1)

    def put(name, at, value, err):
        out[name][0][at], out[name][1][at] = value, err

    if z is not None:
        sg = torch.sigmoid(z)
        rel = (2 * z.abs() + 9) * U
        silu, slope = z * sg, sg * (1 + z * (1 - sg))
        e_slope = (1 + z.abs()) * sg * rel + 3 * U * sg * (1 + z.abs() * (1 - sg))
    for n, (b, lo, hi) in enumerate(spans):
        h = t["h0"][n] if t["h0"] is not None else zero(D, N)
        eh = zero(D, N)
        kept = []
        for s in range(lo, hi):
            raw = dt[b, s] + (bias if bias is not None else 0)
            e_raw = U * raw.abs()
            if softplus:
                d = torch.logaddexp(raw, torch.zeros_like(raw))
                ed = torch.sigmoid(raw) * e_raw + 8 * U * d + 2.0 ** -126
            else:
                d, ed = raw, e_raw
            F = torch.exp(d[:, None] * A)
            r = aA * ed[:, None] + (3 + chunk) * U * aA * d.abs()[:, None] + 4 * U
            xs = x[b, s]
            step = d * xs
            e_step = xs.abs() * ed + U * step.abs()
            bb, cc = wide(Bm[b, s]), wide(Cm[b, s])
            inc = step[:, None] * bb
            before, e_before = h, eh
            h = F * h + inc
            eh = F * eh + (F * before).abs() * r + bb.abs() * e_step[:, None] + U * inc.abs() + U * h.abs()
            pre = (cc * h).sum(1)
            e_pre = (cc.abs() * eh).sum(1) + 14 * U * (cc * h).abs().sum(1)
            if skip is not None:
                pre = pre + skip * xs
                e_pre = e_pre + U * pre.abs()
            y, ey = pre, e_pre
            if z is not None:
                y = pre * silu[b, s]
                ey = silu[b, s].abs() * e_pre + y.abs() * (rel[b, s] + U)
            put("y", (b, s), y, ey)
            kept.append((raw, e_raw, d, ed, F, r, step, e_step, before, e_before, h, eh, pre, e_pre))
        put("ht", n, h, eh)
        g = grads["dht"][n] if dht else zero(D, N)
        eg, gabs = zero(D, N), g.abs()
        for s in range(hi - 1, lo - 1, -1):
            raw, e_raw, d, ed, F, r, step, e_step, before, e_before, h, eh, pre, e_pre = kept[s - lo]
            xs, bb, cc, dy = x[b, s], wide(Bm[b, s]), wide(Cm[b, s]), grads["dy"][b, s]
            go, ego = dy, torch.zeros_like(dy)
            if z is not None:
                go = dy * silu[b, s]
                ego = go.abs() * (rel[b, s] + U)
            g = cc * go[:, None] + g
            eg = cc.abs() * ego[:, None] + eg + U * g.abs()
            gabs = (cc * go[:, None]).abs() + gabs
            carry = g * F
            e_carry = F * eg + carry.abs() * (r + U)
            gabs = gabs * F
            if (s - lo) % chunk == 0:
                e_carry = e_carry + chunk * U * gabs
            sB = (g * bb).sum(1)
            e_sB = (bb.abs() * eg).sum(1) + 14 * U * (g * bb).abs().sum(1)
            q = carry * before
            eq = carry.abs() * e_before + before.abs() * e_carry + U * q.abs()
            qA = (q * A).sum(1)
            e_qA = (aA * eq).sum(1) + 18 * U * (q * A).abs().sum(1)
            dx = d * sB
            e_dx = sB.abs() * ed + d.abs() * e_sB + U * dx.abs()
            if skip is not None:
                e_dx = e_dx + skip.abs() * ego + 2 * U * ((skip * go).abs() + dx.abs())
                dx = dx + skip * go
            put("dx", (b, s), dx, e_dx)
            dd = xs * sB + qA
            e_dd = xs.abs() * e_sB + e_qA + U * dd.abs() + U * qA.abs()
            if softplus:
                sr = torch.sigmoid(raw)
                e_dd = sr * e_dd + dd.abs() * sr * ((1 - sr) * e_raw + (2 * raw.abs() + 9) * U)
                dd = dd * sr
            put("ddt", (b, s), dd, e_dd)
            if z is not None:
                dz = dy * pre * slope[b, s]
                put("dz", (b, s), dz,
                    dy.abs() * (slope[b, s].abs() * e_pre + pre.abs() * e_slope[b, s]) + 2 * U * dz.abs())
            for name, v, ev in (("dB", step[:, None] * g, step.abs()[:, None] * eg + g.abs() * e_step[:, None]),
                                ("dC", go[:, None] * h, go.abs()[:, None] * eh + h.abs() * ego[:, None])):
                put(name, (b, s), joined(v), joined(ev) + (16 + D / G / 8) * U * joined(v.abs()))
            for name, v, ev in (("dA", d[:, None] * q, d.abs()[:, None] * eq + q.abs() * ed[:, None]),
                                ("dD", go * xs, xs.abs() * ego), ("ddt_bias", dd, e_dd)):
                out[name][0] += v
                out[name][1] += ev
                terms[name] += v.abs()
            g, eg = carry, e_carry
        put("dh0", n, g, eg)
    for name in ("dA", "dD", "ddt_bias"):
        out[name][1] += (chunk + slots + 20) * U * terms[name]
    return {k: (v, 1.05 * e) for k, (v, e) in out.items()}


def within(got, want, label):
    """got against (value, bound): the bound, and half a step of a 16-bit type."""
    value, bound = want
    g = got.detach().double().cpu()
    assert g.shape == value.shape, (label, g.shape, value.shape)
    if g.numel() == 0:
        return
    assert torch.isfinite(g).all(), label
    half = torch.finfo(got.dtype).eps / 2 if got.dtype != torch.float32 else 0.0
    off = (g - value).abs()
    # values that fp32 or the 16-bit type holds with fewer bits, or not at all, lie below 2^-120
    limit = half * value.abs() + (1 + half) * bound + 2.0 ** -120
    worst = (off / limit).max()
    assert worst <= 1, (label, "off by", float(worst), "times the bound")
