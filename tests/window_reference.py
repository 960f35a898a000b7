"""Attention over a sliding window with sinks in 64 bits, its gradients from their formulas, each
value with a bound on what the kernels' arithmetic may be off.

With u = 2^-24 (half a step of fp32) and r = half a step of the tensors' type where that is bf16, else 0:

* a score is a sum of d products: off by (d + 4) u of scale sum |q k|, and its product with log2 e, the
  difference with the maximum and the exponential by 4 u of their sizes, 4 units: E in all.  A weight
  p = e^{s - lse} is off by 2 E + (n + 16) u of itself (lse's sum over n keys, joined in any order), and by r
  where it is an operand of a product in bf16;
* o = sum p v: each term off by p's error, sums of n terms by n u of sum p |v|; then r of itself;
* dP = do . v: (d + 4) u of sum |do v|; D = do . o: the o that is read is off by its bound;
* dS = p (dP - D): p's error on |dP - D|, p times the errors of dP and D, and r of itself as an operand;
* dq = scale sum dS k, dk = scale sum dS q, dv = sum p do: their terms' errors, n u of the sums of absolute
  values, r of itself.

5 % on all of it covers terms of second order."""
from __future__ import annotations

import torch

import layer_reference as ref

U = 2.0 ** -24


def seen_mask(T, window, sinks):
    t = torch.arange(T)[:, None]
    j = torch.arange(T)[None, :]
    return (j <= t) & ((t - j < window) | (j < sinks))


def attention(q, k, v, window, sinks, lengths=None, scale=None, do=None, half=0.0):
    """{name: (value, bound)} of o and lse, and with `do` of dq, dk and dv; operands in 64 bits on the CPU."""
    B, T, Nq, d = q.shape
    Nk = k.shape[2]
    G = Nq // Nk
    scale = d ** -0.5 if scale is None else scale
    zero = q.new_zeros
    out = {n: [zero(s), zero(s)] for n, s in dict(o=q.shape, lse=(B, T, Nq)).items()}
    if do is not None:
        out.update({n: [zero(s), zero(s)] for n, s in dict(dq=q.shape, dk=k.shape, dv=v.shape).items()})
    absum = {n: zero(k.shape) for n in ("dk", "dv")}
    for b, lo, hi in ref.spans(B, T, lengths):
        n = hi - lo
        if n == 0:
            continue
        seen = seen_mask(n, window, sinks)
        for h in range(Nq):
            Q, K, V = q[b, lo:hi, h], k[b, lo:hi, h // G], v[b, lo:hi, h // G]
            # what no pair sees is not looked at: a masked key may hold anything
            S = torch.where(seen, scale * (Q @ K.T), torch.tensor(-torch.inf, dtype=Q.dtype))
            size = torch.where(seen, scale * (Q.abs() @ K.abs().T), torch.tensor(0.0, dtype=Q.dtype))
            lse = torch.logsumexp(S, -1)
            P = torch.exp(S - lse[:, None])
            keys = min(n, window + sinks)
            top = torch.where(seen, S.abs(), torch.tensor(0.0, dtype=Q.dtype)).amax(-1, keepdim=True)
            E = (d + 4) * U * size.amax(-1, keepdim=True) + 4 * U * (top + lse.abs()[:, None]) + 4 * U
            rel = 2 * E + (keys + 16) * U
            eP = P * (rel + half)
            O = P @ V
            eO = eP @ V.abs() + keys * U * (P @ V.abs())
            out["o"][0][b, lo:hi, h] = O
            eO = eO + half * (O.abs() + eO)
            out["o"][1][b, lo:hi, h] = eO
            out["lse"][0][b, lo:hi, h] = lse
            out["lse"][1][b, lo:hi, h] = (rel[:, 0] + 8 * U * (1 + lse.abs()))
            if do is None:
                continue
            g = do[b, lo:hi, h]
            dP = torch.where(seen, g @ V.T, torch.tensor(0.0, dtype=Q.dtype))
            D = (g * O).sum(-1, keepdim=True)
            eD = (g.abs() * eO).sum(-1, keepdim=True) + (d + 4) * U * (g.abs() * O.abs()).sum(-1, keepdim=True)
            dS = P * (dP - D)
            edS = P * rel * (dP - D).abs() + P * ((d + 4) * U * (g.abs() @ V.abs().T) + eD + 2 * U * (dP - D).abs())
            edS = torch.where(seen, edS, torch.tensor(0.0, dtype=Q.dtype))
            edS = edS + half * (dS.abs() + edS)
            dq = scale * (dS @ K)
            e = scale * (edS @ K.abs() + keys * U * (dS.abs() @ K.abs()))
            out["dq"][0][b, lo:hi, h] = dq
            out["dq"][1][b, lo:hi, h] = e + (half + 2 * U) * (dq.abs() + e)
            span = slice(lo, hi)
            out["dk"][0][b, span, h // G] += scale * (dS.T @ Q)
            out["dk"][1][b, span, h // G] += scale * (edS.T @ Q.abs())
            absum["dk"][b, span, h // G] += scale * (dS.abs().T @ Q.abs())
            out["dv"][0][b, span, h // G] += P.T @ g
            out["dv"][1][b, span, h // G] += eP.T @ g.abs()
            absum["dv"][b, span, h // G] += P.T @ g.abs()
        for name in ("dk", "dv") if do is not None else ():
            value, bound = out[name][0][b, lo:hi], out[name][1][b, lo:hi]
            e = bound + (n * G + 16) * U * absum[name][b, lo:hi]
            out[name][1][b, lo:hi] = e + (half + 2 * U) * (value.abs() + e)
    return {n: (x, 1.05 * e + 1e-30) for n, (x, e) in out.items()}


def close(got, want, label=""):
    value, bound = want
    g = got.detach().double().cpu()
    assert g.shape == value.shape, (label, g.shape, value.shape)
    assert torch.isfinite(g).all(), label
    if not g.numel():
        return
    over = (g - value).abs() - bound
    assert float(over.max()) <= 0, (label, "over by", float(over.max()), "largest error", float((g - value).abs().max()))


def slot(p, sinks, ring):
    return p if p < sinks else sinks + (p - sinks) % ring


def cache_of(rows, had, sinks, ring, cache):
    """The cache [Nk, sinks + ring, d] after rows [T, Nk, d] at positions `had` on, token by token."""
    cache = cache.clone()
    for i in range(rows.shape[0]):
        cache[:, slot(had + i, sinks, ring)] = rows[i]
    return cache
