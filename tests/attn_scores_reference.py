"""Attention in 64 bits with capped scores, a bias by distance and prefixes, straight from its
definition, sequence by sequence and head by head, and bounds of what the kernels' rounding can do
to it. Shared by the CPU and GPU tests.

Bounds. With u half the storage type's step: a score errs by
    e_ij = D 2^-24 scale sum_d |q k|  +  2^-21 |capped score|  +  2^-22 (|score| + |bias|)
(the fp32 sum over D, whose error a tanh does not enlarge; the roundings of scale / cap, of its
product, of the tanh, within 2^-22, and of cap log2 e, six half steps in all; the roundings of
slope log2 e, its product with the distance and the sum, at most 3 half steps of either part). It moves the weight
P_ij by a relative e_ij and, through the normalizer, all weights of the row by the mean
E_i = sum_j P_ij e_ij. The weights are rounded to the storage type (u), their sum over n keys errs by
n 2^-24, exp2 and the division by a few 2^-23, and the output is rounded once:
    |out - exact| <= sum_j P_ij (u + e_ij + E_i + (n + 32) 2^-23) |v_j| + u |exact|
up to second order, for which 1% is added. Backward, P is formed again from the scores and the rounded
lse (|lse| 2^-22 + 2^-21 more), dP errs by D 2^-24 sum |do v|, D_i, where it is formed from the rounded output
(prefixes alone), by sum |do| times the output's bound, and else, a sum of P dP, by what P and dP are
off and n 2^-23 of its magnitudes; r = 1 - t^2 by 2 |t| times what t is off, (1 - t^2) e / cap + |t| 2^-21, and
2^-24; dS = P (dP - D_i) r is rounded once (for dq of changed scores up to D = 64, in two parts, u^2), sums
over c terms err by c 2^-24 of their magnitudes and outputs are rounded once.
"""
import torch

import attn_reference
from attn_reference import F64, check, half_step, sequences  # noqa: F401


def tiny(dtype):
    return 0.0 if dtype == F64 else attn_reference.tiny(dtype)


def head(q, k, v, scale, before, held, cap=None, slope=None, prefix=0, gone=None):
    """One head: q [n, D] at positions before .. before + n - 1 of a sequence that holds `held` tokens,
    whose first keys are k and v [m, D]; `gone` [m]: keys that nobody sees. A dict of 64-bit tensors."""
    n, D = q.shape
    m = k.shape[0]
    q, k, v = q.to(F64), k.to(F64), v.to(F64)
    i = before + torch.arange(n, device=q.device)[:, None]
    j = torch.arange(m, device=q.device)[None]
    seen = ((j <= i) | (j < prefix)) & (j < held) & (i >= 0)
    if gone is not None:
        seen = seen & ~gone[None]
        k, v = k.masked_fill(gone[:, None], 0.0), v.masked_fill(gone[:, None], 0.0)
    s = q @ k.T * scale
    e = D * 2.0 ** -24 * (q.abs() @ k.abs().T * scale)
    t = None
    if cap is not None:
        t = torch.tanh(s / cap)
        s = cap * t
        e = e + 2.0 ** -21 * s.abs()
    if slope is not None:
        bias = slope * (i - j).abs().to(F64)
        e = e + 2.0 ** -22 * (s.abs() + bias.abs())
        s = s - bias
    s = s.masked_fill(~seen, float("-inf"))
    lse = torch.logsumexp(s, -1) if m else torch.full((n,), float("-inf"), dtype=F64, device=q.device)
    p = torch.exp(s - torch.where(lse == float("-inf"), 0.0, lse)[:, None]).masked_fill(~seen, 0.0)
    e = e.masked_fill(~seen, 0.0)
    mean = (p * e).sum(-1, keepdim=True)
    return dict(out=p @ v, lse=lse, p=p, t=t, e=e, mean=mean, seen=seen, k=k, v=v,
                rel=e + mean + (m + 32) * 2.0 ** -23)


def out_bound(h, u, dtype):
    return 1.01 * ((h["p"] * (u + h["rel"])) @ h["v"].abs() + u * h["out"].abs()) + tiny(dtype)


def lse_bound(h):
    """The mean error of the scores, the sum, the logarithm and the rounding of lse itself."""
    lse = h["lse"].masked_fill(h["lse"] == float("-inf"), 0.0)
    n = h["p"].shape[-1]
    return 1.01 * (h["mean"][:, 0] + (n + 32) * 2.0 ** -24 + (4.0 + lse.abs()) * 2.0 ** -22)


def _head_args(h, slopes, cap):
    return dict(cap=cap, slope=None if slopes is None else float(slopes[h]))


def forward(q, k, v, seqs, scale, cap=None, slopes=None, prefixes=None):
    """(out, lse, bound of out, bound of lse) of packed sequences; rows of none are 0 and -inf."""
    T, Hq, _ = q.shape
    G = Hq // k.shape[1]
    u = half_step(q.dtype)
    out, tol = (torch.zeros(q.shape, dtype=F64, device=q.device) for _ in range(2))
    lse = torch.full((T, Hq), float("-inf"), dtype=F64, device=q.device)
    ltol = torch.zeros_like(lse)
    for s, (a, n) in enumerate(seqs):
        if n == 0:
            continue
        sl = slice(a, a + n)
        for h in range(Hq):
            r = head(q[sl, h], k[sl, h // G], v[sl, h // G], scale, 0, n, **_head_args(h, slopes, cap),
                     prefix=0 if prefixes is None else int(prefixes[s]))
            out[sl, h], lse[sl, h] = r["out"], r["lse"]
            tol[sl, h], ltol[sl, h] = out_bound(r, u, q.dtype), lse_bound(r)
    return out, lse, tol, ltol


def paged(q, k_cache, v_cache, table, cu, lens, scale, cap=None, slopes=None, prefixes=None):
    """The same of the new tokens over a paged cache; keys behind the table or on no page are seen
    by nobody."""
    T, Hq, _ = q.shape
    pages, page, Hkv, _ = k_cache.shape
    u = half_step(q.dtype)
    out, tol = (torch.zeros(q.shape, dtype=F64, device=q.device) for _ in range(2))
    lse = torch.full((T, Hq), float("-inf"), dtype=F64, device=q.device)
    ltol = torch.zeros_like(lse)
    for s, (a, n) in enumerate(sequences(cu, T)):
        m = min(max(int(lens[s]), 0), table.shape[1] * page)
        if n == 0 or m == 0:
            continue
        at = torch.arange(m, device=q.device)
        number = table[s].to(q.device).long()[at // page]
        gone = (number < 0) | (number >= pages)
        number = number.masked_fill(gone, 0)
        for h in range(Hq):
            k, v = (c[number, at % page, h // (Hq // Hkv)] for c in (k_cache, v_cache))
            r = head(q[a:a + n, h], k, v, scale, int(lens[s]) - n, int(lens[s]), **_head_args(h, slopes, cap),
                     prefix=0 if prefixes is None else int(prefixes[s]), gone=gone)
            out[a:a + n, h], lse[a:a + n, h] = r["out"], r["lse"]
            tol[a:a + n, h], ltol[a:a + n, h] = out_bound(r, u, q.dtype), lse_bound(r)
    return out, lse, tol, ltol


def backward(do, q, k, v, seqs, scale, dtype, cap=None, slopes=None, prefixes=None):
    """(dq, dk, dv) and their bounds."""
    u = half_step(dtype)
    G = q.shape[1] // k.shape[1]
    D = q.shape[2]
    grads = [torch.zeros(x.shape, dtype=F64, device=q.device) for x in (q, k, v)]
    tols = [torch.zeros_like(x) for x in grads]
    for s, (a, n) in enumerate(seqs):
        if n == 0:
            continue
        sl = slice(a, a + n)
        for h in range(q.shape[1]):
            g = h // G
            qh, kh, vh, dh = (x.to(F64) for x in (q[sl, h], k[sl, g], v[sl, g], do[sl, h]))
            f = head(qh, kh, vh, scale, 0, n, **_head_args(h, slopes, cap),
                     prefix=0 if prefixes is None else int(prefixes[s]))
            p = f["p"]
            rp = f["rel"] + f["lse"].abs()[:, None] * 2.0 ** -22 + 2.0 ** -21
            dp, delta = dh @ vh.T, (dh * f["out"]).sum(-1, keepdim=True)
            e_dp = D * 2.0 ** -24 * (dh.abs() @ vh.abs().T)
            changed = cap is not None or slopes is not None
            if changed:
                e_delta = (p * ((rp + (n + 32) * 2.0 ** -23) * dp.abs() + e_dp)).sum(-1, keepdim=True)
            else:
                e_delta = (dh.abs() * (out_bound(f, u, dtype) + D * 2.0 ** -24 * f["out"].abs())).sum(-1, keepdim=True)
            r, e_r = 1.0, 0.0
            if cap is not None:
                r = 1 - f["t"] ** 2
                e_r = 2 * f["t"].abs() * (r * f["e"] / cap + f["t"].abs() * 2.0 ** -21) + 2.0 ** -24
            ds = p * (dp - delta) * r
            e_ds = rp * ds.abs() + p * ((e_dp + e_delta) * (r + e_r) + (dp - delta).abs() * e_r) * (1 + rp)
            e_dsq = (u * u if changed and D <= 64 else u) * ds.abs() + e_ds + tiny(dtype)
            e_ds = u * ds.abs() + e_ds + tiny(dtype)
            e_p = (u + rp) * p + tiny(dtype)
            c = (n * G + 64) * 2.0 ** -24
            grads[0][sl, h] = scale * (ds @ kh)
            terms = 2 if changed and D <= 64 else 1
            tols[0][sl, h] = 1.01 * scale * (e_dsq @ kh.abs() + terms * c * (ds.abs() @ kh.abs()))
            grads[1][sl, g] += scale * (ds.T @ qh)
            tols[1][sl, g] += 1.01 * scale * (e_ds.T @ qh.abs() + c * (ds.abs().T @ qh.abs()))
            grads[2][sl, g] += p.T @ dh
            tols[2][sl, g] += 1.01 * (e_p.T @ dh.abs() + c * (p.T @ dh.abs()))
    tols = [t + 1.01 * u * x.abs() + tiny(dtype) for t, x in zip(tols, grads)]
    return grads, tols
