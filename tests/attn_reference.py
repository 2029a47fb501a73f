"""Attention in 64 bits, straight from its definition, sequence by sequence and head by head,
and bounds of what the kernels' rounding can do to it. Shared by the CPU and GPU tests.

Bounds. With u half the storage type's step (one rounding), the kernels round the weights
P_ij once (relative u) and the output once; scores are fp32 sums of D exact products, whose
error is at most D * 2^-24 * scale * sum_d |q k| =: e_ij each and moves a weight by a
relative e_ij, numerator and normalizer alike; the weights' fp32 sum over n keys errs by a
relative n * 2^-24, and exp2, the scaling by exp2(m) and the division by a few 2^-23. So
    |out - exact| <= u (A + |exact|) + (2 max e + (n + 32) 2^-23) A,   A = sum_j P_ij |v_j|,
up to second order, for which the bound is widened by 1%. The gradients' bounds follow the
same way, term by term (see backward_bounds).
"""
import torch

F64 = torch.float64


def sequences(cu, T, seqused=None):
    """(start, length) of each sequence as the kernels read cu_seqlens."""
    out, top = [], 0
    starts = []
    for c in cu:
        top = max(top, min(max(int(c), 0), T))
        starts.append(top)
    for s in range(len(cu) - 1):
        end = min(max(int(cu[s + 1]), starts[s]), T)
        n = end - starts[s]
        if seqused is not None:
            n = min(n, max(0, int(seqused[s])))
        out.append((starts[s], n))
    return out


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def head_forward(q, k, v, scale, before, gone=None):
    """One head: q [n, D] at positions before .. before + n - 1, k and v [m, D]; keys of the
    mask `gone` [m] are seen by nobody. Returns (out, lse, weights, bound of the relative
    error of the weights)."""
    n, D = q.shape
    m = k.shape[0]
    q, k, v = q.to(F64), k.to(F64), v.to(F64)
    hidden = torch.arange(m, device=q.device)[None] > before + torch.arange(n, device=q.device)[:, None]
    if gone is not None:
        hidden = hidden | gone[None]
        k, v = k.masked_fill(gone[:, None], 0.0), v.masked_fill(gone[:, None], 0.0)
    s = (q @ k.T * scale).masked_fill(hidden, float("-inf"))
    lse = torch.logsumexp(s, -1) if m else torch.full((n,), float("-inf"), dtype=F64, device=q.device)
    p = torch.exp(s - torch.where(lse == float("-inf"), 0.0, lse)[:, None])
    p = p.masked_fill(hidden, 0.0)
    out = p @ v
    worst = (q.abs() @ k.abs().T * scale).masked_fill(hidden, 0.0)
    e = D * 2.0 ** -24 * worst.amax(-1, keepdim=True) if m else torch.zeros((n, 1), dtype=F64,
                                                                            device=q.device)
    rel = 2 * e + (m + 32) * 2.0 ** -23
    return out, lse, p, rel


def forward(q, k, v, seqs, scale):
    """(out, lse, bound of out) of packed sequences; rows of none are 0 and -inf."""
    T, Hq, D = q.shape
    G = Hq // k.shape[1]
    u = half_step(q.dtype)
    out = torch.zeros((T, Hq, D), dtype=F64, device=q.device)
    tol = torch.zeros_like(out)
    lse = torch.full((T, Hq), float("-inf"), dtype=F64, device=q.device)
    for a, n in seqs:
        if n == 0:
            continue
        for h in range(Hq):
            o, l, p, rel = head_forward(q[a:a + n, h], k[a:a + n, h // G], v[a:a + n, h // G], scale, 0)
            spread = p @ v[a:a + n, h // G].to(F64).abs()
            out[a:a + n, h], lse[a:a + n, h] = o, l
            tol[a:a + n, h] = 1.01 * (u * (spread + o.abs()) + rel * spread)
    return out, lse, tol + tiny(q.dtype)


def paged(q, k_cache, v_cache, table, cu, lens, scale):
    """(out, lse, bound of out) of the new tokens over a paged cache; keys behind the table or
    on no page are seen by nobody."""
    T, Hq, D = q.shape
    pages, page, Hkv, _ = k_cache.shape
    u = half_step(q.dtype)
    out = torch.zeros((T, Hq, D), dtype=F64, device=q.device)
    tol = torch.zeros_like(out)
    lse = torch.full((T, Hq), float("-inf"), dtype=F64, device=q.device)
    for s, (a, n) in enumerate(sequences(cu, T)):
        m = min(max(int(lens[s]), 0), table.shape[1] * page)
        if n == 0 or m == 0:
            continue
        at = torch.arange(m, device=q.device)
        number = table[s].to(q.device).long()[at // page]
        gone = (number < 0) | (number >= pages)
        number = number.masked_fill(gone, 0)
        for h in range(Hq):
            k, v = k_cache[number, at % page, h // (Hq // Hkv)], v_cache[number, at % page, h // (Hq // Hkv)]
            o, l, p, rel = head_forward(q[a:a + n, h], k, v, scale, int(lens[s]) - n, gone)
            spread = p @ v.to(F64).masked_fill(gone[:, None], 0.0).abs()
            out[a:a + n, h], lse[a:a + n, h] = o, l
            tol[a:a + n, h] = 1.01 * (u * (spread + o.abs()) + rel * spread)
    return out, lse, tol + tiny(q.dtype)


def tiny(dtype):
    """What the smallest numbers of the type are off by (subnormal weights and outputs)."""
    return {torch.bfloat16: 2.0 ** -126, torch.float16: 2.0 ** -20, torch.float32: 2.0 ** -126}[dtype]


def check(got, want, tol, what):
    """got within tol of want, element by element."""
    assert got.shape == want.shape, (what, got.shape, want.shape)
    err = (got.to(F64) - want).abs()
    ok = (err <= tol) | (got.to(F64) == want)
    if not bool(ok.all()):
        i = int((~ok).to(torch.uint8).flatten().argmax())
        raise AssertionError(f"{what}: {int((~ok).sum())} of {ok.numel()} values are off, the first at {i}: "
                             f"{float(got.flatten()[i])} for {float(want.flatten()[i])}, "
                             f"allowed {float(tol.flatten()[i])}")


def check_lse(got, lse, D, worst):
    """lse: a sum's logarithm in fp32. The scores' error bound is `worst` (max scale sum |q k|)
    * D * 2^-24; the logarithm and the sum add a few 2^-22 and the rounding of lse itself."""
    tol = 1.01 * (D * 2.0 ** -24 * worst + (4.0 + lse.abs().masked_fill(lse == float("-inf"), 0)) * 2.0 ** -22
                  + 4096 * 2.0 ** -24)
    check(got, lse, tol, "lse")


def backward(do, q, k, v, seqs, scale, dtype):
    """(dq, dk, dv) and their bounds.

    P is formed again from the scores and the rounded lse: relative error rp = e + |lse| 2^-22
    + 2^-21. dP errs by D 2^-24 sum |do v|, and D_i by sum |do| times what the rounded
    forward output is off (the forward's bound). dS = P (dP - D_i) is rounded once, and so
    is P for dV; sums over c terms err by c 2^-24 of the sum of magnitudes; outputs are
    rounded once."""
    u = half_step(dtype)
    G = q.shape[1] // k.shape[1]
    D = q.shape[2]
    grads = [torch.zeros(x.shape, dtype=F64, device=q.device) for x in (q, k, v)]
    tols = [torch.zeros_like(x) for x in grads]
    for a, n in seqs:
        if n == 0:
            continue
        sl = slice(a, a + n)
        for h in range(q.shape[1]):
            g = h // G
            qh, kh, vh, dh = (x.to(F64) for x in (q[sl, h], k[sl, g], v[sl, g], do[sl, h]))
            o, lse, p, rel = head_forward(qh, kh, vh, scale, 0)
            spread = p @ vh.abs()
            tol_o = 1.01 * (u * (spread + o.abs()) + rel * spread) + tiny(dtype)
            rp = rel + lse.abs()[:, None] * 2.0 ** -22 + 2.0 ** -21
            dp, delta = dh @ vh.T, (dh * o).sum(-1, keepdim=True)
            e_dp = D * 2.0 ** -24 * (dh.abs() @ vh.abs().T)
            e_delta = (dh.abs() * (tol_o + D * 2.0 ** -24 * o.abs())).sum(-1, keepdim=True)
            ds = p * (dp - delta)
            e_ds = (u + rp) * ds.abs() + p * (e_dp + e_delta) * (1 + rp) + tiny(dtype)
            e_p = (u + rp) * p + tiny(dtype)
            c = (n * G + 64) * 2.0 ** -24
            grads[0][sl, h] = scale * (ds @ kh)
            tols[0][sl, h] = 1.01 * scale * (e_ds @ kh.abs() + c * (ds.abs() @ kh.abs()))
            grads[1][sl, g] += scale * (ds.T @ qh)
            tols[1][sl, g] += 1.01 * scale * (e_ds.T @ qh.abs() + c * (ds.abs().T @ qh.abs()))
            grads[2][sl, g] += p.T @ dh
            tols[2][sl, g] += 1.01 * (e_p.T @ dh.abs() + c * (p.T @ dh.abs()))
    tols = [t + 1.01 * u * x.abs() + tiny(dtype) for t, x in zip(tols, grads)]
    return grads, tols
