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


def head_forward(q, k, v, scale, before):
    """One head: q [n, D] at positions before .. before + n - 1, k and v [m, D]. Returns
    (out, lse, weights, bound of out, bound of the relative error of the weights)."""
    n, D = q.shape
    m = k.shape[0]
    q, k, v = q.to(F64), k.to(F64), v.to(F64)
    hidden = torch.arange(m, device=q.device)[None] > before + torch.arange(n, device=q.device)[:, None]
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
