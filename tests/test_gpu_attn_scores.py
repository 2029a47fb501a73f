"""GPU tests of the attention with capped scores, a bias by distance and prefixes, packed and over
a paged cache, against its definition in 64 bits (attn_scores_reference)."""
import pytest
import torch

import attn_scores_reference as ref

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
BF16, F16 = torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def rope():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import packed_varlen_rotary_rope_amd as m
    return m


def normal(shape, seed, dtype, size=1.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return (torch.randn(shape, generator=g, device=DEV) * size).to(dtype)


def int32(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def slopes_of(Hq, flat=False):
    """A falling series; `flat`: one that grows with the distance too, and a head without any."""
    s = [2.0 ** (-8.0 * (h + 1) / Hq) for h in range(Hq)]
    if flat:
        s = [0.0 if h == 0 else -x / 64 if h % 2 else x for h, x in enumerate(s)]
    return torch.tensor(s, dtype=torch.float32, device=DEV)


# what scores go through: cap, slopes, prefixes (per cent of a sequence's length; every third has none)
FORMS = {"cap": (20.0, None, None), "low_cap": (1.5, None, None), "slopes": (None, False, None),
         "both": (30.0, True, None), "prefix": (None, None, 55), "all": (8.0, False, 40),
         "whole": (None, True, 100), "cap_prefix": (50.0, None, 30)}

SHAPES = [  # cu_seqlens, T, Hq, Hkv, D, dtype
    ([0, 1], 1, 1, 1, 8, BF16),
    ([0, 5, 22, 25, 64], 64, 4, 2, 16, F16),
    ([0, 64, 65, 192, 193], 193, 4, 4, 64, BF16),
    ([0, 127, 255, 384, 384, 600], 600, 8, 2, 128, BF16),
    ([3, 40, 140], 150, 5, 1, 96, F16),       # rows before and behind the sequences
    ([0, 301, 412], 412, 7, 1, 72, BF16),     # groups that divide no tile
    ([0, 1000], 1000, 8, 1, 128, F16),
    ([0, 900, 1037], 1037, 2, 1, 64, BF16),
    ([0, 500], 500, 2, 1, 160, BF16),
    ([0, 450], 450, 4, 2, 256, F16),
    ([0] + list(range(1, 41)), 40, 32, 8, 128, BF16),  # one token each
    ([0, 1100], 1100, 160, 1, 32, BF16),      # more heads in a group than a tile has rows
]


def case_id(c):
    return f"T{c[1]}_{c[2]}_{c[3]}_{c[4]}_{str(c[5])[6:]}"


def form_args(form, cu, Hq):
    cap, flat, percent = FORMS[form]
    prefixes = None
    if percent is not None:
        prefixes = [0 if s % 3 == 2 else (b - a) * percent // 100 + (percent == 100) * 7
                    for s, (a, b) in enumerate(zip(cu, cu[1:]))]
    return cap, None if flat is None else slopes_of(Hq, flat), prefixes


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("case", SHAPES, ids=case_id)
def test_forward_and_backward(rope, case, form):
    cu, T, Hq, Hkv, D, dtype = case
    print(f"[attn scores] {case_id(case)} {form}", flush=True)
    cap, slopes, prefixes = form_args(form, cu, Hq)
    q, k, v = normal((T, Hq, D), 1, dtype, 3.0 if cap else 1.0), normal((T, Hkv, D), 2, dtype), normal((T, Hkv, D), 3, dtype)
    plan = rope.attn_plan(int32(cu), T, Hq, Hkv, prefix_lens=None if prefixes is None else int32(prefixes))
    more = dict(softcap=cap, slopes=slopes)
    out, lse = rope.attn_fwd(q, k, v, plan, **more)
    seqs = ref.sequences(cu, T)
    args = (seqs, D ** -0.5)
    want, wlse, tol, ltol = ref.forward(q, k, v, *args, cap, slopes, prefixes)
    ref.check(out, want, tol, "out")
    ref.check(lse, wlse, ltol, "lse")
    if D > 128:
        return
    do = normal((T, Hq, D), 4, dtype)
    grads = rope.attn_bwd(do, q, k, v, out, lse, plan, **more)
    for name, got, x, t in zip(("dq", "dk", "dv"), grads, *ref.backward(do, q, k, v, *args, dtype, cap, slopes, prefixes)):
        ref.check(got, x, t, name)


# new tokens, held tokens, Hq, Hkv, D, page, dtype
STEPS = [
    ([1], [1], 1, 1, 8, 1, BF16),
    ([1, 1, 1, 1], [5, 4099, 64, 1000], 8, 2, 128, 16, BF16),
    ([1, 1], [2000, 33], 8, 8, 64, 7, F16),
    ([4, 3, 1], [513, 64, 90], 16, 2, 80, 48, F16),
    ([100, 200], [100, 1700], 8, 2, 128, 64, BF16),
    ([257, 1, 31, 1], [3001, 500, 31, 8], 12, 4, 96, 24, BF16),
    ([0, 2, 0], [40, 50, 0], 6, 3, 72, 5, F16),
    ([1, 40], [700, 777], 4, 2, 256, 16, BF16),
    ([1, 33], [150, 1030], 4, 4, 192, 16, F16),
    ([5], [3], 4, 2, 64, 16, BF16),   # fewer held than new: the first two see no key
    ([16], [9000], 160, 2, 128, 64, BF16),
]


def pool(lens, page, Hkv, D, dtype, seed):
    """(k_cache, v_cache, table): pages in a shuffled order, NaN where no sequence is."""
    g = torch.Generator().manual_seed(seed)
    used = [-(-max(m, 0) // page) for m in lens]
    order = torch.randperm(sum(used) + 2, generator=g)
    table = torch.full((len(lens), max([1] + used)), -7, dtype=torch.int32)
    caches = [torch.full((sum(used) + 2, page, Hkv, D), float("nan"), dtype=dtype, device=DEV) for _ in range(2)]
    at = 0
    for s, m in enumerate(lens):
        table[s, :used[s]] = order[at:at + used[s]].int()
        at += used[s]
        if m > 0:
            pos = torch.arange(m)
            where = table[s].long()[pos // page].to(DEV), (pos % page).to(DEV)
            for i, c in enumerate(caches):
                c[where] = normal((m, Hkv, D), 1000 * seed + 2 * s + i, dtype)
    return caches[0], caches[1], table.to(DEV)


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("case", STEPS, ids=lambda c: f"n{sum(c[0])}_m{max(c[1])}_{c[2]}_{c[3]}_{c[4]}_{c[5]}_{str(c[6])[6:]}")
def test_paged(rope, case, form):
    new, held, Hq, Hkv, D, page, dtype = case
    print(f"[attn_paged scores] {str(case)[:120]} {form}", flush=True)
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    cap, slopes, _ = form_args(form, cu, Hq)
    prefixes = None
    if FORMS[form][2] is not None:
        prefixes = [0 if s % 3 == 2 else m * FORMS[form][2] // 100 for s, m in enumerate(held)]
    k, v, table = pool(held, page, Hkv, D, dtype, 5)
    q = normal((cu[-1], Hq, D), 3, dtype, 3.0 if cap else 1.0)
    plan = rope.paged_plan(int32(cu), int32(held), cu[-1], Hq, Hkv,
                           prefix_lens=None if prefixes is None else int32(prefixes))
    out, lse = rope.attn_paged(q, k, v, table, plan, softcap=cap, slopes=slopes)
    want, wlse, tol, ltol = ref.paged(q, k, v, table, cu, held, D ** -0.5, cap, slopes, prefixes)
    ref.check(out, want, tol, "out")
    ref.check(lse, wlse, ltol, "lse")


def bits(t):
    return t.contiguous().view(torch.int32 if t.dtype == torch.float32 else torch.int16)


def same(a, b):
    return torch.equal(bits(a), bits(b))


def test_nothing_changed_is_the_plain_attention(rope):
    """Bit for bit, with prefixes of 0 and 1 and without."""
    T, cu = 500, [0, 3, 250, 500]
    q, k, v, do = (normal((T, h, 64), i, BF16) for i, h in enumerate((6, 2, 2, 6)))
    want = None
    for prefixes in (None, [0, 0, 0], [1, 0, -5]):
        plan = rope.attn_plan(int32(cu), T, 6, 2, prefix_lens=None if prefixes is None else int32(prefixes))
        out, lse = rope.attn_fwd(q, k, v, plan)
        got = (out, lse, *rope.attn_bwd(do, q, k, v, out, lse, plan))
        want = want or got
        assert all(same(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("size", [1.0, 30.0, 1000.0])
def test_scores_beyond_the_cap(rope, dtype, size):
    """Small, large and saturated scores side by side, forward and backward."""
    cu, T, Hq, Hkv, D = [0, 130, 400], 400, 4, 2, 128
    q, k, v, do = (normal((T, h, D), 10 + i, dtype) for i, h in enumerate((Hq, Hkv, Hkv, Hq)))
    q[::3] *= size
    k[::5] *= 0.01
    plan = rope.attn_plan(int32(cu), T, Hq, Hkv)
    out, lse = rope.attn_fwd(q, k, v, plan, softcap=7.0)
    seqs = ref.sequences(cu, T)
    want, wlse, tol, ltol = ref.forward(q, k, v, seqs, D ** -0.5, 7.0)
    ref.check(out, want, tol, "out")
    ref.check(lse, wlse, ltol, "lse")
    grads = rope.attn_bwd(do, q, k, v, out, lse, plan, softcap=7.0)
    for name, got, x, t in zip(("dq", "dk", "dv"), grads, *ref.backward(do, q, k, v, seqs, D ** -0.5, dtype, 7.0)):
        ref.check(got, x, t, name)


def test_infinite_scores_are_capped(rope):
    """Scores past fp32 count as plus or minus the cap. Weights are then known: e^c and e^-c for the
    signs of the keys; they err by their rounding, half a step, and a few 2^-22."""
    T, D, c = 50, 64, 3.0
    q = torch.full((T, 1, D), 3e38, dtype=BF16, device=DEV)
    sign = torch.where(torch.arange(T, device=DEV) % 3 == 0, 1.0, -1.0)
    k = sign.to(BF16)[:, None, None].expand(T, 1, D).contiguous()
    v = normal((T, 1, D), 1, BF16)
    plan = rope.attn_plan(int32([0, T]), T, 1, 1)
    out, lse = rope.attn_fwd(q, k, v, plan, softcap=c)
    w = torch.exp(c * sign.double()).expand(T, T).tril()
    p = w / w.sum(-1, keepdim=True)
    want = p @ v[:, 0].double()
    u = ref.half_step(BF16)
    ref.check(out[:, 0], want, 1.01 * ((u + 64 * 2.0 ** -22) * (p @ v[:, 0].double().abs()) + u * want.abs()), "out")
    grads = rope.attn_bwd(v, q, k, v, out, lse, plan, softcap=c)
    assert not bool(grads[0].any()) and not bool(grads[1].any()) and bool(torch.isfinite(grads[2]).all())


@pytest.mark.parametrize("form", ["cap", "slopes", "all"])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("D", [64, 128])
def test_hidden_values_have_no_influence(rope, form, value, D):
    """Of the last token of either sequence: its key and value reach the rows that see it alone, its query and
    upstream gradient the keys that it sees, which are all."""
    cu, T, Hq, Hkv = [0, 70, 240], 240, 4, 2
    cap, slopes, prefixes = form_args(form, cu, Hq)
    plan = rope.attn_plan(int32(cu), T, Hq, Hkv, prefix_lens=None if prefixes is None else int32(prefixes))
    more = dict(softcap=cap, slopes=slopes)
    q, k, v, do = (normal((T, h, D), i, BF16) for i, h in enumerate((Hq, Hkv, Hkv, Hq)))

    def run(k, v):
        out, lse = rope.attn_fwd(q, k, v, plan, **more)
        return (out, lse, *rope.attn_bwd(do, q, k, v, out, lse, plan, **more))

    want = run(k, v)
    rest = torch.ones(T, dtype=torch.bool, device=DEV)
    rest[[69, 239]] = False
    for which in range(2):
        x = [k.clone(), v.clone()]
        x[which][~rest, :, 3] = value
        got = run(*x)
        for a, b in zip(got[:3], want[:3]):  # out, lse, dq
            assert same(a[rest], b[rest])
    # rows of no sequence behind the last, and a sequence cut by seqused
    seqused = int32([50, 170])
    plan2 = rope.attn_plan(int32(cu), T, Hq, Hkv, seqused=seqused,
                           prefix_lens=None if prefixes is None else int32([min(p, 50) for p in prefixes]))
    k[50:70], v[50:70], q[50:70], do[50:70] = value, value, value, value
    out, lse = rope.attn_fwd(q, k, v, plan2, **more)
    grads = rope.attn_bwd(do, q, k, v, out, lse, plan2, **more)
    assert not bool(out[50:70].any()) and bool((lse[50:70] == float("-inf")).all())
    for g in grads:
        assert not bool(g[50:70].any()) and bool(torch.isfinite(g).all())


@pytest.mark.parametrize("D,form", [(64, "all"), (128, "cap_prefix"), (32, "whole"), (96, "both")])
def test_long_sequence_of_one_head(rope, D, form):
    """The work of its key tiles is cut between workgroups, in the prefix and behind it."""
    T, cu = 4001, [0, 3900, 4001]
    cap, slopes, prefixes = form_args(form, cu, 1)
    q, k, v, do = (normal((T, 1, D), i, BF16) for i in range(4))
    plan = rope.attn_plan(int32(cu), T, 1, 1, prefix_lens=None if prefixes is None else int32(prefixes))
    more = dict(softcap=cap, slopes=slopes)
    out, lse = rope.attn_fwd(q, k, v, plan, **more)
    args = (ref.sequences(cu, T), D ** -0.5)
    want, wlse, tol, ltol = ref.forward(q, k, v, *args, cap, slopes, prefixes)
    ref.check(out, want, tol, "out")
    ref.check(lse, wlse, ltol, "lse")
    grads = rope.attn_bwd(do, q, k, v, out, lse, plan, **more)
    for name, got, x, t in zip(("dq", "dk", "dv"), grads, *ref.backward(do, q, k, v, *args, BF16, cap, slopes, prefixes)):
        ref.check(got, x, t, name)


def test_many_sequences_with_prefixes(rope):
    """More sequences than a plan's chunk, of 0 to 9 tokens, prefixes of any size."""
    g = torch.Generator().manual_seed(3)
    lens = torch.randint(0, 10, (2300,), generator=g)
    cu = [0] + lens.cumsum(0).tolist()
    T, D = cu[-1], 16
    prefixes = torch.randint(-3, 12, (2300,), generator=g).tolist()
    q, k, v, do = (normal((T, 1, D), i, F16) for i in range(4))
    plan = rope.attn_plan(int32(cu), T, 1, 1, prefix_lens=int32(prefixes))
    out, lse = rope.attn_fwd(q, k, v, plan)
    grads = rope.attn_bwd(do, q, k, v, out, lse, plan)
    # one product for all of them, with what belongs to others hidden; the bounds of a sequence of 16
    seq = torch.repeat_interleave(torch.arange(2300), lens).to(DEV)
    pos = torch.arange(T, device=DEV) - int32(cu).long()[seq]
    pre = int32(prefixes).long()[seq]
    seen = (seq[:, None] == seq[None]) & ((pos[None] <= pos[:, None]) | (pos[None] < pre[:, None]))
    x, y, z, w = (t[:, 0].double() for t in (q, k, v, do))
    s = (x @ y.T * D ** -0.5).masked_fill(~seen, float("-inf"))
    p = s.softmax(-1)
    o, dp = p @ z, w @ z.T
    ds = p * (dp - (w * o).sum(-1, keepdim=True)) * D ** -0.5
    u = 2.0 ** -11
    ref.check(out[:, 0], o, 4 * u * (p @ z.abs() + o.abs()) + 2.0 ** -20, "out")
    # dS errs by its rounding, the weights', and D_i's, which is the output's
    e = 4 * u * (ds.abs() + p * D ** -0.5 * (w.abs() @ z.abs().T + (w.abs() * (p @ z.abs())).sum(-1, keepdim=True)))
    for name, got, want, tol in (("dq", grads[0], ds @ y, e @ y.abs()), ("dk", grads[1], ds.T @ x, e.T @ x.abs()),
                                 ("dv", grads[2], p.T @ w, 4 * u * (p.T @ w.abs()))):
        ref.check(got[:, 0], want, tol + u * want.abs() + 2.0 ** -20, name)


def test_gradients_through_a_fused_projection(rope):
    """rope_qkv_axes and attn_qkv together, as a layer of a model that sees images has them: the gradient of
    the fused projection against autograd's of the formula in 64 bits, from the rotated values in storage
    precision (their rounding is the rotation's); within the attention's bounds and one more rounding."""
    import packed_varlen_rotary_rope_amd.functional as F
    cu, T, Hq, Hkv, D, sections = [0, 90, 220], 220, 4, 2, 64, (12, 10, 10)
    prefixes, cap, slopes = [40, 0], 9.0, slopes_of(4)
    g = torch.Generator().manual_seed(5)
    pos = torch.randint(0, 300, (3, T), generator=g).int().to(DEV)
    qkv = normal((T, Hq + 2 * Hkv, D), 1, BF16).requires_grad_()
    do = normal((T, Hq, D), 2, BF16)
    plan = rope.attn_plan(int32(cu), T, Hq, Hkv, prefix_lens=int32(prefixes))
    turned = F.rope_qkv_axes(qkv * 1.0, Hq, Hkv, pos, sections, 1e4, "interleaved")
    kept = turned.detach().clone()
    out = F.attn_qkv(turned, Hq, Hkv, plan, softcap=cap, slopes=slopes)
    out.backward(do)
    q, k, v = kept[:, :Hq], kept[:, Hq:Hq + Hkv], kept[:, Hq + Hkv:]
    seqs = ref.sequences(cu, T)
    want, _, tol, _ = ref.forward(q, k, v, seqs, D ** -0.5, cap, slopes, prefixes)
    ref.check(out.detach(), want, tol, "out")
    grads, tols = ref.backward(do, q, k, v, seqs, D ** -0.5, BF16, cap, slopes, prefixes)
    # the transposed rotation of both, in 64 bits: errors of a pair are mixed
    d, e = torch.cat(grads, 1), torch.cat(tols, 1)
    ones = torch.ones_like(d[:, :Hq + Hkv], dtype=torch.float32)
    c = rope.qk_apply_axes(torch.cat([ones[..., :D // 2], 0 * ones[..., D // 2:]], -1)[:, :Hq].contiguous(),
                           ones[:, Hq:].contiguous(), pos, sections, 1e4, -1, "interleaved")[0][:, :1].double()
    cos, sin = c[..., :D // 2], c[..., D // 2:]  # of the rotation by minus the angle
    a, b = d[:, :Hq + Hkv].chunk(2, -1)
    ea, eb = e[:, :Hq + Hkv].chunk(2, -1)
    turned_back = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    bound = torch.cat([ea * cos.abs() + eb * sin.abs(), eb * cos.abs() + ea * sin.abs()], -1)
    u = ref.half_step(BF16)
    ref.check(qkv.grad[:, :Hq + Hkv], turned_back, 1.01 * (bound + 2 * u * turned_back.abs()) + 1e-6, "dq, dk")
    ref.check(qkv.grad[:, Hq + Hkv:], d[:, Hq + Hkv:], e[:, Hq + Hkv:], "dv")
    # the same on three tensors, with an expanded upstream gradient
    three = [t.contiguous().requires_grad_() for t in (q, k, v)]
    o = F.attn(*three, cu_seqlens=int32(cu), prefix_lens=int32(prefixes), softcap=cap, slopes=slopes)
    assert same(o.detach(), out.detach())
    o.sum().backward()
    again = ref.backward(torch.ones_like(do), q, k, v, seqs, D ** -0.5, BF16, cap, slopes, prefixes)
    for t, x, y in zip(three, *again):
        ref.check(t.grad, x, y, "gradients of a sum")


def test_gradients_against_differences(rope):
    """The loss sum(w out) along random directions: the central difference in 64 bits of the formula, whose
    slope the kernel's gradient must have up to its bounds."""
    cu, T, H, D, cap = [0, 33, 80], 80, 2, 32, 4.0
    slopes, prefixes = slopes_of(2), [20, 5]
    q, k, v, w = (normal((T, H, D), i, F16, 2.0) for i in range(4))
    plan = rope.attn_plan(int32(cu), T, H, H, prefix_lens=int32(prefixes))
    out, lse = rope.attn_fwd(q, k, v, plan, softcap=cap, slopes=slopes)
    got = rope.attn_bwd(w, q, k, v, out, lse, plan, softcap=cap, slopes=slopes)
    seqs = ref.sequences(cu, T)
    _, tols = ref.backward(w, q, k, v, seqs, D ** -0.5, F16, cap, slopes, prefixes)

    def loss(*x):
        total = 0.0
        for s, (a, n) in enumerate(seqs):
            for h in range(H):
                r = ref.head(*(t[a:a + n, h] for t in x), D ** -0.5, 0, n, cap, float(slopes[h]), prefixes[s])
                total = total + (r["out"] * w[a:a + n, h].double()).sum()
        return float(total)

    base = [t.double() for t in (q, k, v)]
    for i in range(3):
        step = torch.randn(base[i].shape, generator=torch.Generator(device=DEV).manual_seed(i), device=DEV,
                           dtype=torch.float64)
        h = 1e-6
        plus, minus = list(base), list(base)
        plus[i], minus[i] = base[i] + h * step, base[i] - h * step
        slope = (loss(*plus) - loss(*minus)) / (2 * h)
        assert abs(float((got[i].double() * step).sum()) - slope) <= float((tols[i] * step.abs()).sum()) + 1e-4


def test_saved_values_that_change_are_noticed(rope):
    import packed_varlen_rotary_rope_amd.functional as F
    q = normal((64, 4, 64), 1, BF16).requires_grad_()
    slopes, cu = slopes_of(4), int32([0, 64])
    out = F.attn(q, q, q, cu_seqlens=cu, slopes=slopes)
    slopes.mul_(2)
    with pytest.raises(RuntimeError, match="modified"):
        out.sum().backward()
    plan = rope.attn_plan(cu, 64, 4, 4)
    out = F.attn(q, q, q, plan)
    rope.attn_plan(cu, 64, 4, 4, out=plan, prefix_lens=int32([9]))
    with pytest.raises(RuntimeError, match="modified"):
        out.sum().backward()


def test_refusals(rope):
    import packed_varlen_rotary_rope_amd.functional as F
    q = normal((64, 4, 64), 1, BF16)
    cu = int32([0, 64])
    plan = rope.attn_plan(cu, 64, 4, 4, prefix_lens=int32([3]))
    good = slopes_of(4)
    for bad in (0, -3.0, float("nan"), float("inf")):
        with pytest.raises(ValueError):
            rope.attn_fwd(q, q, q, plan, softcap=bad)
    with pytest.raises(rope.RopeError):
        rope.attn_fwd(q, q, q, plan, softcap=1e35)
    for bad in (good.double(), good.cpu(), slopes_of(8)[::2]):
        with pytest.raises(TypeError):
            rope.attn_fwd(q, q, q, plan, slopes=bad)
    for bad in (slopes_of(3), good[None]):
        with pytest.raises(ValueError):
            rope.attn_fwd(q, q, q, plan, slopes=bad)
    with pytest.raises(ValueError):
        rope.attn_plan(cu, 64, 4, 4, prefix_lens=int32([3, 4]))
    with pytest.raises(TypeError):
        rope.attn_plan(cu, 64, 4, 4, prefix_lens=torch.tensor([3], device=DEV))
    with pytest.raises(ValueError):
        rope.paged_plan(cu, int32([64]), 64, 4, 4, prefix_lens=int32([]))
    with pytest.raises(ValueError, match="not both"):
        F.attn(q, q, q, plan, prefix_lens=int32([3]))
    with pytest.raises(ValueError, match="gradient"):
        F.attn(q, q, q, plan, slopes=good.clone().requires_grad_())


def test_captured_training_step(rope):
    """Forward and backward with a new plan, prefixes and slopes in a graph: each replay, with eager work between, gives what
    eager calls give."""
    T, H, D = 300, 4, 64
    q, k, v, do = (normal((T, H, D), i, BF16) for i in range(4))
    cu, prefixes, slopes = int32([0, 100, 300]), int32([20, 30]), slopes_of(H)
    plan = rope.attn_plan(cu, T, H, H, prefix_lens=prefixes)
    res = [torch.empty_like(q), torch.empty((T, H), device=DEV)] + [torch.empty_like(q) for _ in range(3)]

    def step():
        rope.attn_plan(cu, T, H, H, out=plan, prefix_lens=prefixes)
        rope.attn_fwd(q, k, v, plan, out=res[0], lse=res[1], zero_rest=True, softcap=5.0, slopes=slopes)
        rope.attn_bwd(do, q, k, v, res[0], res[1], plan, None, *res[2:], zero_rest=True, softcap=5.0, slopes=slopes)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i, (bounds, pre) in enumerate((([0, 100, 300], [90, 0]), ([0, 299, 299], [150, 7]), ([10, 11, 200], [1, 50]))):
        cu.copy_(int32(bounds))
        prefixes.copy_(int32(pre))
        slopes.mul_(0.5)
        q.copy_(normal((T, H, D), 20 + i, BF16))
        graph.replay()
        got = [t.clone() for t in res]
        fresh = rope.attn_plan(int32(bounds), T, H, H, prefix_lens=int32(pre))
        out, lse = rope.attn_fwd(q, k, v, fresh, softcap=5.0, slopes=slopes)
        want = (out, lse, *rope.attn_bwd(do, q, k, v, out, lse, fresh, softcap=5.0, slopes=slopes))
        torch.cuda.synchronize()
        assert all(same(a, b) for a, b in zip(got, want))


def test_repeatable_and_concurrent(rope):
    """The same bits in every run, also while another stream runs the other forms."""
    cu, T, Hq, Hkv, D = [0, 700, 1500], 1500, 8, 2, 128
    q, k, v, do = (normal((T, h, D), i, BF16) for i, h in enumerate((Hq, Hkv, Hkv, Hq)))
    runs = {}
    for form in ("cap", "slopes", "all"):
        cap, slopes, prefixes = form_args(form, cu, Hq)
        plan = rope.attn_plan(int32(cu), T, Hq, Hkv, prefix_lens=None if prefixes is None else int32(prefixes))
        runs[form] = (plan, dict(softcap=cap, slopes=slopes))

    def run(form):
        plan, more = runs[form]
        out, lse = rope.attn_fwd(q, k, v, plan, **more)
        return (out, lse, *rope.attn_bwd(do, q, k, v, out, lse, plan, **more))

    want = {form: run(form) for form in runs}
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in runs]
    got = []
    for _ in range(3):
        for stream, form in zip(streams, runs):
            with torch.cuda.stream(stream):
                got.append((form, run(form)))
    torch.cuda.synchronize()
    for form, x in got:
        assert all(same(a, b) for a, b in zip(x, want[form]))


def test_paged_pages_that_are_none_and_rows_of_no_sequence(rope):
    """Keys behind the table or on no page are seen by nobody, inside of a prefix too; rows before and
    behind the sequences are left."""
    held, new, page, D = [90, 40], [3, 40], 16, 64
    k, v, table = pool(held, page, 2, D, BF16, 3)
    table[0, 2] = -1
    table[1, 1] = 2 ** 31 - 1
    table = table[:, :5]  # 80 keys of the first
    cu, T = [2, 5, 45], 50
    q = normal((T, 4, D), 1, BF16)
    slopes = slopes_of(4, True)
    plan = rope.paged_plan(int32(cu), int32(held), T, 4, 2, prefix_lens=int32([500, 30]))
    out, lse = torch.full((T, 4, D), 7.0, dtype=BF16, device=DEV), torch.full((T, 4), 7.0, device=DEV)
    rope.attn_paged(q, k, v, table, plan, out=out, lse=lse, softcap=6.0, slopes=slopes)
    want, wlse, tol, ltol = ref.paged(q, k, v, table, cu, held, D ** -0.5, 6.0, slopes, [500, 30])
    ref.check(out[2:45], want[2:45], tol[2:45], "out")
    ref.check(lse[2:45], wlse[2:45], ltol[2:45], "lse")
    for t in (out, lse):
        assert bool((t[:2] == 7).all()) and bool((t[45:] == 7).all())


def test_bias_over_a_very_long_cache(rope):
    """17 million keys, whose distances 24 bits just hold: every block of the table is the same page. Weights
    are sums over the repeats, e^(-slope distance); in fp32 the largest biases err by 2^-22 of 17."""
    page, D, n = 4096, 8, 4097
    held = page * n - 3
    k, v = (normal((1, page, 1, D), i, F16) for i in range(2))
    table = torch.zeros((1, n), dtype=torch.int32, device=DEV)
    q, slope = normal((1, 1, D), 3, F16), 1e-6
    plan = rope.paged_plan(int32([0, 1]), int32([held]), 1, 1, 1)
    out, lse = rope.attn_paged(q, k, v, table, plan, slopes=torch.tensor([slope], device=DEV))
    slope = float(torch.tensor(slope, dtype=torch.float32))
    s = (k[0, :, 0].double() @ q[0, 0].double()) * D ** -0.5
    total, weighted = 0.0, torch.zeros(D, dtype=torch.float64, device=DEV)
    top = float(s.max())
    for first in range(0, held, page * 64):
        j = torch.arange(first, min(first + page * 64, held), device=DEV)
        w = torch.exp(s[j % page] - top - slope * (held - 1 - j).double())
        total += float(w.sum())
        weighted += w @ v[0, :, 0].double()[j % page]
    want = weighted / total
    # weights: u each, of random sign over millions; sums of 17e6 values in some thousand parts; the bias
    mean = float(v.double().abs().max())
    assert float((out[0, 0].double() - want).abs().max()) <= 2.0 ** -11 * (mean + float(want.abs().max())) + 1e-4
    assert abs(float(lse[0, 0]) - (top + torch.log(torch.tensor(total, dtype=torch.float64)).item())) <= 1e-4


def test_a_service_with_images(rope):
    """Requests with an image in front, served chunk by chunk: pages taken, keys rotated by three axes and written to
    their slots, attention over the cache with the image as a prefix and capped scores. Each request's
    last chunk gives what the packed attention of the whole request gives, within the bounds of both."""
    import attn_scores_reference as r
    Hq, Hkv, D, page, sections, cap = 8, 2, 64, 16, (12, 10, 10), 12.0
    lengths, images = [150, 37, 333], [100, 0, 200]
    B, g = len(lengths), torch.Generator().manual_seed(4)
    pos = [torch.randint(0, 400, (3, n), generator=g).int().to(DEV) for n in lengths]
    qkv = [normal((n, Hq + 2 * Hkv, D), 30 + i, BF16) for i, n in enumerate(lengths)]
    pool_, table = rope.page_pool(60), torch.full((B, 24), -1, dtype=torch.int32, device=DEV)
    kc, vc = (torch.full((60, page, Hkv, D), float("nan"), dtype=BF16, device=DEV) for _ in range(2))
    held, done = int32([0] * B), [0] * B
    last = [None] * B
    # the image is taken in as a whole, the rest in chunks and single tokens
    chunks = [[100, 30, 1, 1, 18], [20, 16, 1, 0, 0], [200, 64, 64, 1, 4]]
    for turn in range(5):
        new = [c[turn] for c in chunks]
        rows = torch.cat([x[d:d + n] for x, d, n in zip(qkv, done, new)])
        ids = torch.cat([p[:, d:d + n] for p, d, n in zip(pos, done, new)], 1)
        T = rows.shape[0]
        step = rope.page_step(pool_, table, held, int32(new), T, page)
        pool_.state, held = step.state, step.held
        q = rope.kv_append_slots_(rows[:, Hq:Hq + Hkv], rows[:, Hq + Hkv:], kc, vc, step.slots, ids, 1e4, sections,
                                  q=rows[:, :Hq])
        plan = rope.paged_plan(step.cu_seqlens, step.kv_lens, T, Hq, Hkv, prefix_lens=int32(images))
        out, lse = rope.attn_paged(q, kc, vc, table, plan, softcap=cap)
        at = 0
        for s, n in enumerate(new):
            done[s] += n
            if n:
                last[s] = (done[s] - n, out[at:at + n], lse[at:at + n])
            at += n
    assert done == lengths and held.tolist() == lengths
    for s, (first, out, lse) in enumerate(last):
        q, k = rope.qk_apply_axes(qkv[s][:, :Hq], qkv[s][:, Hq:Hq + Hkv], pos[s], sections, 1e4)
        args = (q, k, qkv[s][:, Hq + Hkv:], [(0, lengths[s])], D ** -0.5, cap, None, [images[s]])
        want, wlse, tol, ltol = r.forward(*args)
        r.check(out, want[first:], tol[first:], "out")
        r.check(lse, wlse[first:], ltol[first:], "lse")
        plan = rope.attn_plan(int32([0, lengths[s]]), lengths[s], Hq, Hkv, prefix_lens=int32([images[s]]))
        packed, _ = rope.attn_fwd(q, k, qkv[s][:, Hq + Hkv:], plan, softcap=cap)
        r.check(packed, want, tol, "packed")


def test_captured_layer(rope):
    """Plan, rotation, attention and their gradients through autograd in a graph: replays with other inputs,
    positions, sequences and prefixes give the eager bits."""
    import packed_varlen_rotary_rope_amd.functional as F
    T, Hq, Hkv, D, sections = 260, 4, 2, 64, (12, 10, 10)
    cu, prefixes, slopes = int32([0, 100, 260]), int32([30, 0]), slopes_of(Hq)
    pos = torch.zeros((3, T), dtype=torch.int32, device=DEV)
    x = normal((T, Hq + 2 * Hkv, D), 1, BF16).requires_grad_()
    do = normal((T, Hq, D), 2, BF16)
    plan = rope.attn_plan(cu, T, Hq, Hkv, prefix_lens=prefixes)

    def layer():
        qkv = F.rope_qkv_axes(x * 1.0, Hq, Hkv, pos, sections, 1e4)
        out = F.attn_qkv(qkv, Hq, Hkv, plan, softcap=10.0, slopes=slopes)
        return out, *torch.autograd.grad(out, (x,), do)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        rope.attn_plan(cu, T, Hq, Hkv, out=plan, prefix_lens=prefixes)
        res = layer()
    for i, (bounds, pre) in enumerate((([0, 100, 260], [50, 160]), ([0, 1, 2], [1, 0]), ([20, 200, 260], [0, 9]))):
        with torch.no_grad():
            x.copy_(normal(x.shape, 40 + i, BF16))
        cu.copy_(int32(bounds))
        prefixes.copy_(int32(pre))
        pos.copy_(torch.randint(0, 999, (3, T), device=DEV))
        graph.replay()
        got = [t.detach().clone() for t in res]
        with torch.no_grad():
            y = x.detach().clone()
            q, k, v = y[:, :Hq], y[:, Hq:Hq + Hkv], y[:, Hq + Hkv:]
            rope.qk_apply_axes(q, k, pos, sections, 1e4, q_out=q, k_out=k)
            fresh = rope.attn_plan(int32(bounds), T, Hq, Hkv, prefix_lens=int32(pre))
            more = dict(softcap=10.0, slopes=slopes)
            out, lse = rope.attn_fwd(q, k, v, fresh, **more)
            dq, dk, dv = rope.attn_bwd(do, q, k, v, out, lse, fresh, **more)
            dq, dk = rope.qk_apply_axes(dq, dk, pos, sections, 1e4, -1)
            grad = torch.cat([dq, dk, dv], 1)
        torch.cuda.synchronize()
        assert same(got[0], out) and same(got[1], grad)


@pytest.mark.parametrize("cap", [1e-3, 1e4, 1e9, 1e25])
def test_caps_of_any_size(rope, cap):
    """Far below the scores, and far above them, where it changes nothing."""
    cu, T, H, D = [0, 100, 170], 170, 2, 64
    q, k, v, do = (normal((T, H, D), i, F16) for i in range(4))
    plan = rope.attn_plan(int32(cu), T, H, H)
    out, lse = rope.attn_fwd(q, k, v, plan, softcap=cap)
    args = (ref.sequences(cu, T), D ** -0.5)
    want, wlse, tol, ltol = ref.forward(q, k, v, *args, cap)
    ref.check(out, want, tol, "out")
    ref.check(lse, wlse, ltol, "lse")
    grads = rope.attn_bwd(do, q, k, v, out, lse, plan, softcap=cap)
    for name, got, x, t in zip(("dq", "dk", "dv"), grads, *ref.backward(do, q, k, v, *args, F16, cap)):
        ref.check(got, x, t, name)


@pytest.mark.parametrize("Hq,Hkv,D,count,most", [(5, 5, 72, 24, 9), (8, 2, 128, 40, 130), (6, 1, 64, 9, 40), (2, 2, 32, 300, 200)])
def test_small_batches_whose_key_tiles_are_cut(rope, Hq, Hkv, D, count, most):
    """Work below a full chip's, of many lengths: pieces of key tiles of every size, in f16."""
    lens = torch.randint(1, most, (count,), generator=torch.Generator().manual_seed(count)).tolist()
    lens[0] = 517
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    T, slopes = cu[-1], slopes_of(Hq)
    q, k, v, do = (normal((T, h, D), i, F16) for i, h in enumerate((Hq, Hkv, Hkv, Hq)))
    prefixes = [n * (s % 3) // 4 for s, n in enumerate(lens)]
    plan = rope.attn_plan(int32(cu), T, Hq, Hkv, prefix_lens=int32(prefixes))
    out, lse = rope.attn_fwd(q, k, v, plan, slopes=slopes)
    grads = rope.attn_bwd(do, q, k, v, out, lse, plan, slopes=slopes)
    want = ref.backward(do, q, k, v, ref.sequences(cu, T), D ** -0.5, F16, None, slopes, prefixes)
    for name, got, x, t in zip(("dq", "dk", "dv"), grads, *want):
        ref.check(got, x, t, name)
