"""GPU tests of packed causal attention against its definition in 64 bits (attn_reference)."""
import pytest
import torch

import attn_reference as ref

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
BF16, F16 = torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def rope():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import packed_varlen_rotary_rope_amd as m
    return m


def normal(shape, seed, dtype):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randn(shape, generator=g, device=DEV).to(dtype)


def batch(T, Hq, Hkv, D, dtype, seed=0):
    return (normal((T, Hq, D), 3 * seed + 1, dtype), normal((T, Hkv, D), 3 * seed + 2, dtype),
            normal((T, Hkv, D), 3 * seed + 3, dtype))


def int32(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def worst_score(q, k, scale):
    """An upper bound of scale * sum |q k| over all pairs."""
    return float(q.double().norm(dim=-1).max() * k.double().norm(dim=-1).max() * scale)


SHAPES = [  # cu_seqlens, T, Hq, Hkv, D, dtype
    ([0, 1], 1, 1, 1, 8, BF16),
    ([0, 5, 22, 25, 64], 64, 4, 2, 16, F16),
    ([0, 64, 65, 192, 193], 193, 4, 4, 64, BF16),
    ([0, 127, 255, 384, 384, 600], 600, 8, 2, 128, BF16),
    ([0, 129], 129, 6, 2, 80, F16),
    ([3, 40, 140], 150, 5, 1, 96, BF16),      # rows before and behind the sequences
    ([0, 301], 301, 7, 1, 72, BF16),          # groups that divide no tile
    ([0, 33, 66], 66, 24, 2, 40, F16),
    ([0, 1000], 1000, 8, 1, 128, F16),
    ([0, 700], 700, 3, 3, 112, BF16),
    ([0, 500], 500, 2, 1, 160, BF16),
    ([0, 90, 333], 333, 2, 2, 192, F16),
    ([0, 450], 450, 4, 2, 256, BF16),
    ([0, 200], 200, 4, 1, 248, F16),
    ([0] + list(range(1, 41)), 40, 32, 8, 128, BF16),  # one token each
    ([0, 2300], 2300, 160, 1, 32, BF16),      # more heads in a group than a tile has rows
]


@pytest.mark.parametrize("case", SHAPES, ids=lambda c: f"T{c[1]}_{c[2]}_{c[3]}_{c[4]}_{str(c[5])[6:]}")
def test_forward(rope, case):
    cu, T, Hq, Hkv, D, dtype = case
    print(f"[attn_fwd] {case}", flush=True)
    q, k, v = batch(T, Hq, Hkv, D, dtype, seed=len(cu) + D)
    plan = rope.attn_plan(int32(cu), T, Hq, Hkv)
    scale = D ** -0.5
    out, lse = rope.attn_fwd(q, k, v, plan)
    want, wlse, tol = ref.forward(q, k, v, ref.sequences(cu, T), scale)
    ref.check(out, want, tol, "out")
    ref.check_lse(lse, wlse, D, worst_score(q, k, scale))


@pytest.mark.parametrize("case", [c for c in SHAPES if c[4] <= 128],
                         ids=lambda c: f"T{c[1]}_{c[2]}_{c[3]}_{c[4]}_{str(c[5])[6:]}")
def test_backward(rope, case):
    cu, T, Hq, Hkv, D, dtype = case
    print(f"[attn_bwd] {case}", flush=True)
    q, k, v = batch(T, Hq, Hkv, D, dtype, seed=len(cu) + D)
    do = normal((T, Hq, D), 77, dtype)
    plan = rope.attn_plan(int32(cu), T, Hq, Hkv)
    out, lse = rope.attn_fwd(q, k, v, plan)
    got = rope.attn_bwd(do, q, k, v, out, lse, plan)
    want, tols = ref.backward(do, q, k, v, ref.sequences(cu, T), D ** -0.5, dtype)
    for name, g, w, tol in zip(("dq", "dk", "dv"), got, want, tols):
        ref.check(g, w, tol, name)


def bits(t):
    return t.contiguous().view(torch.int32 if t.dtype == torch.float32 else torch.int16)


def same(a, b):
    return torch.equal(bits(a), bits(b))


@pytest.mark.parametrize("D,G,dtype", [(64, 1, BF16), (128, 4, F16), (80, 3, BF16), (192, 2, BF16)])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("where", ["k", "v"])
def test_hidden_values_have_no_influence(rope, D, G, dtype, value, where):
    """A key or value that is not finite changes no row before it and no other sequence; rows
    that see it have the result of the definition."""
    print(f"[hidden] D={D} G={G} {dtype} {value} {where}", flush=True)
    cu, T, at = [0, 150, 400], 400, 101
    q, k, v = batch(T, 2 * G, 2, D, dtype, seed=D)
    plan = rope.attn_plan(int32(cu), T, 2 * G, 2)
    out0, lse0 = rope.attn_fwd(q, k, v, plan)
    {"k": k, "v": v}[where][at, 1, 3] = value
    out, lse = rope.attn_fwd(q, k, v, plan)
    hit = torch.zeros(T, dtype=torch.bool, device=DEV)
    hit[at:150] = True
    assert same(out[~hit], out0[~hit]) and same(lse[~hit], lse0[~hit])
    assert same(out[:, :G], out0[:, :G])  # the other key/value head
    if where == "v":
        want = torch.full_like(out[hit][:, G:, 3], value)
        got = out[hit][:, G:, 3]
        assert torch.equal(got.isnan(), want.isnan()) and torch.equal(got[~got.isnan()], want[~want.isnan()])
        rest = torch.arange(D, device=DEV) != 3
        assert same(out[hit][:, G:, rest], out0[hit][:, G:, rest])
    elif value != value:
        assert bool(out[hit][:, G:].isnan().all())


@pytest.mark.parametrize("D,G,dtype", [(64, 1, BF16), (128, 4, F16), (80, 3, BF16)])
@pytest.mark.parametrize("where", ["q", "k", "v", "do"])
def test_hidden_values_and_gradients(rope, D, G, dtype, where):
    """The same for the gradients: a row that is not finite reaches only keys that it sees, and
    a key only rows that see it (and what they reach)."""
    print(f"[hidden gradients] D={D} G={G} {dtype} {where}", flush=True)
    cu, T, at = [0, 150, 400], 400, 101
    q, k, v = batch(T, 2 * G, 2, D, dtype, seed=D)
    do = normal((T, 2 * G, D), 5, dtype)
    plan = rope.attn_plan(int32(cu), T, 2 * G, 2)

    def grads():
        out, lse = rope.attn_fwd(q, k, v, plan)
        return rope.attn_bwd(do, q, k, v, out, lse, plan)

    dq0, dk0, dv0 = grads()
    {"q": q, "k": k, "v": v, "do": do}[where][at, G if where in ("q", "do") else 1, 2] = float("inf")
    dq, dk, dv = grads()
    t = torch.arange(T, device=DEV)
    if where in ("q", "do"):  # one row: its own dq, and the keys up to it
        assert same(dq[t != at], dq0[t != at])
        clean = (t > at) | (t >= 150)
        assert same(dk[clean], dk0[clean]) and same(dv[clean], dv0[clean])
        assert not bool(dv[:at + 1, 1].isfinite().all())
    else:  # one key: the rows from it on, and through them every key of the sequence
        clean = (t < at) | (t >= 150)
        assert same(dq[clean], dq0[clean])
        assert same(dk[150:], dk0[150:]) and same(dv[150:], dv0[150:])
    assert same(dk[:, 0], dk0[:, 0]) and same(dv[:, 0], dv0[:, 0])  # the other key/value head


@pytest.mark.parametrize("dtype", [BF16, F16])
def test_rows_of_no_sequence(rope, dtype):
    """Padded layout: rows that seqused leaves out, and rows before and behind the sequences,
    hold NaN everywhere; results are those of the packed batch, the rows themselves are zeroed
    in new outputs and left alone in given ones."""
    cu, used, T = [5, 105, 205, 335], [100, 0, 70], 350
    print(f"[padded] {dtype}", flush=True)
    q, k, v = batch(T, 6, 2, 96, dtype, seed=3)
    do = normal((T, 6, 96), 9, dtype)
    rows = torch.zeros(T, dtype=torch.bool, device=DEV)
    for a, n in ref.sequences(cu, T, used):
        rows[a:a + n] = True
    for x in (q, k, v, do):
        x[~rows] = float("nan")
    plan = rope.attn_plan(int32(cu), T, 6, 2, seqused=int32(used))
    out, lse = rope.attn_fwd(q, k, v, plan)
    grads = rope.attn_bwd(do, q, k, v, out, lse, plan)
    n = int(rows.sum())
    packed = rope.attn_plan(int32([0, 100, 170]), n, 6, 2)
    out1, lse1 = rope.attn_fwd(q[rows], k[rows], v[rows], packed)
    grads1 = rope.attn_bwd(do[rows], q[rows], k[rows], v[rows], out1, lse1, packed)
    assert same(out[rows], out1) and same(lse[rows], lse1)
    assert bool((out[~rows] == 0).all()) and bool((lse[~rows] == float("-inf")).all())
    assert all(bool((g[~rows] == 0).all()) for g in grads)
    assert same(grads[0][rows], grads1[0])
    # dk and dv are summed in shares of the whole batch's work, whose cuts differ between the two
    # layouts: either is within the bounds of the exact sums
    wants, tols = ref.backward(do[rows], q[rows], k[rows], v[rows], [(0, 100), (100, 70)], 96 ** -0.5, dtype)
    for got in (grads, grads1):
        for g, w, t in zip(got, wants, tols):
            ref.check(g[rows] if g.shape[0] == T else g, w, t, "gradient")
    keep = [torch.full_like(x, 7.0) for x in (out, lse, *grads)]
    rope.attn_fwd(q, k, v, plan, out=keep[0], lse=keep[1])
    rope.attn_bwd(do, q, k, v, out, lse, plan, None, *keep[2:])
    for x, y in zip(keep, (out, lse, *grads)):
        assert same(x[rows], y[rows]) and bool((x[~rows] == 7).all())
    rope.attn_fwd(q, k, v, plan, out=keep[0], lse=keep[1], zero_rest=True)
    assert same(keep[0], out) and same(keep[1], lse)


def test_sequences_that_overlap_or_leave_the_tensor(rope):
    """cu_seqlens that are no cu_seqlens: read as the header says, nothing else touched."""
    T = 200
    q, k, v = batch(T, 4, 2, 64, BF16, seed=8)
    for cu in ([0, 120, 60, 150, 200], [-50, 40, 1000, 90], [300, 400], [7], [0, 0, 0], [50, 20]):
        print(f"[cu_seqlens] {cu}", flush=True)
        out, lse = rope.attn_fwd(q, k, v, rope.attn_plan(int32(cu), T, 4, 2))
        want, wlse, tol = ref.forward(q, k, v, ref.sequences(cu, T), 0.125)
        ref.check(out, want, tol, "out")
        grads = rope.attn_bwd(q, q, k, v, out, lse, rope.attn_plan(int32(cu), T, 4, 2))
        wants, tols = ref.backward(q, q, k, v, ref.sequences(cu, T), 0.125, BF16)
        for g, w, t in zip(grads, wants, tols):
            ref.check(g, w, t, "gradient")


def test_refusals(rope):
    q, k, v = batch(64, 4, 2, 64, BF16)
    plan = rope.attn_plan(int32([0, 64]), 64, 4, 2)
    out, lse = rope.attn_fwd(q, k, v, plan)
    for a in ((q.float(), k.float(), v.float()), (q, k.half(), v), (q.cpu(), k, v)):
        with pytest.raises(TypeError):
            rope.attn_fwd(*a, plan)
    for a in ((q[:60], k[:60], v[:60]), (q[:, :2], k, v), (q, k, v[:, :, :32]), (q[:, :, :60], k[:, :, :60], v[:, :, :60]),
              (q[:, :, ::2], k[:, :, ::2], v[:, :, ::2]), (q[:, :, 4:36], k[:, :, 4:36], v[:, :, 4:36])):
        with pytest.raises(ValueError):
            rope.attn_fwd(*a, plan)
    with pytest.raises(ValueError):
        rope.attn_fwd(q, k, v, plan, out=out)
    with pytest.raises(ValueError):
        rope.attn_fwd(q, k, v, plan, out=out[:, :2], lse=lse)
    with pytest.raises(rope.RopeError):
        rope.attn_fwd(q, k, v, plan, scale=-1.0)
    with pytest.raises(ValueError):
        rope.attn_bwd(q, q, k, v, out, lse, plan, dq=q)
    with pytest.raises(ValueError):
        rope.attn_plan(int32([0, 64]), 64, 4, 3)
    with pytest.raises(ValueError):
        rope.attn_plan(int32([0, 64]), 65, 4, 2, out=plan)
    with pytest.raises(TypeError):
        rope.attn_plan(torch.tensor([0, 64], device=DEV), 64, 4, 2)
    big = batch(64, 2, 1, 256, BF16)
    o2, l2 = rope.attn_fwd(*big, rope.attn_plan(int32([0, 64]), 64, 2, 1))
    with pytest.raises(ValueError):
        rope.attn_bwd(o2, *big, o2, l2, rope.attn_plan(int32([0, 64]), 64, 2, 1))


def test_plan_of_another_batch_writes_nothing(rope):
    q, k, v = batch(64, 4, 2, 64, BF16)
    other = rope.attn_plan(int32([0, 32, 80]), 80, 4, 2)
    fake = rope.AttnPlan(64, 2, 4, 2, other.buffer)
    out, lse = torch.full_like(q, 3.0), torch.full((64, 4), 3.0, device=DEV)
    rope.attn_fwd(q, k, v, fake, out=out, lse=lse)
    grads = [torch.full_like(x, 3.0) for x in (q, k, v)]
    rope.attn_bwd(q, q, k, v, out, lse, fake, None, *grads)
    assert all(bool((x == 3).all()) for x in (out, lse, *grads))


def test_gradients_against_differences(rope):
    """<dq, x> + <dk, y> + <dv, z> is the derivative of <out, do> along (x, y, z): against central
    differences of the definition in 64 bits (their own error is of order step^2)."""
    cu, T, Hq, Hkv, D = [0, 3, 70, 71, 150], 150, 6, 2, 48
    q, k, v = batch(T, Hq, Hkv, D, F16, seed=21)
    do = normal((T, Hq, D), 4, F16)
    plan = rope.attn_plan(int32(cu), T, Hq, Hkv)
    out, lse = rope.attn_fwd(q, k, v, plan)
    grads = rope.attn_bwd(do, q, k, v, out, lse, plan)
    _, tols = ref.backward(do, q, k, v, ref.sequences(cu, T), D ** -0.5, F16)
    for i in range(3):
        x = [q.double(), k.double(), v.double()]
        d = normal(x[i].shape, 40 + i, torch.float32).double()
        step, value = 1e-4, []
        for sign in (1, -1):
            y = list(x)
            y[i] = x[i] + sign * step * d
            o = torch.zeros_like(x[0])
            for a, n in ref.sequences(cu, T):
                for h in range(Hq):
                    g = h // (Hq // Hkv)
                    o[a:a + n, h] = ref.head_forward(y[0][a:a + n, h], y[1][a:a + n, g], y[2][a:a + n, g],
                                                     D ** -0.5, 0)[0]
            value.append(float((o * do.double()).sum()))
        slope = (value[0] - value[1]) / (2 * step)
        got = float((grads[i].double() * d).sum())
        assert abs(got - slope) <= float((tols[i] * d.abs()).sum()) + 1e-5 * abs(slope), (i, got, slope)


@pytest.mark.parametrize("D,Hq,Hkv", [(128, 8, 2), (64, 4, 4), (80, 6, 2)])
def test_rotation_and_attention_of_a_fused_projection(rope, D, Hq, Hkv):
    """A layer's middle as a model has it: rope_qkv, then attn_qkv, both on the fused output,
    against attention in 64 bits of the rotated values; the gradient through both against the
    transposed rotation of the exact gradient."""
    import packed_varlen_rotary_rope_amd.functional as F
    cu, T = [0, 33, 200, 201, 390], 390
    print(f"[fused] D={D} {Hq}+{Hkv}", flush=True)
    H = Hq + 2 * Hkv
    x = normal((T, H * D), 2, BF16).requires_grad_()
    do = normal((T, Hq, D), 3, BF16)
    plan = rope.attn_plan(int32(cu), T, Hq, Hkv)
    qkv = F.rope_qkv(x * 1, Hq, Hkv, int32(cu), 1e4)
    out = F.attn_qkv(qkv, Hq, Hkv, plan)
    turned = qkv.detach().clone().view(T, H, D)
    out.backward(do)
    q, k, v = turned[:, :Hq], turned[:, Hq:Hq + Hkv], turned[:, Hq + Hkv:]
    seqs = ref.sequences(cu, T)
    want, _, tol = ref.forward(q, k, v, seqs, D ** -0.5)
    ref.check(out.detach(), want, tol, "out")
    (dq, dk, dv), (tq, tk, tv) = ref.backward(do, q, k, v, seqs, D ** -0.5, BF16)
    got = x.grad.view(T, H, D)
    ref.check(got[:, Hq + Hkv:], dv, tv, "dv")
    c, s = rope.cos_sin_table(400, D, 1e4)
    pos = torch.cat([torch.arange(n) for _, n in seqs]).to(DEV)
    c, s = c[pos].double()[:, None], s[pos].double()[:, None]

    def back(g):
        lo, hi = g.chunk(2, -1)
        return torch.cat([lo * c + hi * s, hi * c - lo * s], -1)

    def spread(t):  # the rotation mixes the halves' errors
        lo, hi = t.chunk(2, -1)
        m = lo + hi
        return torch.cat([m, m], -1)

    u = ref.half_step(BF16)
    for name, g, w, t in (("dq", got[:, :Hq], dq, tq), ("dk", got[:, Hq:Hq + Hkv], dk, tk)):
        w = back(w)
        ref.check(g, w, (spread(t) + u * w.abs()) * 1.01, name)
    # separate tensors, and a plan made on the way: the same bits
    leaves = [y.detach().clone().requires_grad_() for y in (q, k, v)]
    again = F.attn(*leaves, cu_seqlens=int32(cu))
    assert same(again.detach(), out.detach())
    again.backward(do)
    assert same(leaves[2].grad, got[:, Hq + Hkv:].contiguous())


def test_plan_written_over_before_backward(rope):
    import packed_varlen_rotary_rope_amd.functional as F
    q, k, v = (x.requires_grad_() for x in batch(100, 4, 2, 64, BF16))
    plan = rope.attn_plan(int32([0, 100]), 100, 4, 2)
    out = F.attn(q, k, v, plan)
    rope.attn_plan(int32([0, 50]), 100, 4, 2, out=plan)
    with pytest.raises(RuntimeError):
        out.sum().backward()


def test_expanded_gradient_and_frozen_inputs(rope):
    import packed_varlen_rotary_rope_amd.functional as F
    q, k, v = batch(130, 4, 2, 64, BF16)
    q.requires_grad_()
    plan = rope.attn_plan(int32([0, 130]), 130, 4, 2)
    F.attn(q, k, v, plan).sum().backward()  # an expanded upstream gradient
    out, lse = rope.attn_fwd(q.detach(), k, v, plan)
    dq, _, _ = rope.attn_bwd(torch.ones_like(out), q.detach(), k, v, out, lse, plan)
    assert same(q.grad, dq)


def test_repeatable_and_concurrent(rope):
    """The same bits every time, also with one plan in use on two streams at once."""
    cu, T = [0, 700, 750, 2000], 2000
    q, k, v = batch(T, 8, 2, 128, BF16, seed=6)
    q2, k2, v2 = batch(T, 8, 2, 128, BF16, seed=7)
    plan = rope.attn_plan(int32(cu), T, 8, 2)

    def all_of(q, k, v):
        out, lse = rope.attn_fwd(q, k, v, plan)
        return (out, lse, *rope.attn_bwd(q, q, k, v, out, lse, plan))

    one, two = all_of(q, k, v), all_of(q2, k2, v2)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        got = []
        for st, a in zip(streams, ((q, k, v), (q2, k2, v2))):
            with torch.cuda.stream(st):
                got.append(all_of(*a))
        torch.cuda.synchronize()
        assert all(same(a, b) for a, b in zip(got[0] + got[1], one + two))


def test_captured_step(rope):
    """Plan, forward and backward in a HIP graph: replays with other inputs and other sequences
    give the eager bits."""
    import packed_varlen_rotary_rope_amd.functional as F
    T, Hq, Hkv, D = 500, 8, 2, 64
    cu = int32([0, 100, 500])
    q, k, v = (x.requires_grad_() for x in batch(T, Hq, Hkv, D, BF16))
    do = normal((T, Hq, D), 5, BF16)
    plan = rope.attn_plan(cu, T, Hq, Hkv)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.autograd.grad(F.attn(q, k, v, plan), (q, k, v), do)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        rope.attn_plan(cu, T, Hq, Hkv, out=plan)
        out = F.attn(q, k, v, plan)
        grads = torch.autograd.grad(out, (q, k, v), do)
    for i, lengths in enumerate(([0, 100, 500], [0, 1, 2], [250, 490, 500])):
        with torch.no_grad():
            for x, y in zip((q, k, v), batch(T, Hq, Hkv, D, BF16, seed=30 + i)):
                x.copy_(y)
        cu.copy_(int32(lengths))
        graph.replay()
        got = [x.detach().clone() for x in (out, *grads)]
        with torch.no_grad():
            fresh = rope.attn_plan(cu, T, Hq, Hkv)
            o, l = rope.attn_fwd(q, k, v, fresh)
            want = (o, *rope.attn_bwd(do, q, k, v, o, l, fresh))
        torch.cuda.synchronize()
        assert all(same(a, b) for a, b in zip(got, want)), lengths


def test_offsets_beyond_32_bits(rope):
    """524288 rows of 32 + 8 heads of 128 (q has 2^31 elements) as sequences of 100 to 300
    tokens: the first, the last and one between against the definition."""
    T, Hq, Hkv, D = 524288, 32, 8, 128
    print("[64-bit offsets]", flush=True)
    cu = [0]
    i = 0
    while cu[-1] < T:
        cu.append(min(T, cu[-1] + 100 + (37 * i) % 201))
        i += 1
    qkv = torch.empty((T, Hq + 2 * Hkv, D), dtype=BF16, device=DEV)
    for a in range(0, T, 65536):
        qkv[a:a + 65536] = normal((65536, Hq + 2 * Hkv, D), a + 1, BF16)
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    plan = rope.attn_plan(int32(cu), T, Hq, Hkv)
    out, lse = rope.attn_fwd(q, k, v, plan)
    grads = rope.attn_bwd(q, q, k, v, out, lse, plan)
    torch.cuda.synchronize()
    for s in (0, len(cu) // 2, len(cu) - 2):
        a, b = cu[s], cu[s + 1]
        rows = slice(a, b)
        seqs = [(0, b - a)]
        want, _, tol = ref.forward(q[rows], k[rows], v[rows], seqs, D ** -0.5)
        ref.check(out[rows], want, tol, f"out of sequence {s}")
        wants, tols = ref.backward(q[rows], q[rows], k[rows], v[rows], seqs, D ** -0.5, BF16)
        for g, w, t in zip(grads, wants, tols):
            ref.check(g[rows], w, t, f"gradient of sequence {s}")


def test_long_sequence_rows(rope):
    """One sequence of 20000 tokens: sampled rows of out, dq, dk and dv against the definition."""
    T, Hq, Hkv, D = 20000, 2, 1, 64
    print("[long]", flush=True)
    q, k, v = batch(T, Hq, Hkv, D, BF16, seed=12)
    do = normal((T, Hq, D), 13, BF16)
    plan = rope.attn_plan(int32([0, T]), T, Hq, Hkv)
    out, lse = rope.attn_fwd(q, k, v, plan)
    grads = rope.attn_bwd(do, q, k, v, out, lse, plan)
    want, wlse, tol = ref.forward(q, k, v, [(0, T)], D ** -0.5)
    ref.check(out, want, tol, "out")
    wants, tols = ref.backward(do, q, k, v, [(0, T)], D ** -0.5, BF16)
    for g, w, t in zip(grads, wants, tols):
        ref.check(g, w, t, "gradient")


def test_many_sequences(rope):
    """More sequences than a plan reads at a time, empty ones among them."""
    lengths = [(7 * i) % 5 for i in range(3001)]
    cu = [0]
    for n in lengths:
        cu.append(cu[-1] + n)
    T = cu[-1] + 9
    q, k, v = batch(T, 4, 2, 64, BF16, seed=15)
    plan = rope.attn_plan(int32(cu), T, 4, 2)
    out, lse = rope.attn_fwd(q, k, v, plan)
    dq, dk, dv = rope.attn_bwd(q, q, k, v, out, lse, plan)
    # sequences of like length are alike: each length as one batched problem in 64 bits
    for n in range(1, 5):
        at = torch.tensor([c for c, m in zip(cu, lengths) if m == n], device=DEV)[:, None] + torch.arange(n, device=DEV)
        for h in range(4):
            qh, kh, vh = q[at][:, :, h].double(), k[at][:, :, h // 2].double(), v[at][:, :, h // 2].double()
            s = (qh @ kh.transpose(1, 2).contiguous() * 0.125).masked_fill(
                torch.ones(n, n, dtype=torch.bool, device=DEV).triu(1), float("-inf"))
            p = torch.softmax(s, -1)
            o = p @ vh
            tol = 1.02 * ref.half_step(BF16) * (p @ vh.abs() + o.abs()) + 1e-4 * (p @ vh.abs())
            ref.check(out[at][:, :, h], o, tol, f"length {n}")
    assert bool((out[cu[-1]:] == 0).all()) and bool((dk[cu[-1]:] == 0).all())


def test_tokens_that_overlap_are_refused(rope):
    """An expanded tensor has token stride 0, which the C ABI reads as dense rows."""
    q, k, v = batch(64, 4, 2, 64, BF16)
    plan = rope.attn_plan(int32([0, 64]), 64, 4, 2)
    out, lse = rope.attn_fwd(q, k, v, plan)
    inputs = [q, q, k, v, out]
    for i in range(5):
        a = list(inputs)
        a[i] = a[i][:1].expand_as(a[i])
        with pytest.raises(ValueError, match="overlap"):
            rope.attn_bwd(*a, lse, plan)
        if 0 < i < 4:
            with pytest.raises(ValueError, match="overlap"):
                rope.attn_fwd(*a[1:4], plan)
    half = torch.as_strided(q, (64, 4, 64), (128, 64, 1))
    for kw in (dict(out=half, lse=lse), dict(out=q[:1].expand_as(q), lse=lse)):
        with pytest.raises(ValueError, match="overlap"):
            rope.attn_fwd(q, k, v, plan, **kw)
    one = rope.attn_plan(int32([0, 1]), 1, 4, 2)  # one token: its stride says nothing
    a = [torch.as_strided(x, (1, *x.shape[1:]), (0, 64, 1)) for x in (q, k, v)]
    got, ref1 = rope.attn_fwd(*a, one), rope.attn_fwd(q[:1], k[:1], v[:1], one)
    assert same(got[0], ref1[0]) and same(got[1], ref1[1])


def test_plan_of_another_kind_is_refused(rope):
    q, k, v = batch(64, 4, 2, 64, BF16)
    cu = int32([0, 64])
    packed, paged = rope.attn_plan(cu, 64, 4, 2), rope.paged_plan(cu, int32([64]), 64, 4, 2)
    cache, table = k.reshape(4, 16, 2, 64), int32([[0, 1, 2, 3]])
    with pytest.raises(TypeError, match="attn_plan"):
        rope.attn_fwd(q, k, v, paged)
    with pytest.raises(TypeError, match="paged_plan"):
        rope.attn_paged(q, cache, cache, table, packed)
    out, lse = torch.full_like(q, 3.0), torch.full((64, 4), 3.0, device=DEV)
    grads = [torch.full_like(x, 3.0) for x in (q, k, v)]
    fake = rope.AttnPlan(64, 1, 4, 2, paged.buffer)  # the kernels look, too
    rope.attn_fwd(q, k, v, fake, out=out, lse=lse)
    rope.attn_bwd(q, q, k, v, out, lse, fake, None, *grads)
    rope.attn_paged(q, cache, cache, table, rope.PagedPlan(64, 1, 4, 2, packed.buffer), out=out, lse=lse)
    assert all(bool((x == 3).all()) for x in (out, lse, *grads))


def test_no_tokens_and_no_sequences(rope):
    from packed_varlen_rotary_rope_amd import functional as F
    q, k, v = batch(0, 4, 2, 64, BF16)
    for cu in ([0], [0, 0, 0]):
        plan = rope.attn_plan(int32(cu), 0, 4, 2)
        out, lse = rope.attn_fwd(q, k, v, plan)
        assert out.shape == (0, 4, 64) and lse.shape == (0, 4)
        assert [g.shape for g in rope.attn_bwd(q, q, k, v, out, lse, plan)] == [q.shape, k.shape, v.shape]
    q, k, v = (x.requires_grad_() for x in batch(130, 4, 2, 64, BF16))
    out = F.attn(q, k, v, cu_seqlens=int32([0]))
    out.sum().backward()
    assert all(bool((x == 0).all()) for x in (out, q.grad, k.grad, v.grad))


def test_no_second_derivative(rope):
    from packed_varlen_rotary_rope_amd import functional as F
    q, k, v = (x.requires_grad_() for x in batch(40, 2, 1, 64, BF16))
    (g,) = torch.autograd.grad(F.attn(q, k, v, cu_seqlens=int32([0, 40])).float().square().sum(), q,
                               create_graph=True)
    with pytest.raises(RuntimeError):
        g.float().sum().backward()


LARGE = [(BF16, 20, 12), (BF16, 8, 8), (BF16, 40, 40), (F16, 10, 4), (F16, 5, 5), (F16, 15, 7)]


@pytest.mark.parametrize("D", [64, 128, 192])
@pytest.mark.parametrize("dtype,a,b", LARGE)
@pytest.mark.parametrize("sign", [1, -1])
def test_very_large_scores(rope, D, dtype, a, b, sign):
    """Scores sign * n 2^(a+b) D^0.5 with distinct integers n, exact in fp32: each row's softmax is
    one key's. That weight is 1, or 2^e rounded with its sum 2^e unrounded, |e| <= 4: out is off by
    its half step and the output's. lse is the score, scaled twice and multiplied by ln 2."""
    print(f"[large] D={D} {dtype} {a} {b} {sign}", flush=True)
    T, cu = 256, [0, 100, 256]
    n = (torch.randperm(T, generator=torch.Generator().manual_seed(D + a)) + 1).to(DEV)
    q = torch.full((T, 4, D), 2.0 ** a, device=DEV).to(dtype)
    k = (sign * n[:, None, None] * 2.0 ** b).expand(T, 2, D).to(dtype).contiguous()
    v = normal((T, 2, D), 5, dtype)
    out, lse = rope.attn_fwd(q, k, v, rope.attn_plan(int32(cu), T, 4, 2))
    for s, e in zip(cu, cu[1:]):
        m = torch.cummax(sign * n[s:e], 0)
        want = v[s:e][m.indices].repeat_interleave(2, 1).double()
        ref.check(out[s:e], want, want.abs() * 2.1 * ref.half_step(dtype), "out")
        score = (m.values.double() * 2.0 ** (a + b) * D ** 0.5)[:, None].expand(-1, 4)
        ref.check(lse[s:e], score, score.abs() * 2.0 ** -21, "lse")


@pytest.mark.parametrize("D,G,dtype", [(32, 2, F16), (40, 1, BF16), (64, 1, BF16), (64, 3, F16), (80, 3, BF16), (128, 4, F16)])
def test_rows_that_are_not_finite_among_short_sequences(rope, D, G, dtype):
    """1200 sequences of 11 to 60 tokens, so that a workgroup of the dK/dV pass walks several key
    tiles one behind the other, and in every third sequence one row of dout with an infinity: every
    other column of dv keeps its bits, also in the keys that the row sees, and so does all that the
    row does not reach. Several times: waves must not run into each other's tiles."""
    print(f"[short, not finite] D={D} G={G} {dtype}", flush=True)
    cu = [0]
    for i in range(1200):
        cu.append(cu[-1] + 11 + (7 * i) % 50)
    T, Hkv = cu[-1], 2
    q, k, v = batch(T, Hkv * G, Hkv, D, dtype, seed=D + G)
    do = normal((T, Hkv * G, D), 5, dtype)
    plan = rope.attn_plan(int32(cu), T, Hkv * G, Hkv)
    out, lse = rope.attn_fwd(q, k, v, plan)
    dq0, dk0, dv0 = rope.attn_bwd(do, q, k, v, out, lse, plan)
    reached = torch.zeros(T, dtype=torch.bool)
    rows = torch.zeros(T, dtype=torch.bool)
    for s in range(0, 1200, 3):
        at = cu[s] + (5 * s) % (cu[s + 1] - cu[s])
        rows[at] = True
        reached[cu[s]:at + 1] = True
    rows, reached = rows.to(DEV), reached.to(DEV)
    do[rows, G, 2] = float("inf")  # of the second key/value head's first query head
    rest = torch.arange(D, device=DEV) != 2
    for _ in range(4):
        dq, dk, dv = rope.attn_bwd(do, q, k, v, out, lse, plan)
        assert same(dv[:, :, rest], dv0[:, :, rest])
        assert same(dv[~reached], dv0[~reached]) and same(dk[~reached], dk0[~reached])
        assert same(dv[:, 0], dv0[:, 0]) and same(dk[:, 0], dk0[:, 0])
        assert same(dq[~rows], dq0[~rows])
        assert not bool(dv[reached][:, 1, 2].isfinite().any())


def first_large_then_ordinary(T, D, dtype, H, seed):
    """Keys of which the first 64 have scores below -2^28 (f16) or -2^31 (bf16) once scaled and the
    others scores of exactly 0, so that a query of the later ones weighs those alike."""
    a = 5736.0 if dtype == F16 else 17536.0
    q = torch.full((T, 2, D), a, dtype=dtype, device=DEV)
    k = torch.zeros((T, H, D), dtype=dtype, device=DEV)
    k[:64] = -a
    return q, k, normal((T, H, D), seed, dtype)


@pytest.mark.parametrize("D", [64, 128, 192])
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("H", [1, 2])
def test_very_large_scores_before_ordinary_ones(rope, D, dtype, H):
    """A maximum that was large and is small in the end. n keys of score 0 have the weight 1 / n
    each, exactly formed; their fp32 sum of n products errs by n 2^-23 of its spread, and out is
    rounded once. The rows before see equal scores too, however large."""
    print(f"[large first] D={D} {dtype} H={H}", flush=True)
    T = 400
    q, k, v = first_large_then_ordinary(T, D, dtype, H, 6)
    out, lse = rope.attn_fwd(q, k, v, rope.attn_plan(int32([0, T]), T, 2, H))
    v64 = v.repeat_interleave(2 // H, 1).double()
    for a, b in ((0, 64), (64, T)):
        n = torch.arange(1, b - a + 1, device=DEV, dtype=torch.float64)[:, None, None]
        mean, spread = v64[a:b].cumsum(0) / n, v64[a:b].abs().cumsum(0) / n
        ref.check(out[a:b], mean, 1.01 * (ref.half_step(dtype) * mean.abs() + T * 2.0 ** -23 * spread) +
                  ref.tiny(dtype), f"out from {a}")
    n = torch.arange(1, T - 63, device=DEV, dtype=torch.float64)[:, None].expand(-1, 2)
    ref.check(lse[64:], n.log(), (n.log() + 1) * 2.0 ** -21, "lse")


def test_gradient_at_an_odd_address(rope):
    """Outputs that go into one flat buffer behind something else: their gradient is contiguous and
    not aligned."""
    import packed_varlen_rotary_rope_amd.functional as F
    cu = int32([0, 20, 50])
    leaves = [x.requires_grad_() for x in batch(50, 4, 2, 64, BF16)]
    plan = rope.attn_plan(cu, 50, 4, 2)
    weights = normal((3 + 50 * 4 * 64,), 8, BF16)
    (torch.cat([torch.zeros(3, dtype=BF16, device=DEV), F.attn(*leaves, plan).flatten()]) * weights).sum().backward()
    q, k, v = (x.detach() for x in leaves)
    out, lse = rope.attn_fwd(q, k, v, plan)
    do = weights[3:].view(50, 4, 64).clone()
    for x, g in zip(leaves, rope.attn_bwd(do, q, k, v, out, lse, plan)):
        assert same(x.grad, g)
    fused = torch.cat([x.flatten(1) for x in (q, k, v)], 1).requires_grad_()
    (torch.cat([torch.zeros(3, dtype=BF16, device=DEV), F.attn_qkv(fused, 4, 2, plan).flatten()]) * weights).sum().backward()
    assert same(fused.grad, torch.cat([x.grad.flatten(1) for x in leaves], 1))


def test_many_sequences_gradients(rope):
    """The gradients of 3001 sequences of up to 4 tokens, several of them in each tile of a
    workgroup's share, each against the formula in 64 bits (on the CPU: they are many and small)."""
    lengths = [(7 * i) % 5 for i in range(3001)]
    cu = [0]
    for n in lengths:
        cu.append(cu[-1] + n)
    T = cu[-1] + 9
    q, k, v = batch(T, 4, 2, 64, BF16, seed=15)
    do = normal((T, 4, 64), 16, BF16)
    plan = rope.attn_plan(int32(cu), T, 4, 2)
    out, lse = rope.attn_fwd(q, k, v, plan)
    got = rope.attn_bwd(do, q, k, v, out, lse, plan)
    want, tols = ref.backward(*(x.cpu() for x in (do, q, k, v)), ref.sequences(cu, T), 0.125, BF16)
    for name, g, w, tol in zip(("dq", "dk", "dv"), got, want, tols):
        assert bool((g[cu[-1]:] == 0).all())
        ref.check(g.cpu(), w, tol, name)


def mixed_scores(n, m, heads, D, dtype, seed):
    """q [n, heads[0], D] and k [m, heads[1], D] of powers of 2 and zeros, each token at a magnitude
    of its own, so that every product of two rows is exact in fp32 and scores run from 1 to 2^60
    (f16: 2^27) side by side."""
    g = torch.Generator().manual_seed(seed)
    tops = torch.tensor([0, 0, 1, 4, 9, 17, 27] if dtype == BF16 else [0, 0, 1, 4, 7, 9, 12])

    def rows(count, h):
        sign = torch.randint(-1, 2, (count, h, D), generator=g).float()
        size = tops[torch.randint(0, len(tops), (count, h), generator=g)].float()
        return (sign * 2.0 ** size[..., None]).to(dtype).to(DEV)

    return rows(n, heads[0]), rows(m, heads[1])


def head_of_any_scores(q, k, v, scale, before, gone=None):
    """One head in 64 bits as attn_reference.head_forward, with the maximum taken off before the
    logarithm: past 2^50 a log-sum-exp of 64 bits no longer holds the logarithm."""
    n, m = q.shape[0], k.shape[0]
    hidden = torch.arange(m, device=DEV)[None] > before + torch.arange(n, device=DEV)[:, None]
    if gone is not None:
        hidden = hidden | gone[None]
        k = k.masked_fill(gone[:, None], 0.0)
    s = (q.double() @ k.double().T * scale).masked_fill(hidden, float("-inf"))
    top = s.amax(-1, keepdim=True)
    e = torch.exp(s - top.masked_fill(top == float("-inf"), 0.0))
    total = e.sum(-1, keepdim=True)
    p = e / total.masked_fill(total == 0.0, 1.0)
    return p @ v, (top + total.log())[:, 0], p


def exact_scores_bound(o, p, v, dtype, n):
    """Bound of out where scores are exact: a weight 2^-x is formed from an exponent that errs by
    2^-22 x (scale, product and join, in fp32), which moves it by 2^-22 x 2^-x < 2^-22 of the
    largest, and is rounded once (subnormal f16 weights by 2^-25 of the largest); sums of n terms
    err by n 2^-23."""
    u = ref.half_step(dtype)
    spread = p @ v.abs()
    largest = p.amax(-1, keepdim=True) * v.abs().sum(0)
    return 1.01 * (u * (o.abs() + spread) + (n + 32) * 2.0 ** -23 * spread + 2.0 ** -21 * largest) + ref.tiny(dtype)


@pytest.mark.parametrize("seed", range(4))
@pytest.mark.parametrize("D,Hq,Hkv", [(32, 4, 1), (64, 4, 2), (128, 2, 2), (192, 3, 1)])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_scores_of_all_sizes(rope, seed, D, Hq, Hkv, dtype):
    """Ordinary, large and very large scores in one batch, in any order and with ties."""
    print(f"[all sizes] {seed} D={D} {Hq}+{Hkv} {dtype}", flush=True)
    cu, T = [0, 5, 150, 151, 480], 480
    q, k = mixed_scores(T, T, (Hq, Hkv), D, dtype, seed)
    v = normal((T, Hkv, D), seed, dtype)
    out, lse = rope.attn_fwd(q, k, v, rope.attn_plan(int32(cu), T, Hq, Hkv))
    for a, n in ref.sequences(cu, T):
        rows = slice(a, a + n)
        for h in range(Hq):
            v64 = v[rows, h // (Hq // Hkv)].double()
            o, l, p = head_of_any_scores(q[rows, h], k[rows, h // (Hq // Hkv)], v64, D ** -0.5, 0)
            ref.check(out[rows, h], o, exact_scores_bound(o, p, v64, dtype, n), "out")
            ref.check(lse[rows, h], l, (l.abs() + 8) * 2.0 ** -21, "lse")
