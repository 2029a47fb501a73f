"""GPU tests of the rotation by positions with several axes and of the append by a slot map: bit for
bit against the rotary kernels with one axis at a time, and against the formula in 64 bits."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
F64 = torch.float64


@pytest.fixture(scope="module")
def rope():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import packed_varlen_rotary_rope_amd as m
    return m


def normal(shape, seed, dtype):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randn(shape, generator=g, device=DEV).to(dtype)


def ids(axes, T, seed, most=5000):
    g = torch.Generator().manual_seed(seed)
    return torch.randint(0, most, (axes, T), generator=g).int().to(DEV)


def bits(t):
    return t.contiguous().view(torch.int32 if t.dtype == F32 else torch.int16)


def same(a, b):
    return torch.equal(bits(a), bits(b))


def axis_of(sections, layout):
    """Of each frequency its axis, from the definition."""
    half, A = sum(sections), len(sections)
    out = []
    for j in range(half):
        if layout == "interleaved":
            out.append(j % A if j < A * sections[j % A] else 0)
        else:
            out.append(next(a for a in range(A) if j < sum(sections[:a + 1])))
    return out


def frequencies(sections, layout, theta, D):
    if layout != "separate":
        e = [-2.0 * j / D for j in range(D // 2)]
    else:
        e = [-i / n for n in sections for i in range(n)]
    return torch.tensor([theta ** x for x in e], dtype=F64).to(F32).to(DEV)


def angles(pos, sections, layout, theta, D, pos_scale=1.0):
    """fp32 angles [T, D/2]: one division, one product, rounded each."""
    p = pos.to(F32)
    if pos_scale != 1.0:
        p = p / torch.tensor(pos_scale, dtype=F32, device=DEV)
    axis = torch.tensor(axis_of(sections, layout), device=DEV)
    return p[axis].t() * frequencies(sections, layout, theta, D)


def turned(x, angle, direction):
    """In 64 bits."""
    c, s = angle.to(F64).cos()[:, None], direction * angle.to(F64).sin()[:, None]
    a, b = x.to(F64).chunk(2, -1)
    return torch.cat([a * c - b * s, b * c + a * s], -1)


def check(got, want, what):
    """Two fp32 ulps, the correctly rounded cos and sin (half an fp32 step of either product) and
    one rounding: |err| <= eps/2 |y| + (2 ulp: 2^-22 |y|) + 2^-24 (|a| + |b|) <= .. with |a|, |b| at most the
    largest value, doubled for second order."""
    u = torch.finfo(got.dtype).eps / 2
    top = float(want.abs().max()) * math.sqrt(2.0)
    err = (got.to(F64) - want).abs()
    tol = (u + 2.0 ** -22) * want.abs() + 2 * 2.0 ** -24 * 2 * top + (2.0 ** -25 if got.dtype == F16 else 0.0)
    assert bool((err <= tol).all()), (what, float((err - tol).max()))


FORMS = [  # T, Hq, Hkv, D, sections, layout, dtype
    (1, 1, 1, 2, (1,), "sections", F32),
    (3, 1, 0, 4, (1, 1), "separate", BF16),
    (37, 4, 2, 16, (4, 2, 2), "sections", F32),
    (1000, 32, 8, 128, (24, 20, 20), "interleaved", BF16),
    (1000, 32, 8, 128, (16, 24, 24), "sections", BF16),
    (501, 16, 16, 80, (20, 20), "separate", F16),
    (77, 3, 1, 50, (9, 8, 8), "interleaved", BF16),
    (2055, 5, 5, 72, (36, 0), "sections", F16),
    (33, 7, 1, 512, (64, 64, 64, 64), "separate", BF16),
    (300, 2, 2, 96, (12, 12, 12, 12), "interleaved", F32),
    (9, 160, 2, 256, (100, 14, 14), "sections", F16),
    (4099, 1, 1, 8, (2, 1, 1), "interleaved", BF16),
]


@pytest.mark.parametrize("case", FORMS, ids=lambda c: f"T{c[0]}_{c[1]}_{c[2]}_{c[3]}_{c[5]}_{str(c[6])[6:]}")
@pytest.mark.parametrize("direction", [1, -1])
def test_against_the_formula(rope, case, direction):
    T, Hq, Hkv, D, sections, layout, dtype = case
    print(f"[axes] {case} {direction}", flush=True)
    q, k, pos = normal((T, Hq, D), 1, dtype), normal((T, Hkv, D), 2, dtype), ids(len(sections), T, 3)
    got = rope.qk_apply_axes(q, k, pos, sections, 1e4, direction, layout, 2.5)
    angle = angles(pos, sections, layout, 1e4, D, 2.5)
    for name, x, y in zip("qk", (q, k), got):
        if x.numel():
            check(y, turned(x, angle, direction), name)
    # in place, and from and into parts of fused tensors
    fused = normal((T, Hq + 2 * Hkv + 1, D), 4, dtype)
    fused[:, :Hq], fused[:, Hq:Hq + Hkv] = q, k
    before = fused.clone()
    a, b = fused[:, :Hq], fused[:, Hq:Hq + Hkv]
    other = torch.zeros_like(fused)
    oa, ob = other[:, :Hq], other[:, Hq:Hq + Hkv]
    rope.qk_apply_axes(a, b, pos, sections, 1e4, direction, layout, 2.5, oa, ob)
    assert same(fused, before) and same(oa, got[0]) and same(ob, got[1]) and not bool(other[:, Hq + Hkv:].any())
    r = rope.qk_apply_axes(a, b, pos, sections, 1e4, direction, layout, 2.5, a, b)
    assert r[0] is a and same(a, got[0]) and same(b, got[1]) and same(fused[:, Hq + Hkv:], before[:, Hq + Hkv:])


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("layout", ["sections", "interleaved"])
def test_equal_positions_are_the_ordinary_rotation(rope, dtype, layout):
    T, D = 700, 128
    q, k = normal((T, 8, D), 1, dtype), normal((T, 2, D), 2, dtype)
    pos = ids(1, T, 3, 2 ** 31 - 1)
    pos[0, ::7] = -1
    want = rope.qk_apply_ex_(q.clone(), k.clone(), 1e6, -1, position_ids=pos[0].contiguous(), pos_scale=4.0)
    got = rope.qk_apply_axes(q, k, pos.expand(3, T).contiguous(), (24, 20, 20), 1e6, -1, layout, 4.0)
    assert same(got[0], want[0]) and same(got[1], want[1])


def test_each_axis_by_itself(rope):
    """Every frequency is the one-axis rotation's at its axis's position, bit for bit."""
    T, D, sections = 400, 64, (14, 10, 8)
    q, k, pos = normal((T, 6, D), 1, BF16), normal((T, 2, D), 2, BF16), ids(3, T, 3)
    for layout in ("sections", "interleaved"):
        got = rope.qk_apply_axes(q, k, pos, sections, 1e6, 1, layout)
        axis = torch.tensor(axis_of(sections, layout) * 2, device=DEV)
        for a in range(3):
            want = rope.qk_apply_ex_(q.clone(), k.clone(), 1e6, 1, position_ids=pos[a].contiguous())
            for x, y in zip(got, want):
                assert torch.equal(bits(x)[..., axis == a], bits(y)[..., axis == a])


def test_negative_positions_are_copied(rope):
    T, D = 130, 80
    q, k, pos = normal((T, 4, D), 1, F16), normal((T, 4, D), 2, F16), ids(2, T, 3)
    pos[0, 5], pos[1, 77], pos[:, 129] = -1, -(2 ** 31), -9
    q[77] = float("nan")
    got = rope.qk_apply_axes(q, k, pos, (30, 10), 1e4, layout="separate")
    still = torch.zeros(T, dtype=torch.bool, device=DEV)
    still[[5, 77, 129]] = True
    assert same(got[0][still], q[still]) and same(got[1][still], k[still])
    assert bool((bits(got[0]) != bits(q))[~still].flatten(1).any(1).all())


def test_odd_addresses_and_strides(rope):
    T, D = 55, 48
    base = [normal((T * 400 + 1,), i, BF16) for i in range(2)]
    q, k = (b[1:].view(T, 400)[:, 3:3 + h * D].unflatten(1, (h, D)) for b, h in zip(base, (5, 2)))
    pos = ids(4, 2 * T, 3)[1:, 1:T + 1]  # rows further apart than T
    got = rope.qk_apply_axes(q, k, pos, (8, 8, 8), 1e4)
    want = rope.qk_apply_axes(q.contiguous(), k.contiguous(), pos.contiguous(), (8, 8, 8), 1e4)
    assert same(got[0], want[0]) and same(got[1], want[1])


def test_empty(rope):
    e = torch.empty((0, 4, 64), dtype=BF16, device=DEV)
    got = rope.qk_apply_axes(e, e, torch.empty((3, 0), dtype=torch.int32, device=DEV), (16, 8, 8), 1e4)
    assert got[0].shape == e.shape


def test_refusals(rope):
    q, k, pos = normal((16, 4, 64), 1, BF16), normal((16, 2, 64), 2, BF16), ids(3, 16, 3)
    ok = (16, 8, 8)
    rope.qk_apply_axes(q, k, pos, ok, 1e4)
    for bad in ((16, 8), (16, 8, 9), (-1, 25, 8), (32, 0, 0, 0, 0), ()):
        with pytest.raises(ValueError):
            rope.qk_apply_axes(q, k, pos, bad, 1e4)
    with pytest.raises(ValueError, match="turns"):
        rope.qk_apply_axes(q, k, pos, (8, 12, 12), 1e4, layout="interleaved")
    with pytest.raises(ValueError, match="layout"):
        rope.qk_apply_axes(q, k, pos, ok, 1e4, layout="mixed")
    for bad in (pos[:2], pos[:, :15], pos.t(), pos[0]):
        with pytest.raises(ValueError, match="position_ids"):
            rope.qk_apply_axes(q, k, bad, ok, 1e4)
    for bad in (pos.long(), pos.cpu()):
        with pytest.raises(TypeError):
            rope.qk_apply_axes(q, k, bad, ok, 1e4)
    with pytest.raises(ValueError, match="contiguous and of its own"):
        rope.qk_apply_axes(q, k, pos[:1].expand(3, 16), ok, 1e4)
    with pytest.raises(rope.RopeError):
        rope.qk_apply_axes(q, k, pos, ok, 0.5)
    with pytest.raises(rope.RopeError):
        rope.qk_apply_axes(q, k, pos, ok, 1e4, direction=2)
    with pytest.raises(rope.RopeError):
        rope.qk_apply_axes(q, k, pos, ok, 1e4, pos_scale=0.5)
    with pytest.raises(TypeError):
        rope.qk_apply_axes(q, k.half(), pos, ok, 1e4)
    with pytest.raises(ValueError):
        rope.qk_apply_axes(q, k[:8], pos, ok, 1e4)
    with pytest.raises(ValueError, match="overlap"):
        rope.qk_apply_axes(q[:1].expand(16, 4, 64), k, pos, ok, 1e4)
    with pytest.raises(ValueError):
        rope.qk_apply_axes(q, k, pos, ok, 1e4, q_out=q[:, :2])


def test_gradients(rope):
    """rope_qk_axes and rope_qkv_axes against the formula's transposed rotation, views and expanded
    gradients among them."""
    import packed_varlen_rotary_rope_amd.functional as F
    T, Hq, Hkv, D, sections = 90, 4, 2, 64, (12, 10, 10)
    pos = ids(3, T, 3)
    angle = angles(pos, sections, "interleaved", 1e4, D)
    x = normal((T, Hq + 2 * Hkv, D), 1, F32).requires_grad_()
    w = normal((T, Hq + 2 * Hkv, D), 2, F32)
    y = F.rope_qkv_axes(x * 1.0, Hq, Hkv, pos, sections, 1e4, "interleaved")
    check(y[:, :Hq + Hkv].detach(), turned(x[:, :Hq + Hkv].detach(), angle, 1), "qkv")
    y.backward(w)
    check(x.grad[:, :Hq + Hkv], turned(w[:, :Hq + Hkv], angle, -1), "dqkv")
    assert torch.equal(x.grad[:, Hq + Hkv:], w[:, Hq + Hkv:])
    x2 = x.detach().clone().requires_grad_()  # a leaf and views of it
    q, k = F.rope_qk_axes(x2[:, :Hq], x2[:, Hq:Hq + Hkv], pos, sections, 1e4, "interleaved")
    assert torch.equal(torch.cat([q, k], 1), y[:, :Hq + Hkv])
    (q.sum() + (k * w[:, Hq:Hq + Hkv]).sum()).backward()
    check(x2.grad[:, :Hq], turned(torch.ones_like(q), angle, -1), "dq")
    check(x2.grad[:, Hq:Hq + Hkv], turned(w[:, Hq:Hq + Hkv], angle, -1), "dk")
    assert not bool(x2.grad[:, Hq + Hkv:].any())


def test_offsets_beyond_32_bits(rope):
    """Rows behind 2^31 elements of a strided tensor."""
    T, D, stride = 300, 64, 1 << 23
    big = torch.zeros((T * stride,), dtype=BF16, device=DEV)
    q = big.as_strided((T, 2, D), (stride, D, 1))
    q.copy_(normal((T, 2, D), 1, BF16))
    k, pos = normal((T, 1, D), 2, BF16), ids(2, T, 3)
    want = rope.qk_apply_axes(q.contiguous(), k, pos, (16, 16), 1e4)
    rope.qk_apply_axes(q, k, pos, (16, 16), 1e4, q_out=q, k_out=k)
    assert same(q, want[0]) and same(k, want[1])


APPENDS = [  # T, Hq, Hkv, D, page, sections, layout, dtype
    (1, 1, 1, 2, 1, (1,), "sections", F32),
    (64, 32, 8, 128, 16, (16, 24, 24), "sections", BF16),
    (1300, 32, 8, 128, 64, (24, 20, 20), "interleaved", BF16),
    (333, 6, 2, 80, 48, (20, 20), "separate", F16),
    (70, 3, 1, 50, 7, (9, 8, 8), "interleaved", BF16),
    (12, 2, 1, 512, 16, (256,), "sections", F32),
]


@pytest.mark.parametrize("case", APPENDS, ids=lambda c: f"T{c[0]}_{c[1]}_{c[2]}_{c[3]}_{c[4]}_{c[6]}_{str(c[7])[6:]}")
@pytest.mark.parametrize("form", ["fused", "by_head", "keys_only", "in_place"])
def test_append(rope, case, form):
    """The cache rows of the slot map are those of the rotation, bit for bit; tokens without a slot and
    the rest of the cache are left as they were; tokens without a position go there as they are."""
    T, Hq, Hkv, D, page, sections, layout, dtype = case
    print(f"[kv_append_slots] {case} {form}", flush=True)
    g = torch.Generator().manual_seed(7)
    pages = -(-T // page) + 3
    shape = (pages, Hkv, page, D) if form == "by_head" else (pages, page, Hkv, D)
    caches = [torch.full(shape, float("nan"), dtype=dtype, device=DEV) for _ in range(2)]
    kc, vc = (c.transpose(1, 2) if form == "by_head" else c for c in caches)
    slots = torch.randperm(pages * page, generator=g)[:T].to(DEV)
    pos = ids(len(sections), T, 3)
    if T > 5:
        slots[3], slots[4] = -1, pages * page
        slots[5] = 2 ** 40
        pos[-1, 2] = -1
    if form == "fused":
        qkv = normal((T, Hq + 2 * Hkv, D), 1, dtype)
        q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    else:
        q, k, v = (normal((T, h, D), i, dtype) for i, h in enumerate((Hq, Hkv, Hkv)))
    want_q, want_k = rope.qk_apply_axes(q, k, pos, sections, 1e6, 1, layout, 2.0)
    want = [c.clone() for c in (kc, vc)]
    on = (slots >= 0) & (slots < pages * page)
    where = slots[on] // page, slots[on] % page
    want[0][where], want[1][where] = want_k[on], v[on]
    kw = {} if form == "keys_only" else dict(q=q, q_out=q) if form == "in_place" else dict(q=q)
    got = rope.kv_append_slots_(k, v, kc, vc, slots, pos, 1e6, sections, layout, pos_scale=2.0, **kw)
    assert same(kc, want[0]) and same(vc, want[1])
    assert got is None if form == "keys_only" else same(got, want_q)


def test_append_is_kv_append_with_one_axis(rope):
    new, held, page = [5, 1, 130], [5, 77, 900], 16
    T, Hq, Hkv, D = sum(new), 6, 2, 64
    cu = torch.tensor([0, 5, 6, 136], dtype=torch.int32, device=DEV)
    lens = torch.tensor(held, dtype=torch.int32, device=DEV)
    table = torch.randperm(200, generator=torch.Generator().manual_seed(3))[:3 * 57].view(3, 57).int().to(DEV)
    q, k, v = (normal((T, h, D), i, BF16) for i, h in enumerate((Hq, Hkv, Hkv)))
    caches = [normal((200, page, Hkv, D), 9, BF16) for _ in range(4)]
    want = rope.kv_append_(k, v, caches[0], caches[1], table, cu, lens, 1e6, q=q)
    pos = torch.cat([torch.arange(m - n, m) for n, m in zip(new, held)]).to(DEV)
    seq = torch.repeat_interleave(torch.arange(3), torch.tensor(new)).to(DEV)
    slots = table.long()[seq, pos // page] * page + pos % page
    got = rope.kv_append_slots_(k, v, caches[2], caches[3], slots, pos.int(), 1e6, q=q)
    assert same(got, want) and same(caches[2], caches[0]) and same(caches[3], caches[1])


def test_append_refusals(rope):
    k = normal((8, 2, 64), 1, BF16)
    cache = torch.zeros((4, 16, 2, 64), dtype=BF16, device=DEV)
    slots, pos = torch.arange(8, device=DEV), ids(1, 8, 2)
    rope.kv_append_slots_(k, k, cache, cache.clone(), slots, pos, 1e4)
    with pytest.raises(TypeError):
        rope.kv_append_slots_(k, k, cache, cache, slots.int(), pos, 1e4)
    with pytest.raises(ValueError):
        rope.kv_append_slots_(k, k, cache, cache, slots[:7], pos, 1e4)
    with pytest.raises(ValueError):
        rope.kv_append_slots_(k, k, cache, cache, slots, pos, 1e4, sections=(16, 16))
    with pytest.raises(ValueError, match="overlap"):
        one = cache[:1].expand(4, 16, 2, 64)
        rope.kv_append_slots_(k, k, one, one, slots, pos, 1e4)
    with pytest.raises(ValueError):
        rope.kv_append_slots_(k, k, cache[:, :, :1], cache[:, :, :1], slots, pos, 1e4)


def test_streams_and_graph(rope):
    """On another stream, and captured: replays write what eager calls write for new inputs."""
    T, D, sections = 200, 64, (12, 10, 10)
    q, k, v = (normal((T, h, D), i, BF16) for i, h in enumerate((4, 2, 2)))
    pos, slots = ids(3, T, 3), torch.randperm(256, device=DEV)[:T]
    kc, vc = (torch.zeros((16, 16, 2, D), dtype=BF16, device=DEV) for _ in range(2))
    q_out, a, b = torch.empty_like(q), torch.empty_like(q), torch.empty_like(k)

    def step():
        rope.kv_append_slots_(k, v, kc, vc, slots, pos, 1e4, sections, q=q, q_out=q_out)
        rope.qk_apply_axes(q, k, pos, sections, 1e4, -1, q_out=a, k_out=b)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in range(3):
        q.copy_(normal(q.shape, 50 + seed, BF16))
        pos.copy_(ids(3, T, 60 + seed))
        slots.copy_(torch.randperm(256, device=DEV)[:T])
        kc.zero_()
        vc.zero_()
        graph.replay()
        got = [x.clone() for x in (q_out, a, b, kc, vc)]
        kc.zero_()
        vc.zero_()
        step()
        torch.cuda.synchronize()
        assert all(same(x, y) for x, y in zip(got, (q_out, a, b, kc, vc)))
