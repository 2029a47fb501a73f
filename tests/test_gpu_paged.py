"""GPU tests of the paged cache: kv_append_ against the rotary kernels and a plain write,
attn_paged against attention in 64 bits (attn_reference). Cache rows that no sequence holds
are NaN throughout, so that a row read by mistake shows."""
import pytest
import torch

import attn_reference as ref

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def rope():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import packed_varlen_rotary_rope_amd as m
    return m


def normal(shape, seed, dtype):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randn(shape, generator=g, device=DEV).to(dtype)


def int32(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def pool(lens, page, Hkv, D, dtype, seed, by_head=False):
    """(k_cache, v_cache, table): pages in a shuffled order, NaN where no sequence is."""
    g = torch.Generator().manual_seed(seed)
    per = max([1] + [-(-max(m, 0) // page) for m in lens])
    used = [-(-max(m, 0) // page) for m in lens]
    pages = sum(used) + 2
    order = torch.randperm(pages, generator=g)
    table = torch.full((len(lens), per), -7, dtype=torch.int32)
    caches = []
    for i in range(2):
        shape = (pages, Hkv, page, D) if by_head else (pages, page, Hkv, D)
        c = torch.full(shape, float("nan"), dtype=dtype, device=DEV)
        caches.append(c.transpose(1, 2) if by_head else c)
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


# new tokens, held tokens, Hq, Hkv, D, page, dtype
STEPS = [
    ([1], [1], 1, 1, 8, 1, BF16),
    ([1], [300], 32, 8, 128, 16, BF16),
    ([1, 1, 1, 1], [5, 4099, 64, 1000], 8, 2, 128, 16, BF16),
    ([1, 1], [2000, 33], 8, 8, 64, 7, F16),
    ([1] * 70, [1 + 13 * i for i in range(70)], 4, 1, 64, 32, BF16),
    ([4, 3, 1], [513, 64, 90], 16, 2, 80, 48, F16),
    ([100, 200], [100, 1700], 8, 2, 128, 64, BF16),
    ([257, 1, 31, 1], [3001, 500, 31, 8], 12, 4, 96, 24, BF16),
    ([0, 2, 0], [40, 50, 0], 6, 3, 72, 5, F16),
    ([33], [33], 2, 1, 40, 256, BF16),
    ([1, 40], [700, 777], 4, 2, 256, 16, BF16),
    ([1, 1], [150, 1030], 4, 4, 192, 16, F16),
    ([5], [3], 4, 2, 64, 16, BF16),   # fewer held than new: the first two see no key
    ([700], [5000], 5, 1, 112, 16, BF16),
    ([16], [9000], 160, 2, 128, 64, BF16),
]


@pytest.mark.parametrize("case", STEPS, ids=lambda c: f"n{sum(c[0])}_m{max(c[1])}_{c[2]}_{c[3]}_{c[4]}_{c[5]}_{str(c[6])[6:]}")
@pytest.mark.parametrize("by_head", [False, True])
def test_paged(rope, case, by_head):
    new, held, Hq, Hkv, D, page, dtype = case
    print(f"[attn_paged] {str(case)[:150]} by_head={by_head}", flush=True)
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    T = cu[-1]
    k, v, table = pool(held, page, Hkv, D, dtype, 5, by_head)
    q = normal((T, Hq, D), 3, dtype)
    plan = rope.paged_plan(int32(cu), int32(held), T, Hq, Hkv)
    out, lse = rope.attn_paged(q, k, v, table, plan)
    scale = D ** -0.5
    want, wlse, tol = ref.paged(q, k, v, table, cu, held, scale)
    ref.check(out, want, tol, "out")
    worst = float(q.double().norm(dim=-1).max()) * float(torch.nan_to_num(k.double()).norm(dim=-1).max()) * scale
    ref.check_lse(lse, wlse, D, worst)


APPENDS = [  # new, held, Hq, Hkv, D, page, dtype
    ([1], [1], 1, 1, 2, 1, F32),
    ([1, 1, 1], [7, 100, 4000], 32, 8, 128, 16, BF16),
    ([5, 0, 130], [5, 3, 900], 6, 2, 80, 48, F16),
    ([64], [64], 4, 4, 64, 64, F32),
    ([300, 9], [1000, 20], 16, 2, 96, 7, BF16),
    ([33], [77], 3, 1, 50, 16, BF16),
    ([12], [40], 2, 1, 512, 16, F16),
]


@pytest.mark.parametrize("case", APPENDS, ids=lambda c: f"n{sum(c[0])}_{c[2]}_{c[3]}_{c[4]}_{c[5]}_{str(c[6])[6:]}")
@pytest.mark.parametrize("form", ["fused", "by_head", "keys_only", "in_place"])
def test_append(rope, case, form):
    """The cache rows are those of the rotary kernel at the same positions, bit for bit, the
    rest of the cache is untouched, and so is the rotated q."""
    new, held, Hq, Hkv, D, page, dtype = case
    print(f"[kv_append] {case} {form}", flush=True)
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    T = cu[-1]
    kc, vc, table = pool(held, page, Hkv, D, dtype, 9, by_head=form == "by_head")
    if form == "fused":
        qkv = normal((T, Hq + 2 * Hkv, D), 1, dtype)
        q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    else:
        q, k, v = (normal((T, h, D), i, dtype) for i, h in enumerate((Hq, Hkv, Hkv)))
    pos = torch.cat([torch.arange(m - n, m) for n, m in zip(new, held)])
    seq = torch.cat([torch.full((n,), s) for s, n in enumerate(new)]).to(DEV)
    want_q, want_k = q.contiguous().clone(), k.contiguous().clone()
    rope.qk_apply_ex_(want_q, want_k, 1e6, 1, position_ids=pos.int().to(DEV), pos_scale=2.0)
    want_kc, want_vc = kc.clone(), vc.clone()
    where = table.long()[seq, pos.to(DEV) // page], pos.to(DEV) % page
    want_kc[where], want_vc[where] = want_k, v
    kw = {} if form == "keys_only" else dict(q=q, q_out=q) if form == "in_place" else dict(q=q)
    got = rope.kv_append_(k, v, kc, vc, table, int32(cu), int32(held), 1e6, pos_scale=2.0, **kw)
    view = torch.int32 if dtype == F32 else torch.int16

    def same(a, b):
        return torch.equal(a.contiguous().view(view), b.contiguous().view(view))

    assert same(kc, want_kc) and same(vc, want_vc)
    assert got is None if form == "keys_only" else same(got, want_q)


def bits(t):
    return t.contiguous().view(torch.int32 if t.dtype == F32 else torch.int16)


def same(a, b):
    return torch.equal(bits(a), bits(b))


@pytest.mark.parametrize("new,held", [([1, 1], [500, 77]), ([300, 1], [500, 77]), ([40], [120])])
def test_pages_that_are_none(rope, new, held):
    """Page numbers out of range anywhere in a sequence, and tables shorter than what a sequence
    holds: those keys are seen by nobody, the others as ever."""
    print(f"[pages] {new} {held}", flush=True)
    Hq, Hkv, D, page = 8, 2, 64, 16
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    k, v, table = pool(held, page, Hkv, D, BF16, 4)
    table[0, 1], table[0, 3], table[-1, 2] = -1, k.shape[0], 2 ** 31 - 1
    q = normal((cu[-1], Hq, D), 3, BF16)
    plan = rope.paged_plan(int32(cu), int32(held), cu[-1], Hq, Hkv)
    for t in (table, table[:, :4], table[:, :1], table[:, :0]):
        out, lse = rope.attn_paged(q, k, v, t, plan)
        want, wlse, tol = ref.paged(q, k, v, t, cu, held, D ** -0.5)
        ref.check(out, want, tol, f"out, {t.shape[1]} pages")
        assert torch.equal(lse == float("-inf"), wlse == float("-inf"))


def test_tokens_that_are_not_appended(rope):
    """No page, behind the table, negative positions, rows of no sequence: the cache keeps its
    bits there, q is rotated where it has a position and copied where it has none."""
    Hq, Hkv, D, page = 4, 2, 64, 16
    kc, vc = normal((6, page, Hkv, D), 1, BF16), normal((6, page, Hkv, D), 2, BF16)
    table = int32([[0, -1, 2], [3, 6, 4]])
    cu, lens, T = [2, 42, 60], [40, 50], 64     # rows 0, 1 and 60 .. 63 belong to nobody
    q, k, v = normal((T, Hq, D), 3, BF16), normal((T, Hkv, D), 4, BF16), normal((T, Hkv, D), 5, BF16)
    want_kc, want_vc, want_q, turned = kc.clone(), vc.clone(), q.clone(), k.clone()
    pos = torch.full((T,), -1, dtype=torch.int32)
    pos[2:42], pos[42:60] = torch.arange(40), torch.arange(32, 50)
    rope.qk_apply_ex_(want_q, turned, 1e4, 1, position_ids=pos.to(DEV))
    for t in range(T):
        p, s = int(pos[t]), 0 if t < 42 else 1
        if p >= 0 and p // page < 3 and 0 <= int(table[s, p // page]) < 6:
            want_kc[int(table[s, p // page]), p % page] = turned[t]
            want_vc[int(table[s, p // page]), p % page] = v[t]
    got = rope.kv_append_(k, v, kc, vc, table, int32(cu), int32(lens), 1e4, q=q)
    assert same(kc, want_kc) and same(vc, want_vc) and same(got, want_q)
    # more new tokens than held ones: the first of them have no position

    got = rope.kv_append_(k, v, kc, vc, table[:1], int32([0, 10]), int32([4]), 1e4, q=q)
    assert same(got[:6], q[:6]) and same(got[10:], q[10:]) and not same(got[8:10], q[8:10])
    assert same(kc[3:], want_kc[3:])
    # no sequence at all
    got = rope.kv_append_(k, v, kc, vc, table[:0], int32([0]), int32([]), 1e4, q=q)
    assert same(got, q)


def test_refusals(rope):
    kc, vc = normal((4, 16, 2, 64), 1, BF16), normal((4, 16, 2, 64), 2, BF16)
    q, k, v = normal((3, 4, 64), 3, BF16), normal((3, 2, 64), 4, BF16), normal((3, 2, 64), 5, BF16)
    table, cu, lens = int32([[0, 1]]), int32([0, 3]), int32([9])

    def append(**kw):
        a = dict(k=k, v=v, k_cache=kc, v_cache=vc, block_table=table, cu_seqlens=cu, kv_lens=lens, theta=1e4)
        a.update(kw)
        return rope.kv_append_(**a)

    for kw in (dict(k=k.half()), dict(v=v.cpu()), dict(k_cache=kc.half()), dict(kv_lens=lens.long()),
               dict(q=q.half()), dict(block_table=table.long())):
        with pytest.raises(TypeError):
            append(**kw)
    for kw in (dict(v=v[:2]), dict(k_cache=kc[:3]), dict(v_cache=vc.transpose(1, 2)), dict(kv_lens=int32([1, 2])),
               dict(q=q[:2]), dict(q_out=q), dict(block_table=int32([[0], [1]])), dict(k=k[:, :1], v=v[:, :1]),
               dict(q=q[:, :, ::2], q_out=None)):
        with pytest.raises(ValueError):
            append(**kw)
    for kw in (dict(theta=0.1), dict(pos_scale=0.5)):
        with pytest.raises(rope.RopeError):
            append(**kw)
    plan = rope.paged_plan(cu, lens, 3, 4, 2)
    with pytest.raises(TypeError):
        rope.attn_paged(q.float(), kc.float(), vc.float(), table, plan)
    for a in ((q[:2], kc, vc, table, plan), (q[:, :2], kc, vc, table, plan), (q, kc, vc[:3], table, plan),
              (q, kc[:, :, :1], vc[:, :, :1], table, plan), (q, kc, vc, int32([[0], [1]]), plan),
              (q, kc[..., :60], vc[..., :60], table, plan)):
        with pytest.raises(ValueError):
            rope.attn_paged(*a)
    with pytest.raises(ValueError):
        rope.paged_plan(cu, lens, 3, 4, 3)
    with pytest.raises(ValueError):
        rope.paged_plan(cu, lens, 4, 4, 2, out=plan)


def test_plan_of_another_batch_writes_nothing(rope):
    kc = normal((4, 16, 2, 64), 1, BF16)
    q = normal((3, 4, 64), 3, BF16)
    other = rope.paged_plan(int32([0, 5]), int32([9]), 5, 4, 2)
    fake = rope.PagedPlan(3, 1, 4, 2, other.buffer)
    out, lse = torch.full_like(q, 3.0), torch.full((3, 4), 3.0, device=DEV)
    rope.attn_paged(q, kc, kc, int32([[0, 1]]), fake, out=out, lse=lse)
    assert bool((out == 3).all()) and bool((lse == 3).all())


def test_rows_of_no_sequence(rope):
    held = [30, 700]
    k, v, table = pool(held, 16, 2, 64, BF16, 2)
    q = normal((400, 4, 64), 3, BF16)
    q[:3] = q[250:] = float("nan")
    plan = rope.paged_plan(int32([3, 4, 250]), int32(held), 400, 4, 2)
    out, lse = rope.attn_paged(q, k, v, table, plan)
    want, wlse, tol = ref.paged(torch.nan_to_num(q), k, v, table, [3, 4, 250], held, 0.125)
    ref.check(out, want, tol, "out")
    keep = torch.full_like(q, 5.0), torch.full((400, 4), 5.0, device=DEV)
    rope.attn_paged(q, k, v, table, plan, out=keep[0], lse=keep[1])
    assert same(keep[0][3:250], out[3:250]) and bool((keep[0][250:] == 5).all()) and bool((keep[1][:3] == 5).all())


@pytest.mark.parametrize("D,page,chunks", [(128, 16, [150, 1, 1, 64, 1, 33, 1]), (80, 7, [1, 1, 300, 2, 5]),
                                           (64, 64, [257, 31, 1])])
def test_serving_a_sequence(rope, D, page, chunks):
    """A prompt in chunks and single tokens, through append and paged attention with one plan
    buffer: every step's output against the packed attention's definition over the whole
    sequence, rotated once by the packed rotation."""
    print(f"[serving] D={D} page={page} {chunks}", flush=True)
    Hq, Hkv, T = 8, 2, sum(chunks)
    q, k, v = normal((T, Hq, D), 1, BF16), normal((T, Hkv, D), 2, BF16), normal((T, Hkv, D), 3, BF16)
    rq, rk = q.clone(), k.clone()
    rope.qk_fwd_(rq, rk, int32([0, T]), 1e5)
    want, _, tol = ref.forward(rq, rk, v, [(0, T)], D ** -0.5)
    pages = -(-T // page)
    g = torch.Generator().manual_seed(1)
    table = torch.randperm(pages + 4, generator=g)[:pages].int()[None].to(DEV)
    kc = torch.full((pages + 4, page, Hkv, D), float("nan"), dtype=BF16, device=DEV)
    vc = kc.clone()
    at = 0
    for n in chunks:
        cu, lens = int32([0, n]), int32([at + n])
        tq = rope.kv_append_(k[at:at + n], v[at:at + n], kc, vc, table, cu, lens, 1e5, q=q[at:at + n])
        assert same(tq, rq[at:at + n])
        out, _ = rope.attn_paged(tq, kc, vc, table, rope.paged_plan(cu, lens, n, Hq, Hkv))
        ref.check(out, want[at:at + n], tol[at:at + n], f"tokens {at} .. {at + n}")
        at += n


def test_captured_decode_step(rope):
    """Append, plan and attention of one step in a HIP graph, replayed with growing lengths."""
    B, Hq, Hkv, D, page = 5, 8, 2, 128, 16
    lens0 = [1, 15, 16, 700, 2047]
    kc, vc, _ = pool([m + 8 for m in lens0], page, Hkv, D, BF16, 6)
    _, _, table = pool([m + 8 for m in lens0], page, Hkv, D, BF16, 6)
    q, k, v = normal((B, Hq, D), 1, BF16), normal((B, Hkv, D), 2, BF16), normal((B, Hkv, D), 3, BF16)
    cu, lens = int32(list(range(B + 1))), int32(lens0)
    plan = rope.paged_plan(cu, lens, B, Hq, Hkv)

    def step(caches, plan):
        tq = rope.kv_append_(k, v, *caches, table, cu, lens, 1e4, q=q)
        rope.paged_plan(cu, lens, B, Hq, Hkv, out=plan)
        return rope.attn_paged(tq, *caches, table, plan)

    step((kc.clone(), vc.clone()), plan)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = step((kc, vc), plan)
    for i in range(4):
        lens.copy_(int32([m + i for m in lens0]))
        q.copy_(normal((B, Hq, D), 50 + i, BF16))
        k.copy_(normal((B, Hkv, D), 60 + i, BF16))
        eager = kc.clone(), vc.clone()
        graph.replay()
        want = step(eager, rope.paged_plan(cu, lens, B, Hq, Hkv))
        torch.cuda.synchronize()
        assert same(out, want[0]) and same(lse, want[1]) and same(kc, eager[0]) and same(vc, eager[1])


def test_repeatable_and_concurrent(rope):
    """The same bits every time, with one plan in use on two streams at once."""
    held, new = [3000, 40, 900, 1], [1, 40, 200, 1]
    cu = [0, 1, 41, 241, 242]
    k, v, table = pool(held, 32, 2, 64, BF16, 8)
    q = normal((242, 8, 64), 1, BF16)
    assert len(new) == 4
    plan = rope.paged_plan(int32(cu), int32(held), 242, 8, 2)
    want = rope.attn_paged(q, k, v, table, plan)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(4):
        got = []
        for st in streams:
            with torch.cuda.stream(st):
                got += rope.attn_paged(q, k, v, table, plan)
        # another plan of the same step has its items and slots in another order
        got += rope.attn_paged(q, k, v, table, rope.paged_plan(int32(cu), int32(held), 242, 8, 2))
        torch.cuda.synchronize()
        assert all(same(a, b) for a, b in zip(got, want * 3))


def test_offsets_beyond_32_bits(rope):
    """A cache of more than 2^31 elements: pages from its far end, written by the append and read
    by the attention."""
    print("[64-bit offsets]", flush=True)
    pages, page, Hkv, D, Hq = 140000, 16, 8, 128, 32
    kc = torch.zeros((pages, page, Hkv, D), dtype=BF16, device=DEV)
    vc = torch.zeros_like(kc)
    n = 50
    table = int32([[pages - 1, 7, pages - 3, 131072], [pages - 2, 1, 131073, 2]])
    q, k, v = normal((2 * n, Hq, D), 1, BF16), normal((2 * n, Hkv, D), 2, BF16), normal((2 * n, Hkv, D), 3, BF16)
    cu, lens = int32([0, n, 2 * n]), int32([n, n])
    tq = rope.kv_append_(k, v, kc, vc, table, cu, lens, 1e4, q=q)
    rq, rk = q.clone(), k.clone()
    rope.qk_fwd_(rq, rk, cu, 1e4)
    assert same(tq, rq)
    at = torch.arange(n, device=DEV)
    for s in range(2):
        where = table[s].long()[at // page], at % page
        assert same(kc[where], rk[s * n:(s + 1) * n]) and same(vc[where], v[s * n:(s + 1) * n])
    out, _ = rope.attn_paged(tq, kc, vc, table, rope.paged_plan(cu, lens, 2 * n, Hq, Hkv))
    want, _, tol = ref.forward(rq, rk, v, [(0, n), (n, n)], D ** -0.5)
    ref.check(out, want, tol, "out")
    # decode, and a stride that a combined cache of keys and values has
    both = torch.zeros((64, 2, page, Hkv, D), dtype=BF16, device=DEV)
    t2 = int32([[63, 0, 30, 1]])
    rope.kv_append_(k[:n], v[:n], both[:, 0], both[:, 1], t2, int32([0, n]), int32([n]), 1e4)
    out1, _ = rope.attn_paged(rq[n - 1:n], both[:, 0], both[:, 1], t2,
                              rope.paged_plan(int32([0, 1]), int32([n]), 1, Hq, Hkv))
    ref.check(out1, want[n - 1:n], tol[n - 1:n], "one token")


def test_tokens_that_overlap_are_refused(rope):
    """An expanded tensor has token stride 0, which the C ABI reads as dense rows."""
    kc, vc = normal((4, 16, 2, 64), 1, BF16), normal((4, 16, 2, 64), 2, BF16)
    q, k, v = normal((3, 4, 64), 3, BF16), normal((3, 2, 64), 4, BF16), normal((3, 2, 64), 5, BF16)
    table, cu, lens = int32([[0, 1]]), int32([0, 3]), int32([9])
    wide = [x[:1].expand_as(x) for x in (q, k, v)]
    for a in ((wide[0], k, v), (q, wide[1], v), (q, k, wide[2])):
        with pytest.raises(ValueError, match="overlap"):
            rope.kv_append_(a[1], a[2], kc, vc, table, cu, lens, 1e4, q=a[0])
    with pytest.raises(ValueError, match="overlap"):
        rope.kv_append_(k, v, kc, vc, table, cu, lens, 1e4, q=q, q_out=wide[0])
    for of in (lambda c: c[:1].expand_as(c), lambda c: c[:, :1].expand_as(c), lambda c: c[:, :, :1].expand_as(c),
               lambda c: torch.as_strided(c, (4, 16, 2, 64), (1024, 128, 64, 1))):
        with pytest.raises(ValueError, match="overlap"):
            rope.kv_append_(k, v, of(kc), of(vc), table, cu, lens, 1e4)
    with pytest.raises(ValueError, match="overlap"):
        rope.attn_paged(wide[0], kc, vc, table, rope.paged_plan(cu, lens, 3, 4, 2))


def test_no_tokens_and_no_sequences(rope):
    kc, vc = normal((4, 16, 2, 64), 1, BF16), normal((4, 16, 2, 64), 2, BF16)
    old = kc.clone()
    for B, T in ((0, 0), (2, 0), (0, 130)):
        q, k, v = normal((T, 4, 64), 3, BF16), normal((T, 2, 64), 4, BF16), normal((T, 2, 64), 5, BF16)
        cu, lens, table = int32([0] * (B + 1)), int32([7] * B), torch.zeros((B, 3), dtype=torch.int32, device=DEV)
        assert same(rope.kv_append_(k, v, kc, vc, table, cu, lens, 1e4, q=q), q)
        out, lse = rope.attn_paged(q, kc, vc, table, rope.paged_plan(cu, lens, T, 4, 2))
        assert out.shape == q.shape and bool((out == 0).all()) and bool((lse == float("-inf")).all())
    none = torch.zeros((1, 0), dtype=torch.int32, device=DEV)  # a table without pages
    q, k, v = normal((3, 4, 64), 3, BF16), normal((3, 2, 64), 4, BF16), normal((3, 2, 64), 5, BF16)
    rope.kv_append_(k, v, kc, vc, none, int32([0, 3]), int32([3]), 1e4)
    out, lse = rope.attn_paged(q, kc, vc, none, rope.paged_plan(int32([0, 3]), int32([3]), 3, 4, 2))
    assert bool((out == 0).all()) and bool((lse == float("-inf")).all()) and same(kc, old)


@pytest.mark.parametrize("D,Hq,new", [(64, 4, 8), (128, 8, 100), (80, 2, 40), (192, 4, 90), (256, 2, 12)])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
def test_hidden_new_tokens_have_no_influence(rope, D, Hq, new, value):
    """A new token whose key or value is not finite changes no query before it and no other
    sequence."""
    print(f"[hidden] D={D} Hq={Hq} new={new} {value}", flush=True)
    held, page, cu = [new + 333, 77], 16, [0, new, new + 1]
    k, v, table = pool(held, page, 2, D, BF16, D)
    q = normal((new + 1, Hq, D), 3, BF16)
    plan = rope.paged_plan(int32(cu), int32(held), new + 1, Hq, 2)
    out0, lse0 = rope.attn_paged(q, k, v, table, plan)
    bad = new // 2
    pos = held[0] - new + bad
    for c in (k, v):
        c[table[0, pos // page].item(), pos % page, 1, 5] = value
    out, lse = rope.attn_paged(q, k, v, table, plan)
    keep = [i for i in range(new + 1) if i < bad or i == new]
    assert same(out[keep], out0[keep]) and same(lse[keep], lse0[keep])
    assert same(out[:, :Hq // 2], out0[:, :Hq // 2])
    assert bool(out0[:new].isfinite().all())


@pytest.mark.parametrize("D,new", [(64, 1), (128, 1), (128, 100), (192, 9), (256, 90)])
@pytest.mark.parametrize("dtype,a,b", [(BF16, 20, 12), (BF16, 40, 40), (F16, 10, 4), (F16, 15, 7)])
@pytest.mark.parametrize("sign", [1, -1])
def test_very_large_scores(rope, D, new, dtype, a, b, sign):
    """As test_gpu_attn's: every score is sign * n 2^(a+b) D^0.5, n distinct, one key takes all;
    of 6 splits or waves each but one has weight 0."""
    print(f"[large] D={D} new={new} {dtype} {a} {b} {sign}", flush=True)
    held, page = 256, 16
    n = (torch.randperm(held, generator=torch.Generator().manual_seed(D + a)) + 1).to(DEV)
    k = (sign * n[:, None, None] * 2.0 ** b).expand(held, 2, D).to(dtype).contiguous()
    v = normal((held, 2, D), 5, dtype)
    q = torch.full((new, 4, D), 2.0 ** a, device=DEV).to(dtype)
    table = torch.arange(16, dtype=torch.int32, device=DEV)[None]
    plan = rope.paged_plan(int32([0, new]), int32([held]), new, 4, 2)
    out, lse = rope.attn_paged(q, k.view(16, page, 2, D), v.view(16, page, 2, D), table, plan)
    m = torch.cummax(sign * n, 0)
    want = v[m.indices[held - new:]].repeat_interleave(2, 1).double()
    ref.check(out, want, want.abs() * 2.1 * ref.half_step(dtype), "out")
    score = (m.values[held - new:].double() * 2.0 ** (a + b) * D ** 0.5)[:, None].expand(-1, 4)
    ref.check(lse, score, score.abs() * 2.0 ** -21, "lse")


@pytest.mark.parametrize("D,new", [(64, 1), (128, 1), (128, 8), (128, 100), (192, 9), (256, 90)])
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("held", [400, 4000])
def test_very_large_scores_before_ordinary_ones(rope, D, new, dtype, held):
    """As test_gpu_attn's: the first 64 keys' scores are below -2^28, the others 0; the new tokens
    weigh the others alike."""
    print(f"[large first] D={D} new={new} {dtype} {held}", flush=True)
    a = 5736.0 if dtype == F16 else 17536.0
    page = 16
    q = torch.full((new, 4, D), a, dtype=dtype, device=DEV)
    k = torch.zeros((held, 2, D), dtype=dtype, device=DEV)
    k[:64] = -a
    v = normal((held, 2, D), 6, dtype)
    table = torch.arange(held // page, dtype=torch.int32, device=DEV)[None]
    plan = rope.paged_plan(int32([0, new]), int32([held]), new, 4, 2)
    out, lse = rope.attn_paged(q, k.view(-1, page, 2, D), v.view(-1, page, 2, D), table, plan)
    v64 = v.repeat_interleave(2, 1).double()[64:]
    n = torch.arange(1, held - 63, device=DEV, dtype=torch.float64)[:, None, None]
    mean, spread = (v64.cumsum(0) / n)[-new:], (v64.abs().cumsum(0) / n)[-new:]
    ref.check(out, mean, 1.01 * (ref.half_step(dtype) * mean.abs() + held * 2.0 ** -23 * spread) + ref.tiny(dtype),
              "out")
    want = n[-new:, :, 0].log().expand(-1, 4)
    ref.check(lse, want, (want + 1) * 2.0 ** -21, "lse")


@pytest.mark.parametrize("D,new", [(64, 1), (128, 8), (256, 3), (64, 300), (256, 200)])
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("c", [83, 101, 127])
def test_very_large_scores_close_together(rope, D, new, dtype, c):
    """One key's score is one step of fp32 above all the others', which are about 2^29: they weigh
    exp(-8) each (D 128: exp(-5.7)), whichever waves and splits they fall in, though scale * s is
    known to half a step of 8 to 16 there. Scores are exact; a weight errs by its rounding and
    2^-18 (an exponent of about 12 in fp32, twice), sums of n terms by n 2^-23 of their spread."""
    print(f"[close] D={D} new={new} {dtype} {c}", flush=True)
    held, page, high = 4000, 16, 1234
    parts = 2 if D == 256 else 1  # the score is c 2^23 for each of these columns
    step = 64.0 * parts
    q, k = torch.zeros((new, 4, D), device=DEV), torch.zeros((held, 2, D), device=DEV)
    q[..., :parts], k[..., :parts] = c * 2.0 ** 8, 2.0 ** 15
    q[..., 40], k[high, :, 40] = 1.0, step
    q, k, v = q.to(dtype), k.to(dtype), normal((held, 2, D), 6, dtype)
    table = torch.arange(held // page, dtype=torch.int32, device=DEV)[None]
    plan = rope.paged_plan(int32([0, new]), int32([held]), new, 4, 2)
    out, lse = rope.attn_paged(q, k.view(-1, page, 2, D), v.view(-1, page, 2, D), table, plan)
    t = torch.arange(held, device=DEV)
    p = torch.full((new, held), -step * D ** -0.5, dtype=torch.float64, device=DEV).exp()
    p[:, high] = 1.0
    p = p.masked_fill(t[None] > held - new + torch.arange(new, device=DEV)[:, None], 0.0)
    p = p / p.sum(-1, keepdim=True)
    u = ref.half_step(dtype)
    for h in range(4):
        want, spread = p @ v[:, h // 2].double(), p @ v[:, h // 2].double().abs()
        ref.check(out[:, h], want, 1.01 * (u * (want.abs() + spread) + (held * 2.0 ** -23 + 2.0 ** -18) * spread) +
                  ref.tiny(dtype), f"out of head {h}")
    score = torch.full((new, 4), c * 2.0 ** 23 * parts * D ** -0.5, dtype=torch.float64, device=DEV)
    ref.check(lse, score, score * 2.0 ** -21, "lse")


def test_sequences_that_leave_the_rows(rope):
    """cu_seqlens with entries outside of the T rows: append and plan both count the rows that are
    there as the last of the held tokens."""
    Hq, Hkv, D, page, T = 4, 2, 64, 16, 8
    q, k, v = normal((T, Hq, D), 3, BF16), normal((T, Hkv, D), 4, BF16), normal((T, Hkv, D), 5, BF16)
    table, lens = int32([[0, 1], [2, 3], [4, 5]]), int32([20, 9, 30])
    got = []
    for cu in ([0, 5, 12, 40], [0, 5, T, T], [-3, 5, 2 ** 31 - 1, 2 ** 31 - 1]):
        print(f"[cu_seqlens] {cu}", flush=True)
        kc, vc = normal((6, page, Hkv, D), 1, BF16), normal((6, page, Hkv, D), 2, BF16)
        tq = rope.kv_append_(k, v, kc, vc, table, int32(cu), lens, 1e4, q=q)
        out, lse = rope.attn_paged(tq, kc, vc, table, rope.paged_plan(int32(cu), lens, T, Hq, Hkv))
        got.append((kc, vc, tq, out, lse))
    assert same(got[0][0][2, 6:9], got[1][0][2, 6:9])  # the second sequence's rows at positions 6 .. 8
    for other in (got[0], got[2]):
        assert all(same(a, b) for a, b in zip(other, got[1]))


@pytest.mark.parametrize("seed", range(4))
@pytest.mark.parametrize("D,Hq,Hkv", [(32, 4, 1), (64, 4, 2), (128, 2, 2), (192, 3, 1), (256, 2, 2)])
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("new,held", [([1, 1, 3], [700, 33, 2500]), ([60, 1, 200], [300, 9, 1111])])
def test_scores_of_all_sizes(rope, seed, D, Hq, Hkv, dtype, new, held):
    """As test_gpu_attn's, over a cache with NaN behind the sequences and a page that is none: parts
    of a row with ordinary and with very large maxima are joined."""
    from test_gpu_attn import exact_scores_bound, head_of_any_scores, mixed_scores
    print(f"[all sizes] {seed} D={D} {Hq}+{Hkv} {dtype} {new}", flush=True)
    page, cu = 16, [0]
    for n in new:
        cu.append(cu[-1] + n)
    k, v, table = pool(held, page, Hkv, D, dtype, 40 + seed)
    q, _ = mixed_scores(cu[-1], 1, (Hq, Hkv), D, dtype, 2 * seed)
    for s, m in enumerate(held):
        at = torch.arange(m, device=DEV)
        k[table[s].long()[at // page], at % page] = mixed_scores(1, m, (Hq, Hkv), D, dtype, 100 * seed + s)[1]
    table[2, 5] = -1
    plan = rope.paged_plan(int32(cu), int32(held), cu[-1], Hq, Hkv)
    out, lse = rope.attn_paged(q, k, v, table, plan)
    for s, (n, m) in enumerate(zip(new, held)):
        rows, at = slice(cu[s], cu[s + 1]), torch.arange(m, device=DEV)
        number = table[s].long()[at // page]
        gone = number < 0
        where = number.clamp_min(0), at % page
        for h in range(Hq):
            kh, vh = k[where][:, h // (Hq // Hkv)], v[where][:, h // (Hq // Hkv)].double()
            vh = vh.masked_fill(gone[:, None], 0.0)
            o, l, p = head_of_any_scores(q[rows, h], kh, vh, D ** -0.5, m - n, gone)
            ref.check(out[rows, h], o, exact_scores_bound(o, p, vh, dtype, m), "out")
            ref.check(lse[rows, h], l, (l.abs() + 8) * 2.0 ** -21, "lse")
