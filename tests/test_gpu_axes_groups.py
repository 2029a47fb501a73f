"""GPU tests of the rotation with several axes and of the append by a slot map where workgroups take several
tokens, and of as many tokens as launches of one token a workgroup do not reach."""
import pytest
import torch

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


def ids(axes, T, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    p = torch.randint(0, 5000, (axes, T), generator=g, device=DEV, dtype=torch.int32)
    p[torch.randint(0, 40, (axes, T), generator=g, device=DEV) == 0] = -1
    return p


def same(a, b):
    view = torch.int32 if a.dtype == F32 else torch.int16
    return torch.equal(a.contiguous().view(view), b.contiguous().view(view))


CASES = [  # T, Hq, Hkv, D, sections, layout, dtype, misaligned
    (2049, 2, 1, 8, (2, 1, 1), "sections", BF16, False),
    (5003, 3, 1, 24, (4, 4, 4), "interleaved", F16, False),  # chunks of 8 bytes
    (5003, 2, 2, 10, (3, 2), "separate", F32, True),         # of one value
    (16387, 1, 1, 16, (8,), "sections", BF16, False),        # 16 tokens a workgroup, and 3 in the last
    (16400, 1, 1, 6, (1, 2), "separate", BF16, True),
    (40001, 1, 1, 256, (48, 40, 40), "interleaved", F32, False),
]


def case_id(c):
    return f"T{c[0]}_{c[1]}_{c[2]}_{c[3]}_{c[5]}_{str(c[6])[6:]}"


def rows(T, H, D, seed, dtype, misaligned):
    """[T, H, D], with `misaligned` one value past an aligned address and with odd strides."""
    if not misaligned:
        return normal((T, H, D), seed, dtype)
    return normal((T, H * D + 3), seed, dtype)[:, 1:1 + H * D].unflatten(1, (H, D))


def one_by_one(rope, q, k, pos, *args):
    """The rotation of calls that are too small for several tokens a workgroup."""
    parts = [rope.qk_apply_axes(q[a:a + 1000], k[a:a + 1000], pos[:, a:a + 1000], *args) for a in range(0, len(q), 1000)]
    return tuple(torch.cat(x) for x in zip(*parts))


@pytest.mark.parametrize("case", CASES, ids=case_id)
def test_rotation_of_many_tokens_is_that_of_few(rope, case):
    """Bit for bit, either way round, out of place and in place."""
    T, Hq, Hkv, D, sections, layout, dtype, misaligned = case
    print(f"[qk_apply_axes] {case}", flush=True)
    q, k = rows(T, Hq, D, 1, dtype, misaligned), rows(T, Hkv, D, 2, dtype, misaligned)
    pos = ids(len(sections), T, 3)
    for direction in (1, -1):
        want = one_by_one(rope, q, k, pos, sections, 1e5, direction, layout, 2.0)
        got = rope.qk_apply_axes(q, k, pos, sections, 1e5, direction, layout, 2.0)
        assert same(got[0], want[0]) and same(got[1], want[1])
        off = (pos < 0).any(0)
        assert bool(off.any()) and same(got[0][off], q[off])
    want = one_by_one(rope, q, k, pos, sections, 1e5)
    rope.qk_apply_axes(q, k, pos, sections, 1e5, q_out=q, k_out=k)
    assert same(q, want[0]) and same(k, want[1])


@pytest.mark.parametrize("case", CASES, ids=case_id)
def test_append_of_many_tokens(rope, case):
    """The cache rows of the slot map are those of the rotation, bit for bit, in groups in which some tokens have
    no slot and some no position; the rest of the cache is left as it was."""
    T, Hq, Hkv, D, sections, layout, dtype, misaligned = case
    print(f"[kv_append_slots] {case}", flush=True)
    page = 24
    pages = -(-T // page) + 3
    g = torch.Generator(device=DEV).manual_seed(4)
    shape = (pages, page, Hkv, D + misaligned)
    kc, vc = (torch.full(shape, float("nan"), dtype=dtype, device=DEV)[..., :D] for _ in range(2))
    slots = torch.randperm(pages * page, generator=g, device=DEV)[:T]
    gone = torch.randint(0, 30, (T,), generator=g, device=DEV)
    slots = torch.where(gone == 0, -1, torch.where(gone == 1, pages * page, slots))
    q, k, v = (rows(T, h, D, i, dtype, misaligned) for i, h in enumerate((Hq, Hkv, Hkv)))
    pos = ids(len(sections), T, 3)
    want_q, want_k = one_by_one(rope, q, k, pos, sections, 1e5, 1, layout)
    want = [c.clone() for c in (kc, vc)]
    on = (slots >= 0) & (slots < pages * page)
    assert 0 < int(on.sum()) < T
    where = slots[on] // page, slots[on] % page
    want[0][where], want[1][where] = want_k[on], v[on]
    got = rope.kv_append_slots_(k, v, kc, vc, slots, pos, 1e5, sections, layout, q=q)
    assert same(got, want_q) and same(kc, want[0]) and same(vc, want[1])


def test_more_tokens_than_workgroups_of_a_launch(rope):
    """33554437 tokens of 257 heads of 2, in place (34 GB): a workgroup, which has work enough with one token,
    takes two. Every token is the first turned to its own position, one of 97."""
    T, H, D, P = 33554437, 257, 2, 97
    if torch.cuda.mem_get_info()[0] < 48 << 30:
        pytest.skip("no room")
    row = normal((1, H, D), 1, BF16)
    q = row.expand(T, H, D).contiguous()
    k = q.new_empty((T, 0, D))
    pos = (torch.arange(T, device=DEV) % P).int()
    want = rope.qk_apply_axes(row.expand(P, H, D).contiguous(), k[:P], pos[:P], (1,), 1e4)[0]
    rope.qk_apply_axes(q, k, pos, (1,), 1e4, q_out=q)
    torch.cuda.synchronize()
    step = P * 10000
    whole = want.repeat(10000, 1, 1)
    for a in range(0, T, step):
        part = q[a:a + step]
        assert same(part, whole[:len(part)]), a
