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
