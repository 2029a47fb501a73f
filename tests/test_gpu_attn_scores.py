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
