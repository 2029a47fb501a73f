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
