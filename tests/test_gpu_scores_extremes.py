"""GPU tests of the attention with changed scores at their extremes: every part of the tanh, caps and biases
that make very large scores, gradients past the storage type."""
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


@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_tanh_of_every_half_precision_score(rope, sign):
    """A token that sees itself alone has its score as lse. Scores are exact under a cap of 1 with scale 1, so
    that lse = tanh(s) errs by the tanh, 4.93 half steps, and by the roundings of log2 e, of its product with the
    tanh, of ln 2 and of the product with that, relatively; the weight, 2 to the residual of the second, and its
    logarithm by 3 half steps of 1."""
    x = torch.arange(0x2400, 0x4900, device=DEV).to(torch.int16).view(F16) * sign  # 2^-6 .. 10
    T = x.numel()
    q, k, v = (torch.zeros((T, 1, 8), dtype=F16, device=DEV) for _ in range(3))
    q[:, 0, 0], k[:, 0, 0] = x, 1.0
    v[:] = normal(v.shape, 1, F16)
    plan = rope.attn_plan(torch.arange(T + 1, dtype=torch.int32, device=DEV), T, 1, 1)
    out, lse = rope.attn_fwd(q, k, v, plan, scale=1.0, softcap=1.0)
    want = torch.tanh(x.double())
    ref.check(lse[:, 0], want, 1.01 * 2.0 ** -24 * (9 * want.abs() + 3), "lse")
    assert torch.equal(out, v)
