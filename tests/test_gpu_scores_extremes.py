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


@pytest.mark.parametrize("form", ["cap", "slopes", "both"])
@pytest.mark.parametrize("D", [16, 64, 72, 128])
def test_gradients_past_half_precision(rope, form, D):
    """dS past 65504 overflows in f16, at any head size alike. Scores are 0 (but for a bias of up to 3e-4), so that
    weights are 1 / n; dP is 4e6 T at even keys and -4e6 T at odd ones, so that dS is past 65504 for every key of the
    rows that see two or more. The keys' signs make each term of a column of dQ the same infinity."""
    T = 300
    dv = 4e6 * T / D / 60000.0  # of V, at do 60000: dP is 4e6 T
    assert dv < 60000.0
    q, k, v, do = (torch.zeros((T, 1, D), dtype=F16, device=DEV) for _ in range(4))
    sign = torch.where(torch.arange(T, device=DEV) % 2 == 0, 1.0, -1.0)[:, None, None]
    k[:], v[:], do[:] = sign * 0.5, sign * dv, 60000.0
    columns = torch.where(torch.arange(D, device=DEV) % 3 == 0, -1.0, 1.0)
    k *= columns
    plan = rope.attn_plan(int32([0, T]), T, 1, 1)
    more = dict(softcap=None if form == "slopes" else 30.0,
                slopes=None if form == "cap" else torch.full((1,), 2.0 ** -20, device=DEV))
    out, lse = rope.attn_fwd(q, k, v, plan, **more)
    dq = rope.attn_bwd(do, q, k, v, out, lse, plan, **more)[0]
    want = (columns * float("inf")).to(F16).expand(T - 1, 1, D)
    assert torch.equal(dq[1:], want)
