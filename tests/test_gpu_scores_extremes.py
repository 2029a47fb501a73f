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


SIZE, SLOPE = 2.0 ** 30, 256.0


def one_hot(levels, before, n, held, form, prefix=0):
    """(key with the largest score, lse and its bound) of the queries at before .. before + n - 1 where scores are
    SIZE levels[j]; that key's is larger than any other by so much that it has all the weight."""
    i = before + torch.arange(n, device=DEV)[:, None]
    j = torch.arange(held, device=DEV)[None]
    s = (SIZE * levels.double())[None].expand(n, held)
    if form != "slopes":
        s = SIZE * torch.tanh(s / SIZE)
    bias = SLOPE * (i - j).abs().double() if form != "cap" else torch.zeros_like(s)
    tol = (s.abs() * 2.0 ** -21 + 2.0 ** -22 * (s.abs() + bias))
    total = (s - bias).masked_fill((j > i) & (j >= prefix), float("-inf"))
    two = total.topk(min(2, held), -1)
    if held > 1:
        assert bool((two.values[:, 0] - two.values[:, 1] > 2.0 ** 20).all())
    top = two.indices[:, 0]
    lse = two.values[:, 0]
    return top, lse, 1.01 * (tol.gather(1, top[:, None])[:, 0] + (4 + lse.abs()) * 2.0 ** -22)


def level_rows(levels, n, H, D):
    """Keys whose products with SIZE in the first column are SIZE times the levels."""
    k = torch.zeros((n, H, D), dtype=BF16, device=DEV)
    k[:, :, 0] = levels[:, None].to(BF16)
    return k


@pytest.mark.parametrize("form", ["cap", "slopes", "both"])
@pytest.mark.parametrize("D", [8, 64, 128, 192])
def test_very_large_scores(rope, form, D):
    """Scores of 2^30 under a cap of 2^30, a bias beside them: the maximum is subtracted before anything is rounded,
    so each row is the value of its largest score, exactly."""
    lens, prefixes, Hq, Hkv = [1, 100, 255 - 100 - 1], [0, 40, 0], 4, 2
    cu = [0, 1, 101, 255]
    T = cu[-1]
    g = torch.Generator().manual_seed(2)
    levels = ((torch.randperm(255, generator=g) - 127) / 128.0).to(DEV)  # exact in bf16
    q, k, v = torch.zeros((T, Hq, D), dtype=BF16, device=DEV), level_rows(levels, T, Hkv, D), normal((T, Hkv, D), 3, BF16)
    q[:, :, 0] = SIZE
    more = dict(scale=1.0, softcap=None if form == "slopes" else SIZE,
                slopes=None if form == "cap" else torch.full((Hq,), SLOPE, device=DEV))
    plan = rope.attn_plan(int32(cu), T, Hq, Hkv, prefix_lens=int32(prefixes))
    out, lse = rope.attn_fwd(q, k, v, plan, **more)
    for a, n, prefix in zip(cu, lens, prefixes):
        top, want, tol = one_hot(levels[a:a + n], 0, n, n, form, prefix)
        for h in range(Hq):
            assert torch.equal(out[a:a + n, h], v[a:a + n, h // 2][top])
            ref.check(lse[a:a + n, h], want, tol, "lse")


@pytest.mark.parametrize("form", ["cap", "slopes", "both"])
@pytest.mark.parametrize("D", [8, 128, 192])
@pytest.mark.parametrize("new", [1, 60])
def test_very_large_scores_over_a_cache(rope, form, D, new):
    """The same over caches that are long enough to be split: one key has the largest level."""
    held, page, Hq, Hkv = [64, 5000], 16, 8, 2
    cu, T = [0, new, 2 * new], 2 * new
    pages = [-(-m // page) for m in held]
    table = torch.full((2, max(pages)), -1, dtype=torch.int32, device=DEV)
    order = torch.randperm(sum(pages), generator=torch.Generator().manual_seed(1)).int().to(DEV)
    table[0, :pages[0]], table[1, :pages[1]] = order[:pages[0]], order[pages[0]:]
    kc, vc = (torch.zeros((sum(pages), page, Hkv, D), dtype=BF16, device=DEV) for _ in range(2))
    kept = []
    for s, m in enumerate(held):
        g = torch.Generator().manual_seed(10 + s)
        levels = torch.randint(-127, 127, (m,), generator=g) / 128.0
        levels[3 if s == 0 else m // 2 + 7] = 1.0
        levels, at = levels.to(DEV), torch.arange(m, device=DEV)
        where = table[s].long()[at // page], at % page
        k, v = level_rows(levels, m, Hkv, D), normal((m, Hkv, D), 20 + s, BF16)
        kc[where], vc[where] = k, v
        kept.append((levels, v))
    q = torch.zeros((T, Hq, D), dtype=BF16, device=DEV)
    q[:, :, 0] = SIZE
    more = dict(scale=1.0, softcap=None if form == "slopes" else SIZE,
                slopes=None if form == "cap" else torch.full((Hq,), SLOPE, device=DEV))
    plan = rope.paged_plan(int32(cu), int32(held), T, Hq, Hkv)
    out, lse = rope.attn_paged(q, kc, vc, table, plan, **more)
    for s, (levels, v) in enumerate(kept):
        a, m = s * new, held[s]
        top, want, tol = one_hot(levels, m - new, new, m, form)
        for h in range(Hq):
            assert torch.equal(out[a:a + new, h], v[:, h // 4][top])
            ref.check(lse[a:a + new, h], want, tol, "lse")
