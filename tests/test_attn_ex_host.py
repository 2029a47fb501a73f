"""Checks of the changed-score attention, the rotation with several axes and the page steps that need
no GPU: the library exports what the headers declare, host-side validation rejects bad arguments
before any HIP call (no kernel is launched here), CPU tensors are refused, and the references that
the GPU tests compare with agree with autograd in 64 bits and notice planted mistakes."""
import ctypes
import os
import re
import subprocess
import sys

import pytest
import torch

import attn_scores_reference as ref
import packed_varlen_rotary_rope_amd as rope
import packed_varlen_rotary_rope_amd.functional as F
from packed_varlen_rotary_rope_amd import attention as A

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, EINVAL, EUNSUPPORTED = 0, -1, -2
FAKE = ctypes.c_void_p(0x10000)  # never dereferenced: every call below fails validation or is empty
OTHER = ctypes.c_void_p(0x20000)


def ints(*values):
    return (ctypes.c_int32 * len(values))(*values)


@pytest.mark.parametrize("header,names", [
    ("attn_ex.h", {"attn_plan_ex", "attn_fwd_ex", "attn_bwd_ex_scratch_floats", "attn_bwd_ex", "paged_plan_ex",
                   "attn_paged_ex"}),
    ("rope_axes.h", {"rope_qk_apply_axes", "kv_append_slots"}),
    ("kv_pages.h", {"kv_page_step", "kv_page_release"})])
def test_exports_every_declared_symbol(header, names):
    text = open(os.path.join(ROOT, "include", header)).read()
    assert set(re.findall(r"^(?:int32_t|int64_t)\s+(\w+)\s*\(", text, re.M)) == names
    out = subprocess.run(["nm", "-D", "--defined-only", A.LIB_PATH], capture_output=True, text=True,
                         check=True).stdout
    assert names <= {ln.split()[-1] for ln in out.splitlines() if " T " in ln}


def test_tanh_constants_are_generated():
    sys.path.insert(0, os.path.join(ROOT, "packed_varlen_rotary_rope_amd", "csrc"))
    try:
        import gen_tanh_constants as gen
        assert open(gen.OUT).read() == gen.text()
    finally:
        sys.path.pop(0)


def fwd(**kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE, out=FAKE, lse=FAKE, T=16, Hq=4, Hkv=2, D=64, qs=0, ks=0, vs=0, os=0,
             plan=FAKE, B=2, scale=0.125, cap=50.0, slopes=FAKE, dtype=1, fill=1)
    a.update(kw)
    return A._lib.attn_fwd_ex(*a.values(), None)


def bwd(**kw):
    a = dict(dout=FAKE, q=FAKE, k=FAKE, v=FAKE, out=FAKE, lse=FAKE, scratch=FAKE, dq=FAKE, dk=FAKE, dv=FAKE,
             T=16, Hq=4, Hkv=2, D=64, dos=0, qs=0, ks=0, vs=0, os=0, dqs=0, dks=0, dvs=0, plan=FAKE, B=2,
             scale=0.125, cap=50.0, slopes=FAKE, dtype=1, fill=1)
    a.update(kw)
    return A._lib.attn_bwd_ex(*a.values(), None)


def paged(**kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE, out=FAKE, lse=FAKE, space=FAKE, T=16, Hq=4, Hkv=2, D=64, qs=0, os=0,
             pages=9, page=16, ps=2048, ss=128, hs=64, table=FAKE, per=4, ts=4, plan=FAKE, B=2, scale=0.125,
             cap=50.0, slopes=FAKE, dtype=1, fill=1)
    a.update(kw)
    return A._lib.attn_paged_ex(*a.values(), None)


@pytest.mark.parametrize("call", [fwd, bwd, paged])
@pytest.mark.parametrize("kw,expect", [
    (dict(cap=-1.0), EINVAL), (dict(cap=float("nan")), EINVAL), (dict(cap=float("inf")), EINVAL),
    (dict(cap=1e31), EINVAL), (dict(cap=1e-32), EINVAL), (dict(scale=1e-37, cap=1.0), EINVAL),
    (dict(scale=0.0), EINVAL), (dict(dtype=0), EUNSUPPORTED), (dict(T=-1), EINVAL), (dict(D=60), EINVAL),
    (dict(Hq=3), EINVAL), (dict(q=None), EINVAL), (dict(lse=None), EINVAL), (dict(plan=None), EINVAL),
    (dict(T=0, cap=0.0, slopes=None), OK), (dict(T=0, q=None, plan=None), OK)])
def test_validation_of_scores(call, kw, expect):
    assert call(**kw) == expect


def test_sizes():
    lib = A._lib
    small, large = (lib.attn_bwd_ex_scratch_floats(100, 2, 8, 2, 64, b) for b in (0, 1))
    assert small == lib.attn_bwd_scratch_floats(100, 2, 8, 2, 64) and large == small + 2 * 100 * 8
    assert lib.attn_bwd_ex_scratch_floats(100, 2, 8, 2, 136, 0) == -1
    assert lib.attn_plan_ex(FAKE, 2, None, FAKE, 16, 4, 2, FAKE, 10, None) == EINVAL  # too small a buffer
    assert lib.paged_plan_ex(FAKE, 2, FAKE, FAKE, 16, 4, 2, FAKE, 10, None) == EINVAL


def axes(**kw):
    a = dict(q=FAKE, q_out=OTHER, k=FAKE, k_out=OTHER, T=16, Hq=4, Hkv=2, D=64, qs=0, qos=0, ks=0, kos=0,
             ids=FAKE, step=16, sections=ints(16, 8, 8), axes=3, layout=0, theta=1e4, pos_scale=1.0, dtype=1,
             direction=1)
    a.update(kw)
    return A._lib.rope_qk_apply_axes(*a.values(), None)


def slots(**kw):
    a = dict(q=FAKE, q_out=OTHER, k=FAKE, v=FAKE, kc=OTHER, vc=OTHER, T=16, Hq=4, Hkv=2, D=64, qs=0, os=0, ks=0,
             vs=0, pages=9, page=16, ps=2048, ss=128, hs=64, slots=FAKE, ids=FAKE, step=16,
             sections=ints(16, 8, 8), axes=3, layout=0, theta=1e4, pos_scale=1.0, dtype=1)
    a.update(kw)
    return A._lib.kv_append_slots(*a.values(), None)


@pytest.mark.parametrize("call", [axes, slots])
@pytest.mark.parametrize("kw,expect", [
    (dict(dtype=3), EUNSUPPORTED), (dict(T=-1), EINVAL), (dict(T=2 ** 31), EINVAL), (dict(Hq=-1), EINVAL),
    (dict(Hkv=4097), EINVAL), (dict(D=63), EINVAL), (dict(D=514), EINVAL), (dict(D=0), EINVAL),
    (dict(theta=0.5), EINVAL), (dict(theta=float("nan")), EINVAL), (dict(pos_scale=0.5), EINVAL),
    (dict(pos_scale=1e300), EINVAL), (dict(qs=255), EINVAL), (dict(ks=64), EINVAL), (dict(ids=None), EINVAL),
    (dict(step=15), EINVAL), (dict(step=2 ** 41), EINVAL), (dict(axes=0), EINVAL), (dict(axes=5), EINVAL),
    (dict(layout=3), EINVAL), (dict(layout=-1), EINVAL), (dict(sections=None), EINVAL),
    (dict(sections=ints(16, 8, 9)), EINVAL), (dict(sections=ints(-8, 32, 8)), EINVAL),
    (dict(sections=ints(2 ** 31 - 1, 2 ** 31 - 1, 34)), EINVAL),
    (dict(layout=1, sections=ints(8, 12, 12)), EINVAL),  # the third axis would need a 36th frequency
    (dict(k=None), EINVAL), (dict(q_out=None), EINVAL), (dict(q_out=FAKE, qs=512), EINVAL),
    (dict(T=0, k=None, q=None, ids=None), OK)])
def test_validation_of_axes(call, kw, expect):
    assert call(**kw) == expect


@pytest.mark.parametrize("kw", [dict(Hq=0, Hkv=0), dict(direction=0), dict(k_out=None), dict(k_out=FAKE, kos=192)])
def test_validation_of_the_rotation(kw):
    assert axes(**kw) == EINVAL


@pytest.mark.parametrize("kw", [dict(Hkv=0), dict(pages=-1), dict(page=0), dict(ps=-1), dict(hs=2 ** 41), dict(v=None),
                                dict(kc=None), dict(slots=None)])
def test_validation_of_the_append(kw):
    assert slots(**kw) == EINVAL


def page_step(**kw):
    a = dict(new=FAKE, held=FAKE, B=2, T=8, page=16, table=FAKE, per=4, ts=4, ring=FAKE, pages=9, state=FAKE,
             cu=OTHER, lens=OTHER, held_out=OTHER, positions=OTHER, slots=OTHER, state_out=OTHER)
    a.update(kw)
    return A._lib.kv_page_step(*a.values(), None)


def release(**kw):
    a = dict(held=FAKE, gone=FAKE, B=2, page=16, table=FAKE, per=4, ts=4, ring=FAKE, pages=9, state=FAKE)
    a.update(kw)
    return A._lib.kv_page_release(*a.values(), None)


@pytest.mark.parametrize("call", [page_step, release])
@pytest.mark.parametrize("kw", [dict(B=-1), dict(B=2 ** 25), dict(page=0), dict(page=2 ** 30 + 1), dict(per=-1), dict(ts=-1),
                                dict(pages=0), dict(pages=2 ** 30 + 1), dict(table=None), dict(ring=None),
                                dict(state=None), dict(held=None)])
def test_validation_of_pages(call, kw):
    assert call(**kw) == EINVAL


@pytest.mark.parametrize("kw", [dict(T=-1), dict(T=2 ** 30 + 1), dict(new=None), dict(cu=None), dict(lens=None),
                                dict(held_out=None), dict(held_out=FAKE), dict(state_out=FAKE), dict(state_out=None),
                                dict(positions=None), dict(slots=None)])
def test_validation_of_the_page_step(kw):
    assert page_step(**kw) == EINVAL


def test_cpu_tensors_are_refused():
    i = torch.arange(4, dtype=torch.int32)
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    cache = torch.zeros(2, 16, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        rope.qk_apply_axes(x, x, i[None], (32,), 1e4)
    with pytest.raises(TypeError):
        rope.kv_append_slots_(x, x, cache, cache, i.long(), i, 1e4)
    with pytest.raises(TypeError):
        rope.PagePool(i, i[:2])
    with pytest.raises(TypeError):
        rope.page_step(None, i[None], i, i, 4, 16)
    with pytest.raises(TypeError):
        rope.page_release_(None, i[None], i, i > 0, 16)
    with pytest.raises(TypeError):
        F.rope_qk_axes(x, x, i[None], (32,), 1e4)


def test_score_arguments():
    dev = torch.device("cpu")
    assert A._scores(None, None, 4, dev) == (0.0, None)
    good = torch.ones(4)
    assert A._scores(30, good, 4, dev) == (30.0, good.data_ptr())
    for cap in (0.0, -1.0, float("nan"), float("inf")):
        with pytest.raises(ValueError):
            A._scores(cap, None, 4, dev)
    for bad in (good.double(), torch.ones(8)[::2], good.to("meta")):
        with pytest.raises(TypeError):
            A._scores(None, bad, 4, dev)
    for bad in (torch.ones(3), torch.ones(1, 4)):
        with pytest.raises(ValueError):
            A._scores(None, bad, 4, dev)
    with pytest.raises(ValueError, match="gradient"):
        F._constant(good.clone().requires_grad_())
    with torch.no_grad():
        F._constant(good.clone().requires_grad_())


def case(seed=0):
    g = torch.Generator().manual_seed(seed)
    T, Hq, Hkv, D = 23, 4, 2, 8
    return [torch.randn((T, h, D), generator=g, dtype=torch.float64) for h in (Hq, Hkv, Hkv, Hq)]


def by_autograd(q, k, v, do, seqs, scale, cap, slopes, prefixes):
    """The formula on whole matrices, with autograd's gradients."""
    q, k, v = (t.clone().requires_grad_() for t in (q, k, v))
    outs = torch.zeros_like(q)
    for s, (a, n) in enumerate(seqs):
        x = q[a:a + n].transpose(0, 1)
        y, z = (t[a:a + n].repeat_interleave(q.shape[1] // k.shape[1], 1).transpose(0, 1) for t in (k, v))
        sc = x @ y.transpose(1, 2) * scale
        if cap is not None:
            sc = cap * torch.tanh(sc / cap)
        i = torch.arange(n)
        if slopes is not None:
            sc = sc - slopes.double()[:, None, None] * (i[:, None] - i[None]).abs()
        hidden = (i[None] > i[:, None]) & (i[None] >= (prefixes[s] if prefixes else 0))
        o = (sc.masked_fill(hidden, float("-inf")).softmax(-1) @ z).transpose(0, 1)
        outs = outs.index_add(0, torch.arange(a, a + n), o)
    outs.backward(do)
    return outs.detach(), (q.grad, k.grad, v.grad)


SEQS, ARGS = [(0, 9), (9, 14)], (2.0, torch.tensor([0.5, 0.25, -0.1, 0.0]), [4, 20])


@pytest.mark.parametrize("which", [(1, 0, 0), (0, 1, 0), (0, 0, 1), (1, 1, 1)])
def test_reference_against_autograd(which):
    q, k, v, do = case()
    args = [a if w else None for a, w in zip(ARGS, which)]
    out, grads = by_autograd(q, k, v, do, SEQS, 0.4, *args)
    got, _, _, _ = ref.forward(q, k, v, SEQS, 0.4, *args)
    assert torch.allclose(got, out, rtol=1e-12, atol=1e-13)
    for x, y in zip(ref.backward(do, q, k, v, SEQS, 0.4, torch.bfloat16, *args)[0], grads):
        assert torch.allclose(x, y, rtol=1e-11, atol=1e-13)


@pytest.mark.parametrize("mistake", [dict(cap=2.05), dict(slopes=ARGS[1] + 0.02), dict(prefixes=[5, 20]), dict(prefixes=[4, 0])])
def test_reference_notices_mistakes(mistake):
    """A cap, slope or prefix that is a little off is outside of the bounds."""
    q, k, v, do = case()
    args = dict(cap=ARGS[0], slopes=ARGS[1], prefixes=ARGS[2])
    out, _, tol, _ = ref.forward(q.bfloat16(), k.bfloat16(), v.bfloat16(), SEQS, 0.4, **args)
    args.update(mistake)
    other, _, _, _ = ref.forward(q.bfloat16(), k.bfloat16(), v.bfloat16(), SEQS, 0.4, **args)
    with pytest.raises(AssertionError):
        ref.check(other, out, tol, "out")
