"""Attention checks that need no GPU: the library exports what include/attn.h declares,
host-side validation rejects bad arguments before any HIP call (no kernel is launched here), the
package refuses tensors that are not on a GPU, and the reference the GPU tests compare with
agrees with plain autograd in 64 bits and notices planted mistakes."""
import ctypes
import glob
import os
import re
import shutil
import subprocess
import sys

import pytest
import torch

import attn_reference as ref
import packed_varlen_rotary_rope_amd as rope
import packed_varlen_rotary_rope_amd.functional as F
from packed_varlen_rotary_rope_amd import attention as A

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, EINVAL, EUNSUPPORTED = 0, -1, -2
FAKE = ctypes.c_void_p(0x10000)  # never dereferenced: every call below fails validation or is empty
ODD = ctypes.c_void_p(0x10004)


def test_exports_every_declared_symbol():
    text = open(os.path.join(ROOT, "include", "attn.h")).read()
    names = re.findall(r"^(?:int32_t|int64_t)\s+(\w+)\s*\(", text, re.M)
    assert set(names) == {"attn_plan_ints", "attn_plan", "attn_fwd", "attn_bwd_scratch_floats", "attn_bwd",
                          "kv_append", "paged_plan_ints", "paged_workspace_floats", "paged_plan",
                          "attn_paged"}
    out = subprocess.run(["nm", "-D", "--defined-only", A.LIB_PATH], capture_output=True, text=True,
                         check=True).stdout
    exported = {ln.split()[-1] for ln in out.splitlines() if " T " in ln}
    assert set(names) <= exported


def fwd(**kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE, out=FAKE, lse=FAKE, T=16, Hq=4, Hkv=2, D=64, qs=0, ks=0, vs=0, os=0,
             plan=FAKE, B=2, scale=0.125, dtype=1, fill=1)
    a.update(kw)
    return A._lib.attn_fwd(*a.values(), None)


def bwd(**kw):
    a = dict(dout=FAKE, q=FAKE, k=FAKE, v=FAKE, out=FAKE, lse=FAKE, scratch=FAKE, dq=FAKE, dk=FAKE, dv=FAKE,
             T=16, Hq=4, Hkv=2, D=64, dos=0, qs=0, ks=0, vs=0, os=0, dqs=0, dks=0, dvs=0, plan=FAKE, B=2,
             scale=0.125, dtype=1, fill=1)
    a.update(kw)
    return A._lib.attn_bwd(*a.values(), None)


def paged(**kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE, out=FAKE, lse=FAKE, space=FAKE, T=16, Hq=4, Hkv=2, D=64, qs=0, os=0,
             pages=9, page=16, ps=2048, ss=128, hs=64, table=FAKE, per=4, ts=4, plan=FAKE, B=2, scale=0.125,
             dtype=1, fill=1)
    a.update(kw)
    return A._lib.attn_paged(*a.values(), None)


def append(**kw):
    a = dict(q=FAKE, q_out=FAKE, k=FAKE, v=FAKE, kc=FAKE, vc=FAKE, T=16, Hq=4, Hkv=2, D=64, qs=0, os=0, ks=0,
             vs=0, pages=9, page=16, ps=2048, ss=128, hs=64, table=FAKE, per=4, ts=4, cu=FAKE, B=2,
             lens=FAKE, theta=1e4, pos_scale=1.0, dtype=1)
    a.update(kw)
    return A._lib.kv_append(*a.values(), None)


COMMON = [
    (dict(dtype=0), EUNSUPPORTED), (dict(dtype=3), EUNSUPPORTED), (dict(T=-1), EINVAL),
    (dict(Hq=0), EINVAL), (dict(Hkv=0), EINVAL), (dict(Hq=3), EINVAL), (dict(Hq=2, Hkv=4), EINVAL),
    (dict(Hq=8192), EINVAL), (dict(D=0), EINVAL), (dict(D=60), EINVAL), (dict(D=264), EINVAL),
    (dict(scale=0.0), EINVAL), (dict(scale=-1.0), EINVAL), (dict(scale=float("nan")), EINVAL),
    (dict(scale=float("inf")), EINVAL), (dict(qs=255), EINVAL), (dict(qs=248), EINVAL),
    (dict(qs=260), EINVAL), (dict(qs=1 << 24), EINVAL), (dict(B=-1), EINVAL), (dict(q=None), EINVAL),
    (dict(k=ODD), EINVAL), (dict(v=None), EINVAL), (dict(out=ODD), EINVAL), (dict(lse=None), EINVAL),
    (dict(plan=None), EINVAL), (dict(T=2 ** 31), EINVAL), (dict(T=2 ** 30, Hq=8), EINVAL),
    (dict(T=0, q=None, plan=None), OK),
]


@pytest.mark.parametrize("kw,expect", COMMON)
def test_validation_forward(kw, expect):
    assert fwd(**kw) == expect


@pytest.mark.parametrize("kw,expect", COMMON + [
    (dict(D=136), EINVAL), (dict(dq=None), EINVAL), (dict(scratch=None), EINVAL), (dict(dos=4), EINVAL),
    (dict(dvs=130), EINVAL), (dict(dout=ODD), EINVAL)])
def test_validation_backward(kw, expect):
    assert bwd(**kw) == expect


@pytest.mark.parametrize("kw,expect", COMMON + [
    (dict(pages=0), EINVAL), (dict(page=0), EINVAL), (dict(per=-1), EINVAL), (dict(ts=-1), EINVAL),
    (dict(ps=4), EINVAL), (dict(hs=-8), EINVAL), (dict(space=None), EINVAL), (dict(table=None), EINVAL)])
def test_validation_paged(kw, expect):
    assert paged(**kw) == expect


@pytest.mark.parametrize("kw,expect", [
    (dict(dtype=3), EUNSUPPORTED), (dict(T=-1), EINVAL), (dict(Hkv=0), EINVAL), (dict(Hq=-1), EINVAL),
    (dict(D=63), EINVAL), (dict(D=514), EINVAL), (dict(theta=0.5), EINVAL), (dict(theta=float("nan")), EINVAL),
    (dict(pos_scale=0.5), EINVAL), (dict(pos_scale=float("nan")), EINVAL), (dict(pos_scale=1e300), EINVAL),
    (dict(ks=64), EINVAL), (dict(qs=1), EINVAL), (dict(page=0), EINVAL), (dict(pages=-1), EINVAL),
    (dict(per=-1), EINVAL), (dict(ps=-1), EINVAL), (dict(k=None), EINVAL), (dict(kc=None), EINVAL),
    (dict(cu=None), EINVAL), (dict(lens=None), EINVAL), (dict(table=None), EINVAL), (dict(q_out=None), EINVAL),
    (dict(qs=512), EINVAL),  # in place (q_out = q) with another stride
    (dict(B=-1), EINVAL), (dict(T=0, k=None), OK)])
def test_validation_append(kw, expect):
    assert append(**kw) == expect


def test_plan_sizes():
    lib = A._lib
    assert lib.attn_plan_ints(0, 0, 1, 1) > 0 and lib.attn_plan_ints(2 ** 31 - 200, 1, 1, 1) > 0
    for bad in ((-1, 1, 1, 1), (1, -1, 1, 1), (1, 1, 3, 2), (1, 1, 1, 0), (2 ** 31, 1, 1, 1), (2 ** 29, 1, 8, 1)):
        assert lib.attn_plan_ints(*bad) == -1 and lib.paged_plan_ints(*bad) == -1
        assert lib.paged_workspace_floats(*bad, 64) == -1 and lib.attn_bwd_scratch_floats(*bad, 64) == -1
    assert lib.attn_plan(FAKE, 2, None, 16, 4, 2, FAKE, 10, None) == EINVAL  # too small a buffer
    assert lib.attn_plan(None, 2, None, 16, 4, 2, FAKE, 1 << 20, None) == EINVAL
    assert lib.attn_plan(FAKE, 2, None, 16, 4, 2, ODD, 1 << 20, None) == EINVAL
    assert lib.paged_plan(FAKE, 2, None, 16, 4, 2, FAKE, 1 << 20, None) == EINVAL
    assert lib.paged_plan(FAKE, 2, FAKE, 16, 4, 2, FAKE, 10, None) == EINVAL


def test_cpu_tensors_are_refused():
    cu = torch.tensor([0, 4], dtype=torch.int32)
    q = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        rope.attn_plan(cu, 4, 2, 2)
    with pytest.raises(TypeError):
        rope.paged_plan(cu, cu[:1], 4, 2, 2)
    plan = rope.AttnPlan(4, 1, 2, 2, torch.zeros(64, dtype=torch.int32))
    with pytest.raises(TypeError):
        rope.attn_fwd(q, q, q, plan)
    cache = torch.zeros(2, 16, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        rope.kv_append_(q, q, cache, cache, cu[None], cu, cu[:1], 1e4)
    with pytest.raises(TypeError):
        rope.attn_paged(q, cache, cache, cu[None], rope.PagedPlan(4, 1, 2, 2, cu))
    for bad in (dict(), dict(plan=plan, cu_seqlens=cu)):
        with pytest.raises(ValueError):
            F.attn(q, q, q, **bad)


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (6, 2), (4, 1)])
def test_reference_gradients_match_autograd(Hq, Hkv):
    torch.manual_seed(0)
    T, D, cu = 23, 8, [0, 1, 9, 9, 20]
    q, k, v, do = (torch.randn(T, h, D, dtype=torch.float64, requires_grad=i < 3)
                   for i, h in enumerate((Hq, Hkv, Hkv, Hq)))
    seqs, scale = ref.sequences(cu, T), 0.4
    out = torch.zeros(T, Hq, D, dtype=torch.float64)
    for a, n in seqs:
        for h in range(Hq):
            s = q[a:a + n, h] @ k[a:a + n, h // (Hq // Hkv)].T * scale
            s = s.masked_fill(torch.ones(n, n, dtype=torch.bool).triu(1), float("-inf"))
            o = torch.softmax(s, -1) @ v[a:a + n, h // (Hq // Hkv)]
            out = out.index_put((torch.arange(a, a + n), torch.tensor(h)), o)
    want = torch.autograd.grad(out, (q, k, v), do)
    plain, _, _ = ref.forward(*(x.detach().float() for x in (q, k, v)), seqs, scale)
    assert torch.allclose(plain, out.detach(), atol=1e-5)
    got, tols = ref.backward(do.detach(), q.detach(), k.detach(), v.detach(), seqs, scale, torch.float16)
    for g, w, tol in zip(got, want, tols):
        assert torch.allclose(g, w, atol=1e-10) and bool((tol > 0).all())
    # mistakes that the bounds must notice
    for name, wrong in (("scale", got[0] / scale), ("sign", -got[1]), ("shift", got[2].roll(1, 0))):
        i = {"scale": 0, "sign": 1, "shift": 2}[name]
        with pytest.raises(AssertionError):
            ref.check(wrong, got[i], tols[i], name)


def test_reference_pages():
    """Keys on no page count for nobody; positions behind the table neither."""
    torch.manual_seed(1)
    k, v = torch.randn(3, 4, 1, 8), torch.randn(3, 4, 1, 8)
    q = torch.randn(2, 1, 8)
    table = torch.tensor([[2, -1]], dtype=torch.int32)
    out, lse, _ = ref.paged(q, k, v, table, [0, 2], [7], 1.0)
    s = (q[:, 0].double() @ k[2, :, 0].double().T)
    assert torch.allclose(lse[:, 0], torch.logsumexp(s, -1))
    assert torch.allclose(out[:, 0], torch.softmax(s, -1) @ v[2, :, 0].double())


def test_package_without_the_attention_library(tmp_path):
    """The rotary and GLU entry points import without libattn.so; the attention's names say what
    is missing."""
    pkg = os.path.join(ROOT, "packed_varlen_rotary_rope_amd")
    there = tmp_path / "packed_varlen_rotary_rope_amd"
    there.mkdir()
    for path in [*glob.glob(os.path.join(pkg, "*.py")), os.path.join(pkg, "librope_qk.so")]:
        shutil.copy(path, there)
    code = ("import packed_varlen_rotary_rope_amd as m\n"
            "from packed_varlen_rotary_rope_amd import functional as F\n"
            "from packed_varlen_rotary_rope_amd import *\n"
            "assert F.rope_qk and m.qk_fwd_ is qk_fwd_ and not hasattr(m, 'nothing')\n"
            "for name in ('attn_fwd', 'kv_append_', 'AttnPlan'):\n"
            "    try:\n"
            "        getattr(m, name)\n"
            "    except ImportError as e:\n"
            "        assert 'build_attn.py' in str(e)\n"
            "    else:\n"
            "        raise SystemExit(name)\n")
    subprocess.run([sys.executable, "-c", code], check=True, cwd=tmp_path, timeout=300,
                   env={**os.environ, "PYTHONPATH": str(tmp_path)})


def test_plans_are_not_written_over_by_the_other_kind(monkeypatch):
    """The two kinds of plan are of different lengths, each longer for some batches: a plan given as
    `out` is of the function's own kind, and its real length reaches the library. No GPU: the
    launch is replaced."""
    launched = []
    monkeypatch.setattr(A, "_gpu", lambda device: None)
    monkeypatch.setattr(A, "_call", lambda device, fn, what, *args: launched.append((what, args[-1])))
    for T, Hq, Hkv in ((64, 4, 2), (2 ** 20, 1, 1)):
        cu, lens = torch.tensor([0, T], dtype=torch.int32), torch.tensor([T], dtype=torch.int32)
        words = A._lib.attn_plan_ints(T, 1, Hq, Hkv), A._lib.paged_plan_ints(T, 1, Hq, Hkv)
        packed = rope.AttnPlan(T, 1, Hq, Hkv, torch.empty(words[0], dtype=torch.int32))
        paged = rope.PagedPlan(T, 1, Hq, Hkv, torch.empty(words[1], dtype=torch.int32))
        for wrong in (paged, packed.buffer, object()):
            with pytest.raises(TypeError, match="attn_plan"):
                rope.attn_plan(cu, T, Hq, Hkv, out=wrong)
        for wrong in (packed, paged.buffer, object()):
            with pytest.raises(TypeError, match="paged_plan"):
                rope.paged_plan(cu, lens, T, Hq, Hkv, out=wrong)
        assert launched == []
        assert rope.attn_plan(cu, T, Hq, Hkv, out=packed) is packed
        assert rope.paged_plan(cu, lens, T, Hq, Hkv, out=paged) is paged
        short = rope.AttnPlan(T, 1, Hq, Hkv, torch.empty(40, dtype=torch.int32))
        rope.attn_plan(cu, T, Hq, Hkv, out=short)  # the library refuses its length
        assert launched == [("attn_plan", words[0]), ("paged_plan", words[1]), ("attn_plan", 40)]
        launched.clear()
        assert A._lib.attn_plan(FAKE, 1, None, T, Hq, Hkv, FAKE, 40, None) == EINVAL


def test_upstream_gradients_of_any_layout_are_laid_out_for_the_kernels():
    """Contiguous rows at an odd address, as behind another tensor of one concatenated buffer, and
    tokens further apart than the kernels take, are copied; what they take is passed on as it is."""
    T, H, D = 5, 2, 16
    flat = torch.arange(T * H * D + 64, dtype=torch.float32).bfloat16()
    flat = flat[(-flat.data_ptr() // 2) % 8:]
    for first in (1, 3, 4):
        t = flat[first:first + T * H * D].view(T, H, D)
        got = F._rows_for_kernel(t)
        assert torch.equal(got, t) and got.data_ptr() % 16 == 0 and got.is_contiguous()
    for t in (flat[:T * H * D].view(T, H, D), flat[8:8 + T * H * D].view(T, H, D), flat[:T * 40].view(T, 40)[:, 8:40].view(T, H, D)):
        assert F._rows_for_kernel(t) is t
    for t in (flat[:1].expand(T, H, D), flat[:T * H * D].view(H, T, D).transpose(0, 1)):
        assert F._rows_for_kernel(t).is_contiguous()
    far = torch.empty((1,), dtype=torch.bfloat16).expand(2, H, D).as_strided((2, H, D), (0, 0, 0))
    wide = torch.empty((2, 1 << 24), dtype=torch.bfloat16)[:, :H * D].view(2, H, D)
    assert F._rows_for_kernel(far).stride(0) == F._rows_for_kernel(wide).stride(0) == H * D


def test_more_pages_than_a_table_can_name_are_refused():
    """Page numbers are int32; a larger count would reach the library cut to its low bits. The
    cache here is one element seen many times, only its shape is read."""
    one = torch.zeros(8, dtype=torch.bfloat16)
    for shape in ((2 ** 32 + 5, 1, 1, 8), (1, 2 ** 31, 1, 8)):
        cache = one.as_strided(shape, (0, 0, 0, 1))
        with pytest.raises(ValueError, match="int32"):
            A._caches(cache, cache, torch.bfloat16, cache.device)
    assert A._caches(one.as_strided((5, 2, 1, 8), (0, 0, 0, 1)), one.as_strided((5, 2, 1, 8), (0, 0, 0, 1)),
                     torch.bfloat16, one.device)[0] == (5, 2, 1, 8)
