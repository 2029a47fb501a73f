"""Attention around the rotary embedding: causal attention over packed sequences (forward
and backward), the append of new keys and values to a paged cache (rotated on the way), and
attention over that cache.

Thin binding over the C ABI of ``include/attn.h`` (libattn.so, built by build_attn.py from
``csrc/attn_*.hip`` and ``csrc/kv_append.hip``), as the package's other entry points are: it checks
tensor metadata and marshals pointers, sizes and the current HIP stream. There is no
fallback: if the library is missing, importing this module raises. The public names are
exported by the package itself; differentiable wrappers live in ``functional``.

The packed batch is the one the Unsloth page describes (section "Packing non contamine": no
sample sees another's tokens).
"""
from __future__ import annotations

import ctypes
import os

import torch

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libattn.so")

_DTYPE_CODE = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}


def _load() -> ctypes.CDLL:
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"{LIB_PATH} is not built; run `python packed_varlen_rotary_rope_amd/build_attn.py` "
            "(hipcc, gfx950). There is no fallback implementation.")
    lib = ctypes.CDLL(LIB_PATH)
    i32, i64, dbl, vp = ctypes.c_int32, ctypes.c_int64, ctypes.c_double, ctypes.c_void_p
    lib.attn_plan_ints.argtypes = [i64, i32, i32, i32]
    lib.attn_plan_ints.restype = i64
    lib.attn_plan.argtypes = [vp, i32, vp, i64, i32, i32, vp, i64, vp]
    lib.attn_fwd.argtypes = [vp, vp, vp, vp, vp, i64, i32, i32, i32, i64, i64, i64, i64, vp, i32, dbl,
                             i32, i32, vp]
    lib.attn_bwd.argtypes = [vp] * 10 + [i64, i32, i32, i32] + [i64] * 8 + [vp, i32, dbl, i32, i32, vp]
    lib.attn_bwd_scratch_floats.argtypes = [i64, i32, i32, i32, i32]
    lib.attn_bwd_scratch_floats.restype = i64
    lib.kv_append.argtypes = ([vp] * 6 + [i64, i32, i32, i32] + [i64] * 4 + [i32, i32] + [i64] * 3 +
                              [vp, i32, i64, vp, i32, vp, dbl, dbl, i32, vp])
    lib.paged_plan_ints.argtypes = [i64, i32, i32, i32]
    lib.paged_plan_ints.restype = i64
    lib.paged_workspace_floats.argtypes = [i64, i32, i32, i32, i32]
    lib.paged_workspace_floats.restype = i64
    lib.paged_plan.argtypes = [vp, i32, vp, i64, i32, i32, vp, i64, vp]
    lib.attn_paged.argtypes = ([vp] * 6 + [i64, i32, i32, i32, i64, i64, i32, i32] + [i64] * 3 +
                               [vp, i32, i64, vp, i32, dbl, i32, i32, vp])
    for name in ("attn_plan", "attn_fwd", "attn_bwd", "kv_append", "paged_plan", "attn_paged"):
        getattr(lib, name).restype = i32
    return lib


_lib = _load()


_HALF = (torch.bfloat16, torch.float16)
_ANY = (torch.float32, torch.bfloat16, torch.float16)
_INT32_MAX = 2 ** 31 - 1


def _call(device: torch.device, fn, what: str, *args) -> None:
    """fn(*args, stream) on `device` and its current stream."""
    index = device.index
    stream = torch._C._cuda_getCurrentRawStream(index)
    if torch._C._cuda_getDevice() == index:
        status = fn(*args, stream)
    else:
        with torch.cuda.device(index):
            status = fn(*args, stream)
    if status != 0:
        from . import RopeError
        raise RopeError(status, what)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _index(t, name: str, device, numel=None):
    """A contiguous int32 tensor on `device`."""
    if t.dtype != torch.int32 or t.device != device or not t.is_contiguous():
        raise TypeError(f"{name} must be a contiguous int32 tensor on {device}")
    if numel is not None and t.numel() != numel:
        raise ValueError(f"{name} must have {numel} entries")
    return t


def _gpu(device: torch.device) -> None:
    if device.type != "cuda":
        raise TypeError("expected tensors on a GPU")


def _token_rows(t, name: str, dtypes) -> int:
    """Token stride of a [T, H, D] tensor whose tokens hold their heads contiguously."""
    shape, stride = t.shape, t.stride()
    if (len(shape) == 3 and stride[2] == 1 and stride[1] == shape[2] and
            stride[0] >= shape[1] * shape[2] and t.is_cuda and t.dtype in dtypes):
        return stride[0]
    _gpu(t.device)
    if t.dtype not in dtypes:
        raise TypeError(f"{name}: expected " + " or ".join(str(d)[6:] for d in dtypes))
    if t.dim() != 3:
        raise ValueError(f"{name}: expected [T, H, D]")
    T, H, D = t.shape
    if t.numel() == 0:
        return H * D
    if (D > 1 and t.stride(2) != 1) or (H > 1 and t.stride(1) != D):
        raise ValueError(f"{name}: the heads of a token must be contiguous "
                         "(stride(2) == 1 and stride(1) == D)")
    if T <= 1:
        return H * D
    if t.stride(0) < H * D:
        raise ValueError(f"{name}: its tokens overlap (an expanded tensor needs a copy)")
    return t.stride(0)


def _heads_last(t, name: str, most: int = 256) -> int:
    """_token_rows of a 16-bit tensor whose rows are aligned for 16-byte accesses and whose head
    size the kernels take."""
    shape, stride = t.shape, t.stride()
    if (len(shape) == 3 and stride[2] == 1 and stride[1] == shape[2] and stride[0] % 8 == 0 and
            stride[0] >= shape[1] * shape[2] and t.data_ptr() % 16 == 0 and t.is_cuda and
            t.dtype in _HALF and shape[2] % 8 == 0 and 8 <= shape[2] <= most):
        return stride[0]
    stride = _token_rows(t, name, _HALF)
    if shape[2] % 8 or not 8 <= shape[2] <= most:
        raise ValueError(f"head size {shape[2]}: expected a multiple of 8, 8 .. {most}")
    if t.data_ptr() % 16 or stride % 8:
        raise ValueError(f"{name}: data pointer and token stride must be multiples of 16 bytes")
    return stride


def _statistic(lse, q, T, Hq) -> None:
    if lse.dtype != torch.float32 or lse.device != q.device or tuple(lse.shape) != (T, Hq) or \
            not lse.is_contiguous():
        raise ValueError(f"lse must be a contiguous float32 [{T}, {Hq}] tensor on {q.device}")


def _like(t, ref, shape, name: str):
    if t.dtype != ref.dtype or t.device != ref.device:
        raise TypeError(f"{name}: dtype or device differs")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: expected shape {tuple(shape)}")
    return t


class AttnPlan:
    """The work items of a packed batch (see attn_plan): one per batch, for every layer."""

    def __init__(self, T, num_seqs, num_q_heads, num_kv_heads, buffer):
        self.T, self.num_seqs = T, num_seqs
        self.num_q_heads, self.num_kv_heads = num_q_heads, num_kv_heads
        self.buffer = buffer  # int32, on the GPU

    def _match(self, q, k, v):
        qs, ks = q.shape, k.shape
        if len(qs) != 3 or len(ks) != 3 or qs[0] != self.T:
            raise ValueError(f"expected q [{self.T}, Hq, D] and k, v [{self.T}, Hkv, D]")
        if qs[1] != self.num_q_heads or ks[1] != self.num_kv_heads:
            raise ValueError(f"the plan was made for {self.num_q_heads} query and "
                             f"{self.num_kv_heads} key/value heads")
        if ks[0] != self.T or ks[2] != qs[2] or v.shape != ks:
            raise ValueError("k and v must be [T, Hkv, D] with q's T and D")
        dtype, device = q.dtype, self.buffer.device
        if k.dtype != dtype or v.dtype != dtype:
            raise TypeError("q, k and v must share one dtype")
        if q.device != device or k.device != device or v.device != device:
            raise TypeError("q, k, v and the plan must be on one device")


def attn_plan(cu_seqlens, T: int, num_q_heads: int, num_kv_heads: int, seqused=None, out=None) -> AttnPlan:
    """The plan of a packed batch of T rows whose sequence s is the rows cu_seqlens[s] ..
    cu_seqlens[s+1] - 1 (int32[B+1] on the GPU; with `seqused`, int32[B], only the first
    seqused[s] of them): one small launch, no host synchronization. It serves every layer
    of the batch, forward and backward.
    `out`: a plan of the same sizes to be written over (for a captured graph's replays)."""
    dev = cu_seqlens.device
    _gpu(dev)
    cu = _index(cu_seqlens, "cu_seqlens", dev)
    num_seqs = cu.numel() - 1
    if num_seqs < 0:
        raise ValueError("cu_seqlens needs at least one entry")
    su = None if seqused is None else _index(seqused, "seqused", dev, num_seqs)
    T, Hq, Hkv = int(T), int(num_q_heads), int(num_kv_heads)
    words = _lib.attn_plan_ints(T, num_seqs, Hq, Hkv)
    if words < 0:
        raise ValueError(f"no plan for T = {T}, {num_seqs} sequences, {Hq} query and {Hkv} "
                         "key/value heads (the query heads must be a multiple)")
    if out is None:
        out = AttnPlan(T, num_seqs, Hq, Hkv, torch.empty(words, dtype=torch.int32, device=dev))
    elif not isinstance(out, AttnPlan):
        raise TypeError("out: expected what attn_plan returns")
    elif (out.T, out.num_seqs, out.num_q_heads, out.num_kv_heads, out.buffer.device) != \
            (T, num_seqs, Hq, Hkv, dev):
        raise ValueError("out: a plan of other sizes or of another device")
    else:
        torch.autograd.graph.increment_version(out.buffer)  # a backward that saved it shall know
    _call(dev, _lib.attn_plan, "attn_plan", _ptr(cu), num_seqs, _ptr(su), T, Hq, Hkv,
          _ptr(out.buffer), out.buffer.numel())
    return out


def attn_fwd(q, k, v, plan: AttnPlan, scale=None, out=None, lse=None, zero_rest=None):
    """Causal attention of the packed batch: q [T, Hq, D], k and v [T, Hkv, D] (bf16 or f16;
    views whose tokens hold their heads contiguously, e.g. parts of a fused projection), D a
    multiple of 8 up to 256, Hq a multiple of Hkv. scale: D ** -0.5 unless given. Returns
    (out [T, Hq, D], lse float32 [T, Hq]), in the given ones or in new ones. zero_rest: whether
    rows of no sequence are written as 0 (-inf in lse) or left as they are; by default new
    outputs are written and given ones left."""
    if not isinstance(plan, AttnPlan):
        raise TypeError("plan: expected what attn_plan returns")
    plan._match(q, k, v)
    T, Hq, D = q.shape
    strides = _heads_last(q, "q"), _heads_last(k, "k"), _heads_last(v, "v")
    if (out is None) != (lse is None):
        raise ValueError("give both out and lse, or neither")
    fill = out is None if zero_rest is None else bool(zero_rest)
    if out is None:
        out = q.new_empty((T, Hq, D))
        lse = q.new_empty((T, Hq), dtype=torch.float32)
        out_stride = 0
    else:
        out_stride = _heads_last(_like(out, q, (T, Hq, D), "out"), "out")
        _statistic(lse, q, T, Hq)
    _call(q.device, _lib.attn_fwd, "attn_fwd", q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
          lse.data_ptr(), T, Hq, k.shape[1], D, *strides, out_stride, plan.buffer.data_ptr(),
          plan.num_seqs, D ** -0.5 if scale is None else float(scale), _DTYPE_CODE[q.dtype], int(fill))
    return out, lse


def attn_bwd(dout, q, k, v, out, lse, plan: AttnPlan, scale=None, dq=None, dk=None, dv=None,
             zero_rest=None):
    """Gradients of attn_fwd for the upstream gradient dout [T, Hq, D], from its inputs and
    outputs and the same scale; D up to 128. Deterministic (no atomics). Returns (dq, dk, dv), in
    the given ones (all three, e.g. parts of one fused gradient) or in new ones. zero_rest as in
    attn_fwd."""
    if not isinstance(plan, AttnPlan):
        raise TypeError("plan: expected what attn_plan returns")
    plan._match(q, k, v)
    T, Hq, D = q.shape
    Hkv = k.shape[1]
    _like(dout, q, (T, Hq, D), "dout")
    _like(out, q, (T, Hq, D), "out")
    _statistic(lse, q, T, Hq)
    strides = [_heads_last(t, name, 128) for t, name in (
        (dout, "dout"), (q, "q"), (k, "k"), (v, "v"), (out, "out"))]
    given = [g is not None for g in (dq, dk, dv)]
    if any(given) != all(given):
        raise ValueError("give all of dq, dk and dv, or none")
    fill = not any(given) if zero_rest is None else bool(zero_rest)
    if not any(given):
        dq, dk, dv = q.new_empty((T, Hq, D)), q.new_empty((T, Hkv, D)), q.new_empty((T, Hkv, D))
        strides += [0, 0, 0]
    else:
        strides += [_heads_last(_like(t, q, (T, h, D), name), name, 128)
                    for t, h, name in ((dq, Hq, "dq"), (dk, Hkv, "dk"), (dv, Hkv, "dv"))]
    scratch = q.new_empty(_lib.attn_bwd_scratch_floats(T, plan.num_seqs, Hq, Hkv, D),
                          dtype=torch.float32)
    _call(q.device, _lib.attn_bwd, "attn_bwd", dout.data_ptr(), q.data_ptr(), k.data_ptr(), v.data_ptr(),
          out.data_ptr(), lse.data_ptr(), scratch.data_ptr(), dq.data_ptr(), dk.data_ptr(),
          dv.data_ptr(), T, Hq, Hkv, D, *strides, plan.buffer.data_ptr(), plan.num_seqs,
          D ** -0.5 if scale is None else float(scale), _DTYPE_CODE[q.dtype], int(fill))
    return dq, dk, dv


# ---------------------------------------------------------------- paged cache

def _caches(k_cache, v_cache, dtype, device):
    """Checked caches [num_pages, page_size, Hkv, D] of one layout; their shape and strides."""
    shape, stride = k_cache.shape, k_cache.stride()
    if k_cache.dtype != dtype or v_cache.dtype != dtype or k_cache.device != device or \
            v_cache.device != device:
        raise TypeError("k_cache or v_cache: dtype or device differs from the new tokens'")
    if len(stride) != 4:
        raise ValueError("k_cache: expected [num_pages, page_size, Hkv, D]")
    if shape != v_cache.shape or stride != v_cache.stride():
        raise ValueError("k_cache and v_cache must have one shape and layout")
    if shape[0] < 1 or shape[1] < 1:
        raise ValueError("the cache needs at least one page of at least one slot")
    if shape[0] > _INT32_MAX or shape[1] > _INT32_MAX:
        raise ValueError("the cache has more pages or slots than int32 numbers name")
    if shape[3] > 1 and stride[3] != 1:
        raise ValueError("the D elements of a cache row must be contiguous")
    return shape, stride


def _table(block_table, num_seqs, device):
    if block_table.dtype != torch.int32 or block_table.device != device or block_table.dim() != 2:
        raise TypeError(f"block_table must be an int32 [B, max_pages] tensor on {device}")
    B, per = block_table.shape
    if B != num_seqs:
        raise ValueError("block_table must have one row per sequence")
    row, step = block_table.stride()
    if per > 1 and step != 1:
        raise ValueError("block_table: a sequence's pages must be contiguous")
    return per, row if B > 1 else per


def kv_append_(k, v, k_cache, v_cache, block_table, cu_seqlens, kv_lens, theta: float, q=None,
               q_out=None, pos_scale: float = 1.0):
    """Append the new tokens' keys (rotated) and values to a paged cache, in place, and rotate
    their queries, in one launch. k, v [T, Hkv, D] and q [T, Hq, D] (bf16, f16 or f32; views
    whose tokens hold their heads contiguously) are the new tokens of B sequences, rows
    cu_seqlens[s] .. cu_seqlens[s+1] - 1 (int32[B+1]) of sequence s, which holds kv_lens[s]
    tokens with them (int32[B]): token i of n goes to position kv_lens[s] - n + i, in page
    block_table[s, position // page_size] (int32 [B, max_pages]) of the caches [num_pages,
    page_size, Hkv, D]. Keys and queries are rotated as qk_apply_ex_ does at that position.
    Tokens at a negative position, of no sequence, behind the table or on a page number that
    is no page are not appended. No two tokens of a call may share a cache row. Returns the
    rotated q, in q_out (a new tensor if None; may be q itself), or None without q."""
    shape, dtype, dev = k.shape, k.dtype, k.device
    if len(shape) != 3 or v.shape != shape:
        raise ValueError("expected k and v [T, Hkv, D]")
    if v.dtype != dtype or v.device != dev:
        raise TypeError("k and v must share one dtype and device")
    k_stride, v_stride = _token_rows(k, "k", _ANY), _token_rows(v, "v", _ANY)
    T, Hkv, D = shape
    Hq, q_stride, out_stride = 0, 0, 0
    if q is not None:
        if q.dtype != dtype or q.device != dev:
            raise TypeError("q: dtype or device differs from k")
        if q.dim() != 3 or q.shape[0] != T or q.shape[2] != D:
            raise ValueError("expected q [T, Hq, D] with k's T and D")
        Hq = q.shape[1]
        if q_out is None:
            q_out, out_stride = q.new_empty((T, Hq, D)), Hq * D
        else:
            out_stride = _token_rows(_like(q_out, q, q.shape, "q_out"), "q_out", _ANY)
        q_stride = _token_rows(q, "q", _ANY)
    elif q_out is not None:
        raise ValueError("q_out without q")
    cache, steps = _caches(k_cache, v_cache, dtype, dev)
    if cache[2] != Hkv or cache[3] != D:
        raise ValueError("the cache must have k's heads and head size")
    if not k_cache.is_contiguous():
        extent = D
        for step, n in sorted(zip(steps[:3], cache)):
            if n > 1 and step < extent:
                raise ValueError("rows of the cache overlap (an expanded tensor cannot be written)")
            extent += (n - 1) * step
    cu = _index(cu_seqlens, "cu_seqlens", dev)
    num_seqs = cu.numel() - 1
    if num_seqs < 0:
        raise ValueError("cu_seqlens needs at least one entry")
    lens = _index(kv_lens, "kv_lens", dev, num_seqs)
    per, table_stride = _table(block_table, num_seqs, dev)
    _call(dev, _lib.kv_append, "kv_append", _ptr(q), _ptr(q_out), k.data_ptr(), v.data_ptr(),
          k_cache.data_ptr(), v_cache.data_ptr(), T, Hq, Hkv, D, q_stride, out_stride, k_stride,
          v_stride, cache[0], cache[1], steps[0], steps[1], steps[2], block_table.data_ptr(), per,
          table_stride, cu.data_ptr(), num_seqs, lens.data_ptr(), float(theta), float(pos_scale),
          _DTYPE_CODE[dtype])
    return q_out


class PagedPlan:
    """How one step of a batch attends to its paged cache (see paged_plan)."""

    def __init__(self, T, num_seqs, num_q_heads, num_kv_heads, buffer):
        self.T, self.num_seqs = T, num_seqs
        self.num_q_heads, self.num_kv_heads = num_q_heads, num_kv_heads
        self.buffer = buffer  # int32, on the GPU


def paged_plan(cu_seqlens, kv_lens, T: int, num_q_heads: int, num_kv_heads: int, out=None) -> PagedPlan:
    """The plan of one step over a paged cache: T new tokens, rows cu_seqlens[s] ..
    cu_seqlens[s+1] - 1 of sequence s (int32[B+1] on the GPU), which holds kv_lens[s] tokens
    with them (int32[B], read now). One small launch, no host synchronization; it serves every
    layer of the step. `out`: a plan of the same sizes to be written over (for the next step,
    or in a captured graph)."""
    dev = cu_seqlens.device
    _gpu(dev)
    cu = _index(cu_seqlens, "cu_seqlens", dev)
    num_seqs = cu.numel() - 1
    if num_seqs < 0:
        raise ValueError("cu_seqlens needs at least one entry")
    lens = _index(kv_lens, "kv_lens", dev, num_seqs)
    T, Hq, Hkv = int(T), int(num_q_heads), int(num_kv_heads)
    words = _lib.paged_plan_ints(T, num_seqs, Hq, Hkv)
    if words < 0:
        raise ValueError(f"no plan for T = {T}, {num_seqs} sequences, {Hq} query and {Hkv} "
                         "key/value heads (the query heads must be a multiple)")
    if out is None:
        out = PagedPlan(T, num_seqs, Hq, Hkv, torch.empty(words, dtype=torch.int32, device=dev))
    elif not isinstance(out, PagedPlan):
        raise TypeError("out: expected what paged_plan returns")
    elif (out.T, out.num_seqs, out.num_q_heads, out.num_kv_heads, out.buffer.device) != \
            (T, num_seqs, Hq, Hkv, dev):
        raise ValueError("out: a plan of other sizes or of another device")
    _call(dev, _lib.paged_plan, "paged_plan", _ptr(cu), num_seqs, _ptr(lens), T, Hq, Hkv,
          _ptr(out.buffer), out.buffer.numel())
    return out


def attn_paged(q, k_cache, v_cache, block_table, plan: PagedPlan, scale=None, out=None, lse=None,
               zero_rest=None):
    """Attention of the new tokens q [T, Hq, D] (bf16 or f16, D a multiple of 8 up to 256) over
    the paged caches [num_pages, page_size, Hkv, D] that hold their sequences (kv_append_),
    causal among themselves; block_table as there, plan from paged_plan. Keys behind the table
    or on a page number that is no page are seen by no query. Returns (out [T, Hq, D], lse
    float32 [T, Hq]), in the given ones or in new ones; a query that sees no key gets 0 (-inf in
    lse). zero_rest, for rows of no sequence, as in attn_fwd."""
    if not isinstance(plan, PagedPlan):
        raise TypeError("plan: expected what paged_plan returns")
    q_stride = _heads_last(q, "q")
    T, Hq, D = q.shape
    if T != plan.T or Hq != plan.num_q_heads or q.device != plan.buffer.device:
        raise ValueError("the plan was made for other new tokens, query heads or another device")
    cache, (page_stride, slot_stride, head_stride, _) = _caches(k_cache, v_cache, q.dtype, q.device)
    num_pages, page_size, Hkv, cache_d = cache
    if Hkv != plan.num_kv_heads or cache_d != D:
        raise ValueError("the cache must have the plan's key/value heads and q's head size")
    if (page_stride | slot_stride | head_stride) % 8 or k_cache.data_ptr() % 16 or v_cache.data_ptr() % 16:
        raise ValueError("the cache's data pointers and strides must be multiples of 16 bytes")
    per, table_stride = _table(block_table, plan.num_seqs, q.device)
    if (out is None) != (lse is None):
        raise ValueError("give both out and lse, or neither")
    fill = out is None if zero_rest is None else bool(zero_rest)
    if out is None:
        out = q.new_empty((T, Hq, D))
        lse = q.new_empty((T, Hq), dtype=torch.float32)
        out_stride = 0
    else:
        out_stride = _heads_last(_like(out, q, (T, Hq, D), "out"), "out")
        _statistic(lse, q, T, Hq)
    space = q.new_empty(_lib.paged_workspace_floats(T, plan.num_seqs, Hq, Hkv, D), dtype=torch.float32)
    _call(q.device, _lib.attn_paged, "attn_paged", q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
          out.data_ptr(), lse.data_ptr(), space.data_ptr(), T, Hq, Hkv, D, q_stride, out_stride,
          num_pages, page_size, page_stride, slot_stride, head_stride, block_table.data_ptr(), per,
          table_stride, plan.buffer.data_ptr(), plan.num_seqs,
          D ** -0.5 if scale is None else float(scale), _DTYPE_CODE[q.dtype], int(fill))
    return out, lse
