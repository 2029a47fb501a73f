"""Attention around the rotary embedding: causal attention over packed sequences (forward
and backward).

Thin binding over the C ABI of ``include/attn.h`` (libattn.so, built by build_attn.py from
``csrc/attn_*.hip``), as the package's other entry points are: it checks
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
_KEY_TILE = 128


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
    for name in ("attn_plan", "attn_fwd", "attn_bwd"):
        getattr(lib, name).restype = i32
    return lib


_lib = _load()


def _check(status: int, what: str) -> None:
    if status != 0:
        from . import RopeError
        raise RopeError(status, what)


def _stream(device: torch.device) -> int:
    return torch.cuda.current_stream(device).cuda_stream


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


def _heads_last(t, name: str, dtypes=(torch.bfloat16, torch.float16)) -> int:
    """Token stride of a [T, H, D] tensor whose tokens hold their heads contiguously."""
    _gpu(t.device)
    if t.dtype not in dtypes:
        raise TypeError(f"{name}: expected " + " or ".join(str(d)[6:] for d in dtypes))
    if t.dim() != 3:
        raise ValueError(f"{name}: expected [T, H, D]")
    T, H, D = t.shape
    if t.numel() == 0:
        return H * D
    if t.stride(2) != 1 or (H > 1 and t.stride(1) != D):
        raise ValueError(f"{name}: the heads of a token must be contiguous "
                         "(stride(2) == 1 and stride(1) == D)")
    stride = t.stride(0) if T > 1 else H * D
    if t.data_ptr() % 16 or stride * t.element_size() % 16:
        raise ValueError(f"{name}: data pointer and token stride must be multiples of 16 bytes")
    return stride


def _head_size(D: int, most: int) -> None:
    if D % 8 or not 8 <= D <= most:
        raise ValueError(f"head size {D}: expected a multiple of 8, 8 .. {most}")


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
        if q.dim() != 3 or k.dim() != 3 or q.shape[0] != self.T:
            raise ValueError(f"expected q [{self.T}, Hq, D] and k, v [{self.T}, Hkv, D]")
        if q.shape[1] * self.num_kv_heads != k.shape[1] * self.num_q_heads:
            raise ValueError("the plan was made for another ratio of query to key/value heads")
        if k.shape[0] != self.T or k.shape[2] != q.shape[2] or v.shape != k.shape:
            raise ValueError("k and v must be [T, Hkv, D] with q's T and D")
        if k.dtype != q.dtype or v.dtype != q.dtype:
            raise TypeError("q, k and v must share one dtype")
        if any(t.device != self.buffer.device for t in (q, k, v)):
            raise TypeError("q, k, v and the plan must be on one device")


def attn_plan(cu_seqlens, T: int, num_q_heads: int, num_kv_heads: int, seqused=None, out=None) -> AttnPlan:
    """The plan of a packed batch of T rows whose sequence s is the rows cu_seqlens[s] ..
    cu_seqlens[s+1] - 1 (int32[B+1] on the GPU; with `seqused`, int32[B], only the first
    seqused[s] of them): one small launch, no host synchronization. It serves every layer
    of the batch, forward and backward, and any head counts of the same ratio.
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
    elif (out.T, out.num_seqs, out.buffer.device) != (T, num_seqs, dev) or \
            out.num_q_heads * Hkv != Hq * out.num_kv_heads:
        raise ValueError("out: a plan of other sizes or of another device")
    with torch.cuda.device(dev):
        _check(_lib.attn_plan(_ptr(cu), num_seqs, _ptr(su), T, Hq, Hkv, _ptr(out.buffer), words,
                              _stream(dev)), "attn_plan")
    return out


def attn_fwd(q, k, v, plan: AttnPlan, scale=None, out=None, lse=None):
    """Causal attention of the packed batch: q [T, Hq, D], k and v [T, Hkv, D] (bf16 or f16;
    views whose tokens hold their heads contiguously, e.g. parts of a fused projection), D a
    multiple of 8 up to 256, Hq a multiple of Hkv. scale: D ** -0.5 unless given. Returns
    (out [T, Hq, D], lse float32 [T, Hq]). Rows of no sequence are 0 (-inf in lse) in new
    outputs; a given `out` and `lse` keep theirs as they are."""
    plan._match(q, k, v)
    strides = [_heads_last(t, name) for t, name in ((q, "q"), (k, "k"), (v, "v"))]
    T, Hq, D = q.shape
    _head_size(D, 256)
    if (out is None) != (lse is None):
        raise ValueError("give both out and lse, or neither")
    fill = out is None
    if fill:
        out = torch.empty((T, Hq, D), dtype=q.dtype, device=q.device)
        lse = torch.empty((T, Hq), dtype=torch.float32, device=q.device)
    _like(out, q, (T, Hq, D), "out")
    if lse.dtype != torch.float32 or lse.device != q.device or tuple(lse.shape) != (T, Hq) or \
            not lse.is_contiguous():
        raise ValueError(f"lse must be a contiguous float32 [{T}, {Hq}] tensor on {q.device}")
    out_stride = _heads_last(out, "out")
    with torch.cuda.device(q.device):
        _check(_lib.attn_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), T, Hq, k.shape[1], D,
                             *strides, out_stride, _ptr(plan.buffer), plan.num_seqs,
                             float(D ** -0.5 if scale is None else scale), _DTYPE_CODE[q.dtype],
                             int(fill), _stream(q.device)), "attn_fwd")
    return out, lse


def attn_bwd(dout, q, k, v, out, lse, plan: AttnPlan, scale=None, dq=None, dk=None, dv=None):
    """Gradients of attn_fwd for the upstream gradient dout [T, Hq, D], from its inputs and
    outputs and the same scale; D up to 128. Deterministic (no atomics). New gradients have
    zeros in rows of no sequence; given dq, dk and dv (all three, e.g. parts of one fused
    gradient) keep theirs as they are. Returns (dq, dk, dv)."""
    plan._match(q, k, v)
    T, Hq, D = q.shape
    Hkv = k.shape[1]
    _head_size(D, 128)
    for t, name in ((dout, "dout"), (out, "out")):
        _like(t, q, (T, Hq, D), name)
    if lse.dtype != torch.float32 or lse.device != q.device or tuple(lse.shape) != (T, Hq) or \
            not lse.is_contiguous():
        raise ValueError(f"lse must be a contiguous float32 [{T}, {Hq}] tensor on {q.device}")
    given = [g is not None for g in (dq, dk, dv)]
    if any(given) != all(given):
        raise ValueError("give all of dq, dk and dv, or none")
    fill = not any(given)
    if fill:
        dq = torch.empty((T, Hq, D), dtype=q.dtype, device=q.device)
        dk = torch.empty((T, Hkv, D), dtype=q.dtype, device=q.device)
        dv = torch.empty_like(dk)
    _like(dq, q, (T, Hq, D), "dq")
    _like(dk, q, (T, Hkv, D), "dk")
    _like(dv, q, (T, Hkv, D), "dv")
    strides = [_heads_last(t, name) for t, name in (
        (dout, "dout"), (q, "q"), (k, "k"), (v, "v"), (out, "out"), (dq, "dq"), (dk, "dk"), (dv, "dv"))]
    scratch = torch.empty((2, T, Hq), dtype=torch.float32, device=q.device)
    with torch.cuda.device(q.device):
        _check(_lib.attn_bwd(_ptr(dout), _ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), _ptr(scratch),
                             _ptr(dq), _ptr(dk), _ptr(dv), T, Hq, Hkv, D, *strides,
                             _ptr(plan.buffer), plan.num_seqs,
                             float(D ** -0.5 if scale is None else scale), _DTYPE_CODE[q.dtype],
                             int(fill), _stream(q.device)), "attn_bwd")
    return dq, dk, dv
