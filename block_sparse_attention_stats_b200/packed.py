"""Python binding of libpisa's packed sequences and paged key/value cache.

As in api.py, each function has the name of the C entry point it calls
(include/pisa.h) and only checks and passes on its arguments.  Packed tensors
are [H, T, d] with d contiguous and any head and row strides that are multiples
of 8 (a [T, H, d] tensor is passed as its transpose(0, 1), a slice of a fused
projection as it is); caches are [num_pages, Hkv, page_size, d] likewise.  The
work runs on the tensors' device, on `stream` or that device's current stream.
"""
from __future__ import annotations

import contextlib
import ctypes
from typing import Optional, Tuple

import torch

from . import _lib as L
from .api import _check, _require

_DT = {torch.bfloat16: L.PISA_BF16, torch.float16: L.PISA_F16}


@contextlib.contextmanager
def _on(device, stream):
    """Makes `device` and `stream` current, so that memory allocated for the call belongs to the
    stream that uses it; yields the stream's handle."""
    if device.type != "cuda":
        raise ValueError("tensors must live on a CUDA device")
    if stream is not None and stream.device != device:
        raise ValueError(f"stream is on {stream.device}, the tensors are on {device}")
    here = torch.cuda.current_device() == device.index
    if stream is None and here:
        yield torch.cuda.current_stream(device).cuda_stream
    else:
        with torch.cuda.device(device):
            with torch.cuda.stream(stream or torch.cuda.current_stream(device)):
                yield (stream or torch.cuda.current_stream(device)).cuda_stream


def _strides_ok(t) -> bool:
    return t.stride(-1) == 1 and t.data_ptr() % 16 == 0 and all(
        n <= 1 or (s >= t.shape[-1] and s % 8 == 0) for n, s in zip(t.shape[:-1], t.stride()))


def _tensor(t, dims, like, name):
    if t.dim() != dims or t.dtype != like.dtype or t.device != like.device:
        raise ValueError(f"{name} must be a {like.dtype} tensor of {dims} dimensions on {like.device}")
    if t.numel() and not _strides_ok(t):
        raise ValueError(f"{name} must have a contiguous last dimension, the other strides multiples "
                         "of 8 that are no smaller than it, and 16-byte aligned data")


def _rows(t, like, name) -> L.PisaRows:
    _tensor(t, 3, like, name)
    return L.PisaRows(t.data_ptr(), t.stride(0), t.stride(1))


def _pages(t, like, name) -> L.PisaPages:
    _tensor(t, 4, like, name)
    return L.PisaPages(t.data_ptr(), t.stride(0), t.stride(1), t.stride(2))


def _ints(t, shape, name, device, dtype=torch.int32):
    if t.device != device:
        raise ValueError(f"{name} must live on {device}")
    _require(t, shape, dtype, name)
    return t.data_ptr()


def _heads(q, k, v):
    if q.dim() != 3 or k.dim() != 3 or k.shape != v.shape or q.shape[1:] != k.shape[1:]:
        raise ValueError("q must be [Hq, T, d] and k, v [Hkv, T, d]")
    if q.dtype not in _DT:
        raise ValueError("q, k, v must share dtype bf16 or float16")
    if k.shape[0] == 0 or q.shape[0] == 0 or q.shape[0] % k.shape[0]:
        raise ValueError("the number of query heads must be a multiple of the number of key heads")
    return (*q.shape, k.shape[0])


def _scratch(workspace, need, device):
    if workspace is None:
        return torch.empty(need, dtype=torch.uint8, device=device)
    if workspace.device != device or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on {device}")
    return workspace


def _size(t) -> int:
    return t.numel() * t.element_size()


def _f32(t, shape, name, device) -> Optional[int]:
    if t is None:
        return None
    if t.device != device:
        raise ValueError(f"{name} must live on {device}")
    _require(t, shape, torch.float32, name)
    return t.data_ptr()


# ---- packed sequences -----------------------------------------------------------

def pisa_varlen_attention(q, k, v, cu_seqlens, causal: bool = True, scale: Optional[float] = None,
                          out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                          out_f32: Optional[torch.Tensor] = None,
                          workspace: Optional[torch.Tensor] = None, stream=None,
                          zero_tail: bool = False) -> torch.Tensor:
    """Attention of every sequence of a packed batch over itself: q [Hq, T, d], k and v
    [Hkv, T, d] (bf16 or float16), cu_seqlens int32 [B + 1] on the device.  `lse` (float32
    [Hq, T]) and `out_f32` (float32 [Hq, T, d]) are written if given; the backward needs both.
    Rows of `out` behind the last sequence keep what they held, or become zero with `zero_tail`."""
    lib = L.load()
    Hq, T, d, Hkv = _heads(q, k, v)
    B = cu_seqlens.numel() - 1
    with _on(q.device, stream) as st:
        out = torch.empty_like(q) if out is None else out
        if out.shape != q.shape:
            raise ValueError("out must have the shape of q")
        ws = _scratch(workspace, lib.pisa_varlen_attention_workspace_bytes(Hq, Hkv, d), q.device)
        flags = (L.PISA_CAUSAL if causal else 0) | (L.PISA_ZERO_TAIL if zero_tail else 0)
        _check("pisa_varlen_attention", lib.pisa_varlen_attention(
            _rows(q, q, "q"), _rows(k, q, "k"), _rows(v, q, "v"), _DT[q.dtype],
            _ints(cu_seqlens, (B + 1,), "cu_seqlens", q.device), B, T, Hq, Hkv, d,
            0.0 if scale is None else float(scale), flags, _rows(out, q, "out"),
            _f32(lse, (Hq, T), "lse", q.device), _f32(out_f32, (Hq, T, d), "out_f32", q.device),
            ws.data_ptr(), _size(ws), st))
    return out


def pisa_varlen_attention_bwd(q, k, v, dout, lse, out_f32, cu_seqlens, causal: bool = True,
                              scale: Optional[float] = None,
                              grads: Optional[Tuple[torch.Tensor, torch.Tensor, torch.Tensor]] = None,
                              workspace: Optional[torch.Tensor] = None, stream=None,
                              zero_tail: bool = False):
    """Gradients (dq, dk, dv) of pisa_varlen_attention (bf16), from the lse and out_f32 of one
    forward call that was given both."""
    lib = L.load()
    Hq, T, d, Hkv = _heads(q, k, v)
    if dout.shape != q.shape:
        raise ValueError("dout must have the shape of q")
    if lse is None or out_f32 is None:
        raise ValueError("the backward takes the forward's lse and out_f32")
    B = cu_seqlens.numel() - 1
    with _on(q.device, stream) as st:
        dq, dk, dv = grads if grads is not None else (torch.empty_like(x) for x in (q, k, v))
        if dq.shape != q.shape or dk.shape != k.shape or dv.shape != v.shape:
            raise ValueError("grads must have the shapes of q, k, v")
        ws = _scratch(workspace, lib.pisa_varlen_attention_bwd_workspace_bytes(T, Hq, Hkv, d), q.device)
        flags = (L.PISA_CAUSAL if causal else 0) | (L.PISA_ZERO_TAIL if zero_tail else 0)
        _check("pisa_varlen_attention_bwd", lib.pisa_varlen_attention_bwd(
            _rows(q, q, "q"), _rows(k, q, "k"), _rows(v, q, "v"), _rows(dout, q, "dout"),
            _DT[q.dtype], _f32(lse, (Hq, T), "lse", q.device),
            _f32(out_f32, (Hq, T, d), "out_f32", q.device),
            _ints(cu_seqlens, (B + 1,), "cu_seqlens", q.device), B, T, Hq, Hkv, d,
            0.0 if scale is None else float(scale), flags, _rows(dq, q, "dq"), _rows(dk, q, "dk"),
            _rows(dv, q, "dv"), ws.data_ptr(), _size(ws), st))
    return dq, dk, dv


class _VarlenAttention(torch.autograd.Function):
    """Packed attention with its backward (every step in libpisa)."""

    @staticmethod
    def forward(ctx, q, k, v, cu_seqlens, causal, scale):
        Hq, T, d, _ = _heads(q, k, v)
        f = dict(dtype=torch.float32, device=q.device)
        lse, o32 = torch.empty((Hq, T), **f), torch.empty((Hq, T, d), **f)
        out = pisa_varlen_attention(q, k, v, cu_seqlens, causal, scale, lse=lse, out_f32=o32,
                                    zero_tail=True)
        ctx.save_for_backward(q, k, v, lse, o32, cu_seqlens)
        ctx.causal, ctx.scale = causal, scale
        return out

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dout):
        q, k, v, lse, o32, cu = ctx.saved_tensors
        dq, dk, dv = pisa_varlen_attention_bwd(q, k, v, _laid_out(dout), lse, o32, cu, ctx.causal,
                                               ctx.scale, zero_tail=True)
        return dq, dk, dv, None, None, None


def _laid_out(t):
    """t itself where the kernels can read it in place, else a contiguous copy."""
    return t if t.numel() == 0 or _strides_ok(t) else t.contiguous()


def varlen_attention(q, k, v, cu_seqlens, causal: bool = True,
                     scale: Optional[float] = None) -> torch.Tensor:
    """Attention over packed sequences, differentiable with respect to q, k and v (bf16; float16
    without gradients).  Rows behind the last sequence are zero, and so are their gradients."""
    q, k, v = (_laid_out(x) for x in (q, k, v))
    if torch.is_grad_enabled() and any(x.requires_grad for x in (q, k, v)):
        if q.dtype != torch.bfloat16:
            raise ValueError("varlen_attention trains on bf16 q, k, v")
        return _VarlenAttention.apply(q, k, v, cu_seqlens, causal, scale)
    return pisa_varlen_attention(q, k, v, cu_seqlens, causal, scale, zero_tail=True)


# ---- the paged cache ----------------------------------------------------------------

def _caches(k_cache, v_cache, like):
    if k_cache.dim() != 4 or k_cache.shape != v_cache.shape:
        raise ValueError("k_cache and v_cache must be [num_pages, Hkv, page_size, d] with equal shapes")
    if like.dtype not in _DT:
        raise ValueError("the tensors must share dtype bf16 or float16")
    return k_cache.shape


def pisa_paged_attention(q, k_cache, v_cache, block_table, cu_seqlens, kv_lens,
                         scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
                         lse: Optional[torch.Tensor] = None,
                         workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Attention of the newest tokens of every request, q [Hq, T, d], over its pages: the tokens
    cu_seqlens[b] .. cu_seqlens[b + 1] - 1 are the last of request b's kv_lens[b] positions.
    block_table int32 [B, width], cu_seqlens int32 [B + 1], kv_lens int32 [B]."""
    lib = L.load()
    pages, Hkv, ps, d = _caches(k_cache, v_cache, q)
    if q.dim() != 3 or q.shape[2] != d or block_table.dim() != 2:
        raise ValueError("q must be [Hq, T, d] with the caches' d, block_table [B, width]")
    Hq, T, _ = q.shape
    B, width = block_table.shape
    with _on(q.device, stream) as st:
        out = torch.empty_like(q) if out is None else out
        if out.shape != q.shape:
            raise ValueError("out must have the shape of q")
        ws = _scratch(workspace, lib.pisa_paged_attention_workspace_bytes(Hq, Hkv, d), q.device)
        _check("pisa_paged_attention", lib.pisa_paged_attention(
            _rows(q, q, "q"), _pages(k_cache, q, "k_cache"), _pages(v_cache, q, "v_cache"),
            _DT[q.dtype], pages, ps, _ints(block_table, (B, width), "block_table", q.device), width,
            _ints(cu_seqlens, (B + 1,), "cu_seqlens", q.device),
            _ints(kv_lens, (B,), "kv_lens", q.device), B, T, Hq, Hkv, d,
            0.0 if scale is None else float(scale), _rows(out, q, "out"),
            _f32(lse, (Hq, T), "lse", q.device), ws.data_ptr(), _size(ws), st))
    return out


def _page_step(past_lens, new_lens, block_table, free_pages, num_free, page_size, T, out):
    if block_table.dim() != 2 or free_pages.dim() != 1:
        raise ValueError("block_table must be [B, width], free_pages one-dimensional")
    dev = block_table.device
    B, width = block_table.shape
    if out is None:
        i32 = dict(dtype=torch.int32, device=dev)
        out = dict(slots=torch.empty(T, dtype=torch.int64, device=dev),
                   cu_seqlens=torch.empty(B + 1, **i32), kv_lens=torch.empty(B, **i32),
                   num_free=torch.empty(1, **i32))
    step = L.PisaPageStep(
        _ints(past_lens, (B,), "past_lens", dev), _ints(new_lens, (B,), "new_lens", dev), B, T,
        _ints(block_table, (B, width), "block_table", dev), width, page_size,
        _ints(free_pages, free_pages.shape, "free_pages", dev), free_pages.numel(),
        _ints(num_free, (1,), "num_free", dev),
        _ints(out["slots"], (T,), "slots", dev, torch.int64),
        _ints(out["cu_seqlens"], (B + 1,), "cu_seqlens", dev),
        _ints(out["kv_lens"], (B,), "kv_lens", dev), _ints(out["num_free"], (1,), "num_free", dev))
    return step, out


def pisa_page_plan(past_lens, new_lens, block_table, free_pages, num_free, page_size: int, T: int,
                   out: Optional[dict] = None, stream=None) -> dict:
    """One step's bookkeeping: enters new pages into block_table [B, width] and returns
    dict(slots int64 [T], cu_seqlens [B + 1], kv_lens [B], num_free [1]).  Pages come from the end
    of free_pages[: num_free]; `out` may pass preallocated results.  All lengths int32."""
    lib = L.load()
    with _on(block_table.device, stream) as st:
        step, out = _page_step(past_lens, new_lens, block_table, free_pages, num_free, page_size, T, out)
        _check("pisa_page_plan", lib.pisa_page_plan(ctypes.byref(step), st))
    return out


def pisa_page_write(k, v, slots, k_cache, v_cache, stream=None) -> None:
    """Rows t of k and v [Hkv, T, d] to slot slots[t] (int64; negative: left out) of the caches."""
    lib = L.load()
    pages, Hkv, ps, d = _caches(k_cache, v_cache, k)
    if k.dim() != 3 or k.shape != v.shape or k.shape[0] != Hkv or k.shape[2] != d:
        raise ValueError("k and v must be [Hkv, T, d] with the caches' Hkv and d")
    T = k.shape[1]
    with _on(k.device, stream) as st:
        _check("pisa_page_write", lib.pisa_page_write(
            _rows(k, k, "k"), _rows(v, k, "v"), _DT[k.dtype],
            _ints(slots, (T,), "slots", k.device, torch.int64), T, Hkv, d,
            _pages(k_cache, k, "k_cache"), _pages(v_cache, k, "v_cache"), pages, ps, st))


def pisa_paged_step(q, k, v, k_cache, v_cache, past_lens, new_lens, block_table, free_pages, num_free,
                    scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
                    plan: Optional[dict] = None, lse: Optional[torch.Tensor] = None,
                    workspace: Optional[torch.Tensor] = None, stream=None):
    """The whole step of a server: plan, write of k and v, attention of q over the pages.
    Returns (out, plan), plan as from pisa_page_plan; `plan` may pass preallocated results."""
    lib = L.load()
    pages, Hkv, ps, d = _caches(k_cache, v_cache, q)
    Hq, T, dq, hk = _heads(q, k, v)
    if dq != d or hk != Hkv:
        raise ValueError("q, k, v must have the caches' Hkv and d")
    if block_table.device != q.device:
        raise ValueError(f"block_table must live on {q.device}")
    with _on(q.device, stream) as st:
        out = torch.empty_like(q) if out is None else out
        if out.shape != q.shape:
            raise ValueError("out must have the shape of q")
        step, plan = _page_step(past_lens, new_lens, block_table, free_pages, num_free, ps, T, plan)
        ws = _scratch(workspace, lib.pisa_paged_attention_workspace_bytes(Hq, Hkv, d), q.device)
        _check("pisa_paged_step", lib.pisa_paged_step(
            ctypes.byref(step), _rows(q, q, "q"), _rows(k, q, "k"), _rows(v, q, "v"),
            _pages(k_cache, q, "k_cache"), _pages(v_cache, q, "v_cache"), _DT[q.dtype], pages, Hq, Hkv,
            d, 0.0 if scale is None else float(scale), _rows(out, q, "out"),
            _f32(lse, (Hq, T), "lse", q.device), ws.data_ptr(), _size(ws), st))
    return out, plan
