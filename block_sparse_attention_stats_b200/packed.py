"""Python binding of libpisa's packed sequences and paged key/value cache.

As in api.py, each function has the name of the C entry point it calls
(include/pisa.h) and only checks and passes on its arguments.  Packed tensors
are [H, T, d] with d contiguous and any head and row strides that are multiples
of 8 (a [T, H, d] tensor is passed as its transpose(0, 1), a slice of a fused
projection as it is); caches are [num_pages, Hkv, page_size, d] likewise.  The
work runs on the tensors' device, on `stream` or that device's current stream.
A `scale` of None or 0 is 1 / sqrt(d), as in the C calls.  varlen_attention is
differentiable; results of the pisa_ calls carry no graph.
"""
from __future__ import annotations

import ctypes
from typing import Optional, Tuple

import torch
from torch.autograd import forward_ad

from . import _lib as L
from .api import _check, _require

_DT = {torch.bfloat16: L.PISA_BF16, torch.float16: L.PISA_F16}


def _elsewhere(t, stream):
    """A context that makes the tensor's device and `stream` current, so that memory allocated for
    the call belongs to the stream that uses it; None where they are already."""
    if not t.is_cuda:
        raise ValueError("tensors must live on a CUDA device")
    if stream is None:
        if _current_device() == t.get_device():
            return None
        with torch.cuda.device(t.device):
            stream = torch.cuda.current_stream()
    elif stream.device != t.device:
        raise ValueError(f"stream is on {stream.device}, the tensors are on {t.device}")
    # entering a stream's context makes its device current too
    return torch.cuda.stream(stream)


def _current_stream(index) -> int:
    return torch.cuda.current_stream(index).cuda_stream


# the current device, and the stream's handle without an object around it, where this torch has them
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", _current_stream)


def _strides_ok(t) -> bool:
    return t.stride(-1) == 1 and t.data_ptr() % 16 == 0 and all(
        n <= 1 or (s >= t.shape[-1] and s % 8 == 0) for n, s in zip(t.shape[:-1], t.stride()))


def _refuse(t, dims, like, name):
    """Why t cannot be taken; returns where only the quick check failed it."""
    if t.dim() != dims or t.dtype != like.dtype or t.device != like.device:
        raise ValueError(f"{name} must be a {like.dtype} tensor of {dims} dimensions on {like.device}")
    if t.numel() and not _strides_ok(t):
        raise ValueError(f"{name} must have a contiguous last dimension, the other strides multiples "
                         "of 8 that are no smaller than it, and 16-byte aligned data")


def _rows(t, like, name) -> L.PisaRows:
    ptr = t.data_ptr()
    st = t.stride()
    if len(st) == 3:
        h, r, c = st
        if (c == 1 and not (h | r) & 7 and not ptr & 15 and h >= 8 and r >= 8 and t.dtype is like.dtype
                and t.get_device() == like.get_device()):
            d = t.shape[2]
            if h >= d and r >= d:
                return L.PisaRows(ptr, h, r)
    _refuse(t, 3, like, name)
    return L.PisaRows(ptr, st[0], st[1])


def _pages(t, like, name) -> L.PisaPages:
    ptr = t.data_ptr()
    st = t.stride()
    if len(st) == 4:
        p, h, r, c = st
        if (c == 1 and not (p | h | r) & 7 and not ptr & 15 and t.dtype is like.dtype
                and t.get_device() == like.get_device()):
            d = t.shape[3]
            if p >= d and h >= d and r >= d:
                return L.PisaPages(ptr, p, h, r)
    _refuse(t, 4, like, name)
    return L.PisaPages(ptr, st[0], st[1], st[2])


def _dense(t, shape, dtype, name, like) -> Optional[int]:
    """Pointer of a dense array of that shape on like's device (None for None)."""
    if t is None:
        return None
    if (t.dtype is not dtype or t.shape != shape or not t.is_contiguous()
            or t.get_device() != like.get_device()):
        if t.device != like.device:
            raise ValueError(f"{name} must live on {like.device}")
        _require(t, shape, dtype, name)
    return t.data_ptr()


def _ints(t, shape, name, like):
    if t is None:
        raise ValueError(f"{name} is needed")
    return _dense(t, shape, torch.int32, name, like)


def _heads(q, k, v):
    qs, ks = q.shape, k.shape
    if len(qs) != 3 or len(ks) != 3 or ks != v.shape or qs[1:] != ks[1:]:
        raise ValueError("q must be [Hq, T, d] and k, v [Hkv, T, d]")
    if q.dtype not in _DT:
        raise ValueError("q, k, v must share dtype bf16 or float16")
    hq, T, d = qs
    hkv = ks[0]
    if hkv == 0 or hq == 0 or hq % hkv:
        raise ValueError("the number of query heads must be a multiple of the number of key heads")
    return hq, T, d, hkv


_sizes = {}


def _scratch(workspace, size, like, *args):
    """(tensor, pointer, bytes) of the call's scratch memory; size(*args) bytes are needed."""
    if workspace is None:
        need = _sizes.get((size, args))
        if need is None:
            if len(_sizes) > 1000:
                _sizes.clear()
            need = _sizes[size, args] = getattr(L.load(), size)(*args)
        workspace = torch.empty(need, dtype=torch.uint8, device=like.device)
        return workspace, workspace.data_ptr(), need
    if workspace.device != like.device or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on {like.device}")
    return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()


# ---- packed sequences -----------------------------------------------------------

def pisa_varlen_attention(q, k, v, cu_seqlens, causal: bool = True, scale: Optional[float] = None,
                          out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                          out_f32: Optional[torch.Tensor] = None,
                          workspace: Optional[torch.Tensor] = None, stream=None,
                          zero_tail: bool = False) -> torch.Tensor:
    """Attention of every sequence of a packed batch over itself: q [Hq, T, d], k and v
    [Hkv, T, d] (bf16 or float16), cu_seqlens int32 [B + 1] on the device.  `lse` (float32
    [Hq, T]) and `out_f32` (float32 [Hq, T, d]) are written if given; the backward needs both.
    Rows of `out` that belong to no sequence (behind the last, before the first) keep what they held,
    or become zero with `zero_tail`."""
    Hq, T, d, Hkv = _heads(q, k, v)
    away = _elsewhere(q, stream)
    if away is not None:
        with away:
            return pisa_varlen_attention(q, k, v, cu_seqlens, causal, scale, out, lse, out_f32, workspace,
                                         zero_tail=zero_tail)
    B = cu_seqlens.numel() - 1
    if out is None:
        out = torch.empty_like(q)
    elif out.shape != q.shape:
        raise ValueError("out must have the shape of q")
    ws, ptr, size = _scratch(workspace, "pisa_varlen_attention_workspace_bytes", q, Hq, Hkv, d)
    status = L.load().pisa_varlen_attention(
        _rows(q, q, "q"), _rows(k, q, "k"), _rows(v, q, "v"), _DT[q.dtype],
        _ints(cu_seqlens, (B + 1,), "cu_seqlens", q), B, T, Hq, Hkv, d, 0.0 if scale is None else float(scale),
        (L.PISA_CAUSAL if causal else 0) | (L.PISA_ZERO_TAIL if zero_tail else 0), _rows(out, q, "out"),
        _dense(lse, (Hq, T), torch.float32, "lse", q),
        _dense(out_f32, (Hq, T, d), torch.float32, "out_f32", q), ptr, size, _current_stream(q.get_device()))
    if status:
        _check("pisa_varlen_attention", status)
    return out


def pisa_varlen_attention_bwd(q, k, v, dout, lse, out_f32, cu_seqlens, causal: bool = True,
                              scale: Optional[float] = None,
                              grads: Optional[Tuple[torch.Tensor, torch.Tensor, torch.Tensor]] = None,
                              workspace: Optional[torch.Tensor] = None, stream=None,
                              zero_tail: bool = False):
    """Gradients (dq, dk, dv) of pisa_varlen_attention (bf16), from the lse and out_f32 of one
    forward call that was given both."""
    Hq, T, d, Hkv = _heads(q, k, v)
    if dout.shape != q.shape:
        raise ValueError("dout must have the shape of q")
    if lse is None or out_f32 is None:
        raise ValueError("the backward takes the forward's lse and out_f32")
    away = _elsewhere(q, stream)
    if away is not None:
        with away:
            return pisa_varlen_attention_bwd(q, k, v, dout, lse, out_f32, cu_seqlens, causal, scale, grads,
                                             workspace, zero_tail=zero_tail)
    B = cu_seqlens.numel() - 1
    dq, dk, dv = grads if grads is not None else (torch.empty_like(q), torch.empty_like(k), torch.empty_like(v))
    if dq.shape != q.shape or dk.shape != k.shape or dv.shape != v.shape:
        raise ValueError("grads must have the shapes of q, k, v")
    ws, ptr, size = _scratch(workspace, "pisa_varlen_attention_bwd_workspace_bytes", q, T, Hq, Hkv, d)
    status = L.load().pisa_varlen_attention_bwd(
        _rows(q, q, "q"), _rows(k, q, "k"), _rows(v, q, "v"), _rows(dout, q, "dout"), _DT[q.dtype],
        _dense(lse, (Hq, T), torch.float32, "lse", q),
        _dense(out_f32, (Hq, T, d), torch.float32, "out_f32", q),
        _ints(cu_seqlens, (B + 1,), "cu_seqlens", q), B, T, Hq, Hkv, d, 0.0 if scale is None else float(scale),
        (L.PISA_CAUSAL if causal else 0) | (L.PISA_ZERO_TAIL if zero_tail else 0), _rows(dq, q, "dq"),
        _rows(dk, q, "dk"), _rows(dv, q, "dv"), ptr, size, _current_stream(q.get_device()))
    if status:
        _check("pisa_varlen_attention_bwd", status)
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
    if t.is_contiguous() and not t.data_ptr() & 15 and not t.shape[-1] & 7:
        return t
    return t if t.numel() == 0 or _strides_ok(t) else t.contiguous()


def varlen_attention(q, k, v, cu_seqlens, causal: bool = True,
                     scale: Optional[float] = None) -> torch.Tensor:
    """Attention over packed sequences, differentiable with respect to q, k and v (bf16; float16
    without gradients; no forward-mode derivative).  Rows that belong to no sequence are zero, and so are their gradients.
    A training step can be captured into a CUDA graph; as with any autograd function, no eager
    autograd graph of the same leaves may be alive then (autograd would make the capture wait for
    the stream that graph was built on)."""
    if any(forward_ad.unpack_dual(x).tangent is not None for x in (q, k, v)):
        raise ValueError("varlen_attention has no forward-mode derivative")
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
    pages, Hkv, ps, d = _caches(k_cache, v_cache, q)
    if q.dim() != 3 or q.shape[2] != d or block_table.dim() != 2:
        raise ValueError("q must be [Hq, T, d] with the caches' d, block_table [B, width]")
    away = _elsewhere(q, stream)
    if away is not None:
        with away:
            return pisa_paged_attention(q, k_cache, v_cache, block_table, cu_seqlens, kv_lens, scale, out, lse,
                                        workspace)
    Hq, T, _ = q.shape
    B, width = block_table.shape
    if out is None:
        out = torch.empty_like(q)
    elif out.shape != q.shape:
        raise ValueError("out must have the shape of q")
    ws, ptr, size = _scratch(workspace, "pisa_paged_attention_workspace_bytes", q, Hq, Hkv, d)
    status = L.load().pisa_paged_attention(
        _rows(q, q, "q"), _pages(k_cache, q, "k_cache"), _pages(v_cache, q, "v_cache"), _DT[q.dtype], pages, ps,
        _ints(block_table, (B, width), "block_table", q), width, _ints(cu_seqlens, (B + 1,), "cu_seqlens", q),
        _ints(kv_lens, (B,), "kv_lens", q), B, T, Hq, Hkv, d, 0.0 if scale is None else float(scale),
        _rows(out, q, "out"), _dense(lse, (Hq, T), torch.float32, "lse", q), ptr, size,
        _current_stream(q.get_device()))
    if status:
        _check("pisa_paged_attention", status)
    return out


def _page_step(past_lens, new_lens, block_table, free_pages, num_free, page_size, T, out):
    if block_table.dim() != 2 or free_pages.dim() != 1:
        raise ValueError("block_table must be [B, width], free_pages one-dimensional")
    like = block_table
    B, width = like.shape
    if out is None:
        dev = like.device
        # the small results share one allocation
        small, slots = (torch.empty(2 * B + 2, dtype=torch.int32, device=dev),
                        torch.empty(T, dtype=torch.int64, device=dev))
        cu, kv, left = small.split((B + 1, B, 1))
        out = dict(slots=slots, cu_seqlens=cu, kv_lens=kv, num_free=left)
        at = small.data_ptr()
        results = slots.data_ptr(), at, at + 4 * (B + 1), at + 4 * (2 * B + 1)
    else:
        results = (_dense(out["slots"], (T,), torch.int64, "slots", like),
                   _ints(out["cu_seqlens"], (B + 1,), "cu_seqlens", like),
                   _ints(out["kv_lens"], (B,), "kv_lens", like), _ints(out["num_free"], (1,), "num_free", like))
    step = L.PisaPageStep(
        _ints(past_lens, (B,), "past_lens", like), _ints(new_lens, (B,), "new_lens", like), B, T,
        _ints(like, (B, width), "block_table", like), width, page_size,
        _ints(free_pages, free_pages.shape, "free_pages", like), free_pages.numel(),
        _ints(num_free, (1,), "num_free", like), *results)
    return step, out


def pisa_page_plan(past_lens, new_lens, block_table, free_pages, num_free, page_size: int, T: int,
                   out: Optional[dict] = None, stream=None) -> dict:
    """One step's bookkeeping: enters new pages into block_table [B, width] and returns
    dict(slots int64 [T], cu_seqlens [B + 1], kv_lens [B], num_free [1]).  Pages come from the end
    of free_pages[: num_free]; `out` may pass preallocated results.  All lengths int32."""
    away = _elsewhere(block_table, stream)
    if away is not None:
        with away:
            return pisa_page_plan(past_lens, new_lens, block_table, free_pages, num_free, page_size, T, out)
    step, out = _page_step(past_lens, new_lens, block_table, free_pages, num_free, page_size, T, out)
    status = L.load().pisa_page_plan(ctypes.byref(step), _current_stream(block_table.get_device()))
    if status:
        _check("pisa_page_plan", status)
    return out


def pisa_page_write(k, v, slots, k_cache, v_cache, stream=None) -> None:
    """Rows t of k and v [Hkv, T, d] to slot slots[t] (int64; negative: left out) of the caches."""
    pages, Hkv, ps, d = _caches(k_cache, v_cache, k)
    shape = k.shape
    if len(shape) != 3 or shape != v.shape or shape[0] != Hkv or shape[2] != d:
        raise ValueError("k and v must be [Hkv, T, d] with the caches' Hkv and d")
    away = _elsewhere(k, stream)
    if away is not None:
        with away:
            return pisa_page_write(k, v, slots, k_cache, v_cache)
    T = shape[1]
    status = L.load().pisa_page_write(
        _rows(k, k, "k"), _rows(v, k, "v"), _DT[k.dtype], _dense(slots, (T,), torch.int64, "slots", k), T, Hkv, d,
        _pages(k_cache, k, "k_cache"), _pages(v_cache, k, "v_cache"), pages, ps, _current_stream(k.get_device()))
    if status:
        _check("pisa_page_write", status)


def pisa_paged_step(q, k, v, k_cache, v_cache, past_lens, new_lens, block_table, free_pages, num_free,
                    scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
                    plan: Optional[dict] = None, lse: Optional[torch.Tensor] = None,
                    workspace: Optional[torch.Tensor] = None, stream=None):
    """The whole step of a server: plan, write of k and v, attention of q over the pages.
    Returns (out, plan), plan as from pisa_page_plan; `plan` may pass preallocated results."""
    pages, Hkv, ps, d = _caches(k_cache, v_cache, q)
    Hq, T, dq, hk = _heads(q, k, v)
    if dq != d or hk != Hkv:
        raise ValueError("q, k, v must have the caches' Hkv and d")
    if block_table.device != q.device:
        raise ValueError(f"block_table must live on {q.device}")
    away = _elsewhere(q, stream)
    if away is not None:
        with away:
            return pisa_paged_step(q, k, v, k_cache, v_cache, past_lens, new_lens, block_table, free_pages,
                                   num_free, scale, out, plan, lse, workspace)
    if out is None:
        out = torch.empty_like(q)
    elif out.shape != q.shape:
        raise ValueError("out must have the shape of q")
    step, plan = _page_step(past_lens, new_lens, block_table, free_pages, num_free, ps, T, plan)
    ws, ptr, size = _scratch(workspace, "pisa_paged_attention_workspace_bytes", q, Hq, Hkv, d)
    status = L.load().pisa_paged_step(
        ctypes.byref(step), _rows(q, q, "q"), _rows(k, q, "k"), _rows(v, q, "v"),
        _pages(k_cache, q, "k_cache"), _pages(v_cache, q, "v_cache"), _DT[q.dtype], pages, Hq, Hkv, d,
        0.0 if scale is None else float(scale), _rows(out, q, "out"),
        _dense(lse, (Hq, T), torch.float32, "lse", q), ptr, size, _current_stream(q.get_device()))
    if status:
        _check("pisa_paged_step", status)
    return out, plan
