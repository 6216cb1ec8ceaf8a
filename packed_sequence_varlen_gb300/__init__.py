"""GB300 (sm_103a) packed-sequence varlen causal attention.

Python face of the C ABI in ``include/varlen_attn.h``: argument marshalling
only.  PyTorch supplies device memory and the current stream; every step of
the path (planner, metadata, tile scheduler, forward, backward) runs in the
library.  There is no CPU fallback: a missing library raises.

Layout: q [T, Hq, d], k/v [T, Hkv, d] bf16 with the last dim contiguous;
``cu_seqlens`` int32 [B+1] on the device; lse fp32 [Hq, T].
"""
from __future__ import annotations

import contextlib
import ctypes
import math

import numpy as np
import torch

from . import _lib
from ._lib import VarlenError, VaShape, check

__all__ = [
    "pack_next_fit", "pack_best_fit_decreasing", "build_metadata", "validate_cu_seqlens",
    "tile_sizes", "workspace_size", "plan", "varlen_attn_fwd", "varlen_attn_bwd", "varlen_attn",
    "read_status", "VarlenError", "make_shape", "library_path", "loss_targets", "token_ce",
    "IGNORE_INDEX", "unpad_index", "gather_rows", "unpad", "pad", "plan_cross", "varlen_attn_fwd_cross",
    "varlen_attn_bwd_cross", "token_distill", "embed_fwd", "embed_bwd", "embed",
]


def library_path() -> str:
    return _lib.LIB_PATH


# Pointers and streams go to the library as plain integers (ctypes converts them): building torch's
# and ctypes' objects for them costs more host time than the rest of a small call.

def _stream(dev: torch.device | None = None) -> int:
    index = torch._C._cuda_getDevice() if dev is None or dev.index is None else dev.index
    return torch._C._cuda_getCurrentRawStream(index)


def _ptr(t: torch.Tensor | None) -> int:
    return 0 if t is None else t.data_ptr()


def _int32(x) -> int:
    """A window or sink count for the library: a larger one sees no more than the largest (ctypes would
    wrap it around)."""
    return max(-2 ** 31, min(int(x), 2 ** 31 - 1))


def _check_sizes(**sizes):
    for name, n in sizes.items():
        if not 0 <= n < 2 ** 30:
            raise ValueError(f"{name} must be below 2^30")


def _on(dev: torch.device):
    """Makes ``dev`` the current device for a ``with`` block (nothing to do where it is already)."""
    return contextlib.nullcontext() if torch._C._cuda_getDevice() == dev.index else torch.cuda.device(dev)


# ----------------------------------------------------------------- host planner

def _pack(fn, lengths, capacity: int):
    lib = _lib.load()
    src = np.asarray(lengths)
    if src.ndim != 1 or (src.size and src.dtype.kind not in "iu"):
        raise TypeError("lengths: a flat sequence of integers")
    if src.size and (src.min() < np.iinfo(np.int32).min or src.max() > np.iinfo(np.int32).max):
        raise ValueError("lengths: values must fit in int32")
    n = int(src.size)
    arr = np.zeros(max(n, 1), dtype=np.int32)
    arr[:n] = src
    order = np.empty(max(n, 1), dtype=np.int32)
    offs = np.zeros(n + 1, dtype=np.int32)
    npk = ctypes.c_int32(0)
    i32p = ctypes.POINTER(ctypes.c_int32)
    check(getattr(lib, fn)(arr.ctypes.data_as(i32p), n, int(capacity), order.ctypes.data_as(i32p),
                           offs.ctypes.data_as(i32p), ctypes.byref(npk)))
    bounds = offs[:npk.value + 1].tolist()
    flat = order[:n].tolist()
    return [flat[bounds[p]:bounds[p + 1]] for p in range(npk.value)]


def pack_next_fit(lengths, capacity: int):
    """Order-preserving next-fit; packs as lists of document indices."""
    return _pack("varlen_pack_next_fit", lengths, capacity)


def pack_best_fit_decreasing(lengths, capacity: int):
    """Best-fit-decreasing; packs as lists of document indices."""
    return _pack("varlen_pack_best_fit_decreasing", lengths, capacity)


# ----------------------------------------------------------------- metadata

def build_metadata(lengths: torch.Tensor, pad_to: int = 0, T_capacity: int | None = None):
    """Device lengths (int32) -> (cu_seqlens[n+2], position_ids[T], segment_ids[T], max_seqlen[1],
    status[1]), all int32 device tensors.  ``cu_seqlens[n+1] == cu_seqlens[n]`` means no pad."""
    assert lengths.is_cuda and lengths.dtype == torch.int32 and lengths.is_contiguous()
    n = lengths.numel()
    if T_capacity is None:
        T_capacity = max(int(pad_to), 0)
    dev = lengths.device
    cu = torch.empty(n + 2, dtype=torch.int32, device=dev)
    pos = torch.empty(max(T_capacity, 1), dtype=torch.int32, device=dev)
    seg = torch.empty(max(T_capacity, 1), dtype=torch.int32, device=dev)
    mx = torch.empty(1, dtype=torch.int32, device=dev)
    st = torch.empty(1, dtype=torch.int32, device=dev)
    check(_lib.load().varlen_build_metadata(_ptr(lengths), n, int(pad_to), int(T_capacity),
                                            _ptr(cu), _ptr(pos), _ptr(seg), _ptr(mx), _ptr(st),
                                            _stream(dev)))
    return cu, pos[:T_capacity], seg[:T_capacity], mx, st


def validate_cu_seqlens(cu_seqlens: torch.Tensor, T: int, max_seqlen: int,
                        status: torch.Tensor):
    """Enqueue the contract check; a violation sets ``status`` to VA_ERR_BAD_SEQLENS."""
    check(_lib.load().varlen_validate_cu_seqlens(_ptr(cu_seqlens), cu_seqlens.numel() - 1, int(T),
                                                 int(max_seqlen), _ptr(status),
                                                 _stream(cu_seqlens.device)))


def cu_seqlens_from_position_ids(position_ids: torch.Tensor, reset_at_min: bool = False,
                                 strict: bool = False):
    """Device position_ids (int32 [T]) -> (cu_seqlens[T + 1], B[1], max_seqlen[1], status[1]),
    int32 device tensors; cu_seqlens[:B + 1] is the boundary array (unwritten on error)."""
    assert position_ids.is_cuda and position_ids.dtype == torch.int32 and position_ids.is_contiguous()
    T = position_ids.numel()
    dev = position_ids.device
    cu = torch.empty(T + 1, dtype=torch.int32, device=dev)
    B = torch.empty(1, dtype=torch.int32, device=dev)
    mx = torch.empty(1, dtype=torch.int32, device=dev)
    st = torch.empty(1, dtype=torch.int32, device=dev)
    check(_lib.load().varlen_cu_seqlens_from_positions(_ptr(position_ids), T, int(reset_at_min), int(strict),
                                                       _ptr(cu), T + 1, _ptr(B), _ptr(mx), _ptr(st),
                                                       _stream(dev)))
    return cu, B, mx, st


# ----------------------------------------------------------------- shapes, plans

def make_shape(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, B: int, max_seqlen: int,
               out: torch.Tensor | None = None) -> VaShape:
    T, Hq, d = q.shape
    s = VaShape()
    s.T, s.B, s.Hq, s.Hkv, s.d, s.max_seqlen = T, B, Hq, k.shape[1], d, int(max_seqlen)
    s.q_row_stride, s.q_head_stride = q.stride(0), q.stride(1)
    s.k_row_stride, s.k_head_stride = k.stride(0), k.stride(1)
    s.v_row_stride, s.v_head_stride = v.stride(0), v.stride(1)
    o = out if out is not None else q
    s.o_row_stride, s.o_head_stride = o.stride(0), o.stride(1)
    return s


def _contig_shape(T, B, Hq, Hkv, d, max_seqlen) -> VaShape:
    s = VaShape()
    _lib.load().varlen_shape_contiguous(ctypes.byref(s), T, B, Hq, Hkv, d, int(max_seqlen))
    return s


def tile_sizes(kind: int, d: int):
    """(BM, BN) of a tile map kind: 0 forward, 1 backward kv blocks, 2 backward dQ blocks."""
    bm, bn = ctypes.c_int32(), ctypes.c_int32()
    check(_lib.load().varlen_attn_tile_sizes(kind, d, ctypes.byref(bm), ctypes.byref(bn)))
    return bm.value, bn.value


def workspace_size(T, B, Hq, Hkv, d, max_seqlen, for_bwd: bool, window: int | None = None, sinks: int = 0) -> int:
    s = _contig_shape(T, B, Hq, Hkv, d, max_seqlen)
    lib = _lib.load()
    n = lib.varlen_attn_workspace_size_sinks(ctypes.byref(s), -1 if window is None else _int32(window), _int32(sinks),
                                             int(for_bwd))
    if n == 0:  # the shape check failed: the plan entry point reports why
        check(lib.varlen_attn_plan_sinks(ctypes.byref(s), None, 0, 1, -1 if window is None else _int32(window),
                                         _int32(sinks), None, 0, None, None, None))
    return n


def plan(cu_seqlens: torch.Tensor, T: int, Hq: int, Hkv: int, d: int, max_seqlen: int,
         kind: int = 0, causal: bool = True, window: int | None = None, sinks: int = 0):
    """Tile map on the device: (records int32 [n, 4], n).  ``window``: causal local window
    (query i sees keys i - window .. i), None for none; ``sinks``: first tokens of every segment
    that stay visible beyond the window."""
    B = cu_seqlens.numel() - 1
    s = _contig_shape(T, B, Hq, Hkv, d, max_seqlen)
    BM, BN = tile_sizes(kind, d)
    blk = BN if kind == 1 else BM
    heads = Hkv if kind == 1 else Hq
    cap = (T // blk + B) * heads
    tm = torch.empty((max(cap, 1), 4), dtype=torch.int32, device=cu_seqlens.device)
    n = torch.zeros(1, dtype=torch.int32, device=cu_seqlens.device)
    scratch = torch.empty(B + 4, dtype=torch.int32, device=cu_seqlens.device)
    with _on(cu_seqlens.device):
        check(_lib.load().varlen_attn_plan_sinks(ctypes.byref(s), _ptr(cu_seqlens), kind, int(causal),
                                                 -1 if window is None else _int32(window), _int32(sinks), _ptr(tm), cap,
                                                 _ptr(n), _ptr(scratch), _stream(cu_seqlens.device)))
    k = int(n.item())
    return tm[:k], k


def read_status(ws: torch.Tensor) -> int:
    st = ctypes.c_int32(-1)
    check(_lib.load().varlen_read_status(_ptr(ws), ctypes.byref(st), _stream(ws.device)))
    return st.value


def _raise_status(ws: torch.Tensor):
    st = read_status(ws)
    if st != 0:
        raise VarlenError(st, "device-detected error (status word)")


def _check_inputs(*ts):
    for t in ts:
        if not t.is_cuda or t.dtype != torch.bfloat16 or t.dim() != 3 or t.stride(2) != 1:
            raise ValueError("q/k/v/out tensors must be CUDA bf16 [T, H, d] with a contiguous last dim")


# ----------------------------------------------------------------- attention

def varlen_attn_fwd(q, k, v, cu_seqlens, max_seqlen: int, scale: float | None = None,
                    causal: bool = True, out=None, lse=None, workspace=None, check_status=False,
                    window: int | None = None, sinks: int = 0):
    """Forward: returns (out [T,Hq,d] bf16, lse [Hq,T] fp32).  ``window``: causal local window
    (query i sees keys i - window .. i of its segment), None for none.  ``sinks`` (with a
    window): every segment's first tokens that stay visible to all its later queries."""
    win = -1 if window is None else _int32(window)
    _check_inputs(q, k, v)
    T, Hq, d = q.shape
    B = cu_seqlens.numel() - 1
    if out is None:
        out = torch.empty_like(q, memory_format=torch.contiguous_format)
    if lse is None:
        lse = torch.empty((Hq, T), dtype=torch.float32, device=q.device)
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    s = make_shape(q, k, v, B, max_seqlen, out)
    lib = _lib.load()
    need = lib.varlen_attn_workspace_size(ctypes.byref(s), 0)
    if need == 0:  # the shape check failed: the call reports why
        check(lib.varlen_attn_fwd_sinks(_ptr(q), _ptr(k), _ptr(v), _ptr(cu_seqlens), ctypes.byref(s),
                                        scale, int(causal), win, _int32(sinks), _ptr(out), _ptr(lse), _ptr(None), 0,
                                        _stream(q.device)))
    if workspace is None or workspace.numel() < need:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    with _on(q.device):
        check(lib.varlen_attn_fwd_sinks(_ptr(q), _ptr(k), _ptr(v), _ptr(cu_seqlens), ctypes.byref(s), scale,
                                        int(causal), win, _int32(sinks), _ptr(out), _ptr(lse), _ptr(workspace),
                                        workspace.numel(), _stream(q.device)))
    if check_status:
        _raise_status(workspace)
    return out, lse


def varlen_attn_bwd(q, k, v, out, lse, dout, cu_seqlens, max_seqlen: int,
                    scale: float | None = None, causal: bool = True, dq=None, dk=None, dv=None,
                    workspace=None, check_status=False, window: int | None = None, sinks: int = 0):
    """Backward: returns (dq, dk, dv) bf16 with the shapes of q, k, v (``window`` and ``sinks``
    as in the forward that produced out and lse)."""
    _check_inputs(q, k, v, out, dout)
    if out.stride() != dout.stride():
        raise ValueError("out and dout must share strides")
    T, Hq, d = q.shape
    B = cu_seqlens.numel() - 1
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    if dq is None:
        dq = torch.empty_strided(out.shape, out.stride(), dtype=q.dtype, device=q.device)
    if dk is None:
        dk = torch.empty_strided(k.shape, k.stride(), dtype=k.dtype, device=k.device)
    if dv is None:
        dv = torch.empty_strided(k.shape, k.stride(), dtype=k.dtype, device=k.device)
    if dq.stride() != out.stride() or dk.stride() != k.stride() or dv.stride() != k.stride():
        raise ValueError("dq must share out's strides and dk/dv k's strides")
    s = make_shape(q, k, v, B, max_seqlen, out)
    lib = _lib.load()
    win = -1 if window is None else _int32(window)
    need = lib.varlen_attn_workspace_size_sinks(ctypes.byref(s), win, _int32(sinks), 1)
    if workspace is None or workspace.numel() < need:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=q.device)
    with _on(q.device):
        check(lib.varlen_attn_bwd_sinks(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), _ptr(dout),
                                        _ptr(cu_seqlens), ctypes.byref(s), scale, int(causal), win, _int32(sinks),
                                        _ptr(dq), _ptr(dk), _ptr(dv), _ptr(workspace), workspace.numel(),
                                        _stream(q.device)))
    if check_status:
        _raise_status(workspace)
    return dq, dk, dv


class _VarlenAttn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, cu_seqlens, max_seqlen, scale, causal, window, sinks):
        out, lse = varlen_attn_fwd(q, k, v, cu_seqlens, max_seqlen, scale, causal, window=window, sinks=sinks)
        ctx.save_for_backward(q, k, v, out, lse, cu_seqlens)
        ctx.max_seqlen, ctx.scale, ctx.causal, ctx.window, ctx.sinks = max_seqlen, scale, causal, window, sinks
        return out

    @staticmethod
    def backward(ctx, dout):
        q, k, v, out, lse, cu = ctx.saved_tensors
        dout = dout.contiguous() if dout.stride() != out.stride() else dout
        dq, dk, dv = varlen_attn_bwd(q, k, v, out, lse, dout, cu, ctx.max_seqlen, ctx.scale,
                                     ctx.causal, window=ctx.window, sinks=ctx.sinks)
        return dq, dk, dv, None, None, None, None, None, None


def varlen_attn(q, k, v, cu_seqlens, max_seqlen: int, scale: float | None = None,
                causal: bool = True, window: int | None = None, sinks: int = 0):
    """Differentiable packed attention: out [T, Hq, d] (``window``: causal local window;
    ``sinks``: first tokens of every segment that stay visible beyond it)."""
    return _VarlenAttn.apply(q, k, v, cu_seqlens, max_seqlen, scale, causal, window, sinks)


# ----------------------------------------------------------------- cross-attention

def plan_cross(cu_q: torch.Tensor, cu_k: torch.Tensor, Tq: int, Tk: int, Hq: int, Hkv: int, d: int,
               max_seqlen_q: int, kind: int = 0, causal: bool = True):
    """Cross-attention tile map on the device: (records int32 [n, 4], n)."""
    B = cu_q.numel() - 1
    s = _contig_shape(Tq, B, Hq, Hkv, d, max_seqlen_q)
    BM, BN = tile_sizes(kind, d)
    cap = ((Tk // BN) + B) * Hkv if kind == 1 else (Tq // BM + B) * Hq
    tm = torch.empty((max(cap, 1), 4), dtype=torch.int32, device=cu_q.device)
    n = torch.zeros(1, dtype=torch.int32, device=cu_q.device)
    scratch = torch.empty(B + 4, dtype=torch.int32, device=cu_q.device)
    check(_lib.load().varlen_attn_plan_cross(ctypes.byref(s), _ptr(cu_q), _ptr(cu_k), Tk, kind, int(causal),
                                             _ptr(tm), cap, _ptr(n), _ptr(scratch), _stream(cu_q.device)))
    k = int(n.item())
    return tm[:k], k


def varlen_attn_fwd_cross(q, k, v, cu_q, cu_k, max_seqlen_q: int, max_seqlen_k: int, scale: float | None = None,
                          causal: bool = True, out=None, lse=None, workspace=None, check_status=False):
    """Cross-attention forward (q [Tq,Hq,d] against k/v [Tk,Hkv,d], boundaries cu_q / cu_k;
    causal aligned bottom-right): returns (out [Tq,Hq,d] bf16, lse [Hq,Tq] fp32)."""
    _check_inputs(q, k, v)
    Tq, Hq, d = q.shape
    Tk = k.shape[0]
    B = cu_q.numel() - 1
    if out is None:
        out = torch.empty_like(q, memory_format=torch.contiguous_format)
    if lse is None:
        lse = torch.empty((Hq, Tq), dtype=torch.float32, device=q.device)
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    s = make_shape(q, k, v, B, max_seqlen_q, out)
    lib = _lib.load()
    need = lib.varlen_attn_workspace_size_cross(ctypes.byref(s), Tk, 0)
    if workspace is None or workspace.numel() < need:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=q.device)
    check(lib.varlen_attn_fwd_cross(_ptr(q), _ptr(k), _ptr(v), _ptr(cu_q), _ptr(cu_k), ctypes.byref(s), Tk,
                                    int(max_seqlen_k), scale, int(causal), _ptr(out), _ptr(lse), _ptr(workspace),
                                    workspace.numel(), _stream(q.device)))
    if check_status:
        _raise_status(workspace)
    return out, lse


def varlen_attn_bwd_cross(q, k, v, out, lse, dout, cu_q, cu_k, max_seqlen_q: int, max_seqlen_k: int,
                          scale: float | None = None, causal: bool = True, workspace=None, check_status=False):
    """Cross-attention backward: returns (dq, dk, dv) bf16 with the shapes of q, k, v."""
    _check_inputs(q, k, v, out, dout)
    Tq, Hq, d = q.shape
    Tk = k.shape[0]
    B = cu_q.numel() - 1
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    dq = torch.empty_strided(out.shape, out.stride(), dtype=q.dtype, device=q.device)
    dk = torch.empty_strided(k.shape, k.stride(), dtype=k.dtype, device=k.device)
    dv = torch.empty_strided(k.shape, k.stride(), dtype=k.dtype, device=k.device)
    s = make_shape(q, k, v, B, max_seqlen_q, out)
    lib = _lib.load()
    need = lib.varlen_attn_workspace_size_cross(ctypes.byref(s), Tk, 1)
    if workspace is None or workspace.numel() < need:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=q.device)
    check(lib.varlen_attn_bwd_cross(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), _ptr(dout), _ptr(cu_q),
                                    _ptr(cu_k), ctypes.byref(s), Tk, int(max_seqlen_k), scale, int(causal), _ptr(dq),
                                    _ptr(dk), _ptr(dv), _ptr(workspace), workspace.numel(), _stream(q.device)))
    if check_status:
        _raise_status(workspace)
    return dq, dk, dv


# ----------------------------------------------------------------- packed loss

IGNORE_INDEX = -100


def loss_targets(token_ids: torch.Tensor, cu_seqlens: torch.Tensor, ignore_index: int = IGNORE_INDEX):
    """Next-token targets (int32 [T]) of a packed stream of whole documents: pairs formed
    inside each segment, ``ignore_index`` at every segment's last position."""
    if not token_ids.is_cuda or token_ids.dtype != torch.int32 or token_ids.dim() != 1:
        raise ValueError("token_ids must be a CUDA int32 [T] tensor")
    T = token_ids.numel()
    out = torch.empty(T, dtype=torch.int32, device=token_ids.device)
    check(_lib.load().varlen_loss_targets(_ptr(token_ids), _ptr(cu_seqlens), cu_seqlens.numel() - 1, T,
                                          int(ignore_index), _ptr(out), _stream(token_ids.device)))
    return out


def token_ce(logits: torch.Tensor, targets: torch.Tensor, ignore_index: int = IGNORE_INDEX,
             grad: bool | torch.Tensor = True, workspace=None, check_status=False):
    """Token-weighted cross entropy of the packed stream: returns (loss [2] float64 device
    tensor {sum, mean}, count [1] int32, grad or None).  ``logits`` is CUDA fp32 or bf16
    [T, V] with a contiguous last dim; ``grad`` True allocates d(mean)/d(logits) like
    ``logits``, a tensor receives it, False skips it.

    An eligible target outside [0, V), or no eligible target at all, is an error found on the device: loss is
    NaN and the gradient is left as it was (uninitialised where this call allocated it);
    ``check_status`` raises."""
    if not logits.is_cuda or logits.dim() != 2 or logits.stride(1) != 1 or \
            logits.dtype not in (torch.float32, torch.bfloat16):
        raise ValueError("logits must be a CUDA fp32/bf16 [T, V] tensor with a contiguous last dim")
    T, V = logits.shape
    dev = logits.device
    if grad is True:
        g = torch.empty_like(logits, memory_format=torch.contiguous_format)
    elif grad is False or grad is None:
        g = None
    else:
        g = grad
        if g.shape != logits.shape or g.dtype != logits.dtype or g.stride(1) != 1:
            raise ValueError("grad must match logits in shape and dtype, with a contiguous last dim")
    lib = _lib.load()
    need = lib.varlen_token_ce_workspace_size(T)
    if workspace is None or workspace.numel() < need:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    loss = torch.empty(2, dtype=torch.float64, device=dev)
    count = torch.empty(1, dtype=torch.int32, device=dev)
    check(lib.varlen_token_ce(_ptr(logits), 1 if logits.dtype == torch.bfloat16 else 0, logits.stride(0),
                              _ptr(targets), T, V, int(ignore_index), _ptr(loss), _ptr(count), _ptr(g),
                              g.stride(0) if g is not None else 0, _ptr(workspace), workspace.numel(),
                              _stream(dev)))
    if check_status:
        _raise_status(workspace)
    return loss, count, g


def _same_device(dev, **tensors):
    for name, t in tensors.items():
        if t is not None and t.device != dev:
            raise ValueError(f"{name} must be on {dev}")


def _row_stride(t: torch.Tensor) -> int:
    """Elements between rows of a 2-D tensor (one row: any stride is right)."""
    return t.stride(0) if t.shape[0] > 1 else max(t.shape[1], 1)


def token_distill(logits: torch.Tensor, teacher_ids: torch.Tensor, teacher_logits: torch.Tensor,
                  targets: torch.Tensor | None = None, temperature: float = 1.0,
                  ignore_index: int = IGNORE_INDEX, grad: bool | torch.Tensor = True, workspace=None,
                  check_status=False):
    """Distillation from a teacher's top logits over the packed stream: returns (loss [2] fp32
    device tensor {sum, mean}, count [1] int32, grad or None).

    ``logits`` CUDA fp32 or bf16 [T, V]; ``teacher_ids`` int32 [T, K] (negative: no entry) and
    ``teacher_logits`` fp32 or bf16 [T, K]; ``targets`` int32 [T] whose ``ignore_index`` rows are
    skipped (None: no row is).  Row t adds temperature^2 KL(p || q), p the softmax of its teacher
    logits / temperature, q the softmax of all its logits / temperature; the mean is over the rows
    that have a target and an entry.  ``grad`` True allocates d(mean)/d(logits) like ``logits``, a
    tensor receives it (``logits`` itself is fine), False skips it.

    An eligible row that lists a class >= V, or no eligible row at all, is an error found on the device: loss is
    NaN and the gradient is left as it was (uninitialised where this call allocated it);
    ``check_status`` raises."""
    if not logits.is_cuda or logits.dim() != 2 or logits.stride(1) != 1 or \
            logits.dtype not in (torch.float32, torch.bfloat16):
        raise ValueError("logits must be a CUDA fp32/bf16 [T, V] tensor with a contiguous last dim")
    T, V = logits.shape
    _check_sizes(T=T, V=V)
    dev = logits.device
    if teacher_ids.dim() != 2 or teacher_ids.dtype != torch.int32 or teacher_ids.shape[0] != T or \
            (teacher_ids.shape[1] > 1 and teacher_ids.stride(1) != 1):
        raise ValueError("teacher_ids must be an int32 [T, K] tensor with a contiguous last dim")
    if teacher_logits.shape != teacher_ids.shape or teacher_logits.dtype not in (torch.float32, torch.bfloat16) or \
            (teacher_logits.shape[1] > 1 and teacher_logits.stride(1) != 1):
        raise ValueError("teacher_logits must be fp32/bf16 in teacher_ids' shape, with a contiguous last dim")
    if targets is not None and (targets.dtype != torch.int32 or targets.shape != (T,) or not targets.is_contiguous()):
        raise ValueError("targets must be a contiguous int32 [T] tensor")
    if grad is True:
        g = torch.empty_like(logits, memory_format=torch.contiguous_format)
    elif grad is False or grad is None:
        g = None
    else:
        g = grad
        if g.shape != logits.shape or g.dtype != logits.dtype or g.stride(1) != 1:
            raise ValueError("grad must match logits in shape and dtype, with a contiguous last dim")
    _same_device(dev, teacher_ids=teacher_ids, teacher_logits=teacher_logits, targets=targets, grad=g,
                 workspace=workspace)
    lib = _lib.load()
    need = lib.varlen_token_distill_workspace_size(T)
    if workspace is None or workspace.numel() < need:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    loss = torch.empty(2, dtype=torch.float32, device=dev)
    count = torch.empty(1, dtype=torch.int32, device=dev)
    with _on(dev):
        check(lib.varlen_token_distill(_ptr(logits), int(logits.dtype == torch.bfloat16), _row_stride(logits),
                                       _ptr(teacher_ids), _row_stride(teacher_ids), _ptr(teacher_logits),
                                       int(teacher_logits.dtype == torch.bfloat16), _row_stride(teacher_logits),
                                       _ptr(targets), T, V, teacher_ids.shape[1], int(ignore_index),
                                       float(temperature), _ptr(loss), _ptr(count), _ptr(g),
                                       _row_stride(g) if g is not None else 0, _ptr(workspace), workspace.numel(),
                                       _stream(dev)))
    if check_status:
        _raise_status(workspace)
    return loss, count, g


# ----------------------------------------------------------------- embedding

_FLOATS = (torch.float32, torch.bfloat16)


def _check_rows(name: str, t: torch.Tensor):
    if not t.is_cuda or t.dim() != 2 or t.dtype not in _FLOATS or (t.shape[1] > 1 and t.stride(1) != 1):
        raise ValueError(f"{name} must be a CUDA fp32/bf16 matrix with a contiguous last dim")


def _check_ids(ids: torch.Tensor, dev: torch.device):
    if ids.dim() != 1 or ids.dtype != torch.int32 or not ids.is_contiguous():
        raise ValueError("ids must be a contiguous int32 [T] tensor")
    _same_device(dev, ids=ids)


def embed_fwd(table: torch.Tensor, ids: torch.Tensor, scale: float = 1.0, out: torch.Tensor | None = None,
              check_status=False) -> torch.Tensor:
    """out[t] = scale * table[ids[t]]: ``table`` CUDA fp32/bf16 [V, D], ``ids`` int32 [T] (negative:
    a zero row; >= V: a row of NaN, an error with ``check_status``); out [T, D] in table's dtype."""
    _check_rows("table", table)
    dev = table.device
    _check_ids(ids, dev)
    (V, D), T = table.shape, ids.numel()
    _check_sizes(T=T, V=V, D=D)
    if out is None:
        out = torch.empty((T, D), dtype=table.dtype, device=dev)
    else:
        _check_rows("out", out)
        if out.shape != (T, D) or out.dtype != table.dtype:
            raise ValueError("out must be [T, D] in table's dtype")
        _same_device(dev, out=out)
    status = torch.zeros(1, dtype=torch.int32, device=dev) if check_status else None
    with _on(dev):
        check(_lib.load().varlen_embed_fwd(_ptr(table), int(table.dtype == torch.bfloat16), _row_stride(table),
                                           _ptr(ids) if T else 0, T, V, D, float(scale),
                                           _ptr(out) if T else _ptr(table), _row_stride(out), _ptr(status),
                                           _stream(dev)))
    if check_status and int(status.item()) != 0:
        raise VarlenError(int(status.item()), "embed_fwd: a token id is past the table")
    return out


def embed_bwd(dout: torch.Tensor, ids: torch.Tensor, num_rows: int, scale: float = 1.0,
              dtable: torch.Tensor | None = None, accumulate: bool = False, workspace=None,
              check_status=False) -> torch.Tensor:
    """Gradient of ``embed_fwd`` with respect to its table: dtable[v] = scale * the sum of dout[t]
    over ids[t] == v, in token order (deterministic), [num_rows, D].  ``dtable`` None allocates
    one in dout's dtype; an fp32 or bf16 tensor receives it, and with ``accumulate`` it is added to
    what the tensor holds (rows whose id does not occur are not touched)."""
    _check_rows("dout", dout)
    dev = dout.device
    _check_ids(ids, dev)
    T, D, V = ids.numel(), dout.shape[1], int(num_rows)
    _check_sizes(T=T, num_rows=V, D=D)
    if dout.shape[0] != T:
        raise ValueError("dout must be [T, D] with ids [T]")
    if dtable is None:
        if accumulate:
            raise ValueError("accumulate needs the tensor to add to")
        dtable = torch.empty((V, D), dtype=dout.dtype, device=dev)
    else:
        _check_rows("dtable", dtable)
        if dtable.shape != (V, D):
            raise ValueError("dtable must be [num_rows, D]")
    _same_device(dev, dtable=dtable, workspace=workspace)
    lib = _lib.load()
    need = lib.varlen_embed_bwd_workspace_size(T, D)
    if workspace is None or workspace.numel() < need:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=dev)
    with _on(dev):
        check(lib.varlen_embed_bwd(_ptr(dout) if T else 0, int(dout.dtype == torch.bfloat16),
                                   _row_stride(dout), _ptr(ids) if T else 0, T, V, D, float(scale),
                                   _ptr(dtable), int(dtable.dtype == torch.bfloat16), _row_stride(dtable),
                                   int(bool(accumulate)), _ptr(workspace), workspace.numel(), _stream(dev)))
    if check_status:
        _raise_status(workspace)
    return dtable


class _Embed(torch.autograd.Function):
    @staticmethod
    def forward(ctx, table, ids, scale):
        ctx.save_for_backward(ids)
        ctx.num_rows, ctx.scale = table.shape[0], scale
        return embed_fwd(table, ids, scale)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dout):
        (ids,) = ctx.saved_tensors
        return embed_bwd(dout.contiguous(), ids, ctx.num_rows, ctx.scale), None, None


def embed(table: torch.Tensor, ids: torch.Tensor, scale: float = 1.0) -> torch.Tensor:
    """Differentiable token embedding of the packed stream: scale * table[ids], [T, D]."""
    return _Embed.apply(table, ids, scale)


# ----------------------------------------------------------------- padded-batch bridge

def unpad_index(mask: torch.Tensor):
    """Padded batch -> packed stream.  ``mask`` CUDA [Bp, S] (nonzero = real token).  Returns
    (indices [Bp*S], inverse [Bp*S], cu_seqlens [Bp+1] (int32 device tensors), T, max_seqlen);
    T and max_seqlen are read back to the host (one synchronisation), as the attention calls
    take them on the host.  A row without real tokens raises (status VA_ERR_BAD_SEQLENS)."""
    if not mask.is_cuda or mask.dim() != 2:
        raise ValueError("mask must be a CUDA [Bp, S] tensor")
    m = mask.to(torch.int32).contiguous()
    Bp, S = m.shape
    dev = m.device
    indices = torch.empty(Bp * S, dtype=torch.int32, device=dev)
    inverse = torch.empty(Bp * S, dtype=torch.int32, device=dev)
    cu = torch.empty(Bp + 1, dtype=torch.int32, device=dev)
    small = torch.empty(3, dtype=torch.int32, device=dev)  # T, max_seqlen, status
    check(_lib.load().varlen_unpad_index(_ptr(m), Bp, S, _ptr(indices), _ptr(inverse), _ptr(cu),
                                         ctypes.c_void_p(small.data_ptr()),
                                         ctypes.c_void_p(small.data_ptr() + 4),
                                         ctypes.c_void_p(small.data_ptr() + 8), _stream(dev)))
    T, mx, st = (int(x) for x in small.cpu())
    if st != 0:
        raise VarlenError(st, "unpad_index: a row has no real token")
    return indices, inverse, cu, T, mx


def gather_rows(src: torch.Tensor, row_map: torch.Tensor, n_rows: int) -> torch.Tensor:
    """dst[i] = src[row_map[i]] (a zero row where row_map[i] < 0) for i < n_rows; rows are
    src's trailing dims (contiguous, a multiple of 16 bytes)."""
    if not src.is_cuda or src.dim() < 1 or not src[0].is_contiguous():
        raise ValueError("src must be a CUDA tensor with contiguous rows")
    row_bytes = src[0].numel() * src.element_size()
    dst = torch.empty((n_rows,) + tuple(src.shape[1:]), dtype=src.dtype, device=src.device)
    check(_lib.load().varlen_gather_rows(_ptr(src), src.stride(0) * src.element_size(), _ptr(row_map), n_rows,
                                         row_bytes, _ptr(dst), dst.stride(0) * dst.element_size(),
                                         _stream(src.device)))
    return dst


def unpad(x: torch.Tensor, indices: torch.Tensor, T: int) -> torch.Tensor:
    """[Bp, S, ...] -> [T, ...]: the real tokens in row-major order."""
    return gather_rows(x.reshape((-1,) + tuple(x.shape[2:])), indices, T)


def pad(y: torch.Tensor, inverse: torch.Tensor, Bp: int, S: int) -> torch.Tensor:
    """[T, ...] -> [Bp, S, ...]: each token back to its padded position, zeros in the padding."""
    return gather_rows(y, inverse, Bp * S).reshape((Bp, S) + tuple(y.shape[1:]))
