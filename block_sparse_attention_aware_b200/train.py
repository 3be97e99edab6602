"""Training through the block-sparse attention (the C ABI in
include/fvattn_train.h): the forward that keeps the log-sum-exp, the gradient
calls, and the layer as a differentiable torch function.

Conventions are those of fvattn.py: buffers have exactly the documented shape,
argument errors raise before any launch, every call is asynchronous on its
stream.  Tensors of a call live on one device; the call runs there even when
another device is current.  The kv lists are constants: no gradient flows into
routing.
"""
from __future__ import annotations

import contextlib
import ctypes
import math
from typing import Optional

import torch

from . import fvattn
from .fvattn import Geom, _check, _expect, _ptr, _raster, _tiled

EXPORTED = ("fvattn_sparse_attn_lse", "fvattn_sparse_attn_bwd_workspace_size", "fvattn_sparse_attn_bwd")

_lib = None


def load():
    """libfvattn.so with this module's signatures declared (raises if missing)."""
    global _lib
    if _lib is None:
        L = fvattn.load()
        P, I, S, F = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, ctypes.c_float
        G = ctypes.POINTER(Geom)
        L.fvattn_sparse_attn_lse.argtypes = [G, P, P, P, P, P, F, P, P, P, P, S, P]
        L.fvattn_sparse_attn_lse.restype = I
        L.fvattn_sparse_attn_bwd_workspace_size.argtypes = [G]
        L.fvattn_sparse_attn_bwd_workspace_size.restype = S
        L.fvattn_sparse_attn_bwd.argtypes = [G] + [P] * 8 + [F] + [P] * 4 + [S, P]
        L.fvattn_sparse_attn_bwd.restype = I
        _lib = L
    return _lib


@contextlib.contextmanager
def _on(device, stream):
    """Run a call on `device` and on `stream` (None: that device's current
    stream); yields the stream handle.  Outputs and workspaces made inside
    belong to that stream."""
    with torch.cuda.device(device):
        if stream is None:
            yield ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)
        else:
            with torch.cuda.stream(stream):
                yield ctypes.c_void_p(stream.cuda_stream)


def _same_device(first: torch.Tensor, **others):
    for name, t in others.items():
        if t is not None and t.device != first.device:
            raise ValueError(f"{name}: on {t.device}, the call's first tensor is on {first.device}")


def _need(name: str, t, shape, dtype):
    if t is None:
        raise ValueError(f"{name} is required")
    _expect(name, t, shape, dtype)


def _expect_workspace(ws: torch.Tensor, size: int):
    if not ws.is_cuda or not ws.is_contiguous() or ws.dtype != torch.uint8 or ws.numel() < size:
        raise ValueError(f"workspace: expected a contiguous CUDA uint8 tensor of at least {size} elements")


def _expect_lists(g: Geom, kv_idx, kv_cnt):
    _need("kv_idx", kv_idx, (g.B, g.H, g.nb, g.nb), torch.int32)
    _need("kv_cnt", kv_cnt, (g.B, g.H, g.nb), torch.int32)


def sparse_attn_lse(g: Geom, qt, kt, vt, kv_idx, kv_cnt, scale: Optional[float] = None,
                    out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                    sm_stats: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None, stream=None):
    """fvattn_sparse_attn_lse: (tiled O, lse [B, H, Npad] fp32).  A row with
    kv_cnt = 0 gets O = 0, lse = -inf.  `workspace` as fvattn.attn_workspace."""
    for name, t in (("qt", qt), ("kt", kt), ("vt", vt)):
        _need(name, t, _tiled(g), torch.bfloat16)
    _expect_lists(g, kv_idx, kv_cnt)
    _expect("out", out, _tiled(g), torch.bfloat16)
    _expect("lse", lse, (g.B, g.H, g.Npad), torch.float32)
    _same_device(qt, kt=kt, vt=vt, kv_idx=kv_idx, kv_cnt=kv_cnt, out=out, lse=lse, sm_stats=sm_stats,
                 workspace=workspace)
    if sm_stats is not None:
        _expect("sm_stats", sm_stats, (2 * fvattn.num_sms(),), torch.int64)
    L = load()
    if workspace is not None:
        _expect_workspace(workspace, L.fvattn_attn_workspace_size(ctypes.byref(g)))
    with _on(qt.device, stream) as s:
        out = fvattn.tiled_empty(g, qt.device) if out is None else out
        lse = torch.empty((g.B, g.H, g.Npad), dtype=torch.float32, device=qt.device) if lse is None else lse
        workspace = fvattn.attn_workspace(g, qt.device) if workspace is None else workspace
        _check("fvattn_sparse_attn_lse",
               L.fvattn_sparse_attn_lse(ctypes.byref(g), _ptr(qt), _ptr(kt), _ptr(vt), _ptr(kv_idx), _ptr(kv_cnt),
                                        1.0 / math.sqrt(g.D) if scale is None else float(scale), _ptr(out), _ptr(lse),
                                        _ptr(sm_stats), _ptr(workspace), workspace.numel(), s))
    return out, lse


def bwd_workspace(g: Geom, device="cuda") -> torch.Tensor:
    """A workspace for sparse_attn_bwd.  Calls that may overlap on the GPU
    need one each (as do two captured graphs that may run at the same time)."""
    n = load().fvattn_sparse_attn_bwd_workspace_size(ctypes.byref(g))
    return torch.empty(max(n, 256), dtype=torch.uint8, device=device)


def sparse_attn_bwd(g: Geom, qt, kt, vt, ot, dot, lse, kv_idx, kv_cnt, scale: Optional[float] = None,
                    dq: Optional[torch.Tensor] = None, dk: Optional[torch.Tensor] = None,
                    dv: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None, stream=None):
    """fvattn_sparse_attn_bwd: tiled (dQ, dK, dV) from the tensors of a
    sparse_attn_lse call and the tiled gradient `dot` of its output, whose
    padding rows are zero as fvattn.reorder writes them."""
    for name, t in (("qt", qt), ("kt", kt), ("vt", vt), ("ot", ot), ("dot", dot)):
        _need(name, t, _tiled(g), torch.bfloat16)
    _need("lse", lse, (g.B, g.H, g.Npad), torch.float32)
    _expect_lists(g, kv_idx, kv_cnt)
    inputs = [t.data_ptr() for t in (qt, kt, vt, ot, dot)]
    outputs = [t.data_ptr() for t in (dq, dk, dv) if t is not None]
    for name, t in (("dq", dq), ("dk", dk), ("dv", dv)):
        _expect(name, t, _tiled(g), torch.bfloat16)
    if len(set(outputs)) < len(outputs) or set(outputs) & set(inputs):
        raise ValueError("dq, dk and dv must be distinct buffers and no input")
    _same_device(qt, kt=kt, vt=vt, ot=ot, dot=dot, lse=lse, kv_idx=kv_idx, kv_cnt=kv_cnt, dq=dq, dk=dk, dv=dv,
                 workspace=workspace)
    L = load()
    if workspace is not None:
        _expect_workspace(workspace, L.fvattn_sparse_attn_bwd_workspace_size(ctypes.byref(g)))
    with _on(qt.device, stream) as s:
        dq, dk, dv = (fvattn.tiled_empty(g, qt.device) if t is None else t for t in (dq, dk, dv))
        workspace = bwd_workspace(g, qt.device) if workspace is None else workspace
        _check("fvattn_sparse_attn_bwd",
               L.fvattn_sparse_attn_bwd(ctypes.byref(g), _ptr(qt), _ptr(kt), _ptr(vt), _ptr(ot), _ptr(dot), _ptr(lse),
                                        _ptr(kv_idx), _ptr(kv_cnt),
                                        1.0 / math.sqrt(g.D) if scale is None else float(scale), _ptr(dq), _ptr(dk),
                                        _ptr(dv), _ptr(workspace), workspace.numel(), s))
    return dq, dk, dv


class _Attention(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, g, order, tiles, kv_idx, kv_cnt, scale):
        with torch.cuda.device(q.device):
            qt, kt = tiles if tiles is not None else (fvattn.reorder(g, q), fvattn.reorder(g, k))
            vt = fvattn.reorder(g, v)
            ot, lse = sparse_attn_lse(g, qt, kt, vt, kv_idx, kv_cnt, scale)
            out = fvattn.inverse_reorder(g, ot)
        ctx.g, ctx.order, ctx.scale = g, order, scale   # order: the block-order table that g points to
        ctx.save_for_backward(qt, kt, vt, ot, lse, kv_idx, kv_cnt)
        return out

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, do):
        g = ctx.g
        qt, kt, vt, ot, lse, kv_idx, kv_cnt = ctx.saved_tensors
        with torch.cuda.device(qt.device):
            dot = fvattn.reorder(g, do.contiguous())
            grads = sparse_attn_bwd(g, qt, kt, vt, ot, dot, lse, kv_idx, kv_cnt, ctx.scale)
            dq, dk, dv = (fvattn.inverse_reorder(g, t) if need else None
                          for t, need in zip(grads, ctx.needs_input_grad))
        return dq, dk, dv, None, None, None, None, None, None


def attention(g: Geom, q, k, v, kv_idx, kv_cnt, scale: Optional[float] = None, order=None) -> torch.Tensor:
    """Differentiable block-sparse attention of raster q, k, v ([B, N, H, D]
    bf16) on given kv lists: raster O.  The lists are kept for the backward
    pass, and must hold the same values then.  `order`: the table of a
    geometry made with fvattn.with_order, kept alive with the call."""
    for name, t in (("q", q), ("k", k), ("v", v)):
        _need(name, t, _raster(g), torch.bfloat16)
    _expect_lists(g, kv_idx, kv_cnt)
    _same_device(q, k=k, v=v, kv_idx=kv_idx, kv_cnt=kv_cnt)
    if g.order and order is None:
        raise ValueError("a geometry with a block order needs its table: pass order=")
    return _Attention.apply(q, k, v, g, order, None, kv_idx, kv_cnt, scale)


class TrainLayer:
    """One attention layer for training: reorder, route, sparse attention and
    inverse reorder of raster q, k, v, differentiable in q, k and v (the lists
    that routing picks are constants).  Every call has tiles, lists and
    statistics of its own, so several calls may be alive before their backward
    passes, on one stream or several."""

    def __init__(self, g: Geom, p: float, k: int, scale: Optional[float] = None, device="cuda", order: str = "raster"):
        if order not in ("raster", "hilbert"):
            raise ValueError(f"block order {order!r}")
        self.order_table = fvattn.block_order(g, device) if order == "hilbert" else None
        self.g = fvattn.with_order(g, self.order_table)
        self.p, self.k = p, k
        self.scale = 1.0 / math.sqrt(g.D) if scale is None else scale

    def route(self, q, k):
        """(tiled Q, tiled K, RouteOut) of raster q and k, in buffers of their own."""
        return fvattn.reorder_route(self.g, q.detach(), k.detach(), self.p, self.k, self.scale)

    def __call__(self, q, k, v) -> torch.Tensor:
        for name, t in (("q", q), ("k", k), ("v", v)):
            _need(name, t, _raster(self.g), torch.bfloat16)
        _same_device(q, k=k, v=v)
        with torch.cuda.device(q.device):
            qt, kt, routed = self.route(q, k)
        return _Attention.apply(q, k, v, self.g, self.order_table, (qt, kt), routed.kv_idx, routed.kv_cnt, self.scale)
