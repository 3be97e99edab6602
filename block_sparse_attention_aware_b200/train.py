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

from . import build, fvattn
from .fvattn import Geom, _check, _raster

EXPORTED = ("fvattn_sparse_attn_lse", "fvattn_sparse_attn_bwd_workspace_size", "fvattn_sparse_attn_bwd")

_lib = None
_fast = None      # the extension that serves a call's plain case (csrc/binding.cpp)


def native():
    """The extension over the C ABI, which checks and marshals a plain call in
    2 us and answers NotImplemented to any other (raises if it is missing or
    was built for another torch)."""
    global _fast
    if _fast is None:
        remedy = "run `python -m block_sparse_attention_aware_b200.build`"
        try:
            from . import _native
        except ImportError as e:
            raise ImportError(f"_native.so is not built for this torch: {remedy}") from e
        if _native.target != build.native_target():
            raise ImportError(f"_native.so was built for {_native.target}, this is {build.native_target()}: {remedy}")
        _fast = _native
    return _fast


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


# The current stream's handle of a device.  torch.cuda.current_stream makes a
# Stream object for it, which takes 3 us of a call's 12.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda index: torch.cuda.current_stream(index).cuda_stream)


class _on:
    """Run a call on `device` and on `stream` (None: that device's current
    stream); the value is the stream handle.  Outputs and workspaces made
    inside belong to that stream."""
    __slots__ = ("device", "stream", "outer")

    def __init__(self, device: torch.device, stream):
        self.device, self.stream, self.outer = device, stream, None

    def __enter__(self) -> int:
        if self.stream is None and torch.cuda.current_device() == self.device.index:   # nothing to switch
            return _raw_stream(self.device.index)
        self.outer = contextlib.ExitStack()
        self.outer.enter_context(torch.cuda.device(self.device))
        stream = torch.cuda.current_stream(self.device) if self.stream is None else self.stream
        if stream.device != self.device:
            self.outer.close()
            raise ValueError(f"stream: on {stream.device}, the call's tensors are on {self.device}")
        self.outer.enter_context(torch.cuda.stream(stream))
        return stream.cuda_stream

    def __exit__(self, *exc):
        if self.outer is not None:
            self.outer.close()


def _device(name: str, t) -> torch.device:
    """The device of a call, that of its first tensor."""
    if t is None:
        raise ValueError(f"{name} is required")
    if not t.is_cuda:
        raise ValueError(f"{name}: expected a CUDA tensor, got one on {t.device}")
    return t.device


def _need(name: str, t, shape, dtype, device):
    """The kernels read and write dense buffers of exactly this shape."""
    if t is None:
        raise ValueError(f"{name} is required")
    if t.dtype is not dtype or t.shape != shape or t.device != device or not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous {dtype} tensor of shape {tuple(shape)} on {device}, got "
                         f"{t.dtype} {tuple(t.shape)} on {t.device} (contiguous={t.is_contiguous()})")


def _check_call(what: str, rc: int, workspace, size):
    """Raise for a call's error; `size()` is the workspace that it needed."""
    if rc == fvattn.ERR_INVALID and workspace is not None and workspace.numel() < size():
        raise ValueError(f"workspace: expected at least {size()} bytes, got {workspace.numel()}")
    _check(what, rc)


def _need_workspace(ws, device):
    if ws.dtype is not torch.uint8 or ws.device != device or not ws.is_contiguous():
        raise ValueError(f"workspace: expected a contiguous uint8 tensor on {device}")


def _scale(g: Geom, scale) -> float:
    scale = 1.0 / math.sqrt(g.D) if scale is None else float(scale)
    if not (0.0 < scale < math.inf):
        raise ValueError(f"scale: expected a positive finite number, got {scale}")
    return scale


def sparse_attn_lse(g: Geom, qt, kt, vt, kv_idx, kv_cnt, scale: Optional[float] = None,
                    out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                    sm_stats: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None, stream=None):
    """fvattn_sparse_attn_lse: (tiled O, lse [B, H, Npad] fp32).  A row with
    kv_cnt = 0 gets O = 0, lse = -inf.  `workspace` as fvattn.attn_workspace."""
    if stream is None and sm_stats is None:
        done = (_fast or native()).sparse_attn_lse(g, qt, kt, vt, kv_idx, kv_cnt, None if scale is None else float(scale),
                                                   out, lse, workspace)
        if done is not NotImplemented:
            return done
    dev = _device("qt", qt)
    B, H, nb, Npad = g.B, g.H, g.nb, g.Npad
    tiled = (B, H, Npad, g.D)
    for name, t in (("qt", qt), ("kt", kt), ("vt", vt)):
        _need(name, t, tiled, torch.bfloat16, dev)
    _need("kv_idx", kv_idx, (B, H, nb, nb), torch.int32, dev)
    _need("kv_cnt", kv_cnt, (B, H, nb), torch.int32, dev)
    if out is not None:
        _need("out", out, tiled, torch.bfloat16, dev)
        if out.data_ptr() in (qt.data_ptr(), kt.data_ptr(), vt.data_ptr()):
            raise ValueError("out must not be an input")
    if lse is not None:
        _need("lse", lse, (B, H, Npad), torch.float32, dev)
    if sm_stats is not None:
        _need("sm_stats", sm_stats, (2 * fvattn.num_sms(),), torch.int64, dev)
    if workspace is not None:
        _need_workspace(workspace, dev)
    scale = _scale(g, scale)
    L = load()
    with _on(dev, stream) as s:
        out = torch.empty(tiled, dtype=torch.bfloat16, device=dev) if out is None else out
        lse = torch.empty((B, H, Npad), dtype=torch.float32, device=dev) if lse is None else lse
        workspace = fvattn.attn_workspace(g, dev) if workspace is None else workspace
        rc = L.fvattn_sparse_attn_lse(ctypes.byref(g), qt.data_ptr(), kt.data_ptr(), vt.data_ptr(), kv_idx.data_ptr(),
                                      kv_cnt.data_ptr(), scale, out.data_ptr(), lse.data_ptr(),
                                      None if sm_stats is None else sm_stats.data_ptr(), workspace.data_ptr(),
                                      workspace.numel(), s)
    if rc:
        _check_call("fvattn_sparse_attn_lse", rc, workspace, lambda: L.fvattn_attn_workspace_size(ctypes.byref(g)))
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
    if stream is None and dq is None and dk is None and dv is None:
        done = (_fast or native()).sparse_attn_bwd(g, qt, kt, vt, ot, dot, lse, kv_idx, kv_cnt,
                                                   None if scale is None else float(scale), workspace)
        if done is not NotImplemented:
            return done
    dev = _device("qt", qt)
    B, H, nb, Npad = g.B, g.H, g.nb, g.Npad
    tiled = (B, H, Npad, g.D)
    for name, t in (("qt", qt), ("kt", kt), ("vt", vt), ("ot", ot), ("dot", dot)):
        _need(name, t, tiled, torch.bfloat16, dev)
    _need("lse", lse, (B, H, Npad), torch.float32, dev)
    _need("kv_idx", kv_idx, (B, H, nb, nb), torch.int32, dev)
    _need("kv_cnt", kv_cnt, (B, H, nb), torch.int32, dev)
    outputs = [t for t in (dq, dk, dv) if t is not None]
    if outputs:
        for name, t in (("dq", dq), ("dk", dk), ("dv", dv)):
            if t is not None:
                _need(name, t, tiled, torch.bfloat16, dev)
        places = {t.data_ptr() for t in outputs}
        if len(places) < len(outputs) or places & {t.data_ptr() for t in (qt, kt, vt, ot, dot)}:
            raise ValueError("dq, dk and dv must be distinct buffers and no input")
    if workspace is not None:
        _need_workspace(workspace, dev)
    scale = _scale(g, scale)
    L = load()
    with _on(dev, stream) as s:
        dq, dk, dv = (torch.empty(tiled, dtype=torch.bfloat16, device=dev) if t is None else t for t in (dq, dk, dv))
        workspace = bwd_workspace(g, dev) if workspace is None else workspace
        rc = L.fvattn_sparse_attn_bwd(ctypes.byref(g), qt.data_ptr(), kt.data_ptr(), vt.data_ptr(), ot.data_ptr(),
                                      dot.data_ptr(), lse.data_ptr(), kv_idx.data_ptr(), kv_cnt.data_ptr(), scale,
                                      dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), workspace.data_ptr(),
                                      workspace.numel(), s)
    if rc:
        _check_call("fvattn_sparse_attn_bwd", rc, workspace,
                    lambda: L.fvattn_sparse_attn_bwd_workspace_size(ctypes.byref(g)))
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
            do = do.contiguous()
            # a view may start anywhere (the gradient of a concatenation's part), the kernels read 16 bytes at a time
            dot = fvattn.reorder(g, do if do.data_ptr() % 16 == 0 else do.clone())
            grads = sparse_attn_bwd(g, qt, kt, vt, ot, dot, lse, kv_idx, kv_cnt, ctx.scale)
            dq, dk, dv = (fvattn.inverse_reorder(g, t) if need else None
                          for t, need in zip(grads, ctx.needs_input_grad))
        return dq, dk, dv, None, None, None, None, None, None


def attention(g: Geom, q, k, v, kv_idx, kv_cnt, scale: Optional[float] = None, order=None) -> torch.Tensor:
    """Differentiable block-sparse attention of raster q, k, v ([B, N, H, D]
    bf16) on given kv lists: raster O.  The lists are kept for the backward
    pass, and must hold the same values then.  `order`: the table of a
    geometry made with fvattn.with_order, kept alive with the call."""
    dev = _device("q", q)
    for name, t in (("q", q), ("k", k), ("v", v)):
        _need(name, t, _raster(g), torch.bfloat16, dev)
    _need("kv_idx", kv_idx, (g.B, g.H, g.nb, g.nb), torch.int32, dev)
    _need("kv_cnt", kv_cnt, (g.B, g.H, g.nb), torch.int32, dev)
    if g.order and (order is None or order.data_ptr() != g.order):
        raise ValueError("order: a geometry with a block order needs the table that it was made with")
    if g.order and order.device != dev:
        raise ValueError(f"order: expected on {dev}, got {order.device}")
    return _Attention.apply(q, k, v, g, order, None, kv_idx, kv_cnt, scale)


class TrainLayer:
    """One attention layer for training: reorder, route, sparse attention and
    inverse reorder of raster q, k, v, differentiable in q, k and v (the lists
    that routing picks are constants).  Every call has tiles, lists and
    statistics of its own, so several calls may be alive before their backward
    passes, on one stream or several.  A step may be captured into a CUDA graph
    with torch.autograd.grad on leaves that no living eager graph uses: drop
    eager outputs before a capture."""

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
        dev = _device("q", q)
        for name, t in (("q", q), ("k", k), ("v", v)):
            _need(name, t, _raster(self.g), torch.bfloat16, dev)
        if self.order_table is not None and self.order_table.device != dev:
            raise ValueError(f"q: on {dev}, the layer's block order is on {self.order_table.device}")
        with torch.cuda.device(q.device):
            qt, kt, routed = self.route(q, k)
        return _Attention.apply(q, k, v, self.g, self.order_table, (qt, kt), routed.kv_idx, routed.kv_cnt, self.scale)
