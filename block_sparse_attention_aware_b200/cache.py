"""A paged cache of keys and values and the attention of one new token over it
(the C ABI in include/fvattn_cache.h).

    cache = PagedCache.empty(pages=512, Hkv=40, D=128, page=128)
    rot = rotation_table(128, (22, 21, 21), rows=1024)
    ...                                      # per step: pages for the new tokens, lens counts them
    q = cache.append(k, v, table, lens, q=q, pos=pos, rot=rot, axes=(22, 21, 21))
    o, lse = cache.attend(q, table, lens)

Which pages a sequence owns is the caller's bookkeeping: `table` [B, width]
int32 lists them in order and `lens` [B] int32 holds the lengths, both on the
GPU, so that a captured step reads the current ones at every replay.

Conventions are those of fvattn.py.  Tensors of a call live on one device; the
call runs there even when another device is current.
"""
from __future__ import annotations

import ctypes
import math
from typing import Optional, Sequence

import torch

from . import fvattn, train
from .fvattn import _check
from .train import _check_call, _need, _need_workspace, _on

EXPORTED = ("fvattn_cache_append", "fvattn_cache_append_fresh", "fvattn_cache_attn_parts", "fvattn_cache_attn_workspace_size",
            "fvattn_cache_attn")

BF16, I32, F32 = torch.bfloat16, torch.int32, torch.float32


class _Cache(ctypes.Structure):
    """Mirror of fvattn_cache."""
    _fields_ = [(n, ctypes.c_int) for n in ("pages", "Hkv", "D", "page")] + \
               [("k", ctypes.c_void_p), ("v", ctypes.c_void_p)]


class _Rotation(ctypes.Structure):
    """Mirror of fvattn_rotation."""
    _fields_ = [("table", ctypes.c_void_p), ("rows", ctypes.c_int), ("axes", ctypes.c_int),
                ("pairs", ctypes.c_int * 3), ("pos", ctypes.c_void_p), ("halves", ctypes.c_int)]


_lib = None


def load():
    """libfvattn.so with this module's signatures declared (raises if missing)."""
    global _lib
    if _lib is None:
        L = fvattn.load()
        P, I, LL, S = ctypes.c_void_p, ctypes.c_int, ctypes.c_longlong, ctypes.c_size_t
        C, R = ctypes.POINTER(_Cache), ctypes.POINTER(_Rotation)
        for call in (L.fvattn_cache_append, L.fvattn_cache_append_fresh):
            call.argtypes = [C, I, LL, P, P, P, I, P, LL, P, LL, P, LL, I, P, LL, R, P]
            call.restype = I
        L.fvattn_cache_attn_parts.argtypes = [I, I, I, I, LL, ctypes.POINTER(I)]
        L.fvattn_cache_attn_parts.restype = I
        L.fvattn_cache_attn_workspace_size.argtypes = [I, I, I, I, LL]
        L.fvattn_cache_attn_workspace_size.restype = S
        L.fvattn_cache_attn.argtypes = [C, I, I, P, LL, P, I, P, LL, ctypes.c_float, P, P, P, S, P]
        L.fvattn_cache_attn.restype = I
        _lib = L
    return _lib


def rotation_table(D: int, axes: Sequence[int], rows: int, base: float = 10000.0, device="cuda") -> torch.Tensor:
    """Cosines and sines of position * frequency for `append`: [rows, D] fp32,
    pair i of an axis with n pairs having frequency base^(-i/n).  The angles
    are formed in 64 bits, so that far positions keep their phase."""
    if sum(axes) != D // 2:
        raise ValueError(f"axes {tuple(axes)} do not add up to {D // 2} pairs")
    freq = torch.cat([base ** (-torch.arange(n, dtype=torch.float64) / n) for n in axes if n])
    angle = torch.arange(rows, dtype=torch.float64)[:, None] * freq
    return torch.cat([angle.cos(), angle.sin()], 1).to(F32).to(device)


def _vector(name, t, n, dev, dtype=I32):
    if t is None or t.dtype is not dtype or t.device != dev or t.shape != (n,) or not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous {dtype} tensor of shape ({n},) on {dev}")


class PagedCache:
    """Keys and values of many sequences in pages [pages, Hkv, page, D] bf16
    (page 16, 32, 64 or 128; D 64 or 128), in the caller's two tensors."""

    def __init__(self, k_pages: torch.Tensor, v_pages: torch.Tensor):
        for name, t in (("k_pages", k_pages), ("v_pages", v_pages)):
            if t.dtype != BF16 or t.dim() != 4 or not t.is_contiguous() or not t.is_cuda or t.shape != k_pages.shape or \
                    t.device != k_pages.device:
                raise ValueError(f"{name}: expected a contiguous CUDA bf16 tensor [pages, Hkv, page, D], one shape for both")
        self.pages, self.Hkv, self.page, self.D = k_pages.shape
        if self.D not in (64, 128) or self.page not in (16, 32, 64, 128) or self.pages < 1 or self.Hkv < 1:
            raise ValueError(f"unsupported page shape {tuple(k_pages.shape)}")
        if k_pages.data_ptr() == v_pages.data_ptr():
            raise ValueError("k_pages and v_pages must be distinct buffers")
        self.k_pages, self.v_pages, self.device = k_pages, v_pages, k_pages.device
        self._c = _Cache(self.pages, self.Hkv, self.D, self.page, k_pages.data_ptr(), v_pages.data_ptr())

    @classmethod
    def empty(cls, pages: int, Hkv: int, D: int, page: int = 128, device="cuda") -> "PagedCache":
        shape = (pages, Hkv, page, D)
        return cls(torch.empty(shape, dtype=BF16, device=device), torch.empty(shape, dtype=BF16, device=device))

    def _rows(self, name, t, rows, heads):
        """(rows, heads, row stride) of a [rows, heads, D] view whose rows may lie apart (a slice of a wider
        projection)."""
        if t is None:
            raise ValueError(f"{name} is required")
        shape = t.shape
        if t.dtype is not BF16 or t.device != self.device or len(shape) != 3 or \
                (rows is not None and shape[0] != rows) or (heads is not None and shape[1] != heads) or \
                shape[1] < 1 or shape[2] != self.D:
            raise ValueError(f"{name}: expected a bf16 tensor [{'rows' if rows is None else rows}, "
                             f"{'heads' if heads is None else heads}, {self.D}] on {self.device}, got {t.dtype} "
                             f"{tuple(shape)} on {t.device}")
        row = shape[1] * self.D
        sr, sh, sd = t.stride()
        if shape[0] <= 1:
            sr = row
        if sd != 1 or (shape[1] > 1 and sh != self.D) or sr < row or sr % 8:
            raise ValueError(f"{name}: a row's heads must be contiguous and rows a multiple of 8 elements apart, "
                             f"got strides {t.stride()}")
        return shape[0], shape[1], sr

    def _table(self, table):
        if table is None or table.dtype is not I32 or table.device != self.device or table.dim() != 2 or \
                not table.is_contiguous() or table.numel() < 1:
            raise ValueError(f"table: expected a contiguous int32 tensor [B, width] on {self.device}")
        return table.shape

    def append(self, k, v, table, lens, cu=None, q=None, q_out=None, pos=None, rot=None, axes=None,
               halves: bool = False, stream=None):
        """fvattn_cache_append: write new tokens k, v ([rows, Hkv, D], which
        may be slices of one projection's output) to the pages of their
        sequences.  Sequence b's are rows cu[b] .. cu[b+1]-1 (cu None: row b),
        and lens[b] counts them.  With `rot` (rotation_table) and `pos`
        ([rows, len(axes)] int32) the keys, and the queries q ([rows, Hq, D])
        into q_out, are rotated; q_out may be q.  Returns q_out.  Rows of no
        sequence and refused tokens are left alone in a q_out that is given,
        and zero in one made here."""
        if stream is None:
            done = (train._fast or train.native()).append(
                self.k_pages, self.v_pages, k, v, table, lens, cu, q, q_out, pos, rot,
                None if axes is None else tuple(axes), bool(halves))
            if done is not NotImplemented:
                return done
        B, width = self._table(table)
        _vector("lens", lens, B, self.device)
        if cu is not None:
            _vector("cu", cu, B + 1, self.device)
        rows, _, ks = self._rows("k", k, None, self.Hkv)
        _, _, vs = self._rows("v", v, rows, self.Hkv)
        if cu is None and rows < B:
            raise ValueError(f"{rows} rows for {B} sequences: without cu, row b is sequence b's token")
        qs = qos = hq = 0
        if q is not None:
            _, hq, qs = self._rows("q", q, rows, None)
            if q_out is not None:
                _, _, qos = self._rows("q_out", q_out, rows, hq)
                if q_out.data_ptr() == q.data_ptr() and qos != qs:
                    raise ValueError("q_out starts where q does, with other strides")
        elif q_out is not None:
            raise ValueError("q_out without q")
        r = None
        if rot is not None:
            axes = (self.D // 2,) if axes is None else tuple(axes)
            if rot.dtype != F32 or rot.device != self.device or rot.dim() != 2 or rot.shape[1] != self.D or \
                    rot.shape[0] < 1 or not rot.is_contiguous():
                raise ValueError(f"rot: expected a contiguous fp32 tensor [positions, {self.D}] on {self.device}")
            if not 1 <= len(axes) <= 3 or min(axes) < 0 or sum(axes) != self.D // 2:
                raise ValueError(f"axes {axes}: one to three counts adding up to {self.D // 2} pairs")
            if pos is None or pos.dtype != I32 or pos.device != self.device or pos.shape != (rows, len(axes)) or \
                    not pos.is_contiguous():
                raise ValueError(f"pos: expected a contiguous int32 tensor ({rows}, {len(axes)}) on {self.device}")
            r = _Rotation(rot.data_ptr(), rot.shape[0], len(axes), (ctypes.c_int * 3)(*axes), pos.data_ptr(), bool(halves))
        elif pos is not None or axes is not None:
            raise ValueError("pos and axes belong with rot")
        L = load()
        with _on(self.device, stream) as s:
            call = L.fvattn_cache_append
            if q is not None and q_out is None:
                call = L.fvattn_cache_append_fresh
                q_out = torch.empty((rows, hq, self.D), dtype=BF16, device=self.device)
                qos = hq * self.D
            if rows == 0:
                return q_out
            rc = call(ctypes.byref(self._c), B, rows, None if cu is None else cu.data_ptr(),
                      lens.data_ptr(), table.data_ptr(), width, k.data_ptr(), ks, v.data_ptr(), vs,
                      None if q is None else q.data_ptr(), qs, hq, None if q is None else q_out.data_ptr(), qos,
                      None if r is None else ctypes.byref(r), s)
            if rc:
                _check("fvattn_cache_append", rc)
        return q_out

    def attend_workspace(self, B: int, Hq: int, longest: int) -> torch.Tensor:
        """A workspace for `attend`.  Calls that may overlap on the GPU need
        one each (as do two captured graphs that may run at the same time)."""
        with torch.cuda.device(self.device):
            n = load().fvattn_cache_attn_workspace_size(B, Hq, self.Hkv, self.D, longest)
        return torch.empty(max(n, 256), dtype=torch.uint8, device=self.device)

    def attend(self, q, table, lens, scale: Optional[float] = None, longest: Optional[int] = None, out=None, lse=None,
               workspace: Optional[torch.Tensor] = None, stream=None):
        """fvattn_cache_attn: (O [B, Hq, D] bf16, lse [B, Hq] fp32) of one
        query a sequence q [B, Hq, D] over its lens[b] cached tokens; Hq is a
        multiple of Hkv.  `longest`: no sequence is longer (default: what the
        table can hold; a nearer bound splits better)."""
        if stream is None:
            done = (train._fast or train.native()).attend(
                self.k_pages, self.v_pages, q, table, lens, None if scale is None else float(scale),
                None if longest is None else int(longest), out, lse, workspace)
            if done is not NotImplemented:
                return done
        B, width = self._table(table)
        _, hq, qs = self._rows("q", q, B, None)
        if hq % self.Hkv:
            raise ValueError(f"{hq} query heads do not divide over {self.Hkv} key heads")
        _vector("lens", lens, B, self.device)
        longest = width * self.page if longest is None else int(longest)
        if out is not None:
            _need("out", out, q.shape, BF16, self.device)
        if lse is not None:
            _need("lse", lse, (B, hq), F32, self.device)
        if workspace is not None:
            _need_workspace(workspace, self.device)
        scale = 1.0 / math.sqrt(self.D) if scale is None else float(scale)
        if not (0.0 < scale < math.inf) or longest < 0:
            raise ValueError(f"scale {scale}, longest {longest}: expected a positive finite scale and longest >= 0")
        L = load()
        with _on(self.device, stream) as s:
            if workspace is None:
                need = L.fvattn_cache_attn_workspace_size(B, hq, self.Hkv, self.D, longest)
                workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=self.device)
            if out is None:
                out = torch.empty((B, hq, self.D), dtype=BF16, device=self.device)
            if lse is None:
                lse = torch.empty((B, hq), dtype=F32, device=self.device)
            rc = L.fvattn_cache_attn(ctypes.byref(self._c), B, hq, q.data_ptr(), qs, table.data_ptr(), width,
                                     lens.data_ptr(), longest, scale, out.data_ptr(), lse.data_ptr(),
                                     workspace.data_ptr(), workspace.numel(), s)
            if rc:
                _check_call("fvattn_cache_attn", rc, workspace,
                            lambda: L.fvattn_cache_attn_workspace_size(B, hq, self.Hkv, self.D, longest))
        return out, lse
