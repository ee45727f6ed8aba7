"""Layer norm and dropout over a call's layout: binding of include/layernorm_bi.h.

The functions stand beside the RMSNorm ones, take the same CallLayout (and its
plan where parameter gradients are asked for) and keep the same promise: y, h,
dx, dweight, dbias and the dropout mask are bitwise the same for every physical
layout of a logical token multiset.  Rows are bfloat16, float16 or float32 (one
type per call), weight and bias have that type or float32.
"""
from __future__ import annotations

import ctypes
from dataclasses import dataclass

import torch

import invariant_rmsnorm_fwd_gb300 as _rb

_Dropout = _rb._Dropout
_DTYPE = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}


def _index(t) -> int:
    """Device index of a CUDA tensor, -1 for a host tensor."""
    return t.get_device()


def _is_cuda(t) -> bool:
    return t.is_cuda


def _current() -> int:
    return torch.cuda.current_device()


# The raw handle of the current stream, without building a Stream object.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


@dataclass
class Dropout:
    """Dropout with probability p whose mask is a function of the state and the
    logical row and column alone.  state: CUDA int64 tensor (seed, offset), read
    when the kernel runs; a captured graph that is replayed after the state was
    changed in place draws a new mask.  Give each layer and step an offset of
    its own.  The logical row is the call's own (tok_id): ranks that number their
    rows locally need different states, or calls with global ids.  p acts in
    steps of 2^-16; below 2^-17 nothing is dropped."""
    p: float
    state: object

    def struct(self, index: int) -> _Dropout:
        s = self.state
        if not isinstance(s, torch.Tensor) or s.dtype != torch.int64:
            raise TypeError("dropout.state: expected an int64 tensor (seed, offset)")
        if not _is_cuda(s) or _index(s) != index:
            raise ValueError(f"dropout.state: must be a CUDA tensor on the call's device (got {s.device})")
        if s.numel() != 2 or not s.is_contiguous():
            raise ValueError("dropout.state: expected a contiguous tensor of two int64 (seed, offset)")
        if not 0.0 <= self.p <= 1.0:
            raise ValueError(f"dropout.p: {self.p} is not in [0, 1]")
        return _Dropout(s.data_ptr(), self.p)


def _drop(dropout, index: int):
    """The call's dropout for the library."""
    if not isinstance(dropout, Dropout):
        raise TypeError(f"dropout: expected Dropout, got {type(dropout).__name__}")
    return ctypes.byref(dropout.struct(index))


class _Call:
    """The checks of one call's tensors.  The first one (x, h or dy) fixes the
    element type, the device, the shape and the token stride; the others are
    compared with it."""
    __slots__ = ("lay", "H", "index", "dtype", "shape", "strides", "code", "stream")

    def __init__(self, x, name: str, lay, stream):
        if not isinstance(x, torch.Tensor):
            raise TypeError(f"{name}: expected a torch.Tensor, got {type(x).__name__}")
        if not _is_cuda(x):
            raise ValueError(f"{name}: must be a CUDA tensor (got {x.device})")
        self.lay, self.dtype, self.shape, self.strides, self.index = lay, x.dtype, x.shape, x.stride(), _index(x)
        self.code = _DTYPE.get(x.dtype)
        if self.code is None:
            raise TypeError(f"{name}: expected bfloat16, float16 or float32, got {x.dtype}")
        R, nd = lay.rows_per_token, len(self.shape)
        self.H = self.shape[2] if nd == 3 else self.shape[1] // R if nd == 2 else 0
        self._layout_of(name, self.shape, self.strides)
        if self.index != _current():
            raise ValueError(f"{name}: on {x.device}, the current device is cuda:{_current()}")
        if stream is None:
            self.stream = _raw_stream(self.index)
        else:
            if stream.device_index != self.index:
                raise ValueError(f"stream: on {stream.device}, the call's rows are on {x.device}")
            self.stream = stream.cuda_stream

    def _layout_of(self, name, shape, st):
        R, H = self.lay.rows_per_token, self.H
        if len(shape) == 3:
            ok = shape[1] == R and shape[2] == H and st[2] == 1 and (st[1] == H or R == 1)
        else:
            ok = len(shape) == 2 and shape[1] == R * H and st[1] == 1
        if not ok:
            raise ValueError(f"{name}: expected [n_tokens, {R}, hidden] or [n_tokens, {R} * hidden] with unit column "
                             f"stride (hidden {H}), got shape {tuple(shape)} strides {tuple(st)}")
        if shape[0] < self.lay.n_tokens:
            raise ValueError(f"{name}: {shape[0]} token slots, the call's layout has {self.lay.n_tokens}")

    def rows(self, t, name: str) -> int:
        """Address of another tensor of rows."""
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name}: expected a torch.Tensor, got {type(t).__name__}")
        if t.dtype != self.dtype:
            raise TypeError(f"{name}: expected {self.dtype}, got {t.dtype}")
        if not _is_cuda(t) or _index(t) != self.index:
            raise ValueError(f"{name}: must be a CUDA tensor on the call's device (got {t.device})")
        shape, st = t.shape, t.stride()
        if shape != self.shape or st != self.strides:
            self._layout_of(name, shape, st)
            if st[0] != self.strides[0] and self.lay.n_tokens > 1:
                raise ValueError(f"{name}: token stride {st[0]} differs from {self.strides[0]} (one stride per call)")
        return t.data_ptr()

    def params(self, weight, bias=None) -> int:
        code = self.code
        for name, t in (("weight", weight), ("bias", bias)):
            if t is None:
                continue
            if not isinstance(t, torch.Tensor):
                raise TypeError(f"{name}: expected a torch.Tensor, got {type(t).__name__}")
            if t.dtype != self.dtype and t.dtype != torch.float32:
                raise TypeError(f"{name}: expected {self.dtype} or torch.float32, got {t.dtype}")
            if _index(t) != self.index or not _is_cuda(t):
                raise ValueError(f"{name}: must be a CUDA tensor on the call's device (got {t.device})")
            if t.dim() != 1 or t.numel() != self.H or not t.is_contiguous():
                raise ValueError(f"{name}: expected a contiguous [{self.H}] tensor, got shape {tuple(t.shape)}")
            code = _DTYPE[t.dtype]
        if weight is not None and bias is not None and weight.dtype != bias.dtype:
            raise TypeError("weight and bias: expected one type")
        return code

    def stat(self, t, name: str):
        """Address of an optional float32 output of one value per row."""
        if t is None:
            return None
        if not isinstance(t, torch.Tensor) or t.dtype != torch.float32:
            raise TypeError(f"{name}: expected a float32 tensor")
        n = self.lay.n_tokens * self.lay.rows_per_token
        if not _is_cuda(t) or _index(t) != self.index or not t.is_contiguous() or t.numel() < n:
            raise ValueError(f"{name}: expected a contiguous CUDA tensor of at least {n} elements on the call's device")
        return t.data_ptr()

    def workspace(self, ws):
        if ws is None:
            return None
        if not isinstance(ws, LayerNormWorkspace):
            raise TypeError(f"workspace: expected LayerNormWorkspace, got {type(ws).__name__}")
        if _index(ws.buf) != self.index:
            raise ValueError(f"workspace: on {ws.buf.device}, the call's rows are on cuda:{self.index}")
        n = self.lay.n_logical_tokens * self.lay.rows_per_token
        if ws.n_rows != n or ws.hidden != self.H:
            raise ValueError(f"workspace: for {ws.n_rows} rows of {ws.hidden}, the call's multiset has {n} rows of {self.H}")
        return ws.buf.data_ptr()

    def layout(self, plan: bool):
        """The call's descriptor; the plan only where it is used.  A call of at most
        one slot does not use its token stride."""
        lay, n = self.lay, self.lay.n_tokens
        tok = None
        if n:
            t = lay.tok_id
            if not isinstance(t, torch.Tensor) or t.dtype != torch.int32:
                raise TypeError("layout.tok_id: expected an int32 tensor")
            if not _is_cuda(t) or _index(t) != self.index:
                raise ValueError(f"layout.tok_id: must be a CUDA tensor on the call's device (got {t.device})")
            if t.numel() != n or not t.is_contiguous():
                raise ValueError(f"layout.tok_id: expected {n} contiguous ids")
            tok = t.data_ptr()
        addr, items = None, 0
        if plan and lay.plan is not None:
            t, items = lay.plan, lay.plan_items
            if not isinstance(t, torch.Tensor) or t.dtype != torch.uint8:
                raise TypeError("layout.plan: expected a uint8 tensor")
            if not _is_cuda(t) or (items and _index(t) != self.index):
                raise ValueError(f"layout.plan: must be a CUDA tensor on the call's device (got {t.device})")
            if items and (t.numel() < items * _rb.PLAN_ITEM_BYTES or not t.is_contiguous()):
                raise ValueError(f"layout.plan: {items} items need {items * _rb.PLAN_ITEM_BYTES} contiguous bytes")
            addr = t.data_ptr()
        stride = self.strides[0] if n > 1 else lay.rows_per_token * self.H
        return ctypes.byref(_rb._Layout(n, lay.rows_per_token, 0, stride, tok, lay.n_logical_tokens, addr, items))


def _empty(shape, strides, dtype, device, stream):
    """Memory of a new output: of the stream that writes it, for what the current stream
    has given back may still be in use there."""
    if stream is None:
        return torch.empty_strided(shape, strides, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty_strided(shape, strides, dtype=dtype, device=device)


def _new(like, stream):
    """A new output with the shape and strides of `like` (rows past n_tokens and padding are left as they come)."""
    return _empty(like.shape, like.stride(), like.dtype, like.device, stream)


def _p(t):
    return None if t is None else t.data_ptr()


def layernorm_fwd(x, weight, bias, lay, eps: float, y=None, mean=None, rstd=None, stream=None):
    """y = (x - mean) * rstd * weight + bias on every active row.  weight and bias
    may be None; mean and rstd are optional float32 outputs of one value per row."""
    c = _Call(x, "x", lay, stream)
    if y is None:
        y = _new(x, stream)
    params = c.params(weight, bias)
    rc = _rb._load().layernorm_fwd(x.data_ptr(), _p(weight), _p(bias), c.H, eps, c.code, params, c.layout(False),
                                   c.rows(y, "y"), c.stat(mean, "mean"), c.stat(rstd, "rstd"), c.stream)
    if rc:
        _rb._check(rc, "layernorm_fwd")
    return y


def layernorm_add_fwd(x, residual, weight, bias, lay, eps: float, h=None, y=None, mean=None, rstd=None,
                      dropout: Dropout = None, stream=None):
    """Dropout and residual add fused with the norm: h = round(drop(x) + residual),
    y = layer norm of h.  Returns (h, y); h is what the backward pass takes."""
    c = _Call(x, "x", lay, stream)
    if h is None:
        h = _new(x, stream)
    if y is None:
        y = _new(x, stream)
    d = None if dropout is None else _drop(dropout, c.index)
    params = c.params(weight, bias)
    rc = _rb._load().layernorm_add_fwd(x.data_ptr(), c.rows(residual, "residual"), _p(weight), _p(bias), c.H, eps, c.code,
                                       params, c.layout(False), d, c.rows(h, "h"), c.rows(y, "y"),
                                       c.stat(mean, "mean"), c.stat(rstd, "rstd"), c.stream)
    if rc:
        _rb._check(rc, "layernorm_add_fwd")
    return h, y


def layernorm_bwd(x, weight, dy, lay, eps: float, dx=None, workspace=None, stream=None, write_dx: bool = True):
    """dx on every active row; with a workspace the same pass adds the call's rows
    to dweight and dbias (the layout needs its plan)."""
    c = _Call(x, "x", lay, stream)
    at_dy = c.rows(dy, "dy")
    if dx is None and write_dx:
        dx = _new(dy, stream)
    params = c.params(weight)
    rc = _rb._load().layernorm_bwd(x.data_ptr(), _p(weight), at_dy, c.H, eps, c.code, params,
                                   c.layout(workspace is not None), None if dx is None else c.rows(dx, "dx"),
                                   c.workspace(workspace), c.stream)
    if rc:
        _rb._check(rc, "layernorm_bwd")
    return dx


def layernorm_add_bwd(h, weight, dy, lay, eps: float, dres=None, grad_scale: float = 1.0, dropout: Dropout = None,
                      dh=None, dx=None, workspace=None, stream=None):
    """Backward of layernorm_add_fwd (h is its output): dh = round(grad_scale *
    (norm backward) + dres) is the residual's gradient, dx = round(drop(the same
    sum)) is x's.  Returns (dh, dx); without dropout dx is dh.  The workspace's
    terms stay unscaled (scale them at finalize)."""
    c = _Call(h, "h", lay, stream)
    at_dy = c.rows(dy, "dy")
    if dh is None:
        dh = _new(dy, stream)
    d = None
    if dropout is not None:
        if dx is None:
            dx = _new(dy, stream)
        d = _drop(dropout, c.index)
    elif dx is not None:
        raise ValueError("dx: only with a dropout (without one it is dh)")
    params = c.params(weight)
    rc = _rb._load().layernorm_add_bwd(h.data_ptr(), _p(weight), at_dy, None if dres is None else c.rows(dres, "dres"),
                                       c.H, eps, grad_scale, c.code, params, c.layout(workspace is not None), d,
                                       c.rows(dh, "dh"), None if dx is None else c.rows(dx, "dx"),
                                       c.workspace(workspace), c.stream)
    if rc:
        _rb._check(rc, "layernorm_add_bwd")
    return dh, (dh if dropout is None else dx)


def _dropout(fn: str, x, out, in_name: str, out_name: str, lay, dropout, stream):
    c = _Call(x, in_name, lay, stream)
    d = _drop(dropout, c.index)
    if out is None:
        out = _new(x, stream)
    rc = getattr(_rb._load(), fn)(x.data_ptr(), c.H, c.code, c.layout(False), d, c.rows(out, out_name), c.stream)
    if rc:
        _rb._check(rc, fn)
    return out


def dropout_fwd(x, lay, dropout: Dropout, y=None, stream=None):
    """y = drop(x) on every active row: kept elements times 1 / (1 - p), the others 0."""
    return _dropout("dropout_fwd", x, y, "x", "y", lay, dropout, stream)


def dropout_bwd(dy, lay, dropout: Dropout, dx=None, stream=None):
    """dx = drop(dy), with the mask that dropout_fwd made from the same state."""
    return _dropout("dropout_bwd", dy, dx, "dy", "dx", lay, dropout, stream)


class LayerNormWorkspace:
    """Device workspace of one reduction of dweight and dbias (allocated by PyTorch).
    It has no nodes over ranges of blocks: the sharded reduction is the RMSNorm
    workspace's."""

    def __init__(self, n_logical_rows: int, hidden: int, device="cuda"):
        self.n_rows = int(n_logical_rows)
        self.hidden = int(hidden)
        self.bytes = int(_rb._load().layernorm_workspace_bytes(self.n_rows, self.hidden))
        if self.bytes == 0:
            raise _rb.RmsNormError(-2, "layernorm_workspace_bytes")
        self.buf = torch.empty(self.bytes, dtype=torch.uint8, device=device)
        if self.buf.data_ptr() % 256:
            raise RuntimeError("workspace allocation is not 256-byte aligned")

    def _stream(self, stream) -> int:
        index = _index(self.buf)
        if index != _current():
            raise ValueError(f"workspace: on {self.buf.device}, the current device is cuda:{_current()}")
        if stream is None:
            return _raw_stream(index)
        if stream.device_index != index:
            raise ValueError(f"stream: on {stream.device}, the workspace is on {self.buf.device}")
        return stream.cuda_stream

    def _gradient(self, t, name: str, stream):
        if t is None:
            return _empty((self.hidden,), (1,), torch.float32, self.buf.device, stream)
        if not isinstance(t, torch.Tensor) or t.dtype != torch.float32:
            raise TypeError(f"{name}: expected a float32 tensor")
        if _index(t) != _index(self.buf) or not t.is_contiguous() or t.numel() < self.hidden:
            raise ValueError(f"{name}: expected a contiguous tensor of at least {self.hidden} elements on {self.buf.device}")
        return t

    def begin(self, stream=None):
        rc = _rb._load().layernorm_begin(self.buf.data_ptr(), self.bytes, self.n_rows, self.hidden, self._stream(stream))
        if rc:
            _rb._check(rc, "layernorm_begin")

    def finalize(self, dweight=None, dbias=None, stream=None, grad_scale: float = 1.0):
        """(dweight, dbias) of the reduction, each root multiplied once by grad_scale."""
        at = self._stream(stream)
        dweight, dbias = self._gradient(dweight, "dweight", stream), self._gradient(dbias, "dbias", stream)
        rc = _rb._load().layernorm_finalize(self.buf.data_ptr(), self.n_rows, self.hidden, grad_scale,
                                            dweight.data_ptr(), dbias.data_ptr(), at)
        if rc:
            _rb._check(rc, "layernorm_finalize")
        return dweight, dbias

    def status(self, stream=None) -> int:
        out = ctypes.c_int32(0)
        _rb._check(_rb._load().layernorm_status(self.buf.data_ptr(), self._stream(stream), ctypes.byref(out)),
                   "layernorm_status")
        return int(out.value)
