"""Layer norm and dropout over a call's layout: binding of include/layernorm_bi.h.

The functions stand beside the RMSNorm ones, take the same CallLayout (and its
plan where parameter gradients are asked for) and keep the same promise: y, h,
dx, dweight, dbias and the dropout mask are bitwise the same for every physical
layout of a logical token multiset.  Rows are bfloat16, float16 or float32 (one
type per call), weight and bias have that type or float32.
"""
from __future__ import annotations

import ctypes
import math
from dataclasses import dataclass

import torch

import invariant_rmsnorm_fwd_gb300 as _rb

_DTYPE = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}


class _Dropout(ctypes.Structure):
    _fields_ = [("state", ctypes.c_void_p), ("p", ctypes.c_double)]


def signatures(layout_ptr) -> dict:
    """Argument and result types of the library's functions (filled in by the package's loader)."""
    P, I64, I32, F, D, S = (ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_float,
                            ctypes.POINTER(_Dropout), ctypes.c_size_t)
    L, R = layout_ptr, ctypes.c_int
    return {
        "layernorm_fwd": ([P, P, P, I64, F, I32, I32, L, P, P, P, P], R),
        "layernorm_add_fwd": ([P, P, P, P, I64, F, I32, I32, L, D, P, P, P, P, P], R),
        "layernorm_bwd": ([P, P, P, I64, F, I32, I32, L, P, P, P], R),
        "layernorm_add_bwd": ([P, P, P, P, I64, F, F, I32, I32, L, D, P, P, P, P], R),
        "layernorm_workspace_bytes": ([I64, I64], S),
        "layernorm_begin": ([P, S, I64, I64, P], R),
        "layernorm_finalize": ([P, I64, I64, F, P, P, P], R),
        "layernorm_status": ([P, P, ctypes.POINTER(I32)], R),
        "dropout_fwd": ([P, I64, I32, L, D, P, P], R),
        "dropout_bwd": ([P, I64, I32, L, D, P, P], R),
    }


@dataclass
class Dropout:
    """Dropout with probability p whose mask is a function of the state and the
    logical row and column alone.  state: CUDA int64 tensor (seed, offset), read
    when the kernel runs; a captured graph that is replayed after the state was
    changed in place draws a new mask.  Give each layer and step an offset of
    its own.  p acts in steps of 2^-16."""
    p: float
    state: object

    def struct(self, device) -> _Dropout:
        s = self.state
        if not isinstance(s, torch.Tensor) or s.dtype != torch.int64:
            raise TypeError("dropout.state: expected an int64 tensor (seed, offset)")
        if not _is_cuda(s) or s.device != device:
            raise ValueError(f"dropout.state: must be a CUDA tensor on {device} (got {s.device})")
        if s.numel() != 2 or not s.is_contiguous():
            raise ValueError("dropout.state: expected a contiguous tensor of two int64 (seed, offset)")
        if not 0.0 <= self.p <= 1.0:
            raise ValueError(f"dropout.p: {self.p} is not in [0, 1]")
        return _Dropout(s.data_ptr(), self.p)


def _is_cuda(t) -> bool:
    return t.is_cuda


def _rows(t, name: str, lay, H: int, like=None):
    """Checks a [T, rows_per_token, H] or [T, rows_per_token * H] tensor of the
    call (T >= n_tokens); `like` is the call's first tensor, whose type, device
    and token stride the others share."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor, got {type(t).__name__}")
    if not _is_cuda(t):
        raise ValueError(f"{name}: must be a CUDA tensor (got {t.device})")
    if like is None:
        if t.dtype not in _DTYPE:
            raise TypeError(f"{name}: expected bfloat16, float16 or float32, got {t.dtype}")
        if lay.n_tokens and lay.tok_id.device != t.device:
            raise ValueError(f"{name}: on {t.device}, the call's layout is on {lay.tok_id.device}")
    elif t.dtype != like.dtype:
        raise TypeError(f"{name}: expected {like.dtype}, got {t.dtype}")
    elif t.device != like.device:
        raise ValueError(f"{name}: on {t.device}, the call's rows are on {like.device}")
    R, shape, st = lay.rows_per_token, t.shape, t.stride()
    if len(shape) == 3:
        ok = shape[1] == R and shape[2] == H and st[2] == 1 and (st[1] == H or R == 1)
    else:
        ok = len(shape) == 2 and shape[1] == R * H and st[1] == 1
    if not ok:
        raise ValueError(f"{name}: expected [n_tokens, {R}, {H}] or [n_tokens, {R * H}] with unit column stride, "
                         f"got shape {tuple(shape)} strides {tuple(st)}")
    if shape[0] < lay.n_tokens:
        raise ValueError(f"{name}: {shape[0]} token slots, the call's layout has {lay.n_tokens}")
    if like is not None and st[0] != like.stride(0) and lay.n_tokens > 1:
        raise ValueError(f"{name}: token stride {st[0]} differs from {like.stride(0)} (one stride per call)")


def _hidden(x, lay) -> int:
    if not isinstance(x, torch.Tensor):
        raise TypeError(f"x: expected a torch.Tensor, got {type(x).__name__}")
    if x.dim() == 3:
        return x.shape[2]
    if x.dim() == 2 and x.shape[1] % lay.rows_per_token == 0:
        return x.shape[1] // lay.rows_per_token
    raise ValueError(f"x: expected [n_tokens, {lay.rows_per_token}, hidden] or [n_tokens, "
                     f"{lay.rows_per_token} * hidden], got shape {tuple(x.shape)}")


def _new(like, lay, H: int):
    """A new output with the call's token stride (rows past n_tokens and padding are left as they come)."""
    if like.shape[0] <= 1 or like.is_contiguous():
        return torch.empty(like.shape, dtype=like.dtype, device=like.device)
    return torch.empty_strided(like.shape, like.stride(), dtype=like.dtype, device=like.device)


def _params(x, H: int, weight, bias=None) -> int:
    code = None
    for name, t in (("weight", weight), ("bias", bias)):
        if t is None:
            continue
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name}: expected a torch.Tensor, got {type(t).__name__}")
        if t.device != x.device:
            raise ValueError(f"{name}: on {t.device}, the call's rows are on {x.device}")
        if t.dtype != x.dtype and t.dtype != torch.float32:
            raise TypeError(f"{name}: expected {x.dtype} or torch.float32, got {t.dtype}")
        if t.shape != (H,) or not t.is_contiguous():
            raise ValueError(f"{name}: expected a contiguous [{H}] tensor, got shape {tuple(t.shape)}")
        if code is not None and code != _DTYPE[t.dtype]:
            raise TypeError("weight and bias: expected one type")
        code = _DTYPE[t.dtype]
    return _DTYPE[x.dtype] if code is None else code


def _layout(x, lay, H: int):
    """The call's descriptor.  A call of at most one slot does not use its stride."""
    return ctypes.byref(lay.struct(x.stride(0) if lay.n_tokens > 1 else lay.rows_per_token * H))


def _stats(lay, x, mean, rstd):
    n = lay.n_tokens * lay.rows_per_token
    for name, t in (("mean", mean), ("rstd", rstd)):
        if t is not None:
            _rb._f32_out(t, name, n, x.device)


def _ws(workspace, lay, H: int, device):
    if workspace is None:
        return None
    if not isinstance(workspace, LayerNormWorkspace):
        raise TypeError(f"workspace: expected LayerNormWorkspace, got {type(workspace).__name__}")
    if workspace.buf.device != device:
        raise ValueError(f"workspace: on {workspace.buf.device}, the call's rows are on {device}")
    n = lay.n_logical_tokens * lay.rows_per_token
    if workspace.n_rows != n or workspace.hidden != H:
        raise ValueError(f"workspace: for {workspace.n_rows} rows of {workspace.hidden}, the call's multiset has "
                         f"{n} rows of {H}")
    return workspace.buf.data_ptr()


def _p(t):
    return None if t is None else t.data_ptr()


def _s(stream, t):
    """The stream handle; t's device has to be the stream's, and the current one."""
    if t.device.index != torch.cuda.current_device():
        raise ValueError(f"the call's tensors are on {t.device}, the current device is "
                         f"cuda:{torch.cuda.current_device()}")
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if stream.device != t.device:
        raise ValueError(f"stream: on {stream.device}, the call's tensors are on {t.device}")
    return stream.cuda_stream


def layernorm_fwd(x, weight, bias, lay, eps: float, y=None, mean=None, rstd=None, stream=None):
    """y = (x - mean) * rstd * weight + bias on every active row.  weight and bias
    may be None; mean and rstd are optional float32 outputs of one value per row."""
    H = _hidden(x, lay)
    _rows(x, "x", lay, H)
    st = _s(stream, x)
    if y is None:
        y = _new(x, lay, H)
    _rows(y, "y", lay, H, x)
    _stats(lay, x, mean, rstd)
    pd = _params(x, H, weight, bias)
    _rb._check(_rb._load().layernorm_fwd(x.data_ptr(), _p(weight), _p(bias), H, eps, _DTYPE[x.dtype], pd,
                                         _layout(x, lay, H), y.data_ptr(), _p(mean), _p(rstd), st),
               "layernorm_fwd")
    return y


def layernorm_add_fwd(x, residual, weight, bias, lay, eps: float, h=None, y=None, mean=None, rstd=None,
                      dropout: Dropout = None, stream=None):
    """Dropout and residual add fused with the norm: h = round(drop(x) + residual),
    y = layer norm of h.  Returns (h, y); h is what the backward pass takes."""
    H = _hidden(x, lay)
    _rows(x, "x", lay, H)
    st = _s(stream, x)
    if h is None:
        h = _new(x, lay, H)
    if y is None:
        y = _new(x, lay, H)
    for name, t in (("residual", residual), ("h", h), ("y", y)):
        _rows(t, name, lay, H, x)
    _stats(lay, x, mean, rstd)
    pd = _params(x, H, weight, bias)
    d = None if dropout is None else ctypes.byref(dropout.struct(x.device))
    _rb._check(_rb._load().layernorm_add_fwd(x.data_ptr(), residual.data_ptr(), _p(weight), _p(bias), H, eps,
                                             _DTYPE[x.dtype], pd, _layout(x, lay, H), d, h.data_ptr(), y.data_ptr(),
                                             _p(mean), _p(rstd), st), "layernorm_add_fwd")
    return h, y


def layernorm_bwd(x, weight, dy, lay, eps: float, dx=None, workspace=None, stream=None, write_dx: bool = True):
    """dx on every active row; with a workspace the same pass adds the call's rows
    to dweight and dbias (the layout needs its plan)."""
    H = _hidden(x, lay)
    _rows(x, "x", lay, H)
    st = _s(stream, x)
    _rows(dy, "dy", lay, H, x)
    if dx is None and write_dx:
        dx = _new(dy, lay, H)
    if dx is not None:
        _rows(dx, "dx", lay, H, x)
    pd = _params(x, H, weight)
    ws = _ws(workspace, lay, H, x.device)
    _rb._check(_rb._load().layernorm_bwd(x.data_ptr(), _p(weight), dy.data_ptr(), H, eps, _DTYPE[x.dtype], pd,
                                         _layout(x, lay, H), _p(dx), ws, st), "layernorm_bwd")
    return dx


def layernorm_add_bwd(h, weight, dy, lay, eps: float, dres=None, grad_scale: float = 1.0, dropout: Dropout = None,
                      dh=None, dx=None, workspace=None, stream=None):
    """Backward of layernorm_add_fwd (h is its output): dh = round(grad_scale *
    (norm backward) + dres) is the residual's gradient, dx = round(drop(the same
    sum)) is x's.  Returns (dh, dx); without dropout dx is dh.  The workspace's
    terms stay unscaled (scale them at finalize)."""
    H = _hidden(h, lay)
    _rows(h, "h", lay, H)
    st = _s(stream, h)
    _rows(dy, "dy", lay, H, h)
    if dh is None:
        dh = _new(dy, lay, H)
    _rows(dh, "dh", lay, H, h)
    if dres is not None:
        _rows(dres, "dres", lay, H, h)
    d = None
    if dropout is not None:
        if dx is None:
            dx = _new(dy, lay, H)
        _rows(dx, "dx", lay, H, h)
        d = ctypes.byref(dropout.struct(h.device))
    elif dx is not None:
        raise ValueError("dx: only with a dropout (without one it is dh)")
    pd = _params(h, H, weight)
    ws = _ws(workspace, lay, H, h.device)
    _rb._check(_rb._load().layernorm_add_bwd(h.data_ptr(), _p(weight), dy.data_ptr(), _p(dres), H, eps, grad_scale,
                                             _DTYPE[h.dtype], pd, _layout(h, lay, H), d, dh.data_ptr(), _p(dx), ws,
                                             st), "layernorm_add_bwd")
    return dh, (dh if dropout is None else dx)


def _dropout(fn: str, x, out, in_name: str, out_name: str, lay, dropout, stream):
    H = _hidden(x, lay)
    _rows(x, in_name, lay, H)
    st = _s(stream, x)
    if not isinstance(dropout, Dropout):
        raise TypeError(f"dropout: expected Dropout, got {type(dropout).__name__}")
    if out is None:
        out = _new(x, lay, H)
    _rows(out, out_name, lay, H, x)
    d = dropout.struct(x.device)
    _rb._check(getattr(_rb._load(), fn)(x.data_ptr(), H, _DTYPE[x.dtype], _layout(x, lay, H), ctypes.byref(d),
                                        out.data_ptr(), st), fn)
    return out


def dropout_fwd(x, lay, dropout: Dropout, y=None, stream=None):
    """y = drop(x) on every active row: kept elements times 1 / (1 - p), the others 0."""
    return _dropout("dropout_fwd", x, y, "x", "y", lay, dropout, stream)


def dropout_bwd(dy, lay, dropout: Dropout, dx=None, stream=None):
    """dx = drop(dy), with the mask that dropout_fwd made from the same state."""
    return _dropout("dropout_bwd", dy, dx, "dy", "dx", lay, dropout, stream)


class LayerNormWorkspace:
    """Device workspace of one reduction of dweight and dbias (allocated by PyTorch)."""

    def __init__(self, n_logical_rows: int, hidden: int, device="cuda"):
        self.n_rows = int(n_logical_rows)
        self.hidden = int(hidden)
        self.bytes = int(_rb._load().layernorm_workspace_bytes(self.n_rows, self.hidden))
        if self.bytes == 0:
            raise _rb.RmsNormError(-2, "layernorm_workspace_bytes")
        self.buf = torch.empty(self.bytes, dtype=torch.uint8, device=device)
        if self.buf.data_ptr() % 256:
            raise RuntimeError("workspace allocation is not 256-byte aligned")

    def begin(self, stream=None):
        _rb._check(_rb._load().layernorm_begin(self.buf.data_ptr(), self.bytes, self.n_rows, self.hidden,
                                               _s(stream, self.buf)), "layernorm_begin")

    def finalize(self, dweight=None, dbias=None, stream=None, grad_scale: float = 1.0):
        """(dweight, dbias) of the reduction, each root multiplied once by grad_scale."""
        if not math.isfinite(grad_scale):
            raise _rb.RmsNormError(-13, "layernorm_finalize")
        if dweight is None:
            dweight = torch.empty(self.hidden, dtype=torch.float32, device=self.buf.device)
        if dbias is None:
            dbias = torch.empty(self.hidden, dtype=torch.float32, device=self.buf.device)
        _rb._f32_out(dweight, "dweight", self.hidden, self.buf.device)
        _rb._f32_out(dbias, "dbias", self.hidden, self.buf.device)
        _rb._check(_rb._load().layernorm_finalize(self.buf.data_ptr(), self.n_rows, self.hidden, grad_scale,
                                                  dweight.data_ptr(), dbias.data_ptr(), _s(stream, self.buf)),
                   "layernorm_finalize")
        return dweight, dbias

    def status(self, stream=None) -> int:
        out = ctypes.c_int32(0)
        _rb._check(_rb._load().layernorm_status(self.buf.data_ptr(), _s(stream, self.buf), ctypes.byref(out)),
                   "layernorm_status")
        return int(out.value)
