"""Rotary positions of queries and keys, alone and behind an RMS norm of every head:
binding of include/rotary_bi.h.

The functions stand beside the per-head norms and take the same CallLayout, one
row per token slot (rows_per_token = 1, no plan); queries and keys are
[n_tokens, heads, head_dim] tensors with any token and head stride, so slices of a
joined projection and head-major tensors need no copy.  y, dx and the weight
gradients are bitwise the same for every physical layout of a logical token
multiset.  Heads are bfloat16, float16 or float32 (one type per call), weights
have that type or float32.
"""
from __future__ import annotations

import ctypes
import struct

import numpy as np
import torch

import invariant_rmsnorm_fwd_gb300 as _rb

# The C structures as bytes: packing them is quicker than building ctypes ones.
_heads_struct = struct.Struct("QqqQqqQqqQii").pack                   # rmsnorm_heads_t
_rotary_struct = struct.Struct("QQiiif").pack                        # rmsnorm_rotary_t
_layout_struct = struct.Struct("qiiqQqQq").pack                      # rmsnorm_layout_t
_DTYPE = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}


_index = torch.Tensor.get_device                                     # of a CUDA tensor; -1 for a host tensor


def _is_cuda(t) -> bool:
    return t.is_cuda


# The current device, without looking whether CUDA runs (a CUDA tensor is at hand).
_current = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
# The raw handle of the current stream, without building a Stream object.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def rotary_frequencies(rotary_dim: int, base: float = 10000.0, factor: float = 1.0, original_length: float = None,
                       low: float = 1.0, high: float = 32.0) -> np.ndarray:
    """Radians per position of the rotary_dim / 2 pairs: base^(-2i / rotary_dim), in float64.

    factor > 1 stretches the positions for contexts longer than the trained one: all
    pairs alike (f / factor), or, with the original length, by how many turns a pair
    makes over it: pairs of at least `high` turns keep their speed, those of at most
    `low` are stretched in full, in between the two are mixed in proportion."""
    if rotary_dim < 4 or rotary_dim % 4:
        raise ValueError(f"rotary_dim: expected a positive multiple of 4, got {rotary_dim}")
    if not (base > 0 and factor > 0):
        raise ValueError(f"base and factor must be positive, got {base} and {factor}")
    f = float(base) ** (-np.arange(0, rotary_dim, 2, dtype=np.float64) / rotary_dim)
    if original_length is None:
        return f / factor
    if not (original_length > 0 and high > low):
        raise ValueError("original_length must be positive and high above low")
    keep = np.clip((original_length * f / (2 * np.pi) - low) / (high - low), 0.0, 1.0)
    return f * keep + f * (1 - keep) / factor


class Rotary:
    """A rotation that a program keeps: the frequencies on the device, which columns of a
    head turn (rotary_dim of them from `first` on) and which belong together: halves
    (i and i + rotary_dim / 2) or neighbours (interleaved).  inv_freq: radians per position
    of the rotary_dim / 2 pairs (rotary_frequencies by default); scale multiplies cosine
    and sine."""

    def __init__(self, rotary_dim: int, base: float = 10000.0, interleaved: bool = False, first: int = 0, inv_freq=None,
                 scale: float = 1.0, device="cuda"):
        self.rotary_dim, self.first, self.interleaved, self.scale = int(rotary_dim), int(first), bool(interleaved), float(scale)
        if self.rotary_dim < 4 or self.rotary_dim % 4:
            raise ValueError(f"rotary_dim: expected a positive multiple of 4, got {rotary_dim}")
        if self.first < 0 or self.first % 2:
            raise ValueError(f"first: expected an even column, got {first}")
        if inv_freq is None:
            inv_freq = rotary_frequencies(self.rotary_dim, base)
        f = np.ascontiguousarray(inv_freq.cpu() if isinstance(inv_freq, torch.Tensor) else inv_freq, dtype=np.float64)
        if f.shape != (self.rotary_dim // 2,):
            raise ValueError(f"inv_freq: expected {self.rotary_dim // 2} frequencies, got shape {f.shape}")
        turns = np.empty(f.size, dtype=np.uint64)
        _rb._check(_rb._load().rotary_turns(f.ctypes.data, f.size, turns.ctypes.data), "rotary_turns")
        self.turns = torch.from_numpy(turns.view(np.int64)).to(device)

    def struct(self, position, n: int, index: int):
        """The library's descriptor for a call of n slots on device `index`."""
        if not isinstance(position, torch.Tensor) or position.dtype != torch.int32:
            raise TypeError("position: expected an int32 tensor")
        if _index(position) != index:
            raise ValueError(f"position: must be a CUDA tensor on the call's device (got {position.device})")
        shape = position.shape
        if len(shape) != 1 or shape[0] < n or not position.is_contiguous():
            raise ValueError(f"position: expected a contiguous tensor of at least {n} positions, one per token slot")
        turns = self.turns
        if _index(turns) != index:
            raise ValueError(f"rotary: on {turns.device}, the call's heads are on cuda:{index}")
        return _rotary_struct(position.data_ptr(), turns.data_ptr(), self.rotary_dim, self.first, self.interleaved, self.scale)


class _Call:
    """The checks of one call's tensors.  The first one (the queries') fixes the element
    type, the device and the head width; the others are compared with it."""
    __slots__ = ("lay", "n", "D", "index", "dtype", "code", "stream")

    def __init__(self, q, name: str, lay, stream):
        if not isinstance(lay, _rb.CallLayout):
            raise TypeError(f"layout: expected CallLayout, got {type(lay).__name__}")
        if not isinstance(q, torch.Tensor):
            raise TypeError(f"{name}: expected a torch.Tensor, got {type(q).__name__}")
        if not _is_cuda(q):
            raise ValueError(f"{name}: must be a CUDA tensor (got {q.device})")
        if lay.rows_per_token != 1:
            raise ValueError(f"layout: one row per token slot expected (heads are a dimension of the tensors), got "
                             f"rows_per_token {lay.rows_per_token}")
        dtype, shape, index = q.dtype, q.shape, _index(q)
        code = _DTYPE.get(dtype)
        if code is None:
            raise TypeError(f"{name}: expected bfloat16, float16 or float32, got {dtype}")
        if len(shape) != 3:
            raise ValueError(f"{name}: expected [n_tokens, heads, head_dim], got shape {tuple(shape)}")
        if index != _current():
            raise ValueError(f"{name}: on {q.device}, the current device is cuda:{_current()}")
        if stream is None:
            self.stream = _raw_stream(index)
        else:
            if stream.device_index != index:
                raise ValueError(f"stream: on {stream.device}, the call's heads are on {q.device}")
            self.stream = stream.cuda_stream
        self.lay, self.n, self.D, self.index, self.dtype, self.code = lay, lay.n_tokens, shape[2], index, dtype, code

    def refuse(self, t, name: str, heads):
        """Says what is wrong with a tensor of heads."""
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name}: expected a torch.Tensor, got {type(t).__name__}")
        if t.dtype != self.dtype:
            raise TypeError(f"{name}: expected {self.dtype}, got {t.dtype}")
        if _index(t) != self.index:
            raise ValueError(f"{name}: must be a CUDA tensor on the call's device (got {t.device})")
        if len(t.shape) == 3 and t.shape[0] < self.n:
            raise ValueError(f"{name}: {t.shape[0]} token slots, the call's layout has {self.n}")
        raise ValueError(f"{name}: expected [n_tokens, {heads}, {self.D}] with unit column stride, got shape {tuple(t.shape)} "
                         f"strides {tuple(t.stride())}")

    def weight(self, w, name: str):
        if not isinstance(w, torch.Tensor):
            raise TypeError(f"{name}: expected a torch.Tensor, got {type(w).__name__}")
        if w.dtype != self.dtype and w.dtype != torch.float32:
            raise TypeError(f"{name}: expected {self.dtype} or torch.float32, got {w.dtype}")
        if _index(w) != self.index:
            raise ValueError(f"{name}: must be a CUDA tensor on the call's device (got {w.device})")
        if w.shape != (self.D,) or not w.is_contiguous():
            raise ValueError(f"{name}: expected a contiguous [{self.D}] tensor, got shape {tuple(w.shape)}")
        return w.data_ptr()

    def weights(self, q_weight, k_weight):
        """Addresses of both weights (0: ones) and the code of their type, one for both."""
        qw = 0 if q_weight is None else self.weight(q_weight, "q_weight")
        kw = 0 if k_weight is None else self.weight(k_weight, "k_weight")
        w = k_weight if q_weight is None else q_weight
        if w is None:
            return qw, kw, self.code
        if k_weight is not None and k_weight.dtype != w.dtype:
            raise TypeError("q_weight and k_weight: expected one type")
        return qw, kw, _DTYPE[w.dtype]

    def side(self, x, x_name, out, out_name, dy=None, dy_name="", w=0):
        """The library's descriptor of one tensor's heads (None without it)."""
        if x is None:
            return None
        dtype, index, n, D = self.dtype, self.index, self.n, self.D
        if not isinstance(x, torch.Tensor):
            self.refuse(x, x_name, "heads")
        shape, st = x.shape, x.stride()
        if len(shape) != 3 or x.dtype is not dtype or _index(x) != index or shape[2] != D or st[2] != 1 or shape[0] < n:
            self.refuse(x, x_name, "heads")
        heads = shape[1]
        if not isinstance(out, torch.Tensor):
            self.refuse(out, out_name, heads)
        o_shape, o_st = out.shape, out.stride()
        if (o_shape != shape and (len(o_shape) != 3 or o_shape[1] != heads or o_shape[2] != D or o_shape[0] < n)) \
                or out.dtype is not dtype or _index(out) != index or o_st[2] != 1:
            self.refuse(out, out_name, heads)
        if not dy_name:
            return _heads_struct(x.data_ptr(), st[0], st[1], 0, 0, 0, out.data_ptr(), o_st[0], o_st[1], w, heads, 0)
        if not isinstance(dy, torch.Tensor):
            self.refuse(dy, dy_name, heads)
        d_shape, d_st = dy.shape, dy.stride()
        if (d_shape != shape and (len(d_shape) != 3 or d_shape[1] != heads or d_shape[2] != D or d_shape[0] < n)) \
                or dy.dtype is not dtype or _index(dy) != index or d_st[2] != 1:
            self.refuse(dy, dy_name, heads)
        return _heads_struct(x.data_ptr(), st[0], st[1], dy.data_ptr(), d_st[0], d_st[1], out.data_ptr(), o_st[0], o_st[1], w,
                             heads, 0)

    def layout(self):
        n, tok = self.n, 0
        if n:
            t = self.lay.tok_id
            if not isinstance(t, torch.Tensor) or t.dtype != torch.int32:
                raise TypeError("layout.tok_id: expected an int32 tensor")
            if _index(t) != self.index:
                raise ValueError(f"layout.tok_id: must be a CUDA tensor on the call's device (got {t.device})")
            if t.numel() != n or not t.is_contiguous():
                raise ValueError(f"layout.tok_id: expected {n} contiguous ids")
            tok = t.data_ptr()
        return _layout_struct(n, 1, 0, 0, tok, self.lay.n_logical_tokens, 0, 0)

    def rotary(self, rotary, position):
        if not isinstance(rotary, Rotary):
            raise TypeError(f"rotary: expected Rotary, got {type(rotary).__name__}")
        return rotary.struct(position, self.n, self.index)


def _new(like, stream):
    """A new contiguous output with the shape of `like`, allocated on the stream that writes it, for what the
    current stream has given back may still be in use there (rows past n_tokens and padding are left as they come)."""
    if stream is None:
        return torch.empty(like.shape, dtype=like.dtype, device=like.device)
    with torch.cuda.stream(stream):
        return torch.empty(like.shape, dtype=like.dtype, device=like.device)


def _outputs(q, k, q_out, k_out, names, stream):
    """Outputs that the caller did not bring (called where one is missing, or is there without its input)."""
    if k is None:
        if k_out is not None:
            raise ValueError(f"{names[1]}: only with the keys")
    elif not isinstance(k, torch.Tensor):
        raise TypeError(f"{names[0]}: expected a torch.Tensor, got {type(k).__name__}")
    elif k_out is None:
        k_out = _new(k, stream)
    return _new(q, stream) if q_out is None else q_out, k_out


def rotary_fwd(q, k, lay, position, rotary: Rotary, q_out=None, k_out=None, stream=None):
    """Turns the heads of q and k (None: q alone) by their tokens' positions; position: int32, one per token slot.
    Returns (q_out, k_out); in place (q_out is q) columns outside the rotation keep their bits."""
    c = _Call(q, "q", lay, stream)
    if q_out is None or (k_out is None) != (k is None):
        q_out, k_out = _outputs(q, k, q_out, k_out, ("k", "k_out"), stream)
    rc = _rb._load().rotary_fwd(c.side(q, "q", q_out, "q_out"), c.side(k, "k", k_out, "k_out"), c.D, c.code, c.layout(),
                                c.rotary(rotary, position), c.stream)
    if rc:
        _rb._check(rc, "rotary_fwd")
    return q_out, k_out


def rotary_bwd(dq_out, dk_out, lay, position, rotary: Rotary, dq=None, dk=None, stream=None):
    """Gradients of rotary_fwd's inputs from those of its outputs: the heads turned back (times scale)."""
    c = _Call(dq_out, "dq_out", lay, stream)
    if dq is None or (dk is None) != (dk_out is None):
        dq, dk = _outputs(dq_out, dk_out, dq, dk, ("dk_out", "dk"), stream)
    rc = _rb._load().rotary_bwd(c.side(dq_out, "dq_out", dq, "dq"), c.side(dk_out, "dk_out", dk, "dk"), c.D, c.code, c.layout(),
                                c.rotary(rotary, position), c.stream)
    if rc:
        _rb._check(rc, "rotary_bwd")
    return dq, dk


def qk_norm_rotary_fwd(q, k, q_weight, k_weight, lay, position, rotary: Rotary, eps: float, q_out=None, k_out=None,
                       stream=None):
    """RMS norm of every head of q and k (None: q alone) with its weight (None: ones), and the rotation, in one pass
    with one rounding.  Returns (q_out, k_out)."""
    c = _Call(q, "q", lay, stream)
    if k is None and k_weight is not None:
        raise ValueError("k_weight: only with the keys")
    if q_out is None or (k_out is None) != (k is None):
        q_out, k_out = _outputs(q, k, q_out, k_out, ("k", "k_out"), stream)
    qw, kw, param = c.weights(q_weight, k_weight)
    rc = _rb._load().qk_norm_rotary_fwd(c.side(q, "q", q_out, "q_out", w=qw), c.side(k, "k", k_out, "k_out", w=kw), c.D, eps,
                                        c.code, param, c.layout(), c.rotary(rotary, position), c.stream)
    if rc:
        _rb._check(rc, "qk_norm_rotary_fwd")
    return q_out, k_out


def qk_norm_rotary_bwd(q, k, q_weight, k_weight, dq_out, dk_out, lay, position, rotary: Rotary, eps: float, dq=None,
                       dk=None, workspace=None, stream=None):
    """Backward of qk_norm_rotary_fwd (q and k are its inputs).  With a workspace the same pass adds the call's tokens
    to both weight gradients.  Returns (dq, dk); dq may be q or dq_out, dk likewise."""
    c = _Call(q, "q", lay, stream)
    if k is None and (dk_out is not None or k_weight is not None):
        raise ValueError("dk_out and k_weight: only with the keys")
    if dq is None or (dk is None) != (k is None):
        dq, dk = _outputs(q, k, dq, dk, ("k", "dk"), stream)
    qw, kw, param = c.weights(q_weight, k_weight)
    qs = c.side(q, "q", dq, "dq", dq_out, "dq_out", qw)
    ks = c.side(k, "k", dk, "dk", dk_out, "dk_out", kw)
    ws = None
    if workspace is not None:
        if not isinstance(workspace, QkNormWorkspace):
            raise TypeError(f"workspace: expected QkNormWorkspace, got {type(workspace).__name__}")
        if _index(workspace.buf) != c.index:
            raise ValueError(f"workspace: on {workspace.buf.device}, the call's heads are on cuda:{c.index}")
        mine = (lay.n_logical_tokens, q.shape[1], 0 if k is None else k.shape[1], c.D)
        if workspace.sizes != mine:
            raise ValueError(f"workspace: for (tokens, query heads, key heads, head_dim) {workspace.sizes}, the call has {mine}")
        ws = workspace.buf.data_ptr()
    rc = _rb._load().qk_norm_rotary_bwd(qs, ks, c.D, eps, c.code, param, c.layout(), c.rotary(rotary, position), ws, c.stream)
    if rc:
        _rb._check(rc, "qk_norm_rotary_bwd")
    return dq, dk


class QkNormWorkspace:
    """Device workspace of one reduction of the weight gradients of the norms of queries and keys (k_heads = 0:
    queries alone), allocated by PyTorch.  begin, any number of qk_norm_rotary_bwd calls that hold every logical
    token exactly once in all, finalize."""

    def __init__(self, n_logical_tokens: int, q_heads: int, k_heads: int, head_dim: int, device="cuda"):
        self.sizes = (int(n_logical_tokens), int(q_heads), int(k_heads), int(head_dim))
        self.bytes = int(_rb._load().qk_norm_workspace_bytes(*self.sizes))
        if self.bytes == 0:
            raise _rb.RmsNormError(-2, "qk_norm_workspace_bytes")
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
        D = self.sizes[3]
        if t is None:
            if stream is None:
                return torch.empty(D, dtype=torch.float32, device=self.buf.device)
            with torch.cuda.stream(stream):
                return torch.empty(D, dtype=torch.float32, device=self.buf.device)
        if not isinstance(t, torch.Tensor) or t.dtype != torch.float32:
            raise TypeError(f"{name}: expected a float32 tensor")
        if _index(t) != _index(self.buf) or not t.is_contiguous() or t.numel() < D:
            raise ValueError(f"{name}: expected a contiguous tensor of at least {D} elements on {self.buf.device}")
        return t

    def begin(self, stream=None):
        rc = _rb._load().qk_norm_begin(self.buf.data_ptr(), self.bytes, *self.sizes, self._stream(stream))
        if rc:
            _rb._check(rc, "qk_norm_begin")

    def finalize(self, dq_weight=None, dk_weight=None, stream=None, grad_scale: float = 1.0):
        """(dq_weight, dk_weight) of the reduction, each root multiplied once by grad_scale; without keys
        dk_weight is None."""
        at = self._stream(stream)
        dq_weight = self._gradient(dq_weight, "dq_weight", stream)
        if self.sizes[2]:
            dk_weight = self._gradient(dk_weight, "dk_weight", stream)
        elif dk_weight is not None:
            raise ValueError("dk_weight: the workspace has no keys")
        rc = _rb._load().qk_norm_finalize(self.buf.data_ptr(), *self.sizes, grad_scale, dq_weight.data_ptr(),
                                          None if dk_weight is None else dk_weight.data_ptr(), at)
        if rc:
            _rb._check(rc, "qk_norm_finalize")
        return dq_weight, dk_weight

    def status(self, stream=None) -> int:
        out = ctypes.c_int32(0)
        _rb._check(_rb._load().qk_norm_status(self.buf.data_ptr(), self._stream(stream), ctypes.byref(out)),
                   "qk_norm_status")
        return int(out.value)
