"""Layer norm and dropout: what the C entry points and the binding refuse (CPU, no GPU needed)."""
import ctypes

import numpy as np
import pytest
import torch

import invariant_rmsnorm_fwd_gb300 as rb
from invariant_rmsnorm_fwd_gb300 import layernorm as ln

P = ctypes.c_void_p
G, G2 = P(256), P(512)                                    # never dereferenced: checks fail first


def _layout(n=4, rpt=1, stride=64, tok=256, n_logical=4, plan=None, items=0, reserved=0):
    return ctypes.byref(rb._Layout(n, rpt, reserved, stride, tok, n_logical, plan, items))


def _fwd(lib, H=64, x=G, w=G, b=G, eps=1e-5, dt=0, pdt=0, lay=None, y=G):
    return lib.layernorm_fwd(x, w, b, H, eps, dt, pdt, lay or _layout(), y, None, None, None)


def test_forward_refusals():
    lib = rb._load()
    for H in (0, 4, 12, -8, 16392):
        assert _fwd(lib, H=H, lay=_layout(stride=1 << 16)) == -2
    assert _fwd(lib, H=8200, dt=2, pdt=2, lay=_layout(stride=8200)) == -2          # FP32 rows stop at 8192
    assert _fwd(lib, x=None) == -1 and _fwd(lib, y=None) == -1
    assert _fwd(lib, x=P(264)) == -3 and _fwd(lib, w=P(264)) == -3 and _fwd(lib, b=P(260)) == -3
    assert _fwd(lib, lay=_layout(stride=68)) == -3 and _fwd(lib, lay=_layout(stride=56)) == -4
    assert _fwd(lib, lay=_layout(rpt=2)) == -4                                       # stride < 2 rows
    assert _fwd(lib, lay=_layout(rpt=0)) == -5 and _fwd(lib, lay=_layout(reserved=1)) == -5
    assert _fwd(lib, lay=_layout(n=-1)) == -5 and _fwd(lib, lay=_layout(n=1 << 31)) == -5
    assert _fwd(lib, lay=_layout(n=1 << 30, rpt=2, stride=128)) == -5
    assert _fwd(lib, lay=_layout(tok=None)) == -1
    assert _fwd(lib, dt=3, pdt=3) == -14 and _fwd(lib, dt=-1) == -14
    assert _fwd(lib, dt=0, pdt=1) == -14 and _fwd(lib, dt=2, pdt=0) == -14
    for eps in (float("nan"), float("inf"), -1e-5):
        assert _fwd(lib, eps=eps) == -13
    assert _fwd(lib, lay=_layout(n=0, tok=None)) == 0                                # nothing to do, no device
    assert lib.layernorm_fwd(G, G, G, 64, 1e-5, 0, 0, None, G, None, None, None) == -1


def test_add_and_dropout_refusals():
    lib = rb._load()
    d = lambda p, s=256: ctypes.byref(ln._Dropout(s, p))                             # noqa: E731
    add = lambda drop=None, h=G, y=G2, res=G: lib.layernorm_add_fwd(                # noqa: E731
        G, res, G, G, 64, 1e-5, 0, 0, _layout(), drop, h, y, None, None, None)
    assert add(y=G) == -5 and add(res=None) == -1 and add(h=None) == -1
    for p in (-0.1, 1.1, float("nan")):
        assert add(d(p)) == -13
        assert lib.dropout_fwd(G, 64, 0, _layout(), d(p), G, None) == -13
    assert add(d(0.1, None)) == -1 and add(d(0.1, 260)) == -3
    drop = lambda H=64, x=G, y=G, dr=d(0.1), dt=0, lay=None: lib.dropout_bwd(       # noqa: E731
        x, H, dt, lay or _layout(), dr, y, None)
    assert drop(dr=None) == -1 and drop(x=None) == -1 and drop(y=None) == -1
    assert drop(H=12) == -2 and drop(H=(1 << 20) + 8, lay=_layout(stride=1 << 21)) == -2
    assert drop(x=P(264)) == -3 and drop(dt=7) == -14


def test_backward_refusals():
    lib = rb._load()
    d = ctypes.byref(ln._Dropout(256, 0.1))

    def bwd(drop=None, dres=None, dh=G, dx=None, ws=None, scale=1.0, lay=None, dy=G):
        return lib.layernorm_add_bwd(G, G, dy, dres, 64, 1e-5, scale, 0, 0, lay or _layout(), drop, dh, dx, ws, None)

    assert bwd(dh=None) == -1 and bwd(dh=None, dres=G, ws=G) == -1 and bwd(dh=None, drop=d, dx=G2, ws=G) == -1
    assert bwd(drop=d) == -1 and bwd(drop=d, dx=G) == -5
    assert bwd(ws=G) == -7                                                           # no plan
    assert bwd(ws=P(272), lay=_layout(plan=256, items=1)) == -3
    assert bwd(scale=float("nan")) == -13 and bwd(dy=None) == -1
    assert bwd(dres=P(264)) == -3 and bwd(drop=d, dx=P(264)) == -3
    assert lib.layernorm_bwd(G, G, G, 64, 1e-5, 0, 0, _layout(), None, None, None) == -1


def test_workspace_refusals_and_size():
    lib = rb._load()
    assert lib.layernorm_workspace_bytes(64, 12) == 0 and lib.layernorm_workspace_bytes(-1, 64) == 0
    assert lib.layernorm_workspace_bytes(1 << 31, 64) == 0 and lib.layernorm_workspace_bytes(64, 16392) == 0
    n, h = 1000, 128
    assert lib.layernorm_workspace_bytes(n, h) >= 256 + 16 * 8 + n + 16 * 8 * 2 * h * 4 + n * 2 * h * 4
    assert lib.layernorm_workspace_bytes(n, h) % 256 == 0
    assert lib.layernorm_begin(G, 16, 64, 8, None) == -6 and lib.layernorm_begin(P(272), 1 << 20, 64, 8, None) == -3
    assert lib.layernorm_begin(None, 1 << 20, 64, 8, None) == -1
    assert lib.layernorm_finalize(G, 64, 8, 1.0, None, None, None) == -1
    assert lib.layernorm_finalize(G, 64, 8, float("inf"), G, G, None) == -13
    assert lib.layernorm_finalize(G, 64, 8, 1.0, P(260), G, None) == -3
    assert lib.layernorm_finalize(G, 64, 12, 1.0, G, G, None) == -2


def test_binding_refuses_host_tensors_and_wrong_arguments():
    lay = rb.CallLayout(torch.arange(4, dtype=torch.int32), None, 0, 4, 1, 4)
    x, w = torch.zeros(4, 16, dtype=torch.bfloat16), torch.ones(16, dtype=torch.bfloat16)
    drop = rb.Dropout(0.1, torch.zeros(2, dtype=torch.int64))
    with pytest.raises(ValueError, match="CUDA tensor"):
        rb.layernorm_fwd(x, w, w, lay, 1e-5)
    with pytest.raises(ValueError, match="CUDA tensor"):
        rb.layernorm_add_fwd(x, x, w, w, lay, 1e-5)
    with pytest.raises(ValueError, match="CUDA tensor"):
        rb.layernorm_bwd(x, w, x, lay, 1e-5)
    with pytest.raises(ValueError, match="CUDA tensor"):
        rb.layernorm_add_bwd(x, w, x, lay, 1e-5)
    with pytest.raises(ValueError, match="CUDA tensor"):
        rb.dropout_fwd(x, lay, drop)
    with pytest.raises(TypeError, match="torch.Tensor"):
        rb.layernorm_fwd(np.zeros((4, 16)), w, w, lay, 1e-5)
    with pytest.raises(ValueError, match="CUDA"):
        drop.struct(0)


@pytest.fixture
def as_cuda(monkeypatch):
    """Lets host tensors pass as CUDA ones, so that the checks behind that one are reached."""
    monkeypatch.setattr(ln, "_is_cuda", lambda t: True)
    monkeypatch.setattr(ln, "_current", lambda: -1)                   # what a host tensor's index is
    monkeypatch.setattr(ln, "_raw_stream", lambda index: 0)


def test_binding_checks_shapes_types_and_strides(as_cuda):
    lay = rb.CallLayout(torch.arange(4, dtype=torch.int32), None, 0, 4, 1, 4)
    x, w = torch.zeros(4, 16, dtype=torch.bfloat16), torch.ones(16, dtype=torch.bfloat16)
    e = 1e-5
    with pytest.raises(TypeError, match="bfloat16, float16 or float32"):
        rb.layernorm_fwd(x.double(), w, w, lay, e)
    with pytest.raises(TypeError, match="y"):
        rb.layernorm_fwd(x, w, w, lay, e, y=x.float())
    with pytest.raises(ValueError, match="token slots"):
        rb.layernorm_fwd(x[:3], w, w, lay, e)
    with pytest.raises(ValueError, match="token stride"):
        rb.layernorm_fwd(x, w, w, lay, e, y=torch.zeros(4, 32, dtype=x.dtype)[:, :16])
    with pytest.raises(ValueError, match="column stride"):
        rb.layernorm_fwd(torch.zeros(16, 4, dtype=x.dtype).t(), w, w, lay, e)
    with pytest.raises(ValueError, match="expected"):
        rb.layernorm_fwd(x, w, w, lay, e, y=torch.zeros(4, 24, dtype=x.dtype))
    with pytest.raises(ValueError, match="shape"):
        rb.layernorm_fwd(x.reshape(4, 2, 8)[0, 0], w, w, lay, e)
    with pytest.raises(ValueError, match="weight"):
        rb.layernorm_fwd(x, w[:8], w, lay, e)
    with pytest.raises(TypeError, match="weight"):
        rb.layernorm_fwd(x, w.half(), None, lay, e)
    with pytest.raises(TypeError, match="one type"):
        rb.layernorm_fwd(x, w, w.float(), lay, e)
    with pytest.raises(TypeError, match="workspace"):
        rb.layernorm_bwd(x, w, x, lay, e, workspace=x)
    with pytest.raises(ValueError, match="dx: only with a dropout"):
        rb.layernorm_add_bwd(x, w, x, lay, e, dx=x)
    with pytest.raises(TypeError, match="Dropout"):
        rb.dropout_fwd(x, lay, 0.1)
    with pytest.raises(ValueError, match="not in"):
        rb.Dropout(1.5, torch.zeros(2, dtype=torch.int64)).struct(-1)
    with pytest.raises(ValueError, match="two int64"):
        rb.Dropout(0.5, torch.zeros(3, dtype=torch.int64)).struct(-1)
    with pytest.raises(TypeError, match="state"):
        rb.Dropout(0.5, torch.zeros(2)).struct(-1)


def test_tensors_off_the_current_device_are_refused(as_cuda, monkeypatch):
    lay = rb.CallLayout(torch.arange(4, dtype=torch.int32), None, 0, 4, 1, 4)
    x, w = torch.zeros(4, 16, dtype=torch.bfloat16), torch.ones(16, dtype=torch.bfloat16)
    monkeypatch.setattr(ln, "_current", lambda: 1)
    with pytest.raises(ValueError, match="current device"):
        rb.layernorm_fwd(x, w, w, lay, 1e-5)
    with pytest.raises(ValueError, match="current device"):
        rb.dropout_bwd(x, lay, rb.Dropout(0.1, torch.zeros(2, dtype=torch.int64)))


def test_unaligned_statistics_ids_and_plans_are_refused():
    lib = rb._load()
    for mean, rstd in ((P(258), None), (None, P(257))):
        assert lib.layernorm_fwd(G, G, G, 64, 1e-5, 0, 0, _layout(), G, mean, rstd, None) == -3
        assert lib.layernorm_add_fwd(G, G, G, G, 64, 1e-5, 0, 0, _layout(), None, G, G2, mean, rstd, None) == -3
    assert _fwd(lib, lay=_layout(tok=258)) == -3
    assert lib.layernorm_bwd(G, G, G, 64, 1e-5, 0, 0, _layout(plan=258, items=1), G, G, None) == -3
