"""Layer-norm backward of a call of no slots: nothing to do, and no error (a rank or a
sample without tokens).  An empty tensor's address is NULL."""
import ctypes
import itertools

import numpy as np
import pytest

import invariant_rmsnorm_fwd_gb300 as rb
from invariant_rmsnorm_fwd_gb300 import layernorm as ln

G = ctypes.c_void_p(256)                                              # never dereferenced


def _layout(n):
    return ctypes.byref(rb._Layout(n, 1, 0, 64, 256 if n else None, 4, 256, 0))


@pytest.mark.parametrize("dres,drop,workspace", list(itertools.product((False, True), repeat=3)))
def test_entry_points_accept_null_outputs_of_an_empty_call(dres, drop, workspace):
    lib = rb._load()
    d = ctypes.byref(ln._Dropout(256, 0.1)) if drop else None
    args = lambda n: (None, G, None, None, 64, 1e-5, 1.0, 0, 0, _layout(n), d, None, None, G if workspace else None,  # noqa: E731
                      None)
    assert lib.layernorm_add_bwd(*args(0)) == 0
    if not (dres or drop):
        assert lib.layernorm_bwd(None, G, None, 64, 1e-5, 0, 0, _layout(0), None, G if workspace else None, None) == 0
    # what is wrong about an empty call besides is still refused
    assert lib.layernorm_add_bwd(None, G, None, None, 12, 1e-5, 1.0, 0, 0, _layout(0), d, None, None, None, None) == -2
    assert lib.layernorm_add_bwd(None, G, None, None, 64, 1e-5, 1.0, 0, 0, _layout(0), d, None, None,
                                 ctypes.c_void_p(272), None) == -3
    # and so are the NULL outputs of a call with slots
    if drop or not workspace:
        assert lib.layernorm_add_bwd(G, G, G, None, 64, 1e-5, 1.0, 0, 0, _layout(4), d, None, None,
                                     G if workspace else None, None) == -1


@pytest.mark.gpu
@pytest.mark.parametrize("H", [128, 1040])
@pytest.mark.parametrize("slots", [0, 3])
@pytest.mark.parametrize("dres,drop,workspace", list(itertools.product((False, True), repeat=3)))
def test_empty_backward_between_others(H, slots, dres, drop, workspace):
    """slots: of the tensors; the call's layout has none."""
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    n = 70
    g = torch.Generator("cpu").manual_seed(H)
    x, dy = (torch.randn(n, H, generator=g).to("cuda", torch.bfloat16) for _ in range(2))
    w = torch.ones(H, dtype=torch.bfloat16, device="cuda")
    d = rb.Dropout(0.1, torch.tensor([1, 2], dtype=torch.int64, device="cuda")) if drop else None
    empty = rb.call_layout(np.zeros(0, dtype=np.int32), 1, n)
    full = rb.call_layout(np.arange(n, dtype=np.int32), 1, n)
    e = torch.full((slots, H), 7.0, dtype=torch.bfloat16, device="cuda")
    ws = rb.LayerNormWorkspace(n, H)
    got = []
    for with_empty in (False, True):
        ws.begin()
        if with_empty:
            for out in (None, e):
                dx = rb.layernorm_bwd(e, w, e, empty, 1e-5, dx=out, workspace=ws if workspace else None)
                dh, dx2 = rb.layernorm_add_bwd(e, w, e, empty, 1e-5, dres=e if dres else None, dropout=d, dh=out,
                                               dx=None if out is None or not drop else e.clone(),
                                               workspace=ws if workspace else None)
                assert dx.shape == dh.shape == dx2.shape == (slots, H)
            assert bool((e == 7).all())
        dx = rb.layernorm_bwd(x, w, dy, full, 1e-5, workspace=ws)
        got.append((dx,) + tuple(ws.finalize()))
        assert ws.status() == 0
    assert all(torch.equal(u, v) for u, v in zip(*got))
