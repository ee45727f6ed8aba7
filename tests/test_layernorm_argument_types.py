"""CPU: arguments of the wrong kind are named by a TypeError of the binding, whatever the
argument is (not by a missing attribute)."""
import numpy as np
import pytest
import torch

import invariant_rmsnorm_fwd_gb300 as rb
from invariant_rmsnorm_fwd_gb300 import layernorm as ln

X, W, E = torch.zeros(4, 16, dtype=torch.bfloat16), torch.ones(16, dtype=torch.bfloat16), 1e-5
LAY = rb.CallLayout(torch.arange(4, dtype=torch.int32), None, 0, 4, 1, 4)


@pytest.fixture(autouse=True)
def as_cuda(monkeypatch):
    """Lets host tensors pass as CUDA ones, so that the checks behind that one are reached."""
    monkeypatch.setattr(ln, "_is_cuda", lambda t: True)
    monkeypatch.setattr(ln, "_current", lambda: -1)                   # what a host tensor's index is
    monkeypatch.setattr(ln, "_raw_stream", lambda index: 0)


CALLS = {
    "x": lambda v: rb.layernorm_fwd(v, W, W, LAY, E),
    "y": lambda v: rb.layernorm_fwd(X, W, W, LAY, E, y=v),
    "weight": lambda v: rb.layernorm_fwd(X, v, W, LAY, E),
    "bias": lambda v: rb.layernorm_fwd(X, W, v, LAY, E),
    "mean": lambda v: rb.layernorm_fwd(X, W, W, LAY, E, mean=v),
    "residual": lambda v: rb.layernorm_add_fwd(X, v, W, W, LAY, E),
    "weight of the chain": lambda v: rb.layernorm_add_fwd(X, X, v, W, LAY, E),
    "h": lambda v: rb.layernorm_add_fwd(X, X, W, W, LAY, E, h=v),
    "dropout": lambda v: rb.layernorm_add_fwd(X, X, W, W, LAY, E, dropout=v),
    "dy": lambda v: rb.layernorm_bwd(X, W, v, LAY, E),
    "weight of the backward pass": lambda v: rb.layernorm_bwd(X, v, X, LAY, E),
    "dx": lambda v: rb.layernorm_bwd(X, W, X, LAY, E, dx=v),
    "workspace": lambda v: rb.layernorm_bwd(X, W, X, LAY, E, workspace=v),
    "dy of the chain": lambda v: rb.layernorm_add_bwd(X, W, v, LAY, E),
    "weight of the chain's backward pass": lambda v: rb.layernorm_add_bwd(X, v, X, LAY, E),
    "dres": lambda v: rb.layernorm_add_bwd(X, W, X, LAY, E, dres=v),
    "dropout of the backward pass": lambda v: rb.layernorm_add_bwd(X, W, X, LAY, E, dropout=v),
    "dropout alone": lambda v: rb.dropout_fwd(X, LAY, v),
    "dropout alone, backward": lambda v: rb.dropout_bwd(X, LAY, v),
}


@pytest.mark.parametrize("value", [0.5, np.zeros((4, 16), dtype=np.float32), "x"], ids=["number", "array", "text"])
@pytest.mark.parametrize("name", CALLS)
def test_wrong_kinds_are_type_errors(name, value):
    with pytest.raises(TypeError, match=name.split()[0]):
        CALLS[name](value)


@pytest.mark.parametrize("name", ["x", "residual", "dy", "dy of the chain", "dropout alone"])
def test_none_is_refused_where_a_tensor_is_needed(name):
    with pytest.raises(TypeError, match=name.split()[0]):
        CALLS[name](None)
