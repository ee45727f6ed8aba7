"""Two copies of the library in one process do not share state (another build of it, or one
that a program brings along): every copy asks for its own kernels' attributes.

A static of a function template with external linkage is a unique global symbol, one object
for the whole process however the copies are loaded.
"""
import ctypes
import shutil
import subprocess

import numpy as np
import pytest

import invariant_rmsnorm_fwd_gb300 as rb


def test_no_symbol_is_shared_between_copies():
    rb._load()
    nm = shutil.which("nm")
    if nm is None:
        pytest.skip("no nm")
    out = subprocess.run([nm, "-D", "--defined-only", rb.library_path()], capture_output=True, text=True, check=True).stdout
    shared = [line for line in out.splitlines() if line.split()[1] == "u"]
    assert not shared, (len(shared), shared[:2])


@pytest.mark.gpu
@pytest.mark.parametrize("H", [64, 512, 1040, 8192])
def test_both_copies_run(tmp_path, H):
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    n = 200
    product = rb._load()
    path = shutil.copy(rb.library_path(), tmp_path / "copy.so")
    copy = ctypes.CDLL(str(path))
    copy.layernorm_bwd.argtypes = product.layernorm_bwd.argtypes
    copy.layernorm_fwd.argtypes = product.layernorm_fwd.argtypes
    g = torch.Generator("cpu").manual_seed(H)
    x, dy = (torch.randn(n, H, generator=g).to("cuda", torch.bfloat16) for _ in range(2))
    cl = rb.call_layout(np.arange(n, dtype=np.int32), 1, n)
    ws = rb.LayerNormWorkspace(n, H)
    ws.begin()
    want = rb.layernorm_fwd(x, None, None, cl, 1e-5), rb.layernorm_bwd(x, None, dy, cl, 1e-5, workspace=ws)
    grads = ws.finalize()
    y, dx = torch.zeros_like(x), torch.zeros_like(x)
    L = ctypes.byref(rb._Layout(n, 1, 0, H, cl.tok_id.data_ptr(), n, cl.plan.data_ptr(), cl.plan_items))
    s = torch.cuda.current_stream().cuda_stream
    ws.begin()
    assert copy.layernorm_fwd(x.data_ptr(), None, None, H, 1e-5, 0, 0, L, y.data_ptr(), None, None, s) == 0
    assert copy.layernorm_bwd(x.data_ptr(), None, dy.data_ptr(), H, 1e-5, 0, 0, L, dx.data_ptr(), ws.buf.data_ptr(), s) == 0
    assert torch.equal(y, want[0]) and torch.equal(dx, want[1])
    assert all(torch.equal(u, v) for u, v in zip(grads, ws.finalize())) and ws.status() == 0
