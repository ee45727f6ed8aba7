"""GPU: the bounded-wait exit of the streaming layer-norm kernel.

The waits for a row's copies give up after a fixed time: the CTA reports (where it has a
workspace), waits, again with a limit, for copies still in flight, frees its tensor memory
and returns.

The wait that runs out is made by a test-only build of the library (never the product
library): RBI_TEST_WITHHOLD_EMPTY makes the kernel refill no stage, and RBI_WAIT_LIMIT_NS
shortens the limit to 10 ms.  What then happens, read from the kernel:
 * a CTA issues its first S rows, which arrive and are worked on as ever;
 * every thread waits for row S, whose copies nobody issues, and gives up after 10 ms; all
   of them see that behind the next CTA barrier and leave the row loop together;
 * no copy is in flight then, so the second wait returns at once.
The sizes leave every CTA more rows (16 to 24) than stages (at most 13).
"""
import ctypes
import time

import numpy as np
import pytest
import torch

import invariant_rmsnorm_fwd_gb300 as rb
from invariant_rmsnorm_fwd_gb300 import _build

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

N, EPS = 3000, 1e-5


@pytest.fixture(scope="module")
def variant():
    lib = ctypes.CDLL(_build.build_test_variant("waitlimit", {"RBI_TEST_WITHHOLD_EMPTY": None,
                                                              "RBI_WAIT_LIMIT_NS": "10000000ull"}))
    for name in ("layernorm_fwd", "layernorm_add_fwd", "layernorm_add_bwd", "layernorm_begin"):
        fn, product = getattr(lib, name), getattr(rb._load(), name)
        fn.argtypes, fn.restype = product.argtypes, product.restype
    return lib


def _data(H):
    g = torch.Generator("cpu").manual_seed(H)
    x, dy, res = (torch.randn(N, H, generator=g).to("cuda", torch.bfloat16) for _ in range(3))
    return x, dy, res, torch.ones(H, dtype=torch.bfloat16, device="cuda")


def _ended(call):
    """The call's launch ends by itself, soon."""
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    assert call() == 0
    torch.cuda.synchronize()
    assert time.perf_counter() - t0 < 5.0


def _cut_off(got, want):
    """Rows are the product's or untouched, some of each; none is half written."""
    same = (got.view(torch.int16) == want.view(torch.int16)).all(1)
    untouched = (got == 7).all(1)
    assert bool((same | untouched).all()) and bool(same.any()) and bool(untouched.any())


@pytest.mark.parametrize("H", [8192, 16384])
@pytest.mark.parametrize("chain", [False, True])
@pytest.mark.parametrize("grads", [False, True])
def test_backward_that_waits_in_vain_reports_and_returns(variant, H, chain, grads):
    x, dy, res, w = _data(H)
    cl = rb.call_layout(np.arange(N, dtype=np.int32), 1, N)
    drop = rb.Dropout(0.2, torch.tensor([1, 2], dtype=torch.int64, device="cuda")) if chain else None

    def product(ws):
        ws.begin()
        dh, dx = rb.layernorm_add_bwd(x, w, dy, cl, EPS, dres=res if chain else None, dropout=drop,
                                      workspace=ws if grads else None)
        return [dh, dx] + (list(ws.finalize()) if grads else [])

    ws = rb.LayerNormWorkspace(N, H)
    want = product(ws)
    dh, dx = torch.full_like(x, 7.0), torch.full_like(x, 7.0)
    ws.begin()
    L = rb._Layout(N, 1, 0, H, cl.tok_id.data_ptr(), N, cl.plan.data_ptr() if grads else None,
                   cl.plan_items if grads else 0)
    d = ctypes.byref(drop.struct(0)) if chain else None
    stream = torch.cuda.current_stream().cuda_stream
    _ended(lambda: variant.layernorm_add_bwd(x.data_ptr(), w.data_ptr(), dy.data_ptr(), res.data_ptr() if chain else None,
                                             H, EPS, 1.0, 0, 0, ctypes.byref(L), d, dh.data_ptr(),
                                             dx.data_ptr() if chain else None, ws.buf.data_ptr() if grads else None, stream))
    assert ws.status() == (rb.STATUS_TIMEOUT if grads else 0)
    _cut_off(dh, want[0])
    if chain:
        _cut_off(dx, want[1])
    # the context is usable, the tensor memory is free, and a normal call gives the same bits
    again = product(ws)
    assert ws.status() == 0
    assert all(torch.equal(u, v) for u, v in zip(want, again))


@pytest.mark.parametrize("H", [8192, 16384])
@pytest.mark.parametrize("chain", [False, True])
def test_forward_that_waits_in_vain_returns(variant, H, chain):
    """Without a workspace nothing reports it: rows stay unwritten."""
    x, dy, res, w = _data(H)
    cl = rb.call_layout(np.arange(N, dtype=np.int32), 1, N)
    product = lambda: rb.layernorm_add_fwd(x, res, w, None, cl, EPS) if chain else (  # noqa: E731
        rb.layernorm_fwd(x, w, None, cl, EPS),)
    want = product()
    got = [torch.full_like(x, 7.0) for _ in want]
    L = rb._Layout(N, 1, 0, H, cl.tok_id.data_ptr(), N, None, 0)
    stream = torch.cuda.current_stream().cuda_stream
    if chain:
        _ended(lambda: variant.layernorm_add_fwd(x.data_ptr(), res.data_ptr(), w.data_ptr(), None, H, EPS, 0, 0,
                                                 ctypes.byref(L), None, got[0].data_ptr(), got[1].data_ptr(), None, None,
                                                 stream))
    else:
        _ended(lambda: variant.layernorm_fwd(x.data_ptr(), w.data_ptr(), None, H, EPS, 0, 0, ctypes.byref(L),
                                             got[0].data_ptr(), None, None, stream))
    for g, v in zip(got, want):
        _cut_off(g, v)
    assert all(torch.equal(u, v) for u, v in zip(want, product()))
