"""Tensor memory is given back only when the CTA's stores to it have landed (CPU: the
order of the instructions in the sources; GPU: CTAs that wait for each other's columns).

`tcgen05.st` is asynchronous: without `tcgen05.wait::st` in the warp that stored, a store
may land after the columns went to another CTA, in that CTA's sums.  The race shows at
best once in many runs, so the CPU test reads the order in the source.
"""
import os
import re

import numpy as np
import pytest

from invariant_rmsnorm_fwd_gb300 import _build

KERNELS = ["layernorm_stream.cuh", "layernorm_narrow.cuh"]


@pytest.mark.parametrize("name", KERNELS)
def test_every_warp_waits_for_its_stores_before_the_columns_are_freed(name):
    with open(os.path.join(_build.CSRC, name)) as f:
        code = re.sub(r"//[^\n]*", "", f.read())
    calls = re.findall(r"umma::(\w+)\(|\b(__syncthreads)\(", code)
    calls = [a or b for a, b in calls]
    assert calls.count("tmem_dealloc") == calls.count("tmem_alloc") == 1
    at = calls.index("tmem_dealloc")
    assert calls[at - 4:at] == ["wait_st", "fence_before", "__syncthreads", "fence_after"]


@pytest.mark.gpu
@pytest.mark.parametrize("H,p,dtype", [(512, 0.1, "bfloat16"), (128, 0.1, "float16"), (1040, 0.0, "bfloat16"),
                                       (16384, 0.1, "bfloat16"), (8192, 0.0, "float32")])
def test_backward_passes_that_share_an_sms_columns(H, p, dtype):
    """Two backward calls on two streams, each with workspace and outputs of its own, many
    times over: CTAs of one take over the columns that CTAs of the other have freed."""
    import torch
    import invariant_rmsnorm_fwd_gb300 as rb
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    n = max(1500, 2 ** 21 // H)
    g = torch.Generator("cpu").manual_seed(H)
    x, dy, dres = (torch.randn(n, H, generator=g).to("cuda", getattr(torch, dtype)) for _ in range(3))
    w = (1 + 0.1 * torch.randn(H, generator=g)).to("cuda", x.dtype)
    cl = rb.call_layout(np.arange(n, dtype=np.int32), 1, n)
    drop = rb.Dropout(p, torch.tensor([3, 4], dtype=torch.int64, device="cuda")) if p else None

    class Side:
        def __init__(self):
            self.ws = rb.LayerNormWorkspace(n, H)
            self.dh = torch.zeros_like(x)
            self.dx = torch.zeros_like(x) if p else None
            self.dw, self.db = torch.zeros(H, device="cuda"), torch.zeros(H, device="cuda")

        def run(self):
            self.ws.begin()
            rb.layernorm_add_bwd(x, w, dy, cl, 1e-5, dres=dres, dropout=drop, dh=self.dh, dx=self.dx, workspace=self.ws)
            self.ws.finalize(dweight=self.dw, dbias=self.db)

        def outputs(self):
            return [t.clone() for t in (self.dh, self.dx, self.dw, self.db) if t is not None]

    a, b = Side(), Side()
    a.run()
    torch.cuda.synchronize()
    want = a.outputs()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(20):
        for side, stream in zip((a, b), streams):
            with torch.cuda.stream(stream):
                side.run()
    torch.cuda.synchronize()
    for side in (a, b):
        assert side.ws.status() == 0
        assert all(torch.equal(u, v) for u, v in zip(want, side.outputs()))
