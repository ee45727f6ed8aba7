"""GPU: masks of rows that several ranks hold (the ranks run one after the other here).

Under local ids every rank draws the masks of rows 0, 1, 2, ...; under global ids it draws
one device's, and the parameter gradients come from the same rows under local ids.
"""
import numpy as np
import pytest
import torch

import invariant_rmsnorm_fwd_gb300 as rb

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)


def _same(a, b):
    return torch.equal(a.contiguous().view(torch.int16), b.contiguous().view(torch.int16))


@pytest.mark.parametrize("H,R", [(64, 3), (128, 32), (1040, 1), (8200, 1)])
def test_global_ids_give_one_devices_masks(H, R):
    n, cuts = 300, [0, 128, 192, 300]
    g = torch.Generator("cuda").manual_seed(H)
    x, res, dy, dres = (torch.randn(n, R, H, generator=g, device="cuda").to(torch.bfloat16) for _ in range(4))
    w = torch.randn(H, generator=g, device="cuda").to(torch.bfloat16)
    drop = rb.Dropout(0.4, torch.tensor([11, 12], dtype=torch.int64, device="cuda"))
    one = rb.call_layout(np.arange(n, dtype=np.int32), R, n)
    h0, y0 = rb.layernorm_add_fwd(x, res, w, None, one, 1e-5, dropout=drop)
    dh0, dx0 = rb.layernorm_add_bwd(h0, w, dy, one, 1e-5, dres=dres, dropout=drop)
    z0 = rb.dropout_fwd(x, one, drop)
    local_first = []
    for a, b in zip(cuts[:-1], cuts[1:]):
        ids = np.arange(a, b, dtype=np.int32)
        both = rb.call_layout(ids, R, n, with_plan=False)                    # global ids
        v = [t[a:b] for t in (x, res, dy, dres)]
        h, y = rb.layernorm_add_fwd(v[0], v[1], w, None, both, 1e-5, dropout=drop)
        dh, dx = rb.layernorm_add_bwd(h, w, v[2], both, 1e-5, dres=v[3], dropout=drop)
        for got, want in ((h, h0), (y, y0), (dh, dh0), (dx, dx0), (rb.dropout_fwd(v[0], both, drop), z0)):
            assert _same(got, want[a:b])
        # the layout's own count does not matter to calls without a plan
        beyond = rb.CallLayout(both.tok_id, None, 0, b - a, R, b - a)
        assert _same(rb.dropout_fwd(v[0], beyond, drop), z0[a:b])
        # gradients: local ids, no dx
        local = rb.call_layout(np.arange(b - a, dtype=np.int32), R, b - a)
        ws = rb.LayerNormWorkspace((b - a) * R, H)
        ws.begin()
        rb.layernorm_bwd(h0[a:b], w, v[2], local, 1e-5, workspace=ws, write_dx=False)
        ws.finalize()
        assert ws.status() == 0
        ones = torch.ones(64, R, H, dtype=torch.bfloat16, device="cuda")
        local_first.append(rb.dropout_fwd(ones, rb.call_layout(np.arange(64, dtype=np.int32), R, 64, with_plan=False), drop))
    assert all(_same(t, local_first[0]) for t in local_first)               # what local ids give
