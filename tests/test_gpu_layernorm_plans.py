"""GPU: plan items of the layer norm's backward that name blocks outside the workspace.

A plan comes from the caller (through the C ABI or a CallLayout made by hand), so an item
may be stale or made for a larger multiset.  It is reported and contributes nothing; no
kernel forms an address from it.
"""
import numpy as np
import pytest
import torch

import invariant_rmsnorm_fwd_gb300 as rb

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

GUARD = 1 << 20


def _item(kind, block, quarters, rows=None):
    """One plan item; rows: (physical row, logical row) of the used slots, by slot."""
    a = np.full(132, -1, dtype=np.int32)
    a[0:4] = kind, block, len(rows or {}), quarters
    for slot, (prow, lrow) in (rows or {}).items():
        a[4 + slot], a[68 + slot] = prow, lrow
    return a


@pytest.mark.parametrize("H", [8, 64, 256, 512, 1040, 16384])
@pytest.mark.parametrize("chain", [False, True])
@pytest.mark.parametrize("kind,quarters", [(0, 0), (2, 15), (2, 4)])
@pytest.mark.parametrize("block", [3, 4, 70000, -1, -2, 2 ** 31 - 1, -2 ** 31])
def test_items_of_blocks_outside_the_workspace_are_reported(H, chain, kind, quarters, block):
    n = 150                                                           # three blocks: 0, 1, 2
    g = torch.Generator("cpu").manual_seed(H)
    x, dy = (torch.randn(n, H, generator=g).to("cuda", torch.bfloat16) for _ in range(2))
    good = rb.call_layout(np.arange(128, dtype=np.int32), 1, n)       # blocks 0 and 1 whole
    items = good.plan.cpu().numpy().view(np.int32).reshape(-1, 132)[:good.plan_items]
    for rows in ({}, {s: (128 + s, 128 + s) for s in range(22)}):     # without rows, and with rows of the last block
        bad = _item(kind, block, quarters, rows)
        plan = torch.from_numpy(np.concatenate([items, bad[None], bad[None]]).reshape(-1).view(np.uint8).copy()).cuda()
        cl = rb.CallLayout(torch.arange(n, dtype=torch.int32, device="cuda"), plan, len(items) + 2, n, 1, n)
        ws = rb.LayerNormWorkspace(n, H)
        room = torch.full((GUARD + ws.bytes + GUARD,), 0xA5, dtype=torch.uint8, device="cuda")
        ws.buf = room[GUARD:GUARD + ws.bytes]
        assert ws.buf.data_ptr() % 256 == 0
        ws.begin()
        out = torch.full_like(x, 7.0)
        if chain:
            drop = rb.Dropout(0.25, torch.tensor([1, 2], dtype=torch.int64, device="cuda"))
            dx = torch.full_like(x, 7.0)
            rb.layernorm_add_bwd(x, None, dy, cl, 1e-5, dres=dy, dropout=drop, dh=out, dx=dx, workspace=ws)
            assert bool((dx[128:] == 7).all())
        else:
            rb.layernorm_bwd(x, None, dy, cl, 1e-5, dx=out, workspace=ws)
        torch.cuda.synchronize()
        if rows or H <= 512:
            # (rows of more than 512 columns take no address from an item without rows, and
            # need not look at it)
            assert ws.status() & rb.STATUS_PLAN
        assert bool((out[128:] == 7).all()) and not bool((out[:128] == 7).all())
        assert bool((room[:GUARD] == 0xA5).all()) and bool((room[-GUARD:] == 0xA5).all())
        # the good items' sums are there all the same: the last block's rows are missing
        again = rb.LayerNormWorkspace(n, H)
        again.begin()
        if chain:
            rb.layernorm_add_bwd(x, None, dy, good, 1e-5, dres=dy, dropout=drop, workspace=again)
        else:
            rb.layernorm_bwd(x, None, dy, good, 1e-5, workspace=again)
        got, want = ws.finalize(), again.finalize()
        assert ws.status() & rb.STATUS_MISSING
        assert all(torch.equal(u, v) for u, v in zip(got, want))
