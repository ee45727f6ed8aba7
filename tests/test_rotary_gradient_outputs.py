"""The weight gradients of queries and keys are written by CTAs without an order between them, so one buffer for both,
or two that overlap, would hold either's values: refused."""
import ctypes

import pytest
import torch

import invariant_rmsnorm_fwd_gb300 as rb

P = ctypes.c_void_p


@pytest.mark.parametrize("D", [8, 64, 512])
def test_gradients_that_overlap_are_refused(D):
    lib = rb._load()
    at = 1 << 20                                          # addresses that are never dereferenced: the check comes first
    for apart in (0, 4, -4, 4 * D - 4, 4 - 4 * D):
        assert lib.qk_norm_finalize(P(256), 64, 4, 2, D, 1.0, P(at), P(at + apart), None) == -5, apart


@pytest.mark.gpu
def test_gradients_side_by_side_are_written():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    n, D = 40, 64
    g = torch.Generator("cuda").manual_seed(3)
    r = lambda h: torch.randn(n, h, D, generator=g, device="cuda").bfloat16()               # noqa: E731
    q, k, dq, dk, w = r(3), r(2), r(3), r(2), torch.ones(D, device="cuda")
    lay = rb.call_layout(torch.arange(n, dtype=torch.int32).numpy(), 1, n, with_plan=False)
    ws = rb.QkNormWorkspace(n, 3, 2, D)
    ws.begin()
    rb.qk_norm_rotary_bwd(q, k, w, w, dq, dk, lay, torch.arange(n, dtype=torch.int32, device="cuda"), rb.Rotary(D), 1e-6,
                          workspace=ws)
    want = ws.finalize()
    both = torch.zeros(2, D, device="cuda")
    for a, b in ((0, 1), (1, 0)):
        got = ws.finalize(both[a], both[b])
        assert all(torch.equal(u, v) for u, v in zip(got, want))
    with pytest.raises(rb.RmsNormError, match="LAYOUT"):
        ws.finalize(both[0], both[0])
    assert ws.status() == 0
