"""GPU: signs of zeros where dropout meets a residual: a dropped element is +0, so -0 in the
residual becomes +0 there (+0 + -0 = +0), and stays -0 only where -0 was kept."""
import numpy as np
import pytest
import torch

from oracle import layernorm as O
import invariant_rmsnorm_fwd_gb300 as rb

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)


@pytest.mark.parametrize("H", [8, 128, 512, 520, 5120, 8192, 12288])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32], ids=str)
@pytest.mark.parametrize("p", [0.0, 0.5, 1.0])
def test_zeros_have_the_sum_s_sign(H, dtype, p):
    if dtype == torch.float32 and H > 8192:
        pytest.skip("FP32 rows stop at 8192")
    n = 40
    cl = rb.call_layout(np.arange(n, dtype=np.int32), 1, n)
    drop = rb.Dropout(p, torch.tensor([3, 4], dtype=torch.int64, device="cuda"))
    keep = torch.tensor(O.keep_mask(3, 4, np.arange(n), H, p), device="cuda")
    zeros = torch.tensor([0.0, -0.0], dtype=dtype, device="cuda")
    g = torch.Generator("cuda").manual_seed(H)
    pick = lambda: zeros[torch.randint(0, 2, (n, H), generator=g, device="cuda")]            # noqa: E731
    x, res, dy = pick(), pick(), pick()
    word = torch.int32 if dtype == torch.float32 else torch.int16
    zero = torch.zeros((), dtype=dtype, device="cuda")
    h, _ = rb.layernorm_add_fwd(x, res, None, None, cl, 1e-5, dropout=drop)
    want = torch.where(keep, x, zero) + res
    assert torch.equal(h.view(word), want.view(word))
    y = rb.dropout_fwd(x, cl, drop)
    assert torch.equal(y.view(word), torch.where(keep, x, zero).view(word))
    dh, dx = rb.layernorm_add_bwd(x, None, dy, cl, 1e-5, dres=res, dropout=drop)
    assert torch.equal(dx.view(word), torch.where(keep, dh, zero).view(word))
