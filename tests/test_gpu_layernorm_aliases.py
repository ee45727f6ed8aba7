"""GPU: outputs over inputs, every alias that the header allows, at a width of each kernel
form and with more rows than a CTA or a team keeps on its way."""
import itertools

import numpy as np
import pytest
import torch

import invariant_rmsnorm_fwd_gb300 as rb

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

BF, FP16, F32 = torch.bfloat16, torch.float16, torch.float32
# narrow teams, one and two CTAs an SM, 257 to 320 threads, dres staged or read in place
WIDTHS = [(24, BF, 1, 70001), (128, FP16, 4, 4001), (512, F32, 1, 6001), (1040, BF, 2, 4001), (5120, BF, 1, 3001),
          (5128, F32, 1, 1501), (8192, F32, 1, 1501), (16384, BF, 1, 1501)]


def _same(a, b):
    word = torch.int32 if a.element_size() == 4 else torch.int16
    return torch.equal(a.contiguous().view(word), b.contiguous().view(word))


@pytest.mark.parametrize("H,dtype,R,n", WIDTHS, ids=lambda v: str(v).replace("torch.", ""))
@pytest.mark.parametrize("p", [0.0, 0.3])
def test_every_allowed_alias_gives_the_same_bits(H, dtype, R, n, p):
    g = torch.Generator("cuda").manual_seed(H)
    ids = np.insert(np.arange(n), np.arange(0, n, 61), -1).astype(np.int32)
    T = ids.size
    cl = rb.call_layout(ids, R, n)
    rnd = lambda s: (torch.randn(T, R, H, generator=g, device="cuda") * s).to(dtype)         # noqa: E731
    src = {"x": rnd(1.0), "residual": rnd(1.0), "dy": rnd(0.01), "dres": rnd(0.01)}
    w, b = (torch.randn(H, generator=g, device="cuda").to(dtype) for _ in range(2))
    drop = rb.Dropout(p, torch.tensor([9, 1], dtype=torch.int64, device="cuda")) if p else None
    act = cl.tok_id >= 0
    ws = rb.LayerNormWorkspace(n * R, H)

    def check(what, got, want):
        assert _same(got[act], want[act]), what

    # forward
    y0 = rb.layernorm_fwd(src["x"], w, b, cl, 1e-5)
    x = src["x"].clone()
    rb.layernorm_fwd(x, w, b, cl, 1e-5, y=x)
    check("y over x", x, y0)
    assert _same(x[~act], src["x"][~act])
    h0, y0 = rb.layernorm_add_fwd(src["x"], src["residual"], w, b, cl, 1e-5, dropout=drop)
    for at_h, at_y in itertools.product((None, "x", "residual"), repeat=2):
        if at_h == at_y:
            continue
        t = {k: v.clone() for k, v in src.items()}
        h, y = rb.layernorm_add_fwd(t["x"], t["residual"], w, b, cl, 1e-5, h=t.get(at_h), y=t.get(at_y), dropout=drop)
        check(("h", at_h, at_y), h, h0)
        check(("y", at_h, at_y), y, y0)
    src["h"] = h0.clone()
    src["h"][~act] = 3.0
    # backward
    for grads in (False, True):
        def run(t, **kw):
            if grads:
                ws.begin()
            out = rb.layernorm_add_bwd(t["h"], w, t["dy"], cl, 1e-5, dres=t["dres"], dropout=drop,
                                       workspace=ws if grads else None, **kw)
            more = ws.finalize() if grads else ()
            assert not grads or ws.status() == 0
            return out, more
        (dh0, dx0), g0 = run(src)
        for at_h, at_x in itertools.product((None, "h", "dy", "dres"), repeat=2):
            if at_h == at_x or (at_x and not p):
                continue
            t = {k: v.clone() for k, v in src.items()}
            kw = {"dh": t.get(at_h)}
            if p:
                kw["dx"] = t.get(at_x)
            (dh, dx), g1 = run(t, **kw)
            check(("dh", at_h, at_x), dh, dh0)
            check(("dx", at_h, at_x), dx, dx0)
            assert all(_same(u, v) for u, v in zip(g0, g1)), (at_h, at_x)
            for k in (at_h, at_x):
                assert k is None or _same(t[k][~act], src[k][~act]), k
        for at in ("h", "dy"):
            t = {k: v.clone() for k, v in src.items()}
            want = rb.layernorm_bwd(src["h"], w, src["dy"], cl, 1e-5)
            if grads:
                ws.begin()
            got = rb.layernorm_bwd(t["h"], w, t["dy"], cl, 1e-5, dx=t[at], workspace=ws if grads else None)
            check(("layernorm_bwd", at), got, want)
            if grads:
                assert all(_same(u, v) for u, v in zip(g0, ws.finalize()))
