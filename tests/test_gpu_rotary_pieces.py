"""GPU: halves that are not made of whole vectors of 8 columns, whose rows pass through places in shared memory that other
lanes read, in the layouts and aliases that the header allows: bit for bit as packed tensors give them."""
import numpy as np
import pytest
import torch

import invariant_rmsnorm_fwd_gb300 as rb

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

EPS = 1e-6
BF, FP16, F32 = torch.bfloat16, torch.float16, torch.float32


def _same(a, b):
    word = torch.int32 if a.element_size() == 4 else torch.int16
    return torch.equal(a.contiguous().view(word), b.contiguous().view(word))


def _major(t):
    """Heads outside tokens, with room behind every row."""
    n, h, D = t.shape
    out = torch.full((h, n, D + 8), 7.0, dtype=t.dtype, device="cuda")[..., :D].transpose(0, 1)
    return out.copy_(t)


class Case:
    def __init__(self, n, hq, hk, D, rot, first, dtype, param):
        g = torch.Generator("cuda").manual_seed(n + D)
        r = lambda h, s: (torch.randn(n, h, D, generator=g, device="cuda") * s).to(dtype)   # noqa: E731
        self.x, self.dy = (r(hq, 1.5), r(hk, 1.5)), (r(hq, 0.01), r(hk, 0.01))
        self.w = [(1 + 0.1 * torch.randn(D, generator=g, device="cuda")).to(param) for _ in range(2)]
        self.pos = torch.randint(-100, 5000, (n,), generator=g, device="cuda", dtype=torch.int32)
        self.rot = rb.Rotary(rot, first=first, scale=1.1)
        ids = np.arange(n, dtype=np.int32)
        ids[[n // 3, n - 2]] = -1                                     # two slots of padding
        ids[n - 5:n - 2] = ids[n - 5:n - 2][::-1].copy()              # and three tokens out of order
        self.active = torch.from_numpy(ids >= 0).cuda()
        self.lay = rb.call_layout(ids, 1, n, with_plan=False)
        self.sizes = (n, hq, hk, D)

    def fwd(self, x, out=(None, None)):
        return rb.qk_norm_rotary_fwd(*x, *self.w, self.lay, self.pos, self.rot, EPS, q_out=out[0], k_out=out[1])

    def alone(self, x, out=(None, None)):
        return rb.rotary_fwd(*x, self.lay, self.pos, self.rot, q_out=out[0], k_out=out[1])

    def back(self, x, out=(None, None)):
        return rb.rotary_bwd(*x, self.lay, self.pos, self.rot, dq=out[0], dk=out[1])

    def bwd(self, x, dy, out=(None, None)):
        ws = rb.QkNormWorkspace(*self.sizes)
        ws.begin()
        got = rb.qk_norm_rotary_bwd(*x, *self.w, *dy, self.lay, self.pos, self.rot, EPS, dq=out[0], dk=out[1], workspace=ws)
        grads = ws.finalize()
        assert ws.status() == rb.STATUS_MISSING                       # those in padding
        return (*got, *grads)

    def check(self, got, want, before=None):
        """Rows of active tokens have the bits of `want`, padding those of `before`; weight gradients are equal."""
        for i, (a, b) in enumerate(zip(got, want)):
            if a.dim() == 1:
                assert _same(a, b)
                continue
            assert _same(a[self.active], b[self.active])
            if before is not None:
                assert _same(a[~self.active], before[i][~self.active])


#        hq  hk  D    rot  first dtype  (pieces of four columns, then of two; one team a warp to 32)
CASES = [(6, 2, 72, 72, 0, BF, BF), (11, 3, 120, 120, 0, F32, F32), (2, 2, 88, 88, 0, FP16, F32), (5, 1, 512, 504, 4, BF, F32),
         (20, 4, 48, 40, 0, BF, BF), (3, 2, 16, 8, 4, F32, F32), (4, 4, 96, 24, 4, FP16, FP16),
         (6, 2, 184, 72, 6, FP16, F32), (7, 1, 80, 20, 0, F32, F32), (9, 2, 64, 20, 10, BF, BF), (3, 1, 512, 508, 2, F32, F32),
         (12, 12, 40, 36, 2, BF, F32), (3, 1, 8, 4, 2, BF, BF), (10, 2, 160, 100, 30, FP16, FP16), (4, 1, 264, 12, 250, BF, BF)]


@pytest.mark.parametrize("hq,hk,D,rot,first,dtype,param", CASES, ids=lambda v: str(v).replace("torch.", ""))
def test_layouts_and_aliases(hq, hk, D, rot, first, dtype, param):
    n = 61
    c = Case(n, hq, hk, D, rot, first, dtype, param)
    y, turned, back, grads = c.fwd(c.x), c.alone(c.x), c.back(c.dy), c.bwd(c.x, c.dy)
    joined = torch.randn(n, hq + 2 * hk, D, device="cuda").to(dtype)
    values = joined[:, hq + hk:].clone()

    def slices(v):
        joined[:, :hq], joined[:, hq:hq + hk] = v
        return joined[:, :hq], joined[:, hq:hq + hk]

    major = lambda v: tuple(_major(t) for t in v)                                           # noqa: E731
    fresh = lambda v: tuple(torch.full_like(t, 7.0) for t in v)                             # noqa: E731
    for place in (slices, major):
        c.check(c.fwd(place(c.x)), y)
        c.check(c.alone(place(c.x)), turned)
        c.check(c.back(place(c.dy)), back)
        c.check(c.bwd(place(c.x), c.dy), grads)
        c.check(c.bwd(c.x, place(c.dy)), grads)
        for run, want in ((lambda o: c.fwd(c.x, o), y), (lambda o: c.alone(c.x, o), turned), (lambda o: c.back(c.dy, o), back),
                          (lambda o: c.bwd(c.x, c.dy, o), grads)):
            out = fresh(c.x)
            c.check(run(place(out)), want, out)
        # in place: x over y, dy over dx, x over dx
        for run, src, want in ((lambda v: c.fwd(v, v), c.x, y), (lambda v: c.alone(v, v), c.x, turned),
                               (lambda v: c.back(v, v), c.dy, back), (lambda v: c.bwd(c.x, v, v), c.dy, grads),
                               (lambda v: c.bwd(v, c.dy, v), c.x, grads)):
            v = place(src)
            got = run(v)
            assert all(a is b for a, b in zip(got, v))
            c.check(got, want, src)
    assert _same(joined[:, hq + hk:], values)
    # only one of the two in place
    v = (c.x[0].clone(), c.x[1])
    c.check(c.alone(v, (v[0], torch.full_like(v[1], 7.0))), turned)
    # one token, or one head, that all read
    shared = (c.x[0][:, :1].expand(n, hq, D), c.x[1][:1].expand(n, hk, D))
    whole = tuple(t.contiguous() for t in shared)
    c.check(c.fwd(shared), c.fwd(whole))
    c.check(c.alone(shared), c.alone(whole))
    c.check(c.bwd(shared, c.dy), c.bwd(whole, c.dy))
    spread = (c.dy[0][:1].expand(n, hq, D), c.dy[1][:, :1].expand(n, hk, D))
    c.check(c.bwd(c.x, spread), c.bwd(c.x, tuple(t.contiguous() for t in spread)))


def test_many_rows_in_place():
    """Chunks of heads longer than the ring of rows, and several tokens a team: what runs ahead is not what was stored."""
    for D, rot, first, dtype in ((72, 72, 0, BF), (120, 40, 20, FP16), (72, 36, 2, F32), (24, 20, 2, BF)):
        n = 3001
        c = Case(n, 32, 8, D, rot, first, dtype, dtype)
        y, grads = c.fwd(c.x), c.bwd(c.x, c.dy)
        v = tuple(t.clone() for t in c.x)
        c.check(c.fwd(v, v), y, c.x)
        v = tuple(t.clone() for t in c.dy)
        c.check(c.bwd(c.x, v, v), grads, c.dy)
        v = tuple(t.clone() for t in c.x)
        c.check(c.bwd(v, c.dy, v), grads, c.x)
