"""GPU: rotary positions and the norms of queries and keys with rotation, against the FP64
oracle, bit for bit across layouts, and at the sizes, strides and calls where they can go
wrong.

Tolerances: the oracle's own bound of an FP32 evaluation (oracle/rotary.py derives it),
plus half a step of the output's type for its one rounding.
"""
import numpy as np
import pytest
import torch

import invariant_rmsnorm_fwd_gb300 as rb
from invariant_rmsnorm_fwd_gb300 import harness
from invariant_rmsnorm_fwd_gb300 import layout as L
from oracle import rotary as O

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

EPS = 1e-6
BF, FP16, F32 = torch.bfloat16, torch.float16, torch.float32


def _name(dtype):
    return str(dtype).split(".")[1]


def _word(t):
    return t.contiguous().view(torch.int32 if t.element_size() == 4 else torch.int16)


def _same(a, b):
    return torch.equal(_word(a), _word(b))


def _f64(t):
    return t.double().cpu().numpy()


def _within(name, got, ref, bound):
    err = np.abs(got - ref)
    bad = ~(err <= bound)
    assert not bad.any(), (name, int(bad.sum()), float((err / np.maximum(bound, 1e-300)).max()), np.argwhere(bad)[:3].tolist())


class Setup:
    """Inputs of n logical tokens and the rotation, from a seed."""

    def __init__(self, n, hq, hk, D, rot, first, inter, dtype, param=None, scale=1.0, top=5000, seed=0):
        g = torch.Generator("cpu").manual_seed(seed + 31 * D + n)
        r = lambda h, s: (torch.randn(n, h, D, generator=g) * s).to("cuda", dtype)          # noqa: E731
        self.q, self.dq = r(hq, 1.5), r(hq, 0.01)
        self.k, self.dk = (r(hk, 1.5), r(hk, 0.01)) if hk else (None, None)
        w = lambda: (1 + 0.1 * torch.randn(D, generator=g)).to("cuda", param or dtype)      # noqa: E731
        self.qw, self.kw = w(), w() if hk else None
        self.pos = torch.randint(-top // 10, top + 1, (n,), generator=g, dtype=torch.int32).cuda()
        self.freq = rb.rotary_frequencies(rot)
        self.rot = rb.Rotary(rot, interleaved=inter, first=first, scale=scale)
        self.args = (rot, first, inter, scale)
        self.n, self.dtype = n, dtype

    def layout(self, ids=None):
        return rb.call_layout(np.arange(self.n, dtype=np.int32) if ids is None else ids, 1, self.n, with_plan=False)

    def fwd(self, **kw):
        return rb.qk_norm_rotary_fwd(self.q, self.k, self.qw, self.kw, self.layout(), self.pos, self.rot, EPS, **kw)

    def workspace(self):
        return rb.QkNormWorkspace(self.n, self.q.shape[1], 0 if self.k is None else self.k.shape[1], self.q.shape[2])

    def bwd(self, ws=None, **kw):
        return rb.qk_norm_rotary_bwd(self.q, self.k, self.qw, self.kw, self.dq, self.dk, self.layout(), self.pos, self.rot,
                                     EPS, workspace=ws, **kw)

    def check(self, y, dx, dw, x, w, dy, s=1.0, eps=EPS, pos=None):
        pos, nm = _f64(self.pos if pos is None else pos), _name(self.dtype)
        w64 = np.ones(x.shape[-1]) if w is None else _f64(w)
        if y is not None:
            ref, err = O.forward(_f64(x), w64, pos, self.freq, *self.args, eps)
            _within("y", _f64(y), ref, O.rounded(err, ref, nm))
        ref, dw64, err, e_dw = O.backward(_f64(x), w64, _f64(dy), pos, self.freq, *self.args, eps)
        _within("dx", _f64(dx), ref, O.rounded(err, ref, nm))
        if dw is not None:
            _within("dweight", _f64(dw), s * dw64, abs(s) * e_dw + O.U * np.abs(s * dw64))


#        hq  hk  D    rot  first inter dtype params scale
CASES = [(32, 8, 128, 128, 0, False, BF, None, 1.0), (4, 1, 64, 64, 0, True, FP16, F32, 1.0),
         (7, 1, 80, 20, 0, False, F32, None, 1.1), (1, 1, 8, 8, 0, False, BF, None, 1.0),
         (3, 2, 16, 4, 12, True, BF, F32, 0.9), (2, 2, 24, 12, 6, False, FP16, None, 1.0),
         (9, 3, 72, 72, 0, True, F32, None, 1.0), (16, 1, 256, 64, 192, True, FP16, F32, 1.0),
         (10, 5, 96, 48, 16, False, BF, F32, 1.2), (5, 0, 128, 32, 96, False, BF, None, 1.0),
         (17, 9, 40, 24, 2, True, F32, None, 1.0), (2, 1, 512, 512, 0, False, BF, None, 1.0),
         (1, 3, 504, 8, 496, True, FP16, None, 1.0), (3, 1, 512, 20, 490, False, F32, None, 1.0),
         (12, 12, 192, 64, 128, False, BF, None, 1.0), (64, 8, 32, 32, 0, False, FP16, None, 1.0),
         (6, 2, 112, 56, 0, True, BF, None, 1.0), (33, 1, 160, 160, 0, True, BF, F32, 1.0),
         # halves that begin or end inside a vector of 8 columns, on multiples of 4 columns and of 2
         (4, 2, 72, 72, 0, False, BF, None, 1.0), (2, 2, 88, 88, 0, False, FP16, F32, 1.0), (9, 1, 120, 120, 0, False, F32, None, 1.0),
         (8, 4, 96, 24, 4, False, BF, None, 1.1), (2, 1, 64, 8, 52, False, FP16, None, 1.0), (1, 1, 16, 8, 4, False, F32, F32, 1.0),
         (3, 3, 256, 200, 20, False, BF, F32, 1.0), (2, 1, 184, 72, 6, False, FP16, None, 1.0), (5, 1, 48, 40, 0, False, BF, None, 1.0),
         (2, 1, 512, 504, 4, False, BF, F32, 1.0), (2, 2, 512, 508, 2, False, F32, None, 1.0), (3, 1, 8, 4, 2, False, BF, None, 1.0),
         (13, 2, 32, 28, 4, False, FP16, None, 0.8), (3, 1, 144, 8, 60, False, F32, None, 1.0), (1, 0, 176, 172, 4, False, BF, None, 1.0)]


@pytest.mark.parametrize("hq,hk,D,rot,first,inter,dtype,param,scale", CASES,
                         ids=lambda v: str(v).replace("torch.", ""))
def test_norm_and_rotation_match_oracle_and_are_layout_invariant(hq, hk, D, rot, first, inter, dtype, param, scale):
    lengths = np.asarray([70, 3, 130, 1, 64, 9])
    s = Setup(int(lengths.sum()), hq, hk, D, rot, first, inter, dtype, param, scale)
    f = 1.0 / s.n
    runs, lays = {}, {}
    for kind in L.LAYOUT_KINDS + ("permuted_chunked", "padded_right_chunked"):
        lays[kind] = L.make_layout(kind, lengths, chunk=37)
        runs[kind] = harness.run_layout_qk_norm_rotary(lays[kind], s.q, s.k, s.dq, s.dk, s.qw, s.kw, s.pos, s.rot, EPS, f)
    rep = harness.assert_batch_invariant(runs, lays)
    assert rep.green, rep.summary()
    assert all(r.status == 0 and r.untouched_padding for r in runs.values())
    r = runs["full"]
    s.check(r.y, r.dx, r.dweight, s.q, s.qw, s.dq, f)
    if hk:
        s.check(r.k, r.dk, r.dk_weight, s.k, s.kw, s.dk, f)


@pytest.mark.parametrize("hq,hk,D,rot,first,inter,dtype,param,scale", CASES,
                         ids=lambda v: str(v).replace("torch.", ""))
def test_rotation_alone(hq, hk, D, rot, first, inter, dtype, param, scale):
    s = Setup(77, hq, hk, D, rot, first, inter, dtype, param, scale)
    outside = np.ones(D, bool)
    outside[first:first + rot] = False
    special = torch.tensor([float("inf"), float("-inf"), float("nan"), -0.0], dtype=dtype, device="cuda")
    if outside.any():                                                 # values that arithmetic would change
        cols = torch.from_numpy(np.flatnonzero(outside)[:4]).cuda()
        s.q[5, 0, cols] = special[:cols.numel()]
    ids = np.arange(s.n, dtype=np.int32)
    ids[[0, 9, 76]] = -1
    act = ids >= 0
    lay = rb.call_layout(ids, 1, s.n, with_plan=False)
    for back in (False, True):
        fn = rb.rotary_bwd if back else rb.rotary_fwd
        names = ("dq", "dk") if back else ("q_out", "k_out")
        fill = [torch.full_like(t, 7.0) for t in (s.q, s.k) if t is not None]
        out = fn(s.q, s.k, lay, s.pos, s.rot, **dict(zip(names, fill)))
        for x, y in zip((s.q, s.k), out):
            if x is None:
                assert y is None
                continue
            assert bool((y[~act] == 7).all())
            assert _same(y[act][..., outside], x[act][..., outside])
            xf = x.clone()
            xf[..., outside] = 0
            ref, err = O.rotate(_f64(xf)[act], _f64(s.pos)[act], s.freq, rot, first, inter, scale, back)
            _within("y", _f64(y[act])[..., ~outside], ref[..., ~outside], O.rounded(err, ref, _name(dtype))[..., ~outside])
            z = x.clone()                                             # in place: the same bits, padding as it was
            fn(z, None, lay, s.pos, s.rot, **{names[0]: z})
            assert _same(z[act], y[act]) and _same(z[~act], x[~act])


def test_special_bits_outside_the_rotation_are_copied():
    n, D = 5, 64
    for dtype, word, bits in ((BF, torch.int16, [0x7FA5, -0x5B, -0x8000, 0x0001]), (F32, torch.int32, [0x7F800123, -1, 1, -2 ** 31])):
        x = torch.zeros(n, 2, D, dtype=dtype, device="cuda")
        x.view(word)[:, :, 32:36] = torch.tensor(bits, dtype=word, device="cuda")
        x.view(word)[:, :, 60:64] = torch.tensor(bits, dtype=word, device="cuda")
        pos = torch.arange(n, dtype=torch.int32, device="cuda")
        lay = rb.call_layout(np.arange(n, dtype=np.int32), 1, n, with_plan=False)
        for rot in (rb.Rotary(32), rb.Rotary(20, interleaved=True), rb.Rotary(16, first=16), rb.Rotary(24, first=2)):
            y, _ = rb.rotary_fwd(x, None, lay, pos, rot)
            out = torch.ones(D, dtype=torch.bool, device="cuda")
            out[rot.first:rot.first + rot.rotary_dim] = False         # inside, 0 c - 0 s is -0 where c < 0 < s
            assert torch.equal(y.view(word)[..., out], x.view(word)[..., out]) and not y[..., ~out].any()


def test_far_and_negative_positions():
    """Positions over the whole int32 range against the fraction of a turn in exact arithmetic."""
    p = [0, 1, -1, 4095, 2 ** 20 + 3, 2 ** 24 + 1, 123456789, -987654321, 2 ** 31 - 1, -2 ** 31]
    D = 64
    pos = torch.tensor(p, dtype=torch.int32, device="cuda")
    lay = rb.call_layout(np.arange(len(p), dtype=np.int32), 1, len(p), with_plan=False)
    freq = rb.rotary_frequencies(D)
    freq[-1] = -0.7                                                   # turns the other way
    freq[-2] = 3.0
    x = torch.zeros(len(p), 1, D, dtype=F32, device="cuda")
    x[..., ::2] = 1.0
    y, _ = rb.rotary_fwd(x, None, lay, pos, rb.Rotary(D, interleaved=True, inv_freq=freq))
    ref = np.array([[O.cos_sin_far(a, f) for f in freq] for a in p]).reshape(len(p), 1, D)
    _within("cos, sin", _f64(y), ref, np.full_like(ref, O.ANGLE * O.U))


def test_gradient_order_replayed():
    """Leaves that are exact, whose sums differ for every order of the additions: rows of one magnitude (eps 0), no turn."""
    for n, hq, hk, D, inter in ((300, 9, 1, 16, True), (1100, 3, 17, 8, False), (64, 25, 8, 40, True), (4500, 1, 1, 8, True),
                                (2500, 60, 3, 8, False), (2500, 57, 6, 24, True), (700, 5, 2, 80, True), (333, 11, 1, 96, True),
                                (901, 3, 1, 160, True), (450, 2, 2, 48, True), (1500, 37, 2, 72, True), (123, 4, 4, 512, False),
                                (211, 9, 1, 192, False), (611, 30, 9, 128, True), (257, 2, 1, 144, False), (4001, 2, 1, 264, True),
                                (15001, 1, 1, 168, True), (5200, 10, 1, 64, False), (9000, 11, 6, 40, True)):
        g = np.random.default_rng(n)
        for kind, chunk in (("full", None), ("chunked", 61), ("permuted", None), ("padded_left", None)):
            sign = lambda h: np.where(g.random((n, h, D)) < 0.5, -1.0, 1.0) * 2.0 ** g.integers(-3, 4, (n, h, 1))   # noqa: E731
            size = lambda h: (g.integers(1, 2 ** 12, (n, h, D)) * 2.0 ** g.integers(-6, 14, (n, h, D)))             # noqa: E731
            q, k, dq, dk = sign(hq), sign(hk), size(hq), size(hk)
            to = lambda v: torch.from_numpy(v).to("cuda", F32)                                                      # noqa: E731
            lay = L.make_layout(kind, np.asarray([n // 2, n - n // 2 - 5, 5]), chunk=chunk or 1024)
            pos = torch.zeros(n, dtype=torch.int32, device="cuda")
            r = harness.run_layout_qk_norm_rotary(lay, to(q), to(k), to(dq), to(dk), None, None, pos,
                                                  rb.Rotary(8, interleaved=inter), 0.0)
            assert r.status == 0
            for got, want in zip((r.dweight, r.dk_weight), O.grad_replay(dq * np.sign(q), dk * np.sign(k))):
                assert np.array_equal(got.cpu().numpy(), want)


def test_one_token_equals_prefill():
    for dtype, inter in ((BF, False), (F32, True)):
        s = Setup(40, 32, 8, 128, 128, 0, inter, dtype)
        q, k = s.fwd()
        rq, rk = rb.rotary_fwd(s.q, s.k, s.layout(), s.pos, s.rot)
        one = rb.call_layout(np.asarray([0], dtype=np.int32), 1, 1, with_plan=False)
        for t in (0, 17, 39):
            a, b = rb.qk_norm_rotary_fwd(s.q[t:t + 1], s.k[t:t + 1], s.qw, s.kw, one, s.pos[t:t + 1], s.rot, EPS)
            assert _same(a[0], q[t]) and _same(b[0], k[t])
            a, b = rb.rotary_fwd(s.q[t:t + 1], s.k[t:t + 1], one, s.pos[t:t + 1], s.rot)
            assert _same(a[0], rq[t]) and _same(b[0], rk[t])


@pytest.mark.parametrize("dtype,D,rot,inter", [(BF, 128, 128, False), (F32, 80, 20, True), (FP16, 64, 32, True)])
def test_strides_and_aliases(dtype, D, rot, inter):
    n, hq, hk = 53, 6, 2
    s = Setup(n, hq, hk, D, rot, 0, inter, dtype)
    q, k = s.fwd()
    dq, dk = s.bwd()
    joined = torch.randn(n, hq + 2 * hk, D, device="cuda").to(dtype)
    joined[:, :hq], joined[:, hq:hq + hk] = s.q, s.k
    values = joined[:, hq + hk:].clone()
    major = lambda t: t.transpose(0, 1).contiguous().transpose(0, 1)                        # noqa: E731
    pad = torch.zeros(n, hq, D + 8, dtype=dtype, device="cuda")
    pad[..., :D] = s.q
    lay = s.layout()
    run = lambda a, b, **kw: rb.qk_norm_rotary_fwd(a, b, s.qw, s.kw, lay, s.pos, s.rot, EPS, **kw)   # noqa: E731
    for a, b in ((joined[:, :hq], joined[:, hq:hq + hk]), (major(s.q), major(s.k)), (pad[..., :D], s.k)):
        y, z = run(a, b)
        assert _same(y, q) and _same(z, k)
        o = major(torch.zeros_like(s.q))
        y, z = run(a, b, q_out=o)
        assert y is o and _same(y, q) and _same(z, k)
    run(joined[:, :hq], joined[:, hq:hq + hk], q_out=joined[:, :hq], k_out=joined[:, hq:hq + hk])    # in place
    assert _same(joined[:, :hq], q) and _same(joined[:, hq:hq + hk], k) and _same(joined[:, hq + hk:], values)
    # one head and one token read by all; gradients in place of either input
    x1 = s.q[:, :1].expand(n, hq, D)
    y, _ = rb.qk_norm_rotary_fwd(x1, None, s.qw, None, lay, s.pos, s.rot, EPS)
    assert all(_same(y[:, h], q[:, 0]) for h in range(hq))
    y, _ = rb.rotary_fwd(s.q[:1].expand(n, hq, D), None, lay, s.pos, s.rot)
    z, _ = rb.rotary_fwd(s.q[:1].repeat(n, 1, 1), None, lay, s.pos, s.rot)
    assert _same(y, z)
    bwd = lambda a, b, c, d, **kw: rb.qk_norm_rotary_bwd(a, b, s.qw, s.kw, c, d, lay, s.pos, s.rot, EPS, **kw)   # noqa: E731
    ga, gb = s.dq.clone(), s.dk.clone()
    bwd(s.q, s.k, ga, gb, dq=ga, dk=gb)
    assert _same(ga, dq) and _same(gb, dk)
    xa, xb = s.q.clone(), s.k.clone()
    bwd(xa, xb, s.dq, s.dk, dq=xa, dk=xb)
    assert _same(xa, dq) and _same(xb, dk)
    ws = s.workspace()
    ws.begin()
    a, b = bwd(major(s.q), s.k, s.dq, major(s.dk), workspace=ws)
    assert _same(a, dq) and _same(b, dk)
    got = ws.finalize()
    ws.begin()
    s.bwd(ws)
    assert all(_same(u, v) for u, v in zip(got, ws.finalize())) and ws.status() == 0


def test_offsets_past_32_bits():
    """Token stride 2^28 elements: the last slot lies 2^32 elements and more behind the first."""
    n, D, stride = 18, 64, 2 ** 28
    free = torch.cuda.mem_get_info()[0]
    if free < 40 * 2 ** 30:
        pytest.skip("needs 40 GB")
    s = Setup(n, 3, 0, D, D, 0, False, BF)
    big = torch.zeros(n * stride, dtype=BF, device="cuda")
    x = torch.as_strided(big, (n, 3, D), (stride, D, 1))
    x.copy_(s.q)
    q, _ = s.fwd()
    y, _ = rb.qk_norm_rotary_fwd(x, None, s.qw, None, s.layout(), s.pos, s.rot, EPS)
    assert _same(y, q)
    rb.qk_norm_rotary_fwd(s.q, None, s.qw, None, s.layout(), s.pos, s.rot, EPS, q_out=x)
    assert _same(x.contiguous(), q)
    x.copy_(s.q)
    major = torch.as_strided(big, (3, n, D), (2 ** 31, D, 1), 1024 * 64).transpose(0, 1)
    major.copy_(s.q)
    rb.rotary_fwd(major, None, s.layout(), s.pos, s.rot, q_out=major)
    z, _ = rb.rotary_fwd(s.q, None, s.layout(), s.pos, s.rot)
    assert _same(major.contiguous(), z)


def test_a_bad_head_stays_alone():
    """NaN and infinities in one head, and in padding, reach no other head."""
    s = Setup(30, 5, 2, 128, 64, 32, False, BF)
    q0, k0 = s.fwd()
    dq0, dk0 = s.bwd()
    s.q[3, 1, 7], s.q[9, 4, 100], s.k[12, 0, 0] = float("nan"), float("inf"), float("-inf")
    q, k = s.fwd()
    dq, dk = s.bwd()
    okq, okk = torch.ones(30, 5, dtype=torch.bool), torch.ones(30, 2, dtype=torch.bool)
    okq[3, 1] = okq[9, 4] = okk[12, 0] = False
    assert _same(q[okq], q0[okq]) and _same(k[okk], k0[okk]) and _same(dq[okq], dq0[okq]) and _same(dk[okk], dk0[okk])
    assert bool(torch.isnan(q[3, 1].float()).any()) and bool(torch.isnan(dk[12, 0].float()).any())
    z = torch.zeros_like(s.q)                                         # rows of zeros: 0 with eps
    y, _ = rb.qk_norm_rotary_fwd(z, None, s.qw, None, s.layout(), s.pos, s.rot, EPS)
    assert not y.float().abs().any()


def test_an_infinity_spoils_its_own_columns():
    """rstd is 0 in a row with an infinity: the other columns are zeros, it and the one it turns with are NaN."""
    n = 9
    for dtype in (BF, F32):
        for D, rot, first, inter in ((64, 32, 16, False), (72, 24, 4, False), (80, 20, 2, False), (96, 40, 6, True)):
            s = Setup(n, 2, 1, D, rot, first, inter, dtype)
            for col in (0, D - 1, first, first + rot - 1, first + rot // 2):
                x = s.q.clone()
                x[3, 1, col] = float("inf")
                y, _ = rb.qk_norm_rotary_fwd(x, s.k, s.qw, s.kw, s.layout(), s.pos, s.rot, EPS)
                bad, j = {col}, col - first
                if 0 <= j < rot:
                    bad.add(first + (j ^ 1 if inter else (j + rot // 2) % rot))
                assert set(torch.isnan(y[3, 1]).nonzero().flatten().tolist()) == bad, (dtype, D, col)
                assert not y[3, 1, [c for c in range(D) if c not in bad]].any()
                clean = torch.ones(n, 2, dtype=torch.bool, device="cuda")
                clean[3, 1] = False
                assert torch.isfinite(y[clean]).all()


def test_status_bits():
    s = Setup(40, 3, 2, 32, 32, 0, False, BF)
    ws = s.workspace()
    run = lambda ids: rb.qk_norm_rotary_bwd(                                                # noqa: E731
        s.q[:len(ids)], s.k[:len(ids)], s.qw, s.kw, s.dq[:len(ids)], s.dk[:len(ids)],
        rb.call_layout(np.asarray(ids, dtype=np.int32), 1, 40, with_plan=False), s.pos[:len(ids)], s.rot, EPS, workspace=ws)
    ws.buf.zero_()
    run(np.arange(40))
    assert ws.status() & rb.STATUS_HEADER                            # never begun
    ws.begin()
    run(np.arange(40))
    good = ws.finalize()
    again = ws.finalize()
    assert ws.status() == 0 and all(_same(a, b) for a, b in zip(good, again))
    ws.begin()
    run(np.arange(39))
    ws.finalize()
    assert ws.status() == rb.STATUS_MISSING
    for ids in ([*range(40), 5], [7, 7] + [i for i in range(40) if i != 7][:38], list(range(8)) * 2 + list(range(16, 40))):
        ids = ids[:40]
        ws.begin()
        run(ids)
        run([i for i in range(40) if i not in ids] or [5])
        assert ws.status() & rb.STATUS_DOUBLE, ids
    ws.begin()
    dq, _ = run([*range(39), 41])
    assert ws.status() == rb.STATUS_PLAN and bool(torch.isfinite(dq.float()).all())
    other = rb.QkNormWorkspace(40, 3, 2, 64)
    other.begin()
    with pytest.raises(ValueError, match="workspace"):
        s.bwd(other)


def test_empty_single_and_large_head_counts():
    s = Setup(3, 1, 1, 64, 64, 0, False, BF)
    none = rb.call_layout(np.zeros(0, dtype=np.int32), 1, 3, with_plan=False)
    e, p = s.q[:0], s.pos[:0]
    assert rb.rotary_fwd(e, None, none, p, s.rot)[0].numel() == 0
    ws = s.workspace()
    ws.begin()
    assert rb.qk_norm_rotary_bwd(e, s.k[:0], s.qw, s.kw, e, s.k[:0], none, p, s.rot, EPS, workspace=ws)[0].numel() == 0
    s.bwd(ws)
    ws.finalize()
    assert ws.status() == 0
    zero = rb.QkNormWorkspace(0, 2, 1, 64)
    zero.begin()
    dq, dk = zero.finalize()
    assert not dq.any() and not dk.any() and zero.status() == 0
    padding = rb.call_layout(np.full(9, -1, dtype=np.int32), 1, 3, with_plan=False)         # nothing but padding
    x = torch.full((9, 1, 64), 3.0, dtype=BF, device="cuda")
    rb.qk_norm_rotary_fwd(x, None, None, None, padding, torch.zeros(9, dtype=torch.int32, device="cuda"), s.rot, EPS, q_out=x)
    assert bool((x == 3).all())
    b = Setup(2, 2000, 1, 8, 4, 4, False, FP16)
    q, k = b.fwd()
    dq, dk = b.bwd()
    b.check(q, dq, None, b.q, b.qw, b.dq)
    b.check(k, dk, None, b.k, b.kw, b.dk)


def test_graph_streams_and_shared_plan():
    """Captured and replayed with new inputs, on a side stream, two workspaces in one graph."""
    s = Setup(200, 8, 2, 128, 128, 0, False, BF)
    want_q, want_k = s.fwd()
    ws = [s.workspace() for _ in range(2)]
    ws[0].begin()
    s.bwd(ws[0])
    want = ws[0].finalize()
    lay = s.layout()
    outs = [torch.empty_like(t) for t in (s.q, s.k, s.q, s.k)]
    grads = [[torch.empty(128, device="cuda") for _ in range(2)] for _ in range(2)]
    src = [s.q.clone(), s.k.clone(), s.dq.clone(), s.dk.clone()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()

    def body():
        rb.qk_norm_rotary_fwd(src[0], src[1], s.qw, s.kw, lay, s.pos, s.rot, EPS, q_out=outs[0], k_out=outs[1])
        for w, d in zip(ws, grads):
            w.begin()
            rb.qk_norm_rotary_bwd(src[0], src[1], s.qw, s.kw, src[2], src[3], lay, s.pos, s.rot, EPS, dq=outs[2],
                                  dk=outs[3], workspace=w)
            w.finalize(*d)

    with torch.cuda.stream(side):
        body()
        with torch.cuda.graph(g, stream=side):
            body()
    torch.cuda.current_stream().wait_stream(side)
    for t in src[:2]:
        t.mul_(2)
    g.replay()
    for t in src[:2]:
        t.mul_(0.5)
    g.replay()
    torch.cuda.synchronize()
    assert _same(outs[0], want_q) and _same(outs[1], want_k)
    assert all(_same(a, b) for d in grads for a, b in zip(d, want)) and ws[0].status() == ws[1].status() == 0
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    a, b = s.fwd(stream=stream)
    ws[1].begin(stream)
    s.bwd(ws[1], stream=stream)
    c = ws[1].finalize(stream=stream)
    stream.synchronize()
    assert _same(a, want_q) and _same(b, want_k) and all(_same(x, y) for x, y in zip(c, want))


def test_a_block_as_it_is_used():
    """Joined projection -> norms with rotation -> scores -> gradients back through both, next to the two
    separate operators, and cached keys moved to new positions."""
    n, hq, hk, D = 96, 8, 2, 128
    s = Setup(n, hq, hk, D, D, 0, False, F32, top=2000)
    q, k = s.fwd()
    # the norm by itself (per-head RMSNorm in bf16 rows), then the rotation: one more rounding
    b = Setup(n, hq, hk, D, D, 0, False, BF, top=2000)
    heads = rb.call_layout(np.arange(n, dtype=np.int32), hq, n, with_plan=False)
    z = rb.rmsnorm_fwd(b.q, b.qw, heads, EPS)
    y, _ = rb.rotary_fwd(z, None, b.layout(), b.pos, b.rot)
    fused, _ = b.fwd()
    ref, err = O.forward(_f64(b.q), _f64(b.qw), _f64(b.pos), b.freq, *b.args, EPS)
    zs = O._spread(_f64(z), *b.args)
    _within("two steps", _f64(y), ref, O.rounded(err + 2.0 ** -8 * zs * 1.01, ref, "bfloat16"))
    _within("fused", _f64(fused), ref, O.rounded(err, ref, "bfloat16"))
    # gradients of a loss of the scores, against differences along a direction
    gq = hq // hk
    c = torch.randn(hq, n, n, generator=torch.Generator("cpu").manual_seed(1)).double()
    score = lambda a, e: torch.einsum("thd,shd,hts->", a, e.repeat_interleave(gq, 1), c)   # noqa: E731
    a, e = (t.double().cpu().requires_grad_() for t in (q, k))
    score(a, e).backward()
    s.dq, s.dk = a.grad.to("cuda", F32), e.grad.to("cuda", F32)
    ws = s.workspace()
    ws.begin()
    dq, dk = s.bwd(ws)
    dqw, dkw = ws.finalize()
    assert ws.status() == 0
    s.check(q, dq, dqw, s.q, s.qw, s.dq)
    s.check(k, dk, dkw, s.k, s.kw, s.dk)

    def loss(vq, vk, wq, wk):
        f = lambda v, w: torch.from_numpy(O.forward(v, w, _f64(s.pos), s.freq, *s.args, EPS)[0])   # noqa: E731
        return float(score(f(vq, wq), f(vk, wk)))

    base = [_f64(t) for t in (s.q, s.k, s.qw, s.kw)]
    gen = np.random.default_rng(3)
    for i, grad in enumerate((dq, dk, dqw, dkw)):
        d = gen.standard_normal(base[i].shape)
        h = 1e-5
        up, down = ([v + t * h * d if j == i else v for j, v in enumerate(base)] for t in (1, -1))
        slope = (loss(*up) - loss(*down)) / (2 * h)
        got, size = float((_f64(grad) * d).sum()), float(np.abs(_f64(grad) * d).sum())
        # differences: h^2 and rounding of the loss; gradients: a few hundred U of their terms
        assert abs(got - slope) <= 1e-5 * size, (i, got, slope)
    # turning keys that stand in a cache by a distance equals turning them at the moved position
    r1, _ = rb.rotary_fwd(s.k, None, s.layout(), s.pos, s.rot)
    move = torch.full_like(s.pos, -700)
    r2, _ = rb.rotary_fwd(r1, None, s.layout(), move, s.rot)
    ref, err = O.rotate(_f64(s.k), _f64(s.pos) - 700, s.freq, *s.args)
    _within("moved", _f64(r2), ref, 4 * err)
    back, _ = rb.rotary_bwd(r1, None, s.layout(), s.pos, s.rot)
    _, err = O.rotate(_f64(s.k), _f64(s.pos), s.freq, *s.args)
    _within("turned back", _f64(back), _f64(s.k), 4 * err)


@pytest.mark.parametrize("seed", range(4))
def test_sizes_at_random(seed):
    """Sizes, widths, parts of the head and layouts at random: bits across layouts, values, rotation in place."""
    rng = np.random.default_rng(seed)
    pick = lambda v: v[int(rng.integers(len(v)))]                                           # noqa: E731
    for _ in range(12):
        D = pick((8, 16, 24, 40, 56, 64, 72, 80, 88, 96, 120, 128, 136, 160, 192, 200, 256, 264, 384, 512))
        rot = max(4, pick((D, D // 2, D // 4, int(rng.integers(4, D + 1)))) // 4 * 4)
        first = (D - rot) // pick((2, 4, 8)) * 2 if rng.random() < 0.5 else 0
        hq, hk = pick((1, 2, 5, 12, 17, 33)), pick((0, 1, 2, 7))
        dtype, param = pick((BF, FP16, F32)), pick((None, F32))
        lengths = rng.integers(1, pick((4, 40, 200)), pick((2, 5, 9)))
        s = Setup(int(lengths.sum()), hq, hk, D, rot, first, rng.random() < 0.3, dtype, param, pick((1.0, 1.2)))
        lays = {kind: L.make_layout(kind, lengths, chunk=pick((1, 7, 37)))
                for kind in ("full", "padded_left", "permuted", "permuted_chunked", "padded_right_chunked")}
        runs = {kind: harness.run_layout_qk_norm_rotary(lay, s.q, s.k, s.dq, s.dk, s.qw, s.kw, s.pos, s.rot, EPS, 0.5)
                for kind, lay in lays.items()}
        sizes = (s.n, hq, hk, D, s.args, dtype)
        assert harness.assert_batch_invariant(runs, lays).first_failure() is None, sizes
        assert all(r.status == 0 and r.untouched_padding for r in runs.values()), sizes
        r = runs["full"]
        s.check(r.y, r.dx, r.dweight, s.q, s.qw, s.dq, 0.5)
        if hk:
            s.check(r.k, r.dk, r.dk_weight, s.k, s.kw, s.dk, 0.5)
        q, k = rb.rotary_fwd(s.q, s.k, s.layout(), s.pos, s.rot)
        for x, y in ((s.q, q), (s.k, k)):
            if x is not None:
                z = x.clone()
                rb.rotary_fwd(z, None, s.layout(), s.pos, s.rot, q_out=z)
                assert _same(z, y), sizes
