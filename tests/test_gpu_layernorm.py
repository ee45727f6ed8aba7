"""GPU: layer norm and dropout against the FP64 oracle, bit for bit across layouts,
and at the sizes, masks and calls where they can go wrong.

Tolerances: the oracle's own bound of an FP32 evaluation (oracle/layernorm.py
derives it from the lengths of the sums), plus half a step of the output's type
for its one rounding.
"""
import numpy as np
import pytest
import torch

import synth
from oracle import layernorm as O
from invariant_rmsnorm_fwd_gb300 import harness
from invariant_rmsnorm_fwd_gb300 import layout as L
import invariant_rmsnorm_fwd_gb300 as rb

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

EPS = 1e-5
BF, FP16, F32 = torch.bfloat16, torch.float16, torch.float32


def _name(dtype):
    return str(dtype).split(".")[1]


def _word(t):
    return t.contiguous().view(torch.int32 if t.element_size() == 4 else torch.int16)


def _same(a, b):
    return torch.equal(_word(a), _word(b))


def _f64(t):
    return t.double().cpu().numpy()


def _state(seed=0x1234567, offset=9):
    return torch.tensor([seed, offset], dtype=torch.int64, device="cuda")


def _keep(drop, rows, H):
    seed, offset = (int(v) % 2 ** 64 for v in drop.state.cpu())
    return O.keep_mask(seed, offset, rows, H, drop.p)


def _data(n, H, dtype, seed=0, rpt=1, param=None):
    g = torch.Generator("cpu").manual_seed(seed + 7 * H + n)
    r = lambda s: torch.randn(n, rpt, H, generator=g) * s                   # noqa: E731
    shift = torch.randn(n, rpt, 1, generator=g)
    x, res, dy, dres = (r(1.0) + shift), r(1.0), r(0.01), r(0.01)
    p = param or dtype
    w, b = 1 + 0.1 * torch.randn(H, generator=g), 0.1 * torch.randn(H, generator=g)
    return [t.to("cuda", dtype) for t in (x, res, dy, dres)] + [w.to("cuda", p), b.to("cuda", p)]


def _within(name, got, ref, bound):
    err = np.abs(got - ref)
    bad = ~(err <= bound)
    assert not bad.any(), (name, int(bad.sum()), float((err / np.maximum(bound, 1e-300)).max()),
                           np.argwhere(bad)[:3].tolist())


def _check_chain(h, y, dh, dx, dw, db, x, res, dy, dres, w, b, drop, s, dtype, rpt=1, eps=EPS):
    """Everything of a run in logical order against the oracle."""
    H = x.shape[-1]
    n = x.numel() // H
    nm = _name(dtype)
    x64, r64, dy64, dr64 = (_f64(t).reshape(n, H) for t in (x, res, dy, dres))
    w64 = np.ones(H) if w is None else _f64(w)
    b64 = np.zeros(H) if b is None else _f64(b)
    keep, sc = (np.ones((n, H), bool), 1.0) if drop is None else (_keep(drop, np.arange(n), H), O.drop_scale(drop.p))
    h64 = np.where(keep, x64 * sc, 0) + r64
    # h: the factor rounded to FP32, one product-sum, one rounding to the type
    _within("h", _f64(h).reshape(n, H), h64, O.rounded(2 * O.U * (np.abs(x64 * sc) + np.abs(h64)), h64, nm))
    hs = _f64(h).reshape(n, H)                                              # the stored h is what the norm takes
    y64, mean, rstd, e = O.forward(hs, w64, b64, eps)
    _within("y", _f64(y).reshape(n, H), y64, O.rounded(e, y64, nm))
    dn, dw64, db64, e_dx, e_dw, e_db = O.backward(hs, w64, dy64, eps)
    dh64 = s * dn + dr64
    e_dh = abs(s) * e_dx + 3 * O.U * (np.abs(s * dn) + np.abs(dr64))
    _within("dh", _f64(dh).reshape(n, H), dh64, O.rounded(e_dh, dh64, nm))
    if drop is not None:
        dx64 = np.where(keep, dh64 * sc, 0)
        got = _f64(dx).reshape(n, H)
        assert not got[~keep].any()
        _within("dx", got, dx64, O.rounded(e_dh * sc + 2 * O.U * np.abs(dx64), dx64, nm))
    _within("dweight", _f64(dw), s * dw64, abs(s) * e_dw + O.U * np.abs(s * dw64))
    _within("dbias", _f64(db), s * db64, abs(s) * e_db + O.U * np.abs(s * db64))
    return mean, rstd


SIZES = [(8, BF), (24, FP16), (40, F32), (128, BF), (200, F32), (256, FP16), (264, BF), (1000, F32), (1000, BF), (2048, BF),
         (4096, FP16), (4104, BF), (5120, BF), (8192, F32), (8200, BF), (12296, FP16), (16384, BF)]


@pytest.mark.parametrize("H,dtype", SIZES, ids=lambda v: str(v).replace("torch.", ""))
@pytest.mark.parametrize("p", [0.0, 0.1])
def test_chain_matches_oracle_and_is_layout_invariant(H, dtype, p):
    lengths = np.asarray([70, 3, 130, 1, 64, 9])
    n = int(lengths.sum())
    x, res, dy, dres, w, b = _data(n, H, dtype, param=F32 if H % 3 == 0 else None)
    drop = rb.Dropout(p, _state()) if p else None
    s = 1.0 / n
    runs, lays = {}, {}
    for kind in L.LAYOUT_KINDS + ("permuted_chunked", "padded_right_chunked"):
        lays[kind] = L.make_layout(kind, lengths, chunk=37)
        runs[kind] = harness.run_layout_layernorm(lays[kind], x, res, dy, dres, w, b, EPS, s, drop)
    rep = harness.assert_batch_invariant(runs, lays)
    assert rep.green, rep.summary()
    assert all(r.status == 0 and r.untouched_padding for r in runs.values())
    r = runs["full"]
    _check_chain(r.h, r.y, r.dh, r.dx, r.dweight, r.dbias, x, res, dy, dres, w, b, drop, s, dtype)


@pytest.mark.parametrize("H,R,dtype", [(64, 3, BF), (128, 8, FP16), (8, 5, BF), (96, 7, F32), (320, 4, BF), (256, 32, BF)])
def test_heads(H, R, dtype):
    lengths = np.asarray([11, 1, 30, 6])
    n = int(lengths.sum())
    x, res, dy, dres, w, b = _data(n, H, dtype, rpt=R)
    drop = rb.Dropout(0.25, _state(5, 2 ** 40))
    lays = {k: L.make_layout(k, lengths, chunk=5) for k in ("full", "chunked", "padded_left", "permuted")}
    runs = {k: harness.run_layout_layernorm(v, x, res, dy, dres, w, b, EPS, 1.0, drop, rows_per_token=R)
            for k, v in lays.items()}
    rep = harness.assert_batch_invariant(runs, lays)
    assert rep.green, rep.summary()
    r = runs["full"]
    assert r.status == 0
    _check_chain(r.h, r.y, r.dh, r.dx, r.dweight, r.dbias, x, res, dy, dres, w, b, drop, 1.0, dtype)


def test_larger_batch_many_blocks():
    """More blocks than one pass of the final tree takes, whole blocks and cut ones."""
    n, H = 64 * 40 + 13, 512
    x, res, dy, dres, w, b = _data(n, H, BF)
    lays = {"full": L.make_layout("full", [n]), "chunked": L.make_layout("chunked", [n], chunk=1000),
            "halves": L.Layout("halves", [np.arange(1300, n, dtype=np.int32), np.arange(1300, dtype=np.int32)], n)}
    runs = {k: harness.run_layout_layernorm(v, x, res, dy, dres, w, b, EPS) for k, v in lays.items()}
    assert harness.assert_batch_invariant(runs, lays).green and all(r.status == 0 for r in runs.values())
    r = runs["full"]
    _check_chain(r.h, r.y, r.dh, r.dx, r.dweight, r.dbias, x, res, dy, dres, w, b, None, 1.0, BF)


@pytest.mark.parametrize("n", [1, 7, 8, 9, 63, 64, 65, 200, 2085])
def test_gradient_order_is_the_replayed_one(n):
    """Rows of +-2^k (mean 0, variance 4^k, eps 0) have exact xhat = +-1, so the terms
    are exact, and dy straddles 2^24: every order of additions gives another sum."""
    for H in (8, 128, 264, 1024):
        rng = np.random.default_rng(n + H)
        sign = np.where(np.arange(H) % 2 == 0, 1.0, -1.0) * np.where(rng.random((n, 1)) < 0.5, 1.0, -1.0)
        x = sign * 2.0 ** rng.integers(-3, 4, size=(n, 1))
        dy = np.where(rng.random((n, H)) < 0.5, 1.0, 2.0 ** rng.integers(0, 26, size=(n, H))) * \
            np.where(rng.random((n, H)) < 0.5, 1.0, -1.0)
        xt, dyt = torch.tensor(x).to("cuda", BF), torch.tensor(dy).to("cuda", BF)
        w = torch.ones(H, dtype=BF, device="cuda")
        for kind in ("full", "chunked", "permuted_chunked"):
            lay = L.make_layout(kind, [n // 2, n - n // 2], chunk=37)
            ws = rb.LayerNormWorkspace(n, H)
            ws.begin()
            for tok in lay.calls:
                cl = rb.call_layout(tok, 1, n)
                i = cl.tok_id.long()
                rb.layernorm_bwd(xt[i], w, dyt[i], cl, 0.0, workspace=ws)
            dw, db = ws.finalize()
            assert ws.status() == 0
            assert np.array_equal(dw.cpu().numpy(), O.grad_replay(dy, sign)), (H, kind)
            assert np.array_equal(db.cpu().numpy(), O.grad_replay(dy)), (H, kind)


@pytest.mark.parametrize("H,dtype", [(128, BF), (1000, F32), (5120, FP16)], ids=str)
def test_fused_equals_its_parts(H, dtype):
    """The fused forward is dropout, one add and the norm; mean and rstd are the norm's."""
    n = 77
    x, res, dy, dres, w, b = _data(n, H, dtype)
    cl = rb.call_layout(np.arange(n, dtype=np.int32), 1, n)
    mean, rstd = torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda")
    h, y = rb.layernorm_add_fwd(x, res, w, b, cl, EPS, mean=mean, rstd=rstd)
    assert _same(h, (x.float() + res.float()).to(dtype))
    m2, r2 = torch.zeros_like(mean), torch.zeros_like(rstd)
    assert _same(y, rb.layernorm_fwd(h, w, b, cl, EPS, mean=m2, rstd=r2))
    assert _same(mean, m2) and _same(rstd, r2)
    _, mean64, rstd64, _ = O.forward(_f64(h).reshape(n, H), _f64(w), _f64(b), EPS)
    a = np.abs(_f64(h).reshape(n, H)).mean(1)
    _within("mean", _f64(mean), mean64, O.DEPTH * O.U * a)
    _within("rstd", _f64(rstd), rstd64, (O.DEPTH / 2 + 8) * O.U * rstd64)
    # backward without dres, unscaled, is the plain one, and write_dx=False leaves the gradients
    dh, dx = rb.layernorm_add_bwd(h, w, dy, cl, EPS)
    assert dh is dx and _same(dh, rb.layernorm_bwd(h, w, dy, cl, EPS))
    got = []
    for write in (True, False):
        ws = rb.LayerNormWorkspace(n, H)
        ws.begin()
        out = rb.layernorm_bwd(h, w, dy, cl, EPS, workspace=ws, write_dx=write)
        assert (out is None) != write and (not write or _same(out, dh))
        got.append(ws.finalize())
        assert ws.status() == 0
    assert all(_same(u, v) for u, v in zip(*got))


def test_no_weight_no_bias():
    n, H = 20, 264
    x, res, dy, dres, w, b = _data(n, H, BF)
    cl = rb.call_layout(np.arange(n, dtype=np.int32), 1, n)
    one, zero = torch.ones_like(w), torch.zeros_like(b)
    assert _same(rb.layernorm_fwd(x, None, None, cl, EPS), rb.layernorm_fwd(x, one, zero, cl, EPS))
    assert _same(rb.layernorm_fwd(x, w, None, cl, EPS), rb.layernorm_fwd(x, w, zero, cl, EPS))
    assert _same(rb.layernorm_bwd(x, None, dy, cl, EPS), rb.layernorm_bwd(x, one, dy, cl, EPS))


@pytest.mark.parametrize("H,dtype", [(8, BF), (264, F32), (4096, BF)], ids=str)
def test_constant_rows_and_large_offsets(H, dtype):
    """A constant row has xhat 0 up to the mean's rounding; a row far from zero keeps its variance."""
    x = torch.empty(4, 1, H, device="cuda", dtype=dtype)
    x[0], x[1] = 3.0, 0.0
    g = torch.Generator("cpu").manual_seed(1)
    x[2] = (1000 + torch.randn(H, generator=g) * 8).to("cuda", dtype)
    x[3] = (-1e-3 * torch.rand(H, generator=g)).to("cuda", dtype)
    dy = torch.randn(4, 1, H, generator=g).to("cuda", dtype)
    w, b = (torch.full((H,), v, dtype=dtype, device="cuda") for v in (1.5, 0.25))
    cl = rb.call_layout(np.arange(4, dtype=np.int32), 1, 4)
    y, dx = rb.layernorm_fwd(x, w, b, cl, EPS), rb.layernorm_bwd(x, w, dy, cl, EPS)
    x64, dy64 = _f64(x).reshape(4, H), _f64(dy).reshape(4, H)
    y64, _, _, e = O.forward(x64, _f64(w), _f64(b), EPS)
    _within("y", _f64(y).reshape(4, H), y64, O.rounded(e, y64, _name(dtype)))
    dx64, _, _, e, _, _ = O.backward(x64, _f64(w), dy64, EPS)
    _within("dx", _f64(dx).reshape(4, H), dx64, O.rounded(e, dx64, _name(dtype)))


def test_nan_and_infinity_stay_in_their_row():
    n, H = 40, 1024
    x, res, dy, dres, w, b = _data(n, H, BF)
    cl = rb.call_layout(np.arange(n, dtype=np.int32), 1, n)
    y, dx = rb.layernorm_fwd(x, w, b, cl, EPS), rb.layernorm_bwd(x, w, dy, cl, EPS)
    x2 = x.clone()
    x2[3, 0, 5], x2[17, 0, 0] = float("nan"), float("inf")
    y2, dx2 = rb.layernorm_fwd(x2, w, b, cl, EPS), rb.layernorm_bwd(x2, w, dy, cl, EPS)
    ok = [i for i in range(n) if i not in (3, 17)]
    assert _same(y[ok], y2[ok]) and _same(dx[ok], dx2[ok])
    assert torch.isnan(y2[3]).all() and torch.isnan(y2[17]).any() and torch.isnan(dx2[3]).all()


def test_dropped_elements_are_zero_whatever_they_were():
    n, H = 33, 520
    cl = rb.call_layout(np.arange(n, dtype=np.int32), 1, n)
    drop = rb.Dropout(0.5, _state(3, 4))
    keep = torch.tensor(_keep(drop, np.arange(n), H), device="cuda").reshape(n, 1, H)
    for bad in (float("nan"), float("inf"), float("-inf")):
        x = torch.ones(n, 1, H, dtype=BF, device="cuda")
        x[~keep] = bad
        y = rb.dropout_fwd(x, cl, drop)
        assert torch.equal(y.float(), 2.0 * keep)
        res = torch.randn(n, 1, H, device="cuda").to(BF)
        h, _ = rb.layernorm_add_fwd(x, res, None, None, cl, EPS, dropout=drop)
        assert _same(h, (2.0 * keep + res.float()).to(BF))


@pytest.mark.parametrize("H,R,dtype", [(8, 1, BF), (264, 1, F32), (128, 32, FP16), (65536, 1, BF), (24, 5, F32)], ids=str)
@pytest.mark.parametrize("p", [0.0, 1e-9, 0.1, 0.5, 1.0])
def test_dropout_alone(H, R, dtype, p):
    lengths = np.asarray([5, 1, 8])
    n = int(lengths.sum())
    x = _data(n, H, dtype, rpt=R)[0]
    drop = rb.Dropout(p, _state(-5, 2 ** 33 + 1))
    keep = _keep(drop, np.arange(n * R), H).reshape(n, R, H)
    ref = np.where(keep, _f64(x) * O.drop_scale(p), 0)
    outs = []
    for kind in ("full", "padded_left", "permuted"):
        tok = L.make_layout(kind, lengths).calls[0]
        cl = rb.call_layout(tok, R, n, with_plan=False)
        act, ids = cl.tok_id >= 0, cl.tok_id.long()
        xp = torch.full((tok.size, R, H), float("nan"), dtype=dtype, device="cuda")
        xp[act] = x[ids[act]]
        y, dx = torch.full_like(xp, 7.0), torch.full_like(xp, 7.0)
        rb.dropout_fwd(xp, cl, drop, y=y)
        rb.dropout_bwd(xp, cl, drop, dx=dx)
        assert _same(y, dx) and bool((y[~act] == 7).all())
        log = torch.empty_like(x)
        log[ids[act]] = y[act]
        outs.append(log)
        rb.dropout_fwd(xp, cl, drop, y=xp)                                  # in place
        assert _same(xp[act], y[act])
    assert _same(outs[0], outs[1]) and _same(outs[0], outs[2])
    got = _f64(outs[0])
    assert np.array_equal(got != 0, keep & (_f64(x) != 0)) or p == 1.0
    _within("y", got, ref, O.rounded(2 * O.U * np.abs(ref), ref, _name(dtype)))


def test_masks_differ_by_seed_and_offset():
    n, H = 16, 4096
    cl = rb.call_layout(np.arange(n, dtype=np.int32), 1, n, with_plan=False)
    x = torch.ones(n, H, dtype=BF, device="cuda")
    y = [rb.dropout_fwd(x, cl, rb.Dropout(0.5, _state(*s))) for s in ((1, 0), (2, 0), (1, 1), (1 + 2 ** 32, 0), (1, 2 ** 32))]
    for i in range(len(y)):
        for j in range(i):
            share = float((y[i] != y[j]).float().mean())
            assert abs(share - 0.5) < 5 * 0.5 / np.sqrt(n * H)              # five standard deviations


def test_strided_slots_tail_and_in_place():
    """Token slots inside wider rows, tensors with more slots than the call, outputs over inputs."""
    n, H, T = 21, 136, 26
    x, res, dy, dres, w, b = _data(n, H, BF)
    cl = rb.call_layout(np.arange(n, dtype=np.int32), 1, n)
    drop = rb.Dropout(0.1, _state())
    h0, y0 = rb.layernorm_add_fwd(x, res, w, b, cl, EPS, dropout=drop)
    ws = rb.LayerNormWorkspace(n, H)
    ws.begin()
    dh0, dx0 = rb.layernorm_add_bwd(h0, w, dy, cl, EPS, dres=dres, dropout=drop, workspace=ws)
    g0 = ws.finalize()

    def wide(t):
        full = torch.full((T, H + 24), 5.0, dtype=BF, device="cuda")
        v = full[:, 8:8 + H]
        if t is not None:
            v[:n] = t.reshape(n, H)
        return full, v

    (fx, xv), (fr, rv), (fd, dv), (fs, sv) = (wide(t) for t in (x, res, dy, dres))
    rb.layernorm_add_fwd(xv, rv, w, b, cl, EPS, h=rv, y=xv, dropout=drop)   # h over the residual, y over x
    assert _same(rv[:n], h0.reshape(n, H)) and _same(xv[:n], y0.reshape(n, H))
    ws.begin()
    rb.layernorm_add_bwd(rv, w, dv, cl, EPS, dres=sv, dropout=drop, dh=sv, dx=dv, workspace=ws)
    assert _same(sv[:n], dh0.reshape(n, H)) and _same(dv[:n], dx0.reshape(n, H))
    assert all(_same(u, v) for u, v in zip(g0, ws.finalize()))
    for full in (fx, fr, fd, fs):
        assert bool((full[n:] == 5).all()) and bool((full[:, :8] == 5).all()) and bool((full[:, 8 + H:] == 5).all())


def test_empty_calls_and_empty_multiset():
    cl = rb.call_layout(np.zeros(0, dtype=np.int32), 1, 3)
    e = torch.empty(0, 128, dtype=BF, device="cuda")
    w = torch.ones(128, dtype=BF, device="cuda")
    assert rb.layernorm_fwd(e, w, None, cl, EPS).shape == (0, 128)
    assert rb.dropout_fwd(e, cl, rb.Dropout(0.5, _state())).shape == (0, 128)
    none = rb.call_layout(np.full(5, -1, dtype=np.int32), 1, 0)
    x = torch.full((5, 128), float("nan"), dtype=BF, device="cuda")
    ws = rb.LayerNormWorkspace(0, 128)
    ws.begin()
    y, dx = torch.full_like(x, 3.0), torch.full_like(x, 3.0)
    rb.layernorm_fwd(x, w, w, none, EPS, y=y)
    rb.layernorm_bwd(x, w, x, none, EPS, dx=dx, workspace=ws)
    dw, db = ws.finalize()
    assert ws.status() == 0 and dw.shape == db.shape == (128,) and not dw.any() and not db.any()
    assert bool((y == 3).all()) and bool((dx == 3).all())


def test_status_bits():
    n, H = 200, 64
    x, res, dy, dres, w, b = _data(n, H, BF)
    full = rb.call_layout(np.arange(n, dtype=np.int32), 1, n)
    part = rb.call_layout(np.arange(150, dtype=np.int32), 1, n)
    ws = rb.LayerNormWorkspace(n, H)
    ws.begin()
    rb.layernorm_bwd(x, w, dy, part, EPS, workspace=ws)
    ws.finalize()
    assert ws.status() == 2                                                 # rows are missing
    for twice in (full, part):
        ws.begin()
        rb.layernorm_bwd(x, w, dy, full, EPS, workspace=ws)
        rb.layernorm_bwd(x, w, dy, twice, EPS, workspace=ws)
        assert ws.status() & 1                                              # rows contributed twice
    for first in (5, 60):                                                   # spilled rows, then their group
        cut = rb.call_layout(np.arange(first, dtype=np.int32), 1, n)
        for a, c in ((cut, full), (full, cut)):
            ws.begin()
            rb.layernorm_bwd(x, w, dy, a, EPS, workspace=ws)
            rb.layernorm_bwd(x, w, dy, c, EPS, workspace=ws)
            ws.finalize()
            assert ws.status() & 1, (first, a is cut)
    ws.begin()
    rb.layernorm_bwd(x, w, dy, full, EPS, workspace=ws)
    first = ws.finalize()
    again = ws.finalize()
    assert ws.status() == 0 and _same(first[0], again[0]) and _same(first[1], again[1])
    fresh = rb.LayerNormWorkspace(n, H)
    fresh.buf.zero_()
    fresh.finalize()
    assert fresh.status() == 4                                              # never begun
    with pytest.raises(ValueError, match="workspace"):
        rb.layernorm_bwd(x, w, dy, full, EPS, workspace=rb.LayerNormWorkspace(n + 1, H))


def test_stale_plan_is_reported():
    """A plan of a longer call: entries past the call's rows are not followed."""
    n, H = 100, 64
    x, res, dy, dres, w, b = _data(n, H, BF)
    cl = rb.call_layout(np.arange(n, dtype=np.int32), 1, n)
    short = rb.CallLayout(cl.tok_id[:40].contiguous(), cl.plan, cl.plan_items, 40, 1, n)
    ws = rb.LayerNormWorkspace(n, H)
    ws.begin()
    dx = torch.full_like(x, 3.0)
    rb.layernorm_bwd(x, w, dy, short, EPS, dx=dx, workspace=ws)
    assert ws.status() & 8 and bool((dx[40:] == 3).all())


def test_graph_replay_with_a_new_mask_and_new_inputs():
    """The chain captured once: replays follow the state and the inputs in place, and
    two graphs with workspaces of their own do not disturb each other."""
    n, H = 300, 1024
    x, res, dy, dres, w, b = _data(n, H, BF)
    cl = rb.call_layout(np.arange(n, dtype=np.int32), 1, n)
    state = _state(1, 1)
    drop = rb.Dropout(0.2, state)

    def step(ws, o):
        rb.layernorm_add_fwd(x, res, w, b, cl, EPS, h=o["h"], y=o["y"], dropout=drop)
        ws.begin()
        rb.layernorm_add_bwd(o["h"], w, dy, cl, EPS, dres=dres, dropout=drop, dh=o["dh"], dx=o["dx"], workspace=ws)
        ws.finalize(dweight=o["dw"], dbias=o["db"])

    def fresh():
        o = {k: torch.zeros_like(x) for k in ("h", "y", "dh", "dx")}
        return {**o, "dw": torch.zeros(H, device="cuda"), "db": torch.zeros(H, device="cuda")}

    graphs = []
    for _ in range(2):
        ws, o = rb.LayerNormWorkspace(n, H), fresh()
        step(ws, o)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step(ws, o)
        graphs.append((g, ws, o))
    side = torch.cuda.Stream()
    for k in range(3):
        state.copy_(torch.tensor([1, 10 + k]))
        dy.mul_(1.5)
        torch.cuda.synchronize()
        graphs[0][0].replay()
        with torch.cuda.stream(side):
            graphs[1][0].replay()
        torch.cuda.synchronize()
        ws, o = rb.LayerNormWorkspace(n, H), fresh()
        step(ws, o)
        for _, gws, go in graphs:
            assert gws.status() == 0
            assert all(_same(go[t], o[t]) for t in o), k


def test_streams_given_and_current():
    n, H = 500, 2048
    x, res, dy, dres, w, b = _data(n, H, BF)
    cl = rb.call_layout(np.arange(n, dtype=np.int32), 1, n)
    y0 = rb.layernorm_fwd(x, w, b, cl, EPS)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    y1 = rb.layernorm_fwd(x, w, b, cl, EPS, stream=side)
    with torch.cuda.stream(torch.cuda.Stream()):
        y2 = rb.layernorm_fwd(x, w, b, cl, EPS)
    torch.cuda.synchronize()
    assert _same(y0, y1) and _same(y0, y2)


def test_gradients_against_differences():
    """dx, dweight and dbias of the FP32 chain against central differences of the
    kernels' own forward, accumulated in 64 bits."""
    n, H = 3, 16
    x, res, dy, dres, w, b = _data(n, H, F32)
    x, res, dy = x.double().float(), res, dy * 100
    cl = rb.call_layout(np.arange(n, dtype=np.int32), 1, n)
    drop = rb.Dropout(0.3, _state(8, 8))
    eps = 1e-2

    def loss(x, w, b):
        return float((rb.layernorm_add_fwd(x, res, w, b, cl, eps, dropout=drop)[1].double() * dy.double()).sum())

    h, _ = rb.layernorm_add_fwd(x, res, w, b, cl, eps, dropout=drop)
    ws = rb.LayerNormWorkspace(n, H)
    ws.begin()
    _, dx = rb.layernorm_add_bwd(h, w, dy, cl, eps, dropout=drop, workspace=ws)
    dw, db = ws.finalize()
    step = 2.0 ** -7
    for t, grad in ((x, dx), (w, dw), (b, db)):
        flat, gf = t.reshape(-1), grad.reshape(-1)
        for i in range(flat.numel()):
            keep = float(flat[i])
            vals = []
            for d in (step, -step):
                flat[i] = keep + d
                vals.append(loss(x, w, b))
            flat[i] = keep
            num = (vals[0] - vals[1]) / (2 * step)
            # truncation: step^2 / 6 times a third derivative of order 10; rounding: 48 terms of
            # order 1, each 2^-22 off, over 2 step
            assert abs(num - float(gf[i])) < 1e-3, (i, num, float(gf[i]))


# Both sides of every rule that picks a kernel: lanes and octets of a team, a row's
# first CTA, one and two CTAs an SM, vectors a thread, packed weights.
EDGES = [(16, BF), (32, F32), (72, BF), (136, FP16), (248, F32), (504, BF), (512, F32), (520, FP16), (520, F32), (1032, BF),
         (4096, F32), (5112, BF), (5128, BF), (5128, F32), (6144, FP16), (8184, BF), (8192, FP16), (8200, F32), (10240, FP16),
         (12288, BF), (16376, FP16)]


@pytest.mark.parametrize("H,dtype", [e for e in EDGES if e[1] != F32 or e[0] <= 8192], ids=lambda v: str(v).replace("torch.", ""))
def test_chain_at_the_edges_of_the_rules(H, dtype):
    n = 150
    x, res, dy, dres, w, b = _data(n, H, dtype, param=F32 if H % 3 == 0 else None)
    for drop in (None, rb.Dropout(0.3, _state())):
        lays = {k: L.make_layout(k, [n - 20, 20], chunk=37) for k in ("full", "permuted_chunked", "padded_left")}
        runs = {k: harness.run_layout_layernorm(v, x, res, dy, dres, w, b, EPS, 0.5, drop) for k, v in lays.items()}
        rep = harness.assert_batch_invariant(runs, lays)
        assert rep.green, rep.summary()
        r = runs["full"]
        assert r.status == 0
        _check_chain(r.h, r.y, r.dh, r.dx, r.dweight, r.dbias, x, res, dy, dres, w, b, drop, 0.5, dtype)


@pytest.mark.parametrize("H", [48, 400, 1040, 12288])
def test_absent_parameters_are_ones_and_zeros(H):
    n = 9
    x, res, dy, dres, w, b = _data(n, H, BF)
    cl = rb.call_layout(np.arange(n, dtype=np.int32), 1, n)
    for one, zero in ((torch.ones_like(w), torch.zeros_like(b)), (torch.ones_like(w).float(), torch.zeros_like(b).float())):
        assert _same(rb.layernorm_fwd(x, None, None, cl, EPS), rb.layernorm_fwd(x, one, zero, cl, EPS))
        assert _same(rb.layernorm_fwd(x, one, None, cl, EPS), rb.layernorm_fwd(x, one, zero, cl, EPS))
        assert _same(rb.layernorm_fwd(x, None, zero, cl, EPS), rb.layernorm_fwd(x, one, zero, cl, EPS))
        assert _same(rb.layernorm_bwd(x, None, dy, cl, EPS), rb.layernorm_bwd(x, one, dy, cl, EPS))


@pytest.mark.parametrize("n", [64 * 32 + 1, 64 * 300 + 9, 64 * 8200 + 5])
def test_final_tree_of_two_and_three_passes(n):
    """Exact terms (xhat = +-1), sums that round: every order gives another result."""
    H = 8
    rng = np.random.default_rng(n)
    sign = np.where(np.arange(H) % 2 == 0, 1.0, -1.0) * np.where(rng.random((n, 1)) < 0.5, 1.0, -1.0)
    dy = np.where(rng.random((n, H)) < 0.5, 1.0, 2.0 ** rng.integers(0, 26, size=(n, H))) * np.where(rng.random((n, H)) < 0.5, 1.0, -1.0)
    xt, dyt = torch.tensor(sign).to("cuda", BF), torch.tensor(dy).to("cuda", BF)
    cl = rb.call_layout(np.arange(n, dtype=np.int32), 1, n)
    ws = rb.LayerNormWorkspace(n, H)
    ws.begin()
    rb.layernorm_bwd(xt, None, dyt, cl, 0.0, workspace=ws, write_dx=False)
    dw, db = ws.finalize()
    assert ws.status() == 0
    assert np.array_equal(dw.cpu().numpy(), O.grad_replay(dy, sign))
    assert np.array_equal(db.cpu().numpy(), O.grad_replay(dy))


@pytest.mark.parametrize("H,dtype", [(128, BF), (264, F32), (1024, FP16), (9000, BF)], ids=str)
def test_offsets_past_32_bits(H, dtype):
    """Six slots 2^30 elements apart, every tensor a view of one buffer: the last offsets
    are beyond 2^32 elements."""
    n, pitch = 6, 2 ** 30
    x, res, dy, dres, w, b = _data(n, H, dtype)
    cl = rb.call_layout(np.arange(n, dtype=np.int32)[::-1].copy(), 1, n)
    drop = rb.Dropout(0.4, _state())

    def run(t):
        x, res, dy, dres, h, y, dh, dx, z = t
        ws = rb.LayerNormWorkspace(n, H)
        ws.begin()
        rb.layernorm_add_fwd(x, res, w, b, cl, EPS, h=h, y=y, dropout=drop)
        rb.layernorm_add_bwd(h, w, dy, cl, EPS, dres=dres, dropout=drop, dh=dh, dx=dx, workspace=ws)
        rb.dropout_fwd(x, cl, drop, y=z)
        dw, db = ws.finalize()
        assert ws.status() == 0
        return [t.reshape(n, H).clone() for t in (h, y, dh, dx, z)] + [dw, db]

    ins = [t.reshape(n, H) for t in (x, res, dy, dres)]
    near = run(ins + [torch.zeros(n, H, dtype=dtype, device="cuda") for _ in range(5)])
    buf = torch.empty(n, pitch, dtype=dtype, device="cuda")
    far = [buf[:, i * 16384:i * 16384 + H] for i in range(9)]
    for v, t in zip(far, ins):
        v.copy_(t)
    assert all(_same(a, c) for a, c in zip(near, run(far)))


def test_duplicate_ids_in_the_passes_without_gradients():
    """Two slots may hold the same logical row where nothing is reduced: both get its
    result and its mask."""
    for H in (64, 300 * 8):
        ids = np.asarray([3, 0, 3, -1, 1, 3], dtype=np.int32)
        x, res, dy, dres, w, b = _data(4, H, BF)
        cl = rb.call_layout(ids, 1, 4, with_plan=False)
        drop = rb.Dropout(0.5, _state())
        at = torch.tensor(np.maximum(ids, 0), device="cuda").long()
        xs, rs, ds = x[at], res[at], dy[at]
        out = rb.layernorm_add_fwd(xs, rs, w, b, cl, EPS, dropout=drop) + rb.layernorm_add_bwd(xs, w, ds, cl, EPS, dropout=drop) + \
            (rb.dropout_fwd(xs, cl, drop), rb.layernorm_fwd(xs, w, b, cl, EPS))
        for t in out:
            assert _same(t[0], t[2]) and _same(t[0], t[5])
            assert not bool((t[0] == t[1]).all())


def test_runs_next_to_the_other_norm():
    """Two kernels that hold tensor memory, on two streams at once: results as when alone."""
    n, H = 4000, 12296
    x, res, dy, dres, w, b = _data(n, H, BF)
    cl = rb.call_layout(np.arange(n, dtype=np.int32), 1, n)
    R = 10240                                                               # the other norm's widest rows
    ws, rws = rb.LayerNormWorkspace(n, H), rb.DweightWorkspace(n, R)
    rx, rw, rdy = res[..., :R].contiguous(), w[:R].contiguous(), dy[..., :R].contiguous()

    def ln(ws):
        ws.begin()
        dx = rb.layernorm_bwd(x, w, dy, cl, EPS, workspace=ws)
        return (dx,) + tuple(ws.finalize())

    def rms():
        rws.begin()
        dx = rb.rmsnorm_bwd_dx(rx, rw, rdy, cl, EPS, workspace=rws)
        return dx, rws.finalize()

    a0, r0 = ln(ws), rms()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(3):
        r1 = rms()
        with torch.cuda.stream(side):
            a1 = ln(ws)
        torch.cuda.synchronize()
        assert all(_same(u, v) for u, v in zip(a0, a1)) and all(_same(u, v) for u, v in zip(r0, r1))
        assert ws.status() == 0 and rws.status() == 0


def test_outputs_of_a_given_stream_belong_to_it():
    """A block that the current stream has just given back, and may still be writing, is
    not where a call on another stream puts its new outputs."""
    n, H = 600, 2048
    x, res, dy, dres, w, b = _data(n, H, BF)
    cl = rb.call_layout(np.arange(n, dtype=np.int32), 1, n)
    drop = rb.Dropout(0.5, _state())
    side = torch.cuda.Stream()
    ws = rb.LayerNormWorkspace(n, H)
    ws.begin()
    want = (rb.layernorm_fwd(x, w, b, cl, EPS), rb.layernorm_bwd(x, w, dy, cl, EPS, workspace=ws)) + ws.finalize()
    torch.cuda.synchronize()
    given = [torch.empty_like(x) for _ in range(8)] + [torch.empty(H, device="cuda") for _ in range(4)]
    used = {t.data_ptr() for t in given}
    given.clear()
    ws.begin(side)
    outs = (rb.layernorm_fwd(x, w, b, cl, EPS, stream=side), rb.layernorm_bwd(x, w, dy, cl, EPS, workspace=ws, stream=side))
    outs += ws.finalize(stream=side)
    outs += rb.layernorm_add_fwd(x, res, w, b, cl, EPS, dropout=drop, stream=side)
    outs += rb.layernorm_add_bwd(x, w, dy, cl, EPS, dropout=drop, stream=side)
    outs += (rb.dropout_fwd(x, cl, drop, stream=side), rb.dropout_bwd(x, cl, drop, stream=side))
    side.synchronize()
    assert not used & {t.data_ptr() for t in outs}
    assert all(_same(u, v) for u, v in zip(want, outs))
