"""Rotary positions and norms of queries and keys: what the C entry points and the binding refuse, the host's turns per
position and the frequencies (CPU, no GPU needed)."""
import ctypes
from fractions import Fraction

import numpy as np
import pytest
import torch

import invariant_rmsnorm_fwd_gb300 as rb
from invariant_rmsnorm_fwd_gb300 import rotary as R
from oracle import rotary as O

P = ctypes.c_void_p
E = 1e-6
A = [4096 * (i + 1) for i in range(8)]                    # addresses that are never dereferenced: checks fail first


def _layout(n=4, rpt=1, tok=256, n_logical=4, reserved=0):
    return ctypes.byref(rb._Layout(n, rpt, reserved, 0, tok, n_logical, None, 0))


def _heads(at=A[0], out=A[1], dy=A[2], w=A[3], heads=2, token=128, head=64, out_token=128, out_head=64, dy_token=128, dy_head=64,
           reserved=0):
    return ctypes.byref(rb._Heads(at, token, head, dy, dy_token, dy_head, out, out_token, out_head, w, heads, reserved))


def _rot(position=256, turns=256, dim=64, first=0, interleaved=0, scale=1.0):
    return ctypes.byref(rb._Rotary(position, turns, dim, first, interleaved, scale))


def _fwd(q=None, k=None, D=64, eps=E, dt=0, pdt=0, lay=None, rot=None):
    return rb._load().qk_norm_rotary_fwd(q or _heads(), k, D, eps, dt, pdt, lay or _layout(), rot or _rot(), None)


def _bwd(q=None, k=None, D=64, ws=None, dt=0, lay=None):
    return rb._load().qk_norm_rotary_bwd(q or _heads(), k, D, E, dt, dt, lay or _layout(), _rot(), ws, None)


def _alone(q=None, k=None, D=64, dt=0, lay=None, rot=None):
    return rb._load().rotary_fwd(q or _heads(), k, D, dt, lay or _layout(), rot or _rot(), None)


def test_structures_match_the_packed_ones():
    """The binding packs the C structures itself."""
    assert ctypes.sizeof(rb._Heads) == len(R._heads_struct(*range(12))) == 88
    assert ctypes.sizeof(rb._Rotary) == len(R._rotary_struct(1, 2, 3, 4, 5, 6.0)) == 32
    assert ctypes.sizeof(rb._Layout) == len(R._layout_struct(*range(8))) == 56
    assert bytes(rb._Heads(*range(1, 13))) == R._heads_struct(*range(1, 13))
    assert bytes(rb._Rotary(1, 2, 3, 4, 5, 6.0)) == R._rotary_struct(1, 2, 3, 4, 5, 6.0)
    assert bytes(rb._Layout(*range(1, 9))) == R._layout_struct(*range(1, 9))


def test_size_and_type_refusals():
    for D in (0, 4, 12, -8, 520, 1024):
        assert _fwd(D=D) == -2 and _alone(D=D) == -2
    for dim in (0, 2, -4, 6, 62, 68):
        assert _fwd(rot=_rot(dim=dim)) == -2
    for first in (-2, 1, 3, 2, 64):
        assert _fwd(rot=_rot(first=first)) == -2
    assert _fwd(rot=_rot(dim=32, first=34)) == -2 and _alone(rot=_rot(dim=32, first=2 ** 31 - 2)) == -2
    assert _fwd(rot=_rot(interleaved=2)) == -5 and _fwd(rot=_rot(interleaved=-1)) == -5
    for bad in (float("nan"), float("inf")):
        assert _fwd(rot=_rot(scale=bad)) == -13 and _fwd(eps=bad) == -13
    assert _fwd(eps=-1e-6) == -13
    assert _fwd(dt=3, pdt=3) == -14 and _fwd(dt=-1, pdt=-1) == -14 and _fwd(dt=0, pdt=1) == -14 and _fwd(dt=2, pdt=0) == -14
    assert _alone(dt=5) == -14


def test_layout_and_pointer_refusals():
    lib = rb._load()
    assert _fwd(lay=_layout(rpt=2)) == -5 and _fwd(lay=_layout(rpt=0)) == -5 and _fwd(lay=_layout(reserved=1)) == -5
    assert _fwd(lay=_layout(n=-1)) == -5 and _fwd(lay=_layout(n=1 << 31)) == -5 and _fwd(lay=_layout(n_logical=-1)) == -5
    assert _fwd(lay=_layout(n_logical=1 << 31)) == -5
    assert _fwd(q=_heads(heads=0)) == -5 and _fwd(q=_heads(heads=65536)) == -5 and _fwd(q=_heads(reserved=1)) == -5
    assert _fwd(q=_heads(heads=32768, token=1 << 22, out_token=1 << 22), lay=_layout(n=1 << 16)) == -5      # 2^31 rows
    assert _fwd(q=_heads(at=None)) == -1 and _fwd(q=_heads(out=None)) == -1 and _bwd(q=_heads(dy=None)) == -1
    assert _fwd(lay=_layout(tok=None)) == -1 and _fwd(rot=_rot(position=None)) == -1 and _fwd(rot=_rot(turns=None)) == -1
    assert lib.rotary_fwd(None, None, 64, 0, _layout(), _rot(), None) == -1
    assert lib.rotary_fwd(_heads(), None, 64, 0, None, _rot(), None) == -1
    assert lib.rotary_bwd(_heads(), None, 64, 0, _layout(), None, None) == -1
    assert _fwd(q=_heads(at=A[0] + 8)) == -3 and _fwd(q=_heads(out=A[1] + 2)) == -3 and _fwd(q=_heads(w=A[3] + 8)) == -3
    assert _bwd(q=_heads(dy=A[2] + 8)) == -3
    assert _alone(q=_heads(at=A[0] + 16), dt=2) == -3 and _alone(q=_heads(out=A[1] + 16), dt=2) == -3       # FP32: 32 bytes
    assert _fwd(lay=_layout(tok=258)) == -3 and _fwd(rot=_rot(position=258)) == -3 and _fwd(rot=_rot(turns=264)) == -3
    assert _fwd(lay=_layout(n=0, tok=None)) == 0 and _alone(q=_heads(at=None, out=None), lay=_layout(n=0)) == 0


def test_stride_and_overlap_refusals():
    assert _fwd(q=_heads(token=132)) == -3 and _fwd(q=_heads(head=60)) == -3 and _fwd(q=_heads(out_token=130)) == -3
    assert _fwd(q=_heads(token=-128)) == -4 and _fwd(q=_heads(head=-64)) == -4
    # outputs whose rows overlap: heads, slots, neither inside the other
    assert _fwd(q=_heads(out_head=0)) == -4 and _fwd(q=_heads(out_head=56)) == -4 and _fwd(q=_heads(out_token=64)) == -4
    assert _fwd(q=_heads(out_token=64, out_head=192)) == -4 and _fwd(q=_heads(out_token=0, out_head=64)) == -4
    # in place only with the strides of the input
    assert _fwd(q=_heads(out=A[0], out_token=256)) == -4 and _bwd(q=_heads(out=A[2], dy_token=256)) == -4
    # the keys' output is none of the queries' tensors, and the other way round
    k = lambda **kw: _heads(**{"at": A[4], "out": A[5], "dy": A[6], **kw})                   # noqa: E731
    assert _fwd(k=k(out=A[1])) == -5 and _fwd(k=k(out=A[0])) == -5 and _fwd(q=_heads(out=A[4]), k=k()) == -5
    assert _bwd(k=k(out=A[2])) == -5 and _bwd(q=_heads(out=A[6]), k=k()) == -5
    assert _fwd(k=k(heads=0)) == -5 and _fwd(k=k(at=None)) == -1 and _fwd(k=k(out_head=8)) == -4


def test_workspace_refusals_and_size():
    lib = rb._load()
    size = lib.qk_norm_workspace_bytes
    assert size(64, 4, 2, 12) == 0 and size(-1, 4, 2, 64) == 0 and size(1 << 31, 4, 2, 64) == 0
    assert size(64, 0, 2, 64) == 0 and size(64, 4, -1, 64) == 0 and size(64, 65536, 2, 64) == 0 and size(64, 4, 2, 520) == 0
    n, D = 900, 128
    # few tokens: groups of 4 and a partial sum for 4 heads; many: of 8, 40 heads in 4 chunks, keys in the last one too;
    # 10 + 1 in one
    assert 0 <= size(n, 32, 8, D) - (256 + 4 * n + 4 * 225 + 10 * (225 + n) * D * 4) < 2048 and size(n, 32, 8, D) % 256 == 0
    n = 40000
    assert 0 <= size(n, 32, 8, D) - (256 + 4 * n + 4 * 5000 + 5 * (5000 + n) * D * 4) < 2048
    assert 0 <= size(n, 10, 1, D) - (256 + 4 * n + 4 * 5000 + 2 * (5000 + n) * D * 4) < 2048
    big = 1 << 40
    assert lib.qk_norm_begin(P(256), 16, 64, 4, 2, 64, None) == -6 and lib.qk_norm_begin(P(272), big, 64, 4, 2, 64, None) == -3
    assert lib.qk_norm_begin(None, big, 64, 4, 2, 64, None) == -1 and lib.qk_norm_begin(P(256), big, 64, 4, 2, 60, None) == -2
    fin = lambda q=P(512), k=P(1024), hk=2, s=1.0: lib.qk_norm_finalize(P(256), 64, 4, hk, 64, s, q, k, None)   # noqa: E731
    assert fin(q=None, k=None) == -1 and fin(s=float("nan")) == -13 and fin(q=P(514)) == -3 and fin(hk=0) == -5
    assert lib.qk_norm_finalize(None, 64, 4, 2, 64, 1.0, P(512), None, None) == -1
    assert _bwd(ws=P(272)) == -3 and lib.qk_norm_status(None, None, ctypes.byref(ctypes.c_int32())) == -1


def test_turns_are_the_rounded_exact_values():
    lib = rb._load()
    f = np.concatenate([rb.rotary_frequencies(128), rb.rotary_frequencies(64, 500000.0, 8.0, 8192),
                        [0.0, 1e-300, 5e-324, -0.3, 3.0, 2.0 ** -40, 1.7 * 2.0 ** -62, 2147483647.9, -2.0 ** 30 - 0.125]])
    t = np.empty(f.size, dtype=np.uint64)
    assert lib.rotary_turns(f.ctypes.data, f.size, t.ctypes.data) == 0
    for a, b in zip(f, t):
        want = int(O.turns(abs(a)) * 2 ** 64 + Fraction(1, 2)) * (-1 if a < 0 else 1) % 2 ** 64
        assert int(b) == want, a
    for bad in (float("nan"), float("inf"), 2.0 ** 31, -2.0 ** 40):
        x = np.asarray([1.0, bad])
        assert lib.rotary_turns(x.ctypes.data, 2, t.ctypes.data) == -13
    assert lib.rotary_turns(None, 1, t.ctypes.data) == -1 and lib.rotary_turns(None, 0, None) == 0
    assert lib.rotary_turns(f.ctypes.data, -1, t.ctypes.data) == -5


def test_frequencies():
    f = rb.rotary_frequencies(8)
    assert f.dtype == np.float64 and np.allclose(f, [1, 0.1, 0.01, 0.001], rtol=1e-15)
    assert np.allclose(rb.rotary_frequencies(8, factor=4.0), f / 4, rtol=1e-15)
    g = rb.rotary_frequencies(8, factor=4.0, original_length=2 * np.pi * 100, low=1.0, high=20.0)
    # 100, 10, 1 and 0.1 turns over the original length: kept; (10 - 1) / 19 of the way; stretched
    assert np.allclose(g, [f[0], f[1] * (9 / 19 + 10 / 19 / 4), f[2] / 4, f[3] / 4], rtol=1e-14)
    for bad in (lambda: rb.rotary_frequencies(6), lambda: rb.rotary_frequencies(0), lambda: rb.rotary_frequencies(8, base=0),
                lambda: rb.rotary_frequencies(8, factor=0), lambda: rb.rotary_frequencies(8, original_length=0),
                lambda: rb.rotary_frequencies(8, original_length=10, low=4, high=4)):
        with pytest.raises(ValueError):
            bad()


def test_rotary_plan_refusals():
    for kw, err in ((dict(rotary_dim=6), ValueError), (dict(rotary_dim=0), ValueError), (dict(rotary_dim=8, first=3), ValueError),
                    (dict(rotary_dim=8, first=-2), ValueError), (dict(rotary_dim=8, inv_freq=np.ones(3)), ValueError),
                    (dict(rotary_dim=8, inv_freq=np.full(4, np.nan)), rb.RmsNormError)):
        with pytest.raises(err):
            rb.Rotary(device="cpu", **kw)
    r = rb.Rotary(8, inv_freq=torch.ones(4, dtype=torch.float64), device="cpu")
    assert r.turns.dtype == torch.int64 and r.turns.shape == (4,)


# ---------------------------------------------------------------- binding, host tensors let through

LAY = rb.CallLayout(torch.arange(4, dtype=torch.int32), None, 0, 4, 1, 4)
Q, K, W = torch.zeros(4, 3, 16, dtype=torch.bfloat16), torch.zeros(4, 1, 16, dtype=torch.bfloat16), torch.ones(16, dtype=torch.bfloat16)
POS, ROT = torch.zeros(4, dtype=torch.int32), rb.Rotary(16, device="cpu")


def test_binding_refuses_host_tensors():
    for call in (lambda: rb.rotary_fwd(Q, K, LAY, POS, ROT), lambda: rb.rotary_bwd(Q, None, LAY, POS, ROT),
                 lambda: rb.qk_norm_rotary_fwd(Q, K, W, W, LAY, POS, ROT, E),
                 lambda: rb.qk_norm_rotary_bwd(Q, K, W, W, Q, K, LAY, POS, ROT, E)):
        with pytest.raises(ValueError, match="CUDA tensor"):
            call()


@pytest.fixture
def as_cuda(monkeypatch):
    """Lets host tensors pass as CUDA ones, so that the checks behind that one are reached."""
    monkeypatch.setattr(R, "_is_cuda", lambda t: True)
    monkeypatch.setattr(R, "_current", lambda: -1)                    # what a host tensor's index is
    monkeypatch.setattr(R, "_raw_stream", lambda index: 0)


@pytest.mark.parametrize("value", [0.5, np.zeros((4, 3, 16), dtype=np.float32), "x"], ids=["number", "array", "text"])
@pytest.mark.parametrize("name,call", [
    ("q", lambda v: rb.rotary_fwd(v, K, LAY, POS, ROT)), ("k", lambda v: rb.rotary_fwd(Q, v, LAY, POS, ROT)),
    ("q_out", lambda v: rb.rotary_fwd(Q, K, LAY, POS, ROT, q_out=v)), ("k_out", lambda v: rb.rotary_fwd(Q, K, LAY, POS, ROT, k_out=v)),
    ("position", lambda v: rb.rotary_fwd(Q, K, LAY, v, ROT)), ("rotary", lambda v: rb.rotary_fwd(Q, K, LAY, POS, v)),
    ("layout", lambda v: rb.rotary_fwd(Q, K, v, POS, ROT)), ("dq_out", lambda v: rb.rotary_bwd(v, K, LAY, POS, ROT)),
    ("dk", lambda v: rb.rotary_bwd(Q, K, LAY, POS, ROT, dk=v)),
    ("q_weight", lambda v: rb.qk_norm_rotary_fwd(Q, K, v, W, LAY, POS, ROT, E)),
    ("k_weight", lambda v: rb.qk_norm_rotary_fwd(Q, K, W, v, LAY, POS, ROT, E)),
    ("dq_out", lambda v: rb.qk_norm_rotary_bwd(Q, K, W, W, v, K, LAY, POS, ROT, E)),
    ("dk_out", lambda v: rb.qk_norm_rotary_bwd(Q, K, W, W, Q, v, LAY, POS, ROT, E)),
    ("dq", lambda v: rb.qk_norm_rotary_bwd(Q, K, W, W, Q, K, LAY, POS, ROT, E, dq=v)),
    ("workspace", lambda v: rb.qk_norm_rotary_bwd(Q, K, W, W, Q, K, LAY, POS, ROT, E, workspace=v))])
def test_wrong_kinds_are_type_errors(as_cuda, name, call, value):
    with pytest.raises(TypeError, match=name):
        call(value)


def test_binding_checks_shapes_types_and_devices(as_cuda, monkeypatch):
    fwd = lambda q=Q, k=K, qw=W, kw=W, lay=LAY, pos=POS, rot=ROT, **o: rb.qk_norm_rotary_fwd(q, k, qw, kw, lay, pos, rot, E, **o)   # noqa: E731
    for err, match, call in (
            (TypeError, "bfloat16, float16 or float32", lambda: fwd(q=Q.double())),
            (TypeError, "k", lambda: fwd(k=K.float())),
            (TypeError, "q_out", lambda: fwd(q_out=Q.float())),
            (ValueError, "head_dim", lambda: fwd(q=Q[0])),
            (ValueError, "k: expected", lambda: fwd(k=K[0])),
            (ValueError, "k: expected", lambda: fwd(k=torch.zeros(4, 1, 24, dtype=K.dtype))),
            (ValueError, "q_out: expected", lambda: fwd(q_out=torch.zeros(4, 2, 16, dtype=Q.dtype))),
            (ValueError, "token slots", lambda: fwd(q=Q[:3])),
            (ValueError, "token slots", lambda: fwd(k_out=K[:2])),
            (ValueError, "column stride", lambda: fwd(q=torch.zeros(4, 16, 3, dtype=Q.dtype).transpose(1, 2))),
            (ValueError, "q_weight", lambda: fwd(qw=W[:8])),
            (TypeError, "k_weight", lambda: fwd(kw=W.half())),
            (TypeError, "one type", lambda: fwd(qw=W.float())),
            (ValueError, "k_weight", lambda: fwd(k=None)),
            (ValueError, "k_out", lambda: fwd(k=None, kw=None, k_out=K)),
            (ValueError, "rows_per_token", lambda: fwd(lay=rb.CallLayout(LAY.tok_id, None, 0, 4, 2, 4))),
            (TypeError, "tok_id", lambda: fwd(lay=rb.CallLayout(LAY.tok_id.long(), None, 0, 4, 1, 4))),
            (ValueError, "tok_id", lambda: fwd(lay=rb.CallLayout(LAY.tok_id[:3], None, 0, 4, 1, 4))),
            (TypeError, "position", lambda: fwd(pos=POS.long())),
            (ValueError, "position", lambda: fwd(pos=POS[:3])),
            (ValueError, "position", lambda: fwd(pos=torch.zeros(8, dtype=torch.int32)[::2])),
            (rb.RmsNormError, "HIDDEN", lambda: fwd(rot=rb.Rotary(32, device="cpu"))),
            (rb.RmsNormError, "ALIGN", lambda: fwd(q=torch.zeros(4 * 52, dtype=Q.dtype)[4:].as_strided((4, 3, 16), (48, 16, 1)))),
            (rb.RmsNormError, "STRIDE", lambda: fwd(q_out=torch.zeros(4, 1, 16, dtype=Q.dtype).expand(4, 3, 16))),
            (ValueError, "dk_out", lambda: rb.qk_norm_rotary_bwd(Q, None, W, None, Q, K, LAY, POS, ROT, E))):
        with pytest.raises(err, match=match):
            call()
    monkeypatch.setattr(R, "_current", lambda: 1)
    with pytest.raises(ValueError, match="current device"):
        fwd()
