"""GPU: calls that give a warp several steps, full chunks and many windows.  Their rows have the bits of small calls, and
their weight gradients those of every other layout, so what small calls are held to holds for them."""
import numpy as np
import pytest
import torch

import invariant_rmsnorm_fwd_gb300 as rb
from invariant_rmsnorm_fwd_gb300 import harness
from invariant_rmsnorm_fwd_gb300 import layout as L

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

EPS = 1e-6
BF, FP16, F32 = torch.bfloat16, torch.float16, torch.float32


def _word(t):
    return t.contiguous().view(torch.int32 if t.element_size() == 4 else torch.int16)


def _same(a, b):
    return torch.equal(_word(a), _word(b))


def _data(n, heads, D, dtype, scale, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    return (torch.randn(n, heads, D, generator=g, device="cuda") * scale).to(dtype)


#        n       hq hk D    rot  first inter dtype  (steps of a warp: up to 8 forward)
CASES = [(160000, 1, 1, 64, 64, 0, False, BF), (60000, 2, 1, 128, 128, 0, False, BF), (40000, 3, 1, 256, 64, 192, True, FP16),
         (30011, 9, 2, 80, 80, 0, False, BF), (30011, 7, 1, 96, 36, 0, False, FP16), (25000, 12, 3, 72, 72, 0, True, F32),
         (20000, 32, 8, 128, 128, 0, False, BF), (20000, 13, 4, 128, 104, 10, False, F32), (90000, 4, 1, 24, 24, 0, True, BF),
         (9000, 20, 4, 512, 512, 0, False, BF)]


@pytest.mark.parametrize("n,hq,hk,D,rot,first,inter,dtype", CASES, ids=lambda v: str(v).replace("torch.", ""))
def test_rows_of_large_calls_are_those_of_small_ones(n, hq, hk, D, rot, first, inter, dtype):
    gen = np.random.default_rng(n + D)
    ids = gen.permutation(n).astype(np.int32)                         # any order: no row looks at its neighbours
    at = np.arange(n)
    ids[(at // 777) % 3 == 1] = -1                                    # stretches of padding, and single slots of it
    ids[gen.integers(0, n, n // 50)] = -1
    q, k, dq, dk = _data(n, hq, D, dtype, 1.5, 1), _data(n, hk, D, dtype, 1.5, 2), _data(n, hq, D, dtype, 0.01, 3), \
        _data(n, hk, D, dtype, 0.01, 4)
    pos = torch.from_numpy(gen.integers(-10, 100000, n).astype(np.int32)).cuda()
    qw, kw = 1 + _data(1, 1, D, F32, 0.1, 5).reshape(D), 1 + _data(1, 1, D, F32, 0.1, 6).reshape(D)
    r = rb.Rotary(rot, interleaved=inter, first=first, scale=1.1)
    calls = {"fwd": lambda a, b, c, d, lay, p, **o: rb.qk_norm_rotary_fwd(a, b, qw, kw, lay, p, r, EPS, q_out=o["q"], k_out=o["k"]),
             "alone": lambda a, b, c, d, lay, p, **o: rb.rotary_fwd(a, b, lay, p, r, q_out=o["q"], k_out=o["k"]),
             "back": lambda a, b, c, d, lay, p, **o: rb.rotary_bwd(c, d, lay, p, r, dq=o["q"], dk=o["k"]),
             "bwd": lambda a, b, c, d, lay, p, **o: rb.qk_norm_rotary_bwd(a, b, qw, kw, c, d, lay, p, r, EPS, dq=o["q"], dk=o["k"])}
    whole = rb.call_layout(ids, 1, n, with_plan=False)
    parts = [slice(s, s + 45) for s in (0, 700, n // 2 - 7, n - 45)] + [slice(s, s + 1) for s in (1, n - 1)]
    for name, call in calls.items():
        out = {"q": torch.full_like(q, 7.0), "k": torch.full_like(k, 7.0)}
        call(q, k, dq, dk, whole, pos, **out)
        pad = torch.from_numpy(ids < 0).cuda()
        assert bool((out["q"][pad] == 7).all()) and bool((out["k"][pad] == 7).all()), name
        assert bool((out["q"][~pad].flatten(1) != 7).any(1).all()), name                     # every active token was written
        for s in parts:
            some = {"q": torch.full_like(q[s], 7.0), "k": torch.full_like(k[s], 7.0)}
            call(q[s], k[s], dq[s], dk[s], rb.call_layout(ids[s], 1, n, with_plan=False), pos[s], **some)
            assert _same(some["q"], out["q"][s]) and _same(some["k"], out["k"][s]), (name, s)


@pytest.mark.parametrize("hq,hk,D,rot,inter,dtype", [(32, 8, 128, 128, False, BF), (3, 1, 64, 64, True, BF), (10, 1, 256, 128, False, FP16),
                                                     (1, 1, 80, 20, False, F32), (6, 2, 24, 24, True, BF), (32, 8, 80, 80, False, BF),
                                                     (4, 1, 160, 160, True, FP16), (8, 2, 48, 40, False, BF), (5, 1, 96, 96, True, F32)],
                         ids=lambda v: str(v).replace("torch.", ""))
def test_gradients_of_many_tokens_in_every_layout(hq, hk, D, rot, inter, dtype):
    lengths = np.asarray([4099, 17, 3500, 1, 8, 5003, 260])
    n = int(lengths.sum())
    q, k, dq, dk = _data(n, hq, D, dtype, 1.5, 1), _data(n, hk, D, dtype, 1.5, 2), _data(n, hq, D, dtype, 0.01, 3), \
        _data(n, hk, D, dtype, 0.01, 4)
    qw, kw = _data(1, 1, D, dtype, 1.0, 5).reshape(D), _data(1, 1, D, dtype, 1.0, 6).reshape(D)
    pos = torch.arange(n, dtype=torch.int32, device="cuda") % 4099
    r = rb.Rotary(rot, interleaved=inter)
    lays = {kind: L.make_layout(kind, lengths, chunk=1003) for kind in ("full", "chunked", "singleton", "padded_left", "permuted")}
    runs = {kind: harness.run_layout_qk_norm_rotary(v, q, k, dq, dk, qw, kw, pos, r, EPS, 1.0 / n) for kind, v in lays.items()}
    rep = harness.assert_batch_invariant(runs, lays)
    assert rep.green, rep.summary()
    assert all(v.status == 0 and v.untouched_padding for v in runs.values())
    # every token a call of its own order: no group is whole
    order = np.random.default_rng(1).permutation(n).astype(np.int32)
    lay = L.Layout("shuffled", [order[:5000], order[5000:]], n)
    run = harness.run_layout_qk_norm_rotary(lay, q, k, dq, dk, qw, kw, pos, r, EPS, 1.0 / n)
    assert run.status == 0 and _same(run.dweight, runs["full"].dweight) and _same(run.dk_weight, runs["full"].dk_weight)
    assert _same(run.dx, runs["full"].dx) and _same(run.dk, runs["full"].dk)


def test_first_call_inside_a_capture():
    """A kernel's first launch of the process may be in a captured stream."""
    import subprocess
    import sys
    from conftest import ROOT
    program = """
import torch, numpy as np
import invariant_rmsnorm_fwd_gb300 as rb
n, D = 64, 128
q, k = torch.randn(n, 4, D, device="cuda").bfloat16(), torch.randn(n, 2, D, device="cuda").bfloat16()
lay = rb.call_layout(np.arange(n, dtype=np.int32), 1, n, with_plan=False)
pos, r, w = torch.arange(n, dtype=torch.int32, device="cuda"), rb.Rotary(D), torch.ones(D, device="cuda")
ws = rb.QkNormWorkspace(n, 4, 2, D)
g = torch.cuda.CUDAGraph()
torch.cuda.synchronize()
def step():
    y = rb.qk_norm_rotary_fwd(q, k, w, w, lay, pos, r, 1e-6)
    ws.begin()
    d = rb.qk_norm_rotary_bwd(q, k, w, w, *y, lay, pos, r, 1e-6, workspace=ws)
    return (*y, *d, *ws.finalize())
with torch.cuda.graph(g):
    got = step()
g.replay()
want = step()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(got, want)) and ws.status() == 0
"""
    res = subprocess.run([sys.executable, "-c", program], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert res.returncode == 0, res.stderr[-2000:]
