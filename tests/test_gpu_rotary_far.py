"""GPU: rotary positions over the whole int32 range in exact arithmetic, the backward pass of the norms with offsets past
2^32 elements in every tensor and in the workspace, and as many heads as a call may have."""
import numpy as np
import pytest
import torch

import invariant_rmsnorm_fwd_gb300 as rb
from oracle import rotary as O

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

EPS = 1e-6
BF, FP16, F32 = torch.bfloat16, torch.float16, torch.float32


def _same(a, b):
    word = torch.int32 if a.element_size() == 4 else torch.int16
    return torch.equal(a.contiguous().view(word), b.contiguous().view(word))


def _f64(t):
    return t.double().cpu().numpy()


def _within(name, got, ref, bound):
    err = np.abs(got - ref)
    bad = ~(err <= bound)
    assert not bad.any(), (name, int(bad.sum()), float((err / bound).max()), np.argwhere(bad)[:3].tolist())


def _cos_sin(positions, frequencies):
    """Cosine and sine [positions, frequencies]: the fraction of a turn in 2^-192 of one, then float64."""
    one = 1 << 192
    angle = np.empty((len(positions), len(frequencies)))
    for j, f in enumerate(frequencies):
        t = O.turns(f)
        step = t.numerator * one // t.denominator
        for i, p in enumerate(positions):
            a = step * int(p) % one
            angle[i, j] = 2 * np.pi * float((a - one if a >= one // 2 else a) / one)
    return np.cos(angle), np.sin(angle)


@pytest.mark.parametrize("dtype,D,rot,first,inter", [
    (F32, 64, 64, 0, True), (F32, 64, 64, 0, False), (F32, 72, 72, 0, False), (F32, 64, 60, 2, False),
    (BF, 64, 64, 0, False), (BF, 80, 72, 4, False), (FP16, 64, 64, 0, True), (FP16, 64, 60, 2, False), (FP16, 72, 72, 0, False)],
    ids=lambda v: str(v).replace("torch.", ""))
def test_cosine_and_sine_over_the_whole_range(dtype, D, rot, first, inter):
    """Pairs (1, 0) turn into cosine and sine themselves: with scale 1 off by at most 4 U (the oracle's derivation without
    the product with scale) and the rounding to the type.  A third of the frequencies are multiples of an eighth of a
    turn, where quadrants meet, and their neighbours."""
    g = np.random.default_rng(rot + D)
    p = np.concatenate([g.integers(-2 ** 31, 2 ** 31, 1500), g.integers(-5000, 200000, 500), np.arange(-40, 40),
                        2 ** 31 - 1 - np.arange(9), -2 ** 31 + np.arange(9)])
    eighth = np.pi / 4
    freq = rb.rotary_frequencies(rot)
    m = freq.size // 3
    freq[m:2 * m] = eighth * g.integers(1, 9, m) * (1 + g.choice([0.0, 2.0 ** -52, -2.0 ** -50, 2.0 ** -36, -2.0 ** -33], m))
    freq[2 * m:] = g.uniform(-4, 4, freq.size - 2 * m)
    n = len(p)
    a, b = O.pairs(rot, first, inter)
    x = torch.zeros(n, 1, D, dtype=dtype, device="cuda")
    x[..., torch.from_numpy(a).cuda()] = 1.0
    pos = torch.from_numpy(p.astype(np.int32)).cuda()
    lay = rb.call_layout(np.arange(n, dtype=np.int32), 1, n, with_plan=False)
    r = rb.Rotary(rot, interleaved=inter, first=first, inv_freq=freq)
    c, s = _cos_sin(p, freq)
    name = str(dtype).split(".")[1]
    for fn, sign in ((rb.rotary_fwd, 1), (rb.rotary_bwd, -1)):
        y = _f64(fn(x, None, lay, pos, r)[0])[:, 0]
        for got, ref in ((y[:, a], c), (y[:, b], sign * s)):
            _within("cosine, sine", got, ref, O.rounded(np.full_like(ref, 4 * O.U), ref, name))


@pytest.mark.parametrize("dtype,D,rot,first,inter", [(BF, 64, 64, 0, False), (BF, 72, 72, 0, False), (FP16, 80, 20, 2, False),
                                                     (F32, 128, 64, 32, True), (F32, 72, 36, 2, False)],
                         ids=lambda v: str(v).replace("torch.", ""))
def test_backward_offsets_past_32_bits(dtype, D, rot, first, inter):
    """Token stride 2^28 elements, and heads 2^31 apart: x, dy and dx in turn reach past 2^32 elements."""
    n, h, stride = 18, 3, 2 ** 28
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 40 * 2 ** 30:
        pytest.skip("needs 40 GB")
    g = torch.Generator("cuda").manual_seed(D)
    x, dy = ((torch.randn(n, h, D, generator=g, device="cuda") * s).to(dtype) for s in (1.5, 0.01))
    w = 1 + 0.1 * torch.randn(D, generator=g, device="cuda")
    pos = torch.arange(n, dtype=torch.int32, device="cuda") * 77
    lay = rb.call_layout(np.arange(n, dtype=np.int32), 1, n, with_plan=False)
    r = rb.Rotary(rot, interleaved=inter, first=first)

    def bwd(x, dy, dx=None):
        ws = rb.QkNormWorkspace(n, h, 0, D)
        ws.begin()
        got, _ = rb.qk_norm_rotary_bwd(x, None, w, None, dy, None, lay, pos, r, EPS, dq=dx, workspace=ws)
        dw, _ = ws.finalize()
        assert ws.status() == 0
        return got, dw

    want, dw = bwd(x, dy)
    big = torch.zeros(n * stride, dtype=dtype, device="cuda")
    for far in (torch.as_strided(big, (n, h, D), (stride, D, 1)),
                torch.as_strided(big, (h, n, D), (2 ** 31, D, 1), 1024 * 64).transpose(0, 1)):
        for run in (lambda: bwd(far.copy_(x), dy), lambda: bwd(x, far.copy_(dy)), lambda: bwd(x, dy, far),
                    lambda: bwd(far.copy_(x), dy, far), lambda: bwd(x, far.copy_(dy), far)):
            got, got_w = run()
            assert _same(got, want) and _same(got_w, dw)


def test_workspace_offsets_past_32_bits():
    """The last tokens of 4.5 M, two tensors of 512 columns: their sums in the dense area lie 2^32 elements and more
    behind its start.  Leaves are small whole numbers (rows of one magnitude, eps 0, no turn), so the sums are exact."""
    N, D = 4500004, 512                                               # 562,500 groups of 8 and one of 4
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 40 * 2 ** 30:
        pytest.skip("needs 40 GB")
    ws = rb.QkNormWorkspace(N, 1, 1, D)
    assert ws.bytes > 2 * N * D * 4                                   # a dense area for both tensors
    ids = np.concatenate([np.arange(N - 36, N), [3, 2, 1]]).astype(np.int32)      # four whole groups, the last four, cut ones
    n = ids.size
    g = np.random.default_rng(5)
    sign = lambda: np.where(g.random((n, 1, D)) < 0.5, -1.0, 1.0)                           # noqa: E731
    q, k, dq, dk = sign() * 2, sign() * 4, *(g.integers(-100, 100, (n, 1, D)).astype(float) for _ in "qk")
    to = lambda v: torch.from_numpy(v).to("cuda", F32)                                      # noqa: E731
    lay = rb.call_layout(ids, 1, N, with_plan=False)
    ws.begin()
    rb.qk_norm_rotary_bwd(to(q), to(k), None, None, to(dq), to(dk), lay, torch.zeros(n, dtype=torch.int32, device="cuda"),
                          rb.Rotary(8, interleaved=True), 0.0, workspace=ws)
    got = ws.finalize()
    assert ws.status() == rb.STATUS_MISSING
    for v, want in zip(got, ((dq * np.sign(q)).sum((0, 1)), (dk * np.sign(k)).sum((0, 1)))):
        assert np.array_equal(_f64(v), want)


def test_the_most_heads():
    """65,535 query heads beside as many key heads: values, gradients, and rows with the bits of a call of few heads."""
    n, h, D = 2, 65535, 8
    g = torch.Generator("cuda").manual_seed(1)
    q, k, dq, dk = ((torch.randn(n, h, D, generator=g, device="cuda") * s).to(BF) for s in (1.5, 1.5, 0.01, 0.01))
    qw, kw = (1 + 0.1 * torch.randn(D, generator=g, device="cuda") for _ in "qk")
    pos = torch.tensor([12, 345], dtype=torch.int32, device="cuda")
    lay = rb.call_layout(np.arange(n, dtype=np.int32), 1, n, with_plan=False)
    for r in (rb.Rotary(8), rb.Rotary(8, interleaved=True)):
        ws = rb.QkNormWorkspace(n, h, h, D)
        ws.begin()
        y, z = rb.qk_norm_rotary_fwd(q, k, qw, kw, lay, pos, r, EPS)
        a, b = rb.qk_norm_rotary_bwd(q, k, qw, kw, dq, dk, lay, pos, r, EPS, workspace=ws)
        grads = ws.finalize()
        assert ws.status() == 0
        for s in (slice(0, 3), slice(40000, 40005), slice(h - 4, h)):
            few = rb.qk_norm_rotary_fwd(q[:, s], k[:, s], qw, kw, lay, pos, r, EPS)
            assert _same(few[0], y[:, s]) and _same(few[1], z[:, s])
            few = rb.qk_norm_rotary_bwd(q[:, s], k[:, s], qw, kw, dq[:, s], dk[:, s], lay, pos, r, EPS)
            assert _same(few[0], a[:, s]) and _same(few[1], b[:, s])
        for x, w, dy, got in ((q, qw, dq, grads[0]), (k, kw, dk, grads[1])):
            _, ref, _, err = O.backward(_f64(x), _f64(w), _f64(dy), _f64(pos), rb.rotary_frequencies(8), 8, 0, r.interleaved, 1.0, EPS)
            _within("weight gradient", _f64(got), ref, err + O.U * np.abs(ref))
