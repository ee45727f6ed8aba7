"""CPU: the oracle of the rotary operators, pinned by closed forms, differences and worked cases."""
import numpy as np
import pytest

from oracle import rotary as O

RNG = np.random.default_rng(5)


def _freq(r):
    return 10000.0 ** (-np.arange(0, r, 2) / r)


def test_inverse_turn():
    assert abs(float(O.INVERSE_TURN) - 1 / (2 * np.pi)) < 1e-16
    for p, f in ((0, 1.0), (1, 0.5), (100, 0.37), (-1000, 1.0), (12345, -0.001)):
        c, s = O.cos_sin_far(p, f)
        assert abs(c - np.cos(p * f)) < 1e-12 and abs(s - np.sin(p * f)) < 1e-12


def test_worked_cases():
    x = np.arange(1.0, 9.0).reshape(1, 1, 8)
    quarter = np.asarray([np.pi / 2, np.pi])                          # at position 1: a quarter and a half turn
    y, _ = O.rotate(x, [1], quarter, 4, 2, False)                     # halves: columns (2, 4) and (3, 5)
    assert np.allclose(y, [[[1, 2, -5, -4, 3, -6, 7, 8]]], atol=1e-14)
    y, _ = O.rotate(x, [1], quarter, 4, 2, True)                      # neighbours: (2, 3) and (4, 5)
    assert np.allclose(y, [[[1, 2, -4, 3, -5, -6, 7, 8]]], atol=1e-14)
    y, _ = O.rotate(x, [1], quarter, 4, 2, True, scale=2.0, back=True)
    assert np.allclose(y, [[[1, 2, 8, -6, -10, -12, 7, 8]]], atol=1e-14)


@pytest.mark.parametrize("inter", [False, True])
def test_scores_depend_on_the_distance_alone(inter):
    q, k = RNG.standard_normal((2, 1, 1, 16))
    f = _freq(12)
    dot = lambda m, n: float((O.rotate(q, [m], f, 12, 2, inter)[0] * O.rotate(k, [n], f, 12, 2, inter)[0]).sum())   # noqa: E731
    assert abs(dot(7, 3) - dot(104, 100)) < 1e-12 and abs(dot(7, 3) - dot(7, 4)) > 1e-6


def test_back_is_the_transpose_and_the_inverse():
    x, g = RNG.standard_normal((2, 5, 3, 24))
    p, f = RNG.integers(-50, 1000, 5), _freq(16)
    for inter in (False, True):
        y, _ = O.rotate(x, p, f, 16, 4, inter)
        z, _ = O.rotate(g, p, f, 16, 4, inter, back=True)
        assert abs((y * g).sum() - (x * z).sum()) < 1e-11
        assert np.allclose(O.rotate(y, p, f, 16, 4, inter, back=True)[0], x, atol=1e-13)
        assert np.allclose((y * y).sum(-1), (x * x).sum(-1))


@pytest.mark.parametrize("inter,scale,eps", [(False, 1.0, 1e-6), (True, 1.3, 0.1)])
def test_gradients_by_differences(inter, scale, eps):
    x, dy = RNG.standard_normal((2, 3, 2, 16))
    w = 1 + 0.3 * RNG.standard_normal(16)
    p, f, a = np.asarray([0, 3, 11]), _freq(8), (8, 4, inter, scale)
    dx, dw, _, _ = O.backward(x, w, dy, p, f, *a, eps)
    loss = lambda x, w: float((O.forward(x, w, p, f, *a, eps)[0] * dy).sum())                # noqa: E731
    h = 1e-6
    for i in np.ndindex(x.shape):
        d = np.zeros_like(x)
        d[i] = h
        assert abs((loss(x + d, w) - loss(x - d, w)) / (2 * h) - dx[i]) < 1e-7
    for i in range(16):
        d = np.zeros(16)
        d[i] = h
        assert abs((loss(x, w + d) - loss(x, w - d)) / (2 * h) - dw[i]) < 1e-7


def test_norm_closed_forms():
    x = np.full((1, 1, 8), -3.0)
    y, _ = O.forward(x, np.arange(1.0, 9.0), [0], _freq(8), 8, 0, False, 1.0, 0.0)
    assert np.allclose(y, -np.arange(1.0, 9.0))                       # a constant row: w times its sign
    x = RNG.standard_normal((4, 2, 8))
    p = np.asarray([1, 2, 3, 4])
    one = O.forward(x, 1.0, p, _freq(8), 8, 0, True, 1.0, 0.0)[0]
    assert np.allclose((one ** 2).mean(-1), 1) and np.allclose(O.forward(5 * x, 1.0, p, _freq(8), 8, 0, True, 1.0, 0.0)[0], one)


def test_replay_of_small_cases():
    """9 tokens make few groups, so chunks are of two heads, the second one of both kinds: a full group's tokens chunk by
    chunk, then the chunks; then the ninth token's."""
    q, k = RNG.standard_normal((9, 3, 16)).astype(np.float32), RNG.standard_normal((9, 2, 16)).astype(np.float32)
    gq, gk = O.grad_replay(q, k)

    def left(v):
        s = v[0]
        for r in v[1:]:
            s = s + r
        return s

    for got, parts in ((gq, (q[:, :2], q[:, 2:])), (gk, (k[:, :1], k[:, 1:]))):
        tokens = [[left(p[t]) for t in range(9)] for p in parts]               # heads of a chunk
        first = left([left(p[:8]) for p in tokens])                   # width 16: one lane a team, a token a team
        assert np.array_equal(got, first + left([p[8] for p in tokens]))
        assert np.allclose(got, np.concatenate(parts, 1).sum((0, 1)), atol=1e-4)


def test_replay_keeps_many_heads_in_chunks():
    """2,440 tokens of 60 + 3 heads: chunks of 8, the last one with 4 query heads and all key heads.  Leaves are zero but
    in one token, whose sums show the chunks."""
    q, k = np.zeros((2440, 60, 8), np.float32), np.zeros((2440, 3, 8), np.float32)
    big = np.float32(2.0 ** 24)
    q[77, 0], q[77, 1], q[77, 8], q[77, 15] = big, -big, 1.0, big     # (big - big + 3) + (1 + big): 1 is lost in the second chunk
    q[77, 7] = 3.0
    k[77, 0], k[77, 2] = 1.0, 2.0
    gq, gk = O.grad_replay(q, k)
    assert np.array_equal(gq, np.full(8, np.float32(3.0) + (np.float32(1.0) + big))) and np.array_equal(gk, np.full(8, 3.0, np.float32))
