"""CPU: the layer-norm and dropout oracle against hand-worked values, finite
differences and the generator's published vectors."""
import numpy as np
import pytest

from oracle import layernorm as O


def test_philox_published_vectors():
    f = 0xFFFFFFFF
    assert O.philox((0, 0, 0, 0), (0, 0)) == (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8)
    assert O.philox((f, f, f, f), (f, f)) == (0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD)
    assert O.philox((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0)) == \
        (0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1)


def test_mask_is_the_generators_words():
    seed, offset = 0x0123456789ABCDEF, 0xFEDCBA9876543210
    rows = [0, 5, 2 ** 31 - 1]
    keep = O.keep_mask(seed, offset, rows, 24, 0.25)
    for i, g in enumerate(rows):
        for h in range(24):
            w = O.philox((h // 8, g, offset & 0xFFFFFFFF, offset >> 32), (seed & 0xFFFFFFFF, seed >> 32))[h % 8 // 2]
            assert keep[i, h] == ((w >> 16 if h % 2 else w & 0xFFFF) >= 16384)


def test_mask_share_and_borders():
    keep = O.keep_mask(7, 1, np.arange(512), 512, 0.3)
    n = keep.size
    assert abs(keep.mean() - 0.7) < 5 * np.sqrt(0.21 / n)          # five standard deviations
    assert O.keep_mask(7, 1, [1], 64, 0.0).all() and not O.keep_mask(7, 1, [1], 64, 1.0).any()
    assert O.drop_scale(0.5) == 2.0 and O.drop_scale(0.0) == 1.0 and O.drop_scale(1.0) == 0.0


def test_hand_worked_row():
    # mean 3, deviations -2 -1 1 2, variance 2.5, eps 1.5: rstd = 1/2
    x = np.array([[1.0, 2, 4, 5]])
    w, b = np.array([1.0, 2, 1, -1]), np.array([0.0, 0.5, 0, 0])
    y, mean, rstd, _ = O.forward(x, w, b, 1.5)
    assert mean[0] == 3 and rstd[0] == 0.5
    assert np.array_equal(y, [[-1.0, -0.5, 0.5, -1.0]])
    # dy = 1, 1, 0, 0: a = 1, 2, 0, 0; mean a = 3/4; mean a xhat = (-1 - 1) / 4 = -1/2
    dx, dw, db, *_ = O.backward(x, w, np.array([[1.0, 1, 0, 0]]), 1.5)
    assert np.array_equal(dx, [[0.5 * (1 - 0.75 - 0.5), 0.5 * (2 - 0.75 - 0.25), 0.5 * (0 - 0.75 + 0.25),
                                0.5 * (0 - 0.75 + 0.5)]])
    assert np.array_equal(dw, [-1.0, -0.5, 0, 0]) and np.array_equal(db, [1.0, 1, 0, 0])


@pytest.mark.parametrize("H", [2, 3, 8])
def test_central_differences(H):
    rng = np.random.default_rng(H)
    x, dy = rng.normal(size=(3, H)) + 0.7, rng.normal(size=(3, H))
    w, b = rng.normal(size=H), rng.normal(size=H)
    loss = lambda x, w, b: float((dy * O.forward(x, w, b, 1e-3)[0]).sum())   # noqa: E731
    dx, dw, db, *_ = O.backward(x, w, dy, 1e-3)
    step = 1e-6
    for got, at in ((dx, 0), (dw, 1), (db, 2)):
        args = [x, w, b]
        for i in np.ndindex(args[at].shape):
            lo, hi = [a.copy() for a in args], [a.copy() for a in args]
            lo[at][i] -= step
            hi[at][i] += step
            num = (loss(*hi) - loss(*lo)) / (2 * step)
            # truncation ~ step^2 times the third derivative (below 1e3 here), rounding 1e-15 / step
            assert abs(num - got[i]) < 1e-7 * max(1, abs(got[i])) + 1e-8


def test_replay_orders_by_groups_then_blocks():
    # 2^24 + 1 - 2^24: which sums meet first decides whether the 1 survives
    big, col = np.float32(2 ** 24), np.zeros((72, 1), np.float32)
    col[0], col[1], col[2] = big, 1, -big
    assert O.grad_replay(col)[0] == 0                                       # (2^24 + 1) rounds, then - 2^24
    col = np.zeros((72, 1), np.float32)
    col[0], col[8], col[9] = big, 1, -big                                   # group 1: 1 - 2^24, exact
    assert O.grad_replay(col)[0] == 1
    col = np.zeros((130, 1), np.float32)
    col[0], col[64], col[128] = big, 1, -big                                # (block 0 + block 1) + block 2
    assert O.grad_replay(col)[0] == 0
