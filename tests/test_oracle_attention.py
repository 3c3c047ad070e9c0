"""Pins of oracle.attention by hand-worked values, rotations by known angles and torch's float64 softmax (CPU)."""

import numpy as np
import torch

from oracle import attention as A


def test_norm_by_hand():
    x = np.array([[[3.0, 4.0, 0.0, 0.0]]])
    y, size = A.heads(x, np.array([1.0, 2.0, 1.0, 1.0]), 0.0, None, None, False)
    assert np.allclose(y, [[[1.2, 3.2, 0.0, 0.0]]]) and np.array_equal(size, np.abs(y))
    y, _ = A.heads(x, np.ones(4), 93.75, None, None, False)  # 25 / 4 + 93.75 = 100
    assert np.allclose(y, x / 10)


def test_rotation_by_hand():
    x = np.arange(1.0, 7.0).reshape(1, 1, 6)
    quarter = np.array([np.pi / 2])
    y, size = A.heads(x, None, 0.0, [1], quarter, False)  # columns 0 and 1 by a quarter turn, the rest as it is
    assert np.allclose(y, [[[-2, 1, 3, 4, 5, 6]]]) and np.allclose(size[0, 0, :2], 3)
    y, _ = A.heads(x, None, 0.0, [2], np.array([np.pi / 2, np.pi / 4]), False)  # (0, 2) by pi, (1, 3) by pi / 2
    assert np.allclose(y, [[[-1, -4, -3, 2, 5, 6]]])
    y, _ = A.heads(x, None, 0.0, [2], np.array([np.pi / 2, np.pi / 4]), True)   # (0, 1) by pi, (2, 3) by pi / 2
    assert np.allclose(y, [[[-1, -2, -4, 3, 5, 6]]])
    far = 2.0 ** 20 + 1
    y, _ = A.heads(x, None, 0.0, [far], np.array([np.pi]), False)  # an odd number of half turns (pi's own rounding: 1e-10)
    assert np.allclose(y[0, 0, :2], [-1, -2], atol=1e-8)


def test_quantize_by_hand():
    codes, s = A.quantize([[448.0, -224.0, 0.0, 17.0], [0.0, 0.0, 0.0, 0.0]])
    assert s[0] == 1.0 and s[1] == np.float32(2.0 ** -80)
    assert codes[0, 0] == 0x7E and codes[0, 1] == 0xF6 and codes[0, 3] == 0x58 and not codes[1].any()  # 17: a tie, to 16
    assert np.array_equal(A.values(codes, s)[0], [448.0, -224.0, 0.0, 16.0])


def test_attend_by_hand():
    q = np.array([[1.0, 0.0]])
    k = np.array([[np.log(2.0), 5.0], [0.0, -1.0], [9.0, 9.0]])
    v = np.array([[3.0, 0.0], [0.0, 6.0], [np.inf, np.nan]])
    out, spread, noise, reach = A.attend(q, k, v, 1.0, np.array([[True, True, False]]))
    assert np.allclose(out, [[2.0, 2.0]]) and np.allclose(spread, out) and np.allclose(noise, out)
    assert np.allclose(reach, np.log(2.0))
    assert not A.attend(q, k, v, 1.0, np.zeros((1, 3), bool))[0].any()


def test_attend_and_mask_against_torch():
    g = np.random.default_rng(1)
    n, m, D = 5, 9, 16
    q, k, v = g.standard_normal((n, D)), g.standard_normal((m, D)), g.standard_normal((m, D))
    seen = A.causal(n, m)
    assert seen.sum(1).tolist() == [5, 6, 7, 8, 9]
    assert A.causal(4, 2).sum(1).tolist() == [0, 0, 1, 2]
    s = torch.from_numpy(q @ k.T * 0.25).masked_fill(~torch.from_numpy(seen), float("-inf"))
    want = torch.softmax(s, 1).numpy() @ v
    assert np.allclose(A.attend(q, k, v, 0.25, seen)[0], want, atol=1e-14)
