"""Pins of oracle.f8 and oracle.route by hand-worked values, torch's own e4m3 type and finite differences (CPU)."""

import numpy as np
import pytest
import torch

from oracle import f8, route


def test_e4m3_table():
    v = f8.e4m3_values()
    assert v[0x7E] == 448 and v[0x08] == 2.0 ** -6 and v[0x01] == 2.0 ** -9 and v[0x38] == 1.0 and v[0xC0] == -2.0
    assert np.isnan(v[0x7F]) and np.isnan(v[0xFF])
    t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float().numpy().astype(np.float64)
    assert np.array_equal(v, t, equal_nan=True)


def test_encode_ties_and_neighbours():
    v = f8.e4m3_values()[:127]
    assert np.array_equal(f8.encode(v), np.arange(127, dtype=np.uint8))
    mid = (v[1:] + v[:-1]) / 2
    even = np.where(np.arange(126) % 2 == 0, np.arange(126), np.arange(1, 127))
    assert np.array_equal(f8.encode(mid), even)
    assert np.array_equal(f8.encode(mid * (1 + 2.0 ** -50)), np.arange(1, 127))
    assert np.array_equal(f8.encode(mid * (1 - 2.0 ** -50)), np.arange(126))
    assert np.array_equal(f8.encode(-mid), even | 0x80)


def test_quantize_by_hand():
    # the largest value takes 448; 1 / 448 rounds to fp32 once; zeros take the smallest scale
    x = np.zeros((2, 130))
    x[0, 0], x[0, 1], x[0, 128] = 1.0, -0.5, 448.0
    codes, s = f8.quantize_rows(x)
    assert codes.shape == (2, 256) and s.shape == (2, 2)
    assert s[0, 0] == np.float32(1 / 448) and s[1, 0] == 1.0 and s[0, 1] == np.float32(2.0 ** -80)
    assert codes[0, 0] == 0x7E and codes[0, 1] == 0x76 | 0x80 and codes[0, 128] == 0x7E
    assert not codes[1].any() and not codes[0, 130:].any()
    x[1, 5] = np.inf
    assert np.isnan(f8.quantize_rows(x)[1][0, 1])


def test_weight_blocks():
    g = np.random.default_rng(3)
    w = g.standard_normal((200, 150))
    codes, s = f8.quantize_weight(w)
    assert codes.shape == (200, 256) and s.shape == (2, 2)
    assert s[1, 1] == np.float32(np.abs(w[128:, 128:]).max() / 448)
    v = f8.weight_values(codes, s, 150)
    big = np.repeat(np.repeat(s, 128, 0)[:200], 128, 1)[:, :150].astype(np.float64)
    # half a step of a normal value, or of the subnormal spacing
    assert np.all(np.abs(v - w) <= np.maximum(np.abs(w) * 2.0 ** -4, big * 2.0 ** -10) * (1 + 1e-6))
    # a block's transpose is the block of the transpose
    ct, st = f8.quantize_weight(w.T)
    assert np.array_equal(ct[:, :200], codes[:, :150].T) and np.array_equal(st, s.T)


def test_route_by_hand():
    l = np.log(np.array([[1.0, 2.0, 4.0, 1.0], [3.0, 3.0, 1.0, 1.0]]))
    l = np.vstack([l, np.full((1, 4), -np.inf)])
    r = route.route(l, 2, True, 0.5)
    assert r["ids"].tolist() == [[2, 1], [0, 1], [-1, -1]]
    assert np.allclose(r["weights"], [[4 / 6, 2 / 6], [0.5, 0.5], [0, 0]])
    assert r["counts"].tolist() == [1, 2, 1, 0, 2]
    # f = counts * 4 / (2 * 2) = counts; P = column means over the two rows that have an expert
    P = (np.array([1, 2, 4, 1]) / 8 + np.array([3, 3, 1, 1]) / 8) / 2
    assert np.isclose(r["loss"], 0.5 * (np.array([1, 2, 1, 0]) * P).sum())


@pytest.mark.parametrize("normalise", [False, True])
def test_route_backward_against_differences(normalise):
    g = np.random.default_rng(5)
    l, dw = g.standard_normal((3, 7)), g.standard_normal((3, 3))
    r = route.route(l, 3, normalise, 0.1)
    got = route.route_backward(l, r, normalise, 0.1, dw, 2.0)
    f = r["counts"][:7] * 7 / (3 * 3.0)

    def value(x):
        q = route.route(x, 3, normalise, 0.1)
        return (dw * q["weights"]).sum() + 2.0 * 0.1 * (f * q["psum"]).sum() / 3

    for t in range(3):
        for e in range(7):
            h = np.zeros_like(l)
            h[t, e] = 1e-6
            assert np.isclose((value(l + h) - value(l - h)) / 2e-6, got[t, e], atol=1e-8)


def test_combine_leaves_slots_of_weight_zero_out():
    y = np.array([[[1.0, 2.0], [np.nan, np.inf]], [[3.0, 4.0], [5.0, 6.0]]])
    assert np.array_equal(route.combine(y, [[2.0, 0.0], [1.0, -1.0]]), [[2.0, 4.0], [-2.0, -2.0]])
    assert np.isnan(route.combine(y)[0, 0]) and np.isnan(route.combine(y, [[1.0, np.nan], [0.0, 0.0]])[0]).all()
