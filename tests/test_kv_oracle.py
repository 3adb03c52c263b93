"""The float64 oracle of the paged cache against hand-worked and brute-force values (CPU)."""
import math

import numpy as np
import pytest

from oracle import kv_oracle as K


def test_e4m3_values_and_rounding():
    v = K.e4m3_values()
    assert v[0x38] == 1.0 and v[0x7E] == 448.0 and v[1] == 2.0 ** -9 and v[0x08] == 2.0 ** -6 and v[0xB8] == -1.0
    assert np.isnan(v[0x7F]) and np.isnan(v[0xFF])
    codes = np.array([c for c in range(256) if c & 0x7F != 0x7F])
    assert np.array_equal(K.to_e4m3(v[codes]), codes)
    # midpoints go to the even code, anything beside them to the nearer one
    up = v[:0x7F]
    for c in range(0x7E):
        mid, eps = (up[c] + up[c + 1]) / 2, (up[c + 1] - up[c]) / 1e6
        assert K.to_e4m3(np.array([mid, mid - eps, mid + eps])).tolist() == [c + (c & 1), c, c + 1]
    assert K.to_e4m3(np.array([np.nan, np.inf, -np.inf])).tolist() == [0x7F] * 3


def test_torch_rounds_the_same():
    import torch
    x = np.random.default_rng(0).normal(size=4096).astype(np.float32) * 60
    want = torch.from_numpy(np.clip(x, -448, 448)).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(K.to_e4m3(np.clip(x, -448, 448)), want)


@pytest.mark.parametrize("a,s", [(448.0, 1.0), (448.0000001, 2.0), (449.0, 2.0), (224.0, 0.5), (1.0, 2.0 ** -8),
                                 (1.75, 2.0 ** -8), (1.76, 2.0 ** -7), (0.0, 2.0 ** -118), (1e-40, 2.0 ** -118)])
def test_least_scale(a, s):
    assert K.least_scale(a) == s


@pytest.mark.parametrize("style", ["halves", "pairs"])
def test_rotation_keeps_length_and_turns_by_position(style):
    x = np.random.default_rng(1).normal(size=(3, 2, 32))
    f = np.array([1.0, 0.25, 0.125, 0.01, 0.5, 0.3, 0.2, 0.1])
    y = K.rotate(x, np.array([0, 7, 100000]), f, style)
    assert np.array_equal(y[0], x[0]) and np.array_equal(y[:, :, 16:], x[:, :, 16:])
    assert np.allclose(np.linalg.norm(y, axis=-1), np.linalg.norm(x, axis=-1))
    a, b = (0, 8) if style == "halves" else (0, 1)
    assert y[1, 0, a] == pytest.approx(x[1, 0, a] * math.cos(7) - x[1, 0, b] * math.sin(7))
    # the product of two turned vectors depends on the distance alone
    u, w = x[:1], x[1:2]
    for p in (0, 5, 999):
        d = (K.rotate(u, np.array([p + 3]), f, style) * K.rotate(w, np.array([p]), f, style)).sum()
        assert d == pytest.approx((K.rotate(u, np.array([3]), f, style) * w).sum(), abs=1e-9)


def test_visible():
    assert K.visible(5, 8, 0, 0).tolist() == [1, 1, 1, 1, 1, 1, 0, 0]
    assert K.visible(5, 8, 2, 1).tolist() == [1, 0, 0, 0, 1, 1, 0, 0]
    assert not K.visible(-1, 8, 2, 1).any()
    assert K.visible(6, 8, 0, 0, [1, 3, -1], 2).tolist() == [0, 0, 1, 1, 0, 0, 1, 0]
    assert K.visible(6, 8, 1, 1, [], 2).tolist() == [1, 0, 0, 0, 0, 0, 1, 0]


def test_attend_row_by_hand():
    V = np.array([[1.0, 2.0], [3.0, -4.0]])
    out, lse, bound, _ = K.attend_row(np.array([1.0, 0.0]), np.array([[0.0, 9.0], [math.log(3), 9.0]]), V, np.array([True, True]), 1.0)
    assert out == pytest.approx([2.5, -2.5]) and lse == pytest.approx(math.log(4)) and bound == pytest.approx([2.5, 3.5])
    out, lse, _, _ = K.attend_row(np.array([1.0, 0.0]), V, V, np.array([False, False]), 1.0)
    assert out.tolist() == [0, 0] and lse == -math.inf


def test_append_grows_the_scale_of_a_page():
    values, scale = np.zeros((3, 1, 4, 2)), np.ones((3, 1))
    values[2, 0, 0] = [448, 1]
    new = np.array([[[449.0, 0.0]], [[1.0, 0.0]], [[1.0, -2.0]], [[8.0, 0.0]]])
    got, s = K.append_fp8(values, scale, np.array([2, 0]), 1, new)
    assert s[:, 0].tolist() == [2.0 ** -5, 1.0, 2.0]
    assert got[2, 0].tolist() == [[224, 0.5], [224.5, 0], [0.5, 0], [0.5, -1]]
    assert got[0, 0, 0].tolist() == [8 / s[0, 0], 0]
