"""Hand-worked values of kv_more_oracle (CPU)."""
import numpy as np
import pytest

from oracle import kv_more_oracle as M


def test_sees():
    f = lambda *a, **k: np.flatnonzero(M.sees(*a, **k)).tolist()
    assert f(3, 6) == [0, 1, 2, 3]
    assert f(3, 6, doc_start=2) == [2, 3]
    assert f(3, 6, doc_start=4) == []
    assert f(3, 6, prefix_end=5) == [0, 1, 2, 3, 4]
    assert f(3, 6, prefix_end=2) == [0, 1, 2, 3]
    assert f(3, 6, prefix_end=60, doc_start=1) == [1, 2, 3, 4, 5]
    assert f(1, 6, doc_start=3, prefix_end=5) == [3, 4]
    assert f(5, 6, window=2, sinks=1) == [0, 4, 5]
    assert f(5, 6, window=2, sinks=2, doc_start=1) == [1, 4, 5]
    assert f(5, 6, 1, 1, listed=[1], entry_tokens=2) == [0, 2, 3, 5]


def test_scores():
    x = M.scores(np.array([0.0, 3.0, -3.0, 1e30]), 2, softcap=2.0, slope=0.5)
    want = [0 - 1, 2 * np.tanh(1.5) - 0.5, -2 * np.tanh(1.5), 2 - 0.5]
    assert np.allclose(x, want, rtol=1e-15)
    # two keys of equal score, one token apart: the nearer one has e^slope times the weight
    out, lse, *_ = M.attend_row(np.array([1.0]), np.array([[0.5], [0.5]]), np.array([[0.0], [1.0]]), np.ones(2, bool), 1, 1.0, slope=np.log(3))
    assert out == pytest.approx(0.75) and lse == pytest.approx(0.5 + np.log(4 / 3))


def test_kept():
    assert M.kept_positions(10, [1, 3], 2, 2, 1) == [0, 2, 3, 6, 7, 8, 9]
    assert M.kept_positions(5, [], 4, 0, 0) == []
    assert M.kept_positions(3, [9], 4, 100, 0) == [0, 1, 2]
    assert M.kept_positions(6, [1], 4, 0, 5) == [0, 1, 2, 3, 4, 5]


def test_compact_page():
    codes, scale = M.compact_page(np.array([[448.0, -1.0], [np.nan, 2.0 ** -9]]))
    assert scale == 1 and codes.tolist() == [[0x7E, 0xB8], [0x7F, 0x01]]
    codes, scale = M.compact_page(np.array([[450.0]]))
    assert scale == 2 and codes.tolist() == [[0x76]]


def test_pool():
    p = M.Pool([0] * 5, [[-1] * 3 for _ in range(4)], [0, 0, 0, 0], 16)
    assert p.extend([20, 0, 1, -5]) == [0, 0, 0, 0]
    assert p.table == [[0, 1, -1], [-1] * 3, [2, -1, -1], [-1] * 3] and p.refs == [1, 1, 1, 0, 0] and p.kv_len == [20, 0, 1, 0]
    assert p.fork([0, 0, 0, 7], [1, 2, 0, 3]) == ([0, 0, -1, -1], [(1, 2, 4), (1, 3, 4)])
    assert p.refs == [3, 1, 1, 1, 0] and p.table[1:3] == [[0, 2, -1], [0, 3, -1]] and p.kv_len == [20, 20, 20, 0]
    assert p.extend([12, 30, 0, 16]) == [0, -1, 0, 0] and p.refs == [3, 1, 1, 1, 1] and p.kv_len == [32, 20, 20, 16]
    assert p.extend([1, 1, 13, 0]) == [1, 0, 1, 0]
    p.free([0, 0, 9, 2])
    assert p.refs == [1, 0, 1, 0, 1] and p.kv_len == [0, 21, 0, 16] and p.table[0] == [-1] * 3
