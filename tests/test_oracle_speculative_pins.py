"""The definitions in oracle/speculative.py against facts outside them."""

import math

import numpy as np
import pytest

from oracle import speculative as S


def test_rotation_keeps_norms_and_depends_on_the_distance_alone():
    rng = np.random.default_rng(0)
    f, m = S.rope_frequencies(128, 10000.0)
    assert m == 1.0 and f[0] == 1.0 and abs(f[-1] - 10000.0 ** (-126 / 128)) < 1e-18
    q, k = rng.standard_normal((1, 1, 128)), rng.standard_normal((1, 1, 128))
    for inter in (False, True):
        at = lambda x, p: S.rope_rotate(x, np.array([p]), f, m, inter)
        assert abs(np.linalg.norm(at(q, 777)) - np.linalg.norm(q)) < 1e-12
        assert abs((at(q, 900) * at(k, 700)).sum() - (at(q, 205) * at(k, 5)).sum()) < 1e-9
        assert np.array_equal(at(q, 0), q)


def test_a_quarter_turn():
    x = np.zeros((1, 1, 128))
    x[..., 0] = 1.0
    y = S.rope_rotate(x, np.array([1]), np.array([math.pi / 2, 0.0]), 1.0, False)
    assert abs(y[0, 0, 2] - 1) < 1e-15 and abs(y[0, 0, 0]) < 1e-15
    y = S.rope_rotate(x, np.array([1]), np.array([math.pi / 2, 0.0]), 1.0, True)
    assert abs(y[0, 0, 1] - 1) < 1e-15


@pytest.mark.parametrize("kind", ["linear", "ntk", "banded", "yarn"])
def test_scaling_by_one_changes_nothing_and_by_four_slows_the_slowest_pair_fourfold(kind):
    kw = dict(original_max_len=8192.0)
    plain, _ = S.rope_frequencies(128, 10000.0)
    one, m1 = S.rope_frequencies(128, 10000.0, scaling=kind, factor=1.0, **kw)
    assert np.allclose(one, plain, rtol=1e-14) and m1 == 1.0
    four, _ = S.rope_frequencies(128, 10000.0, scaling=kind, factor=4.0, **kw)
    assert abs(four[-1] / plain[-1] - 0.25) < 1e-12
    assert abs(four[0] / plain[0] - (0.25 if kind == "linear" else 1.0)) < 1e-12
    assert (np.diff(four) < 0).all()


def test_tree_rows_of_a_small_tree():
    assert S.tree_rows([-1, 0, 0, 1, -1]) == [{0}, {0, 1}, {0, 2}, {0, 1, 3}, {4}]
    assert S.pack_rows([{0, 33}, set()], 2).tolist() == [[1, 2], [0, 0]]


def test_tree_attention_closed_forms():
    K, V = np.zeros((3, 128)), np.zeros((3, 128))
    V[0], V[1], V[2] = 1.0, 4.0, 100.0
    K[1, 0] = 1.0
    q = np.zeros((2, 1, 128))
    q[:, 0, 0] = math.log(3.0)
    out, lse, spread = S.tree_attention(q, K, V, 1, [{0}, set()], 1.0)
    # weights 1 : 3 for the first draft, the committed token alone for the second
    assert np.allclose(out[0, 0], 13 / 4) and np.allclose(out[1, 0], 1.0)
    assert abs(lse[0, 0] - math.log(4.0)) < 1e-12 and lse[1, 0] == 0.0
    out, lse, _ = S.tree_attention(q, K, V, 0, [set(), {2}], 1.0)
    assert not out[0].any() and lse[0, 0] == -np.inf and np.allclose(out[1], 100.0)


def test_pool_walk():
    p = S.Pool([[5, 2, -1], [-1, -1, -1], [-1, -1, -1]], [6, 0, 0], [0, 0, 1, 0, 0, 1], 4, 12, np.arange(6))
    p.fork([0], [1])
    assert p.table[1].tolist() == [5, 2, -1] and p.refs.tolist() == [0, 0, 2, 0, 0, 2]
    p.resize([9, 7, 0])      # both leave the shared half page: copies 0 and 3, new page 1, page 2 free
    assert p.table.tolist() == [[5, 0, 1], [5, 3, -1], [-1, -1, -1]]
    assert p.refs.tolist() == [1, 1, 0, 1, 0, 2] and p.data.tolist() == [2, 1, 2, 2, 4, 5]
    p.resize([0, 4, 12])     # three pages are wanted, two are free: the third sequence stays empty
    assert p.lens.tolist() == [0, 4, 0] and p.flags == {"NO_PAGES"}
    assert p.refs.tolist() == [0, 0, 0, 0, 0, 1]
