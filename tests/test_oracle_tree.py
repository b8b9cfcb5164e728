"""Pins of the draft-tree oracle: a chain is causal attention, the visible sets
against powers of the parent matrix, windows shorter than the tree is deep by
hand, the rotation against complex products, and moves against a permutation."""
import numpy as np
import pytest

from oracle import attention as A
from oracle import kvstore as K
from oracle import tree as T


def random_parents(rng, n, roots=0.1):
    return [-1 if i == 0 or rng.random() < roots else int(rng.integers(0, i)) for i in range(n)]


@pytest.mark.parametrize("kind,window", [(A.FULL, 0), (A.SLIDING, 5), (A.SLIDING, 0), (A.CHUNKED, 4)])
def test_chain_is_causal(kind, window):
    chain = list(range(-1, 11))
    for prefix in (0, 1, 7, 30):
        for i in range(12):
            assert T.node_columns(kind, window, prefix, chain, i) == list(
                A.key_positions(kind, window, prefix + i))


def test_visible_sets_against_matrix_powers():
    rng = np.random.default_rng(0)
    for n in (1, 2, 9, 33):
        par = random_parents(rng, n)
        step = np.zeros((n, n))
        for i, p in enumerate(par):
            if p >= 0:
                step[i, p] = 1
        reach, power = np.eye(n), np.eye(n)
        for _ in range(n):
            power = power @ step
            reach += power
        for i in range(n):
            assert T.node_columns(A.FULL, 0, 3, par, i) == [0, 1, 2] + [
                3 + j for j in np.flatnonzero(reach[i])]
            assert T.depths(par)[i] == reach[i].sum() - 1


def test_windows_shorter_than_the_path():
    # 0 - 1 - 3 - 4 (depths 0, 1, 2, 3), node 2 beside 1; prefix 10
    par = [-1, 0, 0, 1, 3]
    assert T.node_columns(A.SLIDING, 1, 10, par, 4) == [13, 14]
    assert T.node_columns(A.SLIDING, 3, 10, par, 4) == [10, 11, 13, 14]
    assert T.node_columns(A.SLIDING, 4, 10, par, 4) == [9, 10, 11, 13, 14]
    assert T.node_columns(A.CHUNKED, 4, 10, par, 4) == [13, 14]       # positions 12, 13
    assert T.node_columns(A.CHUNKED, 4, 10, par, 2) == [8, 9, 10, 12]  # position 11


def test_rotation_against_complex_products():
    rng = np.random.default_rng(1)
    x = rng.standard_normal((3, 2, 16))
    ang = rng.standard_normal((5, 4))
    table = np.concatenate([np.cos(ang), np.sin(ang)], 1)
    pos = np.array([4, 0, 2])
    for inter in (False, True):
        y = T.norm_rope(x, None, 0.0, table, pos, 8, inter)
        a, b = (slice(0, 8, 2), slice(1, 8, 2)) if inter else (slice(0, 4), slice(4, 8))
        z = (x[..., a] + 1j * x[..., b]) * np.exp(1j * ang[pos])[:, None]
        np.testing.assert_allclose(y[..., a], z.real, atol=1e-12)
        np.testing.assert_allclose(y[..., b], z.imag, atol=1e-12)
        np.testing.assert_array_equal(y[..., 8:], x[..., 8:])
    w = rng.standard_normal(16)
    y = T.norm_rope(x, w, 0.5, None, None, 0, False)
    np.testing.assert_allclose(y, x * w / np.sqrt((x ** 2).sum(-1, keepdims=True) / 16 + 0.5))


@pytest.mark.parametrize("layout", ["per_layer", "envelope"])
def test_commit_moves_rows_of_both_pools(layout):
    layers = [(A.FULL, 0, 2), (A.SLIDING, 7, 2), (A.FULL, 0, 2)]
    pools = K.OraclePools(layers, 32, 32, 4, 8, "bf16", layout)
    rng = np.random.default_rng(2)
    mapping = np.zeros(37, np.int64)
    row = 4 + rng.permutation(20)
    mapping[row] = 4 + rng.permutation(20)
    mapping[row[0]] = 0                   # left the window
    x = rng.standard_normal((20, 2, 8)).astype(np.float32)
    for l in range(3):
        pools.store(l, x + l, -x - l, row, np.where(mapping[row] > 0, mapping[row], 1))
    before = [pools.read(l, row if layers[l][0] == A.FULL else mapping[row]) for l in range(3)]
    T.commit(pools, mapping, row, 6, [0, 3, 4, 9])
    want = np.arange(20)
    want[6:10] = [6, 9, 10, 15]
    for l in range(3):
        after = pools.read(l, row if layers[l][0] == A.FULL else mapping[row])
        for a, b in zip(after, before[l]):
            np.testing.assert_array_equal(a[1:], b[want][1:])
    T.move_rows(pools, mapping, [(row[0], row[19])])
    k, _ = pools.read(0, row)
    np.testing.assert_array_equal(k[19], before[0][0][0])
    k, _ = pools.read(1, mapping[row])
    np.testing.assert_array_equal(k[19], before[1][0][19])
