"""Pins of oracle/routing.py (CPU only): worked examples, invariants, and gradients
against central differences."""
import numpy as np
import pytest

from oracle import routing


def test_sort_worked_example():
    """Three groups, align 2: group 1 has pairs 0, 3, 4 (rows 2..4, row 5 padding), group 0
    pair 1 (row 0, row 1 padding), group 2 nothing; pair 2 (-1) and pair 5 (7) have no row."""
    off, row_of, pair_of, grp = routing.sort_tokens([[1, 0], [-1, 1], [1, 7]], 3, align=2, rows=9)
    assert off.tolist() == [0, 2, 6, 6]
    assert row_of.tolist() == [[2, 0], [-1, 3], [4, -1]]
    assert pair_of.tolist() == [1, -1, 0, 3, 4, -1, -2, -2, -2]
    assert grp.tolist() == [0, -1, 1, 1, 1, -1, -1, -1, -1]


def test_sort_masked_worked_example():
    off, row_of, pair_of, grp = routing.sort_tokens([[1], [1], [0], [1]], 2, cap=2)
    assert off.tolist() == [1, 2]
    assert row_of.tolist() == [[2], [3], [0], [-1]]
    assert pair_of.tolist() == [2, -2, 0, 1]
    assert grp.tolist() == [0, -1, 1, 1]


@pytest.mark.parametrize("align", [1, 3, 16])
def test_sort_invariants(align):
    r = np.random.default_rng(align)
    T, k, G = 57, 3, 11
    ids = r.integers(-1, G + 1, (T, k))
    off, row_of, pair_of, grp = routing.sort_tokens(ids, G, align)
    assert np.all(np.diff(off) >= 0) and np.all(off % align == 0)
    flat = ids.reshape(-1)
    for p, row in enumerate(row_of.reshape(-1)):
        if 0 <= flat[p] < G:
            assert pair_of[row] == p and grp[row] == flat[p]
            assert off[flat[p]] <= row < off[flat[p] + 1]
        else:
            assert row == -1
    for g in range(G):
        held = [p for p in pair_of[off[g]:off[g + 1]] if p >= 0]
        assert held == [p for p in range(T * k) if flat[p] == g]      # stable
    assert np.all(pair_of[off[G]:] == -2)
    assert off[G] <= len(pair_of)


def _case(seed, T=7, k=3, G=4, H=5, align=4):
    r = np.random.default_rng(seed)
    ids = r.integers(-1, G, (T, k))
    plan = routing.sort_tokens(ids, G, align)
    rows = len(plan[2])
    return r, plan, r.standard_normal((rows, H)), r.standard_normal((T, k)), r.standard_normal((T, H))


def test_combine_of_dispatch_counts_the_rows():
    """Dispatching and combining without weights gives each token times its pairs."""
    r, (off, row_of, pair_of, grp), Y, W, X = _case(1)
    out = routing.dispatch(X, row_of, pair_of, np.full((len(pair_of), X.shape[1]), np.nan))
    assert np.all(out[pair_of == -1] == 0) and np.all(np.isnan(out[pair_of == -2]))
    got, _ = routing.combine(out, row_of)
    assert np.allclose(got, X * (row_of >= 0).sum(1)[:, None], rtol=1e-12)


def test_combine_backward_is_the_derivative():
    r, (off, row_of, pair_of, grp), Y, W, dO = _case(2)
    f = lambda Y, W: float((routing.combine(Y, row_of, W)[0] * dO).sum())
    dY, dW, _ = routing.combine_backward(dO, Y, row_of, pair_of, W, np.zeros_like(Y))
    h = 1e-6
    for idx in np.ndindex(Y.shape):
        e = np.zeros_like(Y); e[idx] = h
        assert abs((f(Y + e, W) - f(Y - e, W)) / (2 * h) - dY[idx]) < 1e-7
    for idx in np.ndindex(W.shape):
        e = np.zeros_like(W); e[idx] = h
        assert abs((f(Y, W + e) - f(Y, W - e)) / (2 * h) - dW[idx]) < 1e-7


def test_combine_without_weights_is_dispatchs_gradient():
    """<dispatch(X), V> and <X, combine(V)> agree: the two are adjoint."""
    r, (off, row_of, pair_of, grp), V, W, X = _case(3)
    V[pair_of < 0] = 7.0                       # padding rows carry no gradient
    out = routing.dispatch(X, row_of, pair_of, np.zeros_like(V))
    back, _ = routing.combine(V, row_of)
    assert np.isclose((out * V).sum(), (X * back).sum(), rtol=1e-12)


def test_lora_is_the_dense_product_of_the_merged_weight():
    r = np.random.default_rng(4)
    T, K, N, G, rank = 6, 9, 5, 3, 2
    X, W = r.standard_normal((T, K)), r.standard_normal((N, K))
    A, B = r.standard_normal((G, rank, K)), r.standard_normal((G, N, rank))
    s = r.standard_normal(G)
    ids = np.array([0, 2, -1, 1, 2, 3])
    out, err = routing.lora(X, A, B, ids, s, X @ W.T)
    for t, g in enumerate(ids):
        merged = W + (s[g] * B[g] @ A[g] if 0 <= g < G else 0)
        assert np.allclose(out[t], merged @ X[t], rtol=1e-12)
    assert np.all(err[[2, 5]] == 0) and np.all(err[[0, 1, 3, 4]] > 0)
