"""The float64 oracle of the microscaled blocks, held to facts that do not depend on it:
hand-worked blocks, the nearest-value property by brute force, and gradients
against central differences."""
import numpy as np
import pytest

from oracle import mx


def _one(block, elem):
    x = np.zeros((1, 32))
    x[0, :len(block)] = block
    c, s = mx.quantize(x, elem)
    return mx.values(c, s, 32, elem)[0, :len(block)], int(s[0, 0])


def test_hand_worked_e2m1_block():
    # largest 6.5 → exponent 2 − 2 = 0: scale 1; 6.5 saturates at 6, ties to the even code
    got, e = _one([6.5, -0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -5.1], "e2m1")
    assert e == 127
    assert got.tolist() == [6.0, -0.0, 1.0, 1.0, 2.0, 2.0, 4.0, 4.0, -6.0]
    # 0.04 = 1.28 · 2^−5 → scale 2^−7: 0.04 · 128 = 5.12 → 6
    got, e = _one([0.04], "e2m1")
    assert e == 120 and got[0] == 6 / 128


def test_hand_worked_int8_block():
    # largest 1.999 → scale 1, units of 1/64: 127.9 saturates at 127; 0.5/64 ties to 0
    got, e = _one([1.999, -1.0, 0.5 / 64, 1.5 / 64], "int8")
    assert e == 127
    assert got.tolist() == [127 / 64, -1.0, 0.0, 2 / 64]


def test_zero_nan_and_extreme_blocks():
    for elem in ("e2m1", "int8"):
        assert _one([0.0, -0.0], elem) == (pytest.approx([0, 0]), 0)
        got, e = _one([1.0, np.nan], elem)
        assert e == 255 and np.isnan(got).all()
        assert _one([np.inf], elem)[1] == 255
        assert _one([2.0 ** -149], elem)[1] == 0
    assert _one([2.0 ** 127], "e2m1")[1] == 252
    assert _one([2.0 ** 127], "int8")[1] == 254


@pytest.mark.parametrize("elem", ["e2m1", "int8"])
def test_no_held_value_is_nearer(elem):
    rng = np.random.default_rng(1)
    x = rng.standard_t(3, size=(40, 70)).astype(np.float32).astype(np.float64)
    c, s = mx.quantize(x, elem)
    v = mx.values(c, s, 70, elem)
    grid = np.concatenate([-mx.E2M1, mx.E2M1]) if elem == "e2m1" else np.arange(-127, 128) / 64.0
    for j in range(70):
        held = grid[None, :] * np.ldexp(1.0, s[:, j // 32].astype(int) - 127)[:, None]
        assert np.array_equal(np.abs(v[:, j] - x[:, j]), np.abs(held - x[:, j:j + 1]).min(axis=1))


def test_quantizing_held_values_changes_nothing():
    rng = np.random.default_rng(2)
    for elem in ("e2m1", "int8"):
        c, s = mx.quantize(rng.standard_normal((9, 100)), elem)
        v = mx.values(c, s, 100, elem)
        c2, s2 = mx.quantize(v, elem)
        assert np.array_equal(mx.values(c2, s2, 100, elem), v)


def test_gradients_against_differences():
    rng = np.random.default_rng(3)
    T, m, n, r = 5, 7, 6, 2
    X, dY = rng.standard_normal((T, n)), rng.standard_normal((T, m))
    U, V, D = rng.standard_normal((m, r)), rng.standard_normal((n, r)), rng.standard_normal((m, n))
    loss = lambda U, V, X: float((dY * (X @ V @ U.T + mx.apply(D, X))).sum())  # noqa: E731
    dU, dV, dXl = mx.factor_grad(X, dY, U, V)
    dX = dXl + mx.apply_t(D, dY)
    h = 1e-6
    for arr, grad, at in ((U, dU, 0), (V, dV, 1), (X, dX, 2)):
        for idx in np.ndindex(arr.shape):
            args = [U, V, X]
            up, down = arr.copy(), arr.copy()
            up[idx] += h
            down[idx] -= h
            args[at] = up
            a = loss(*args)
            args[at] = down
            # the loss is linear in each argument: only rounding (about 1e-16 · |loss| / h) differs
            assert (a - loss(*args)) / (2 * h) == pytest.approx(grad[idx], abs=1e-7, rel=1e-7)
