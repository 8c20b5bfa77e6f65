"""The factor gradients use Z = X V and G = dY U with all the bits of their fp32 sums, and add
over the tokens as fp32 does.

But for the last test every sum below is exact in fp32, and so is every result in bf16: Z (or G) is
1 + 2^-9 + c 2^-20 with a small whole number c, and an output is the difference of two of
them, (c - c') 2^-20.  Held to fewer than 21 bits, 1 + 2^-9 alone remains and the output is 0."""
import numpy as np
import pytest

from test_mx_gpu import blocks, f64, tensor

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def hsl():
    from sparse_rank_linear_03_b200 import hsl as mod
    return mod


SIZES = [(2, 40, 96, 3), (7, 300, 136, 16), (64, 129, 96, 40), (300, 520, 1000, 64), (300, 2048, 96, 129),
         (257, 1001, 777, 200), (500, 19000, 96, 256), (520, 300, 9600, 256)]


def pairs(rows, T):
    """A matrix [T][rows] with a 1 and a -1 in two rows of each column, and where they are."""
    i = np.arange(rows)
    p, q = i % T, (i + 1 + i // T) % T
    q = np.where(q == p, (p + 1) % T, q)
    a = np.zeros((T, rows))
    a[p, i] += 1
    a[q, i] -= 1
    return a, p, q


@pytest.mark.parametrize("T,m,n,r", SIZES)
def test_z_keeps_every_bit(hsl, T, m, n, r):
    c, f = np.arange(T) % 4, 1 + np.arange(r) % 3
    x, v = np.zeros((T, n)), np.zeros((n, r))
    x[:, 0], x[:, 32], x[:, 64] = 1, 1, c
    v[0], v[32], v[64] = 1, 2.0 ** -9, 2.0 ** -20 * f
    X, held = blocks(hsl, x, "int8")
    assert np.array_equal(held, x)
    dY, p, q = pairs(m, T)
    dU, _ = hsl.mx8_factor_grad(X, tensor(dY, "bf16"), tensor(np.zeros((m, r)), "bf16"), tensor(v, "bf16"))
    assert np.array_equal(f64(dU), (c[p] - c[q])[:, None] * f * 2.0 ** -20)


@pytest.mark.parametrize("T,m,n,r", SIZES)
def test_g_keeps_every_bit(hsl, T, m, n, r):
    c, f = np.arange(T) % 4, 1 + np.arange(r) % 3
    dy, u = np.zeros((T, m)), np.zeros((m, r))
    dy[:, 0], dy[:, m // 2], dy[:, m - 1] = 1, 1, c
    u[0], u[m // 2], u[m - 1] = 1, 2.0 ** -9, 2.0 ** -20 * f
    x, p, q = pairs(n, T)
    X, held = blocks(hsl, x, "int8")
    assert np.array_equal(held, x)
    v = np.zeros((n, r))
    j = np.arange(n)
    v[j, j % r] += 1
    v[j, (j + 1) % r] -= 1
    _, dV, dX = hsl.mx8_factor_grad(X, tensor(dy, "bf16"), tensor(u, "bf16"), tensor(v, "bf16"), dx=True)
    assert np.array_equal(f64(dV), (c[p] - c[q])[:, None] * f * 2.0 ** -20)
    assert np.array_equal(f64(dX), c[:, None] * (f[j % r] - f[(j + 1) % r]) * 2.0 ** -20)


@pytest.mark.parametrize("m,n,r", [(160, 96, 64), (19000, 96, 256), (96, 1056, 40)])
def test_long_sums_do_not_drift(hsl, m, n, r):
    """8192 tokens whose second half takes back what the first half adds: dU and dV are 0, and every token's Z (G)
    is bit for bit that of its twin.  A chain of 24 additions that are cut off is off by 24 · 2^-23 of its terms at
    most.  Its 64 chains, of 128 tokens each, are added with an error of 2^-24 of the running sum, which is
    a quarter of all terms on average: 64 / 4 · 2^-24.  (Cut off at each of 512 additions, by half a step of that
    sum, it would be about 46 · 2^-23, all one way.)"""
    T = 8192
    rng = np.random.default_rng(r)
    half = lambda k: 1 + rng.random((T // 2, k))  # noqa: E731
    u, v = (tensor(1 + rng.random((k, r)), "bf16") for k in (m, n))
    a, b = half(n), half(m)
    bound = (24 + 64 / 4 / 2) * 2.0 ** -23 * (1 + 2.0 ** -8)
    X, x = blocks(hsl, np.vstack([a, a]), "int8")
    dY = tensor(np.vstack([b, -b]), "bf16")
    dU, _ = hsl.mx8_factor_grad(X, dY, u, v)
    assert np.all(np.abs(f64(dU)) <= bound * (np.abs(f64(dY)).T @ (x @ f64(v))))
    X, x = blocks(hsl, np.vstack([a, -a]), "int8")
    dY = tensor(np.vstack([b, b]), "bf16")
    _, dV = hsl.mx8_factor_grad(X, dY, u, v)
    assert np.all(np.abs(f64(dV)) <= bound * (np.abs(x).T @ (f64(dY) @ f64(u))))
