"""The products where block scales lie at the ends of their range while the results are ordinary
numbers: one factor near 2^126 or 2^-126, the other one making up for it, for whole
matrices and block by block.  Bounds as in test_mx_gpu, with no allowance for lost small values."""
import numpy as np
import pytest
import torch

from oracle import mx

from test_mx_gpu import blocks, chain, close, f64, tensor, tokens, weights

pytestmark = pytest.mark.gpu

KINDS = ["high", "low", "mixed", "one"]


@pytest.fixture(scope="module")
def hsl():
    from sparse_rank_linear_03_b200 import hsl as mod
    return mod


def powers(kind, nb, seed):
    """Exponents by which the blocks of one factor are scaled up and those of the other down."""
    if kind == "one":                     # most blocks ordinary, a few of them not
        p = np.zeros(nb, np.int64)
        p[nb // 2] = 126
        p[nb // 3] = -126
        return p
    if kind == "mixed":
        return np.random.default_rng(seed).integers(-110, 111, size=nb)
    return np.full(nb, 126 if kind == "high" else -126)


def scaled(a, p):
    """Columns of `a` (|a| < 2 after this) times 2^p of their block."""
    a = a / np.abs(a).max() * 1.9
    return np.ldexp(a, np.repeat(p, 32)[:a.shape[1]])


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("T,m,n", [(1, 48, 320), (1, 40, 4096), (1, 17, 30001), (2, 1000, 777), (4, 130, 2048),
                                   (5, 33, 8200), (8, 256, 4096), (8, 40, 11008), (9, 130, 520), (40, 300, 1100)])
def test_apply(hsl, T, m, n, kind):
    p = powers(kind, -(-n // 32), m)
    w = scaled(weights(m, n, m), p)
    w[::5, :32] = 0.0                     # blocks of nothing
    D, d = blocks(hsl, w, "e2m1")
    x, add = tensor(scaled(tokens(T, n, T), -p), "bf16"), tensor(tokens(T, m, 3), "bf16")
    want, mag = mx.apply(d, f64(x)), mx.apply(np.abs(d), np.abs(f64(x)))
    close(hsl.mx4_apply(D, x), want, mag, n, "bf16")
    want, mag = want + f64(add), mag + np.abs(f64(add))
    close(hsl.mx4_apply(D, x, add=add), want, mag, n, "bf16")
    close(hsl.mx4_apply(D, x, Y=add, add=add), want, mag, n, "bf16")
    hsl.mx_check()


@pytest.mark.parametrize("T,n", [(1, 4096), (3, 8192), (8, 28672), (9, 4096)])
def test_apply_long_sums_of_one_sign(hsl, T, n):
    """Thousands of terms of one sign at scales of 2^119, tokens far below 1."""
    w = 2.0 ** 120 * (1 + np.random.default_rng(n).random((40, n)))
    D, d = blocks(hsl, w, "e2m1")
    x = 2.0 ** -90 * (1 + np.random.default_rng(T).random((T, n)))
    if T > 1:
        x[1, n // 2] = np.nan             # this token's outputs are all NaN, and no other's
    x, keep = tensor(x, "bf16"), np.arange(T) != 1
    want = mx.apply(d, f64(x)[keep])
    y = hsl.mx4_apply(D, x)
    close(y[torch.from_numpy(keep)], want, want, n, "bf16")
    assert torch.isnan(y[torch.from_numpy(~keep)]).all()
    add = tensor(2.0 ** 40 * tokens(T, 40, 1), "bf16")
    kept = f64(add)[keep]
    hsl.mx4_apply(D, x, Y=add, add=add)
    close(add[torch.from_numpy(keep)], want + kept, want + np.abs(kept), n, "bf16")


@pytest.mark.parametrize("top,low", [(127, 100), (100, 75), (60, 40)])
@pytest.mark.parametrize("T,m,n", [(1, 40, 4096), (2, 100, 352), (8, 33, 8192), (9, 130, 520)])
def test_apply_small_scales_beside_a_large_value(hsl, T, m, n, top, low):
    """Weights of 2^-126 and the smallest scale of all; a token's largest value meets weights of zero only,
    and its others decide the result."""
    w = np.ldexp(scaled(weights(m, n, m), np.zeros(-(-n // 32), np.int64)), -127)
    w[:, 64:] *= 0.25                     # scale bytes 0
    w[:, :32] = 0.0
    D, d = blocks(hsl, w, "e2m1")
    x = np.ldexp(scaled(tokens(T, n, T), np.zeros(-(-n // 32), np.int64)), low)
    x[:, 3] = 2.0 ** top
    x = tensor(x, "bf16")
    close(hsl.mx4_apply(D, x), mx.apply(d, f64(x)), mx.apply(np.abs(d), np.abs(f64(x))), n, "bf16")


@pytest.mark.parametrize("T,n", [(1, 320), (2, 4096), (8, 777), (9, 320)])
def test_apply_large_scales_beside_a_large_value(hsl, T, n):
    """Weights of 2^120, tokens of 2^-60 but for one value of 2^100, whose weights, in the same blocks, are 0."""
    w = scaled(weights(40, n, n), np.full(-(-n // 32), 120))
    w[:, 3::32] = 0.0
    D, d = blocks(hsl, w, "e2m1")
    x = np.ldexp(1 + np.random.default_rng(n).random((T, n)), -60)
    x[:, 3] = 2.0 ** 100
    x = tensor(x, "bf16")
    close(hsl.mx4_apply(D, x), mx.apply(d, f64(x)), mx.apply(np.abs(d), np.abs(f64(x))), n, "bf16")


@pytest.mark.parametrize("T", [1, 4, 8, 9])
def test_apply_the_largest_weights(hsl, T):
    """One block of 6 · 2^125 (as large weights are held) against values of 2^-100."""
    D, d = blocks(hsl, np.full((20, 40), 3.0 * 2.0 ** 125), "e2m1")
    x = tensor(np.full((T, 40), 2.0 ** -100), "bf16")
    want = mx.apply(d, f64(x))
    close(hsl.mx4_apply(D, x), want, want, 40, "bf16")


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("T", [1, 3, 40])
def test_apply_f32(hsl, T, kind):
    m, n = 130, 1100
    p = powers(kind, -(-n // 32), m)
    D, d = blocks(hsl, scaled(weights(m, n, m), p), "e2m1")
    x = tensor(scaled(tokens(T, n, T), -p), "f32")
    close(hsl.mx4_apply(D, x), mx.apply(d, f64(x)), mx.apply(np.abs(d), np.abs(f64(x))), n, "f32")


@pytest.mark.parametrize("kind", ["high", "low"])
@pytest.mark.parametrize("T,m,n,dtype", [(1, 48, 320, "bf16"), (33, 1001, 777, "bf16"), (300, 256, 512, "bf16"),
                                         (3, 100, 96, "f32")])
def test_apply_t(hsl, T, m, n, kind, dtype):
    p = powers(kind, -(-n // 32), 0)
    D, d = blocks(hsl, scaled(weights(m, n, m), p), "e2m1")
    dy = tensor(scaled(tokens(T, m, T), np.full(-(-m // 32), -p[0])), dtype)
    close(hsl.mx4_apply_t(D, dy), mx.apply_t(d, f64(dy)), mx.apply_t(np.abs(d), np.abs(f64(dy))), m, dtype)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("T,m,n,dtype", [(1, 48, 320, "bf16"), (33, 1001, 777, "f32"), (300, 256, 2048, "bf16"),
                                         (300, 257, 520, "f32")])
def test_matmul(hsl, T, m, n, kind, dtype):
    p = powers(kind, -(-n // 32), T)
    B, b = blocks(hsl, scaled(weights(m, n, m), p), "e2m1")
    A, a = blocks(hsl, scaled(tokens(T, n, T), -p), "e2m1")
    close(hsl.mx4_matmul(A, B, dtype=dtype), mx.apply(b, a), mx.apply(np.abs(b), np.abs(a)), n, dtype)


@pytest.mark.parametrize("kind", ["high", "low", "mixed"])
@pytest.mark.parametrize("T,m,n,r", [(1, 40, 64, 8), (77, 300, 777, 100), (300, 256, 512, 64)])
def test_factor_grad(hsl, T, m, n, r, kind):
    """X at one end, V and dY U at the other, so that Z, G, dU and dV are all far from it (`mixed`: dV goes with
    the blocks of X).  dX = G V^T leaves the range here."""
    p = powers(kind, -(-n // 32), T)
    X, x = blocks(hsl, scaled(tokens(T, n, T), p), "int8")
    rng = np.random.default_rng(r)
    back = -np.repeat(p, 32)[:n, None] * 100 // 126
    V = tensor(np.ldexp(rng.standard_normal((n, r)), back), "bf16")
    s = 0 if kind == "mixed" else int(back[0, 0]) // 2
    dY, U = (tensor(np.ldexp(rng.standard_normal(sh), s), "bf16") for sh in ((T, m), (m, r)))
    y, u, v = f64(dY), f64(U), f64(V)
    a = np.abs
    dU, dV = hsl.mx8_factor_grad(X, dY, U, V)
    wU, wV, _ = mx.factor_grad(x, y, u, v)
    close(dU, wU, a(y).T @ a(x @ v), T, "bf16", a(y).T @ (chain(n) * (a(x) @ a(v))) * 1.01)
    close(dV, wV, a(x).T @ a(y @ u), T, "bf16", a(x).T @ (chain(m) * (a(y) @ a(u))) * 1.01)
