"""The products where block scales lie at the ends of their range while the results are ordinary
numbers: one factor near 2^126 or 2^-126, the other one making up for it, for whole
matrices and block by block.  Bounds as in test_mx_gpu, with no allowance for lost small values."""
import numpy as np
import pytest
import torch

from oracle import mx

from test_mx_gpu import blocks, close, f64, tensor, tokens, weights

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


@pytest.mark.parametrize("T", [1, 4, 8, 9])
def test_apply_the_largest_weights(hsl, T):
    """One block of 6 · 2^125 (as large weights are held) against values of 2^-100."""
    D, d = blocks(hsl, np.full((20, 40), 3.0 * 2.0 ** 125), "e2m1")
    x = tensor(np.full((T, 40), 2.0 ** -100), "bf16")
    want = mx.apply(d, f64(x))
    close(hsl.mx4_apply(D, x), want, want, 40, "bf16")
