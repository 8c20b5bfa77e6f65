"""Microscaled operators on the GPU against the float64 oracle.

Quantisation is exact: codes and scale bytes are compared bit for bit.  Products
are held to a bound derived from their arithmetic, element by element:

  |y − y*| ≤ u |y*| + c(K) Σ|a||b|,   c(K) = (64 + K/16) · 2^-23

u is half a step of the output type (bf16 2^-8, f32 2^-24); a sum kept in fp32
is folded in chains of at most 64 + K/16 additions, each off by at most 2^-23 of
the partial sums' bound Σ|a||b| (2^-24 for rounding, 2^-23 for truncation inside
the tensor cores).  Operands are exact: bf16 and fp32 inputs, and block values
(at most 8 significant bits) in bf16 or fp32.
"""
import numpy as np
import pytest
import torch

from oracle import mx

pytestmark = pytest.mark.gpu

TDT = {"f32": torch.float32, "bf16": torch.bfloat16}
HALF_STEP = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}


@pytest.fixture(scope="module")
def hsl():
    from sparse_rank_linear_03_b200 import hsl as mod
    return mod


def chain(K):
    return (64 + K / 16) * 2.0 ** -23


def tensor(x, dtype):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).to(TDT[dtype]).cuda()


def f64(t):
    return t.detach().double().cpu().numpy()


def weights(m, n, seed):
    return 0.02 * np.random.default_rng(seed).standard_t(3, size=(m, n))


def tokens(t, n, seed):
    rng = np.random.default_rng(seed)
    return rng.standard_normal((t, n)) * np.where(rng.random(n) < 0.02, 8.0, 1.0)


def blocks(hsl, x, elem):
    """x as blocks on the device (from the oracle's codes) and the float64 values held."""
    c, s = mx.quantize(np.asarray(x, np.float32), elem)
    q = hsl.MX(torch.from_numpy(c).cuda(), torch.from_numpy(s).cuda(), x.shape[1], elem)
    return q, mx.values(c, s, x.shape[1], elem)


def close(got, want, mag, K, dtype, extra=0.0):
    """`mag`: Σ|a||b| (+ |add|) of each element; `extra`: error that the operands carry."""
    err = np.abs(f64(got) - want)
    lim = HALF_STEP[dtype] * np.abs(want) + (chain(K) * mag + extra) * (1 + HALF_STEP[dtype])
    worst = np.max(err - lim)
    assert np.all(np.isfinite(f64(got))) and worst <= 0, f"{worst} over the bound"


# ---------------------------------------------------------------- quantisation

@pytest.mark.parametrize("elem", ["e2m1", "int8"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 31), (3, 32), (5, 33), (7, 40), (2, 511), (9, 1001),
                                       (33, 520), (300, 1024), (1, 70001), (4097, 8)])
def test_quantize_bit_exact(hsl, rows, cols, elem, dtype):
    x = tensor(weights(rows, cols, rows + cols), dtype)
    q = hsl.mx_quantize(x, elem)
    c, s = mx.quantize(f64(x), elem)
    assert np.array_equal(q.codes.cpu().numpy().view(np.uint8), c)
    assert np.array_equal(q.scales.cpu().numpy(), s)
    back = hsl.mx_dequantize(q, dtype)
    assert np.array_equal(f64(back), mx.values(c, s, cols, elem))


@pytest.mark.parametrize("elem", ["e2m1", "int8"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_quantize_special_values(hsl, elem, dtype):
    x = np.zeros((9, 64), np.float32)
    x[0, 3] = np.nan
    x[1, 40] = np.inf
    x[2, 5], x[2, 6] = -np.inf, np.nan
    x[3, :] = -0.0
    x[4, 7] = 2.0 ** -133                      # a subnormal of both types
    x[4, 40] = 2.0 ** -127
    x[5, :] = 2.0 ** 127 * 1.9921875           # the largest bf16
    x[6, :] = np.float32(2.0 ** -126) * np.linspace(0, 3, 64, dtype=np.float32)
    x[7, :32] = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0] * 4   # ties
    x[7, 31] = 7.5
    x[8, ::2] = 2.0 ** 100
    x[8, 1::2] = 2.0 ** -100
    t = tensor(x, dtype)
    q = hsl.mx_quantize(t, elem)
    c, s = mx.quantize(f64(t), elem)
    assert np.array_equal(q.codes.cpu().numpy().view(np.uint8), c)
    assert np.array_equal(q.scales.cpu().numpy(), s)
    for out in ("f32", "bf16"):
        want = mx.values(c, s, 64, elem)
        got = f64(hsl.mx_dequantize(q, out))
        assert np.array_equal(np.isnan(got), np.isnan(want))
        assert np.array_equal(got[~np.isnan(want)], want[~np.isnan(want)])


def test_quantize_unaligned_input(hsl):
    base = tensor(weights(1, 8 * 64 + 1, 5), "bf16").view(-1)
    x = base[1:].view(8, 64)
    q = hsl.mx_quantize(x)
    c, s = mx.quantize(f64(x), "e2m1")
    assert np.array_equal(q.codes.cpu().numpy(), c) and np.array_equal(q.scales.cpu().numpy(), s)


@pytest.mark.parametrize("elem", ["e2m1", "int8"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,cols", [(1, 16), (2, 47), (3, 49), (40, 77), (7, 1003), (3, 4096)])
def test_rows_at_every_offset(hsl, rows, cols, elem, dtype):
    """Rows that start anywhere: the matrix at every offset inside 16 bytes and odd row lengths;
    what lies before and behind it is neither read into the blocks nor written."""
    x = tokens(rows, cols, cols).astype(np.float32)
    for off in range(16 // TDT[dtype].itemsize + 1):
        buf = torch.full((off + rows * cols + 24,), 3.0e30, dtype=TDT[dtype], device="cuda")
        X = buf[off:off + rows * cols].view(rows, cols)
        X.copy_(torch.from_numpy(x))
        c, s = mx.quantize(X.float().cpu().numpy(), elem)
        q = hsl.mx_quantize(X, elem)
        assert np.array_equal(q.codes.cpu().numpy().view(np.uint8), c.view(np.uint8))
        assert np.array_equal(q.scales.cpu().numpy(), s)
        X.zero_()
        assert hsl.lib.hsl_mx_dequantize(q._ref, X.data_ptr(), hsl.DTYPE[dtype],
                                         torch.cuda.current_stream().cuda_stream) == 0
        want = torch.from_numpy(mx.values(c, s, cols, elem)).to(TDT[dtype]).cuda()
        assert torch.equal(X, want)
        assert (buf[:off] == buf[-1]).all() and (buf[off + rows * cols:] == buf[-1]).all()
        assert buf[-1].item() > 2.9e30


def test_quantize_no_rows(hsl):
    q = hsl.mx_quantize(torch.empty(0, 40, device="cuda"))
    assert q.rows == 0 and hsl.mx_dequantize(q, "f32").shape == (0, 40)


# ---------------------------------------------------------------- products

SIZES = [(1, 1, 1), (1, 1, 32), (1, 64, 64), (2, 65, 96), (3, 128, 40), (5, 1000, 777), (8, 256, 512),
         (9, 129, 33), (16, 1024, 1024), (17, 300, 2048), (33, 1001, 777), (64, 257, 520),
         (65, 640, 1056), (130, 511, 1023), (200, 1100, 544), (257, 256, 256), (300, 777, 4096)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,m,n", SIZES)
def test_apply(hsl, T, m, n, dtype):
    D, d = blocks(hsl, weights(m, n, m + n), "e2m1")
    x = tensor(tokens(T, n, T), dtype)
    want, mag = mx.apply(d, f64(x)), mx.apply(np.abs(d), np.abs(f64(x)))
    close(hsl.mx4_apply(D, x), want, mag, n, dtype)
    add = tensor(tokens(T, m, 7), dtype)
    close(hsl.mx4_apply(D, x, add=add), want + f64(add), mag + np.abs(f64(add)), n, dtype)
    kept = f64(add)
    close(hsl.mx4_apply(D, x, Y=add, add=add), want + kept, mag + np.abs(kept), n, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,m,n", SIZES)
def test_apply_t(hsl, T, m, n, dtype):
    D, d = blocks(hsl, weights(m, n, m + n), "e2m1")
    dy = tensor(tokens(T, m, T), dtype)
    want, mag = mx.apply_t(d, f64(dy)), mx.apply_t(np.abs(d), np.abs(f64(dy)))
    close(hsl.mx4_apply_t(D, dy), want, mag, m, dtype)
    add = tensor(tokens(T, n, 7), dtype)
    kept = f64(add)
    close(hsl.mx4_apply_t(D, dy, add=add), want + kept, mag + np.abs(kept), m, dtype)
    close(hsl.mx4_apply_t(D, dy, dX=add, add=add), want + kept, mag + np.abs(kept), m, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,m,n", SIZES)
def test_matmul(hsl, T, m, n, dtype):
    A, a = blocks(hsl, tokens(T, n, T), "e2m1")
    B, b = blocks(hsl, weights(m, n, m + n), "e2m1")
    want, mag = mx.apply(b, a), mx.apply(np.abs(b), np.abs(a))
    close(hsl.mx4_matmul(A, B, dtype=dtype), want, mag, n, dtype)
    add = tensor(tokens(T, m, 7), dtype)
    kept = f64(add)
    close(hsl.mx4_matmul(A, B, dtype=dtype, add=add), want + kept, mag + np.abs(kept), n, dtype)
    close(hsl.mx4_matmul(A, B, Y=add, dtype=dtype, add=add), want + kept, mag + np.abs(kept), n, dtype)


GRAD_SIZES = [(1, 1, 1, 1), (1, 40, 64, 8), (2, 64, 65, 3), (31, 128, 96, 16), (33, 300, 200, 17),
              (64, 256, 512, 64), (77, 1001, 777, 100), (128, 512, 256, 128), (200, 640, 1056, 256),
              (500, 257, 300, 40), (1000, 384, 1100, 33)]


def grad_check(hsl, T, m, n, r, dtype, seed):
    X, x = blocks(hsl, tokens(T, n, seed), "int8")
    rng = np.random.default_rng(seed + 1)
    dY, U, V = (tensor(a, dtype) for a in (0.01 * rng.standard_normal((T, m)),
                                           0.05 * rng.standard_normal((m, r)),
                                           0.05 * rng.standard_normal((n, r))))
    add = tensor(0.01 * rng.standard_normal((T, n)), dtype)
    dy, u, v, ad = f64(dY), f64(U), f64(V), f64(add)
    wU, wV, wX = mx.factor_grad(x, dy, u, v, ad)
    # Z and G carry their own sums' error and 2^-16 from being held as two bf16 parts
    # (f32: 2^-24, within the same bound); it passes through the second products
    a = np.abs
    eZ = chain(n) * (a(x) @ a(v)) + 2.0 ** -16 * a(x @ v)
    eG = chain(m) * (a(dy) @ a(u)) + 2.0 ** -16 * a(dy @ u)
    dU, dV, dX = hsl.mx8_factor_grad(X, dY, U, V, dx=True, add=add)
    close(dU, wU, a(dy).T @ a(x @ v), T, dtype, a(dy).T @ eZ * 1.01)
    close(dV, wV, a(x).T @ a(dy @ u), T, dtype, a(x).T @ eG * 1.01)
    close(dX, wX, a(dy @ u) @ a(v).T + a(ad), r, dtype, eG @ a(v).T * 1.01)
    two = hsl.mx8_factor_grad(X, dY, U, V)
    assert len(two) == 2 and torch.equal(two[0], dU) and torch.equal(two[1], dV)
    plain = hsl.mx8_factor_grad(X, dY, U, V, dx=True)[2]
    close(plain, wX - ad, a(dy @ u) @ a(v).T, r, dtype, eG @ a(v).T * 1.01)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,m,n,r", GRAD_SIZES)
def test_factor_grad(hsl, T, m, n, r, dtype):
    grad_check(hsl, T, m, n, r, dtype, T + m)


def test_no_tokens(hsl):
    D, _ = blocks(hsl, weights(5, 40, 1), "e2m1")
    for dt in (torch.float32, torch.bfloat16):
        assert hsl.mx4_apply(D, torch.empty(0, 40, dtype=dt, device="cuda")).shape == (0, 5)
        assert hsl.mx4_apply_t(D, torch.empty(0, 5, dtype=dt, device="cuda")).shape == (0, 40)
        X = hsl.mx_quantize(torch.empty(0, 40, dtype=dt, device="cuda"), "int8")
        U, V = torch.ones(5, 3, dtype=dt, device="cuda"), torch.ones(40, 3, dtype=dt, device="cuda")
        dU, dV, dX = hsl.mx8_factor_grad(X, torch.empty(0, 5, dtype=dt, device="cuda"), U, V, dx=True)
        assert not dU.any() and not dV.any() and dX.shape == (0, 40)
    E = hsl.mx_quantize(torch.empty(0, 40, device="cuda"))
    assert hsl.mx4_matmul(E, D).shape == (0, 5) and hsl.mx4_matmul(D, E).shape == (5, 0)
    # a D of no rows: the gradient is add, or zero
    dY = torch.empty(3, 0, dtype=torch.bfloat16, device="cuda")
    assert not hsl.mx4_apply_t(E, dY).any()
    one = torch.ones(3, 40, dtype=torch.bfloat16, device="cuda")
    assert torch.equal(hsl.mx4_apply_t(E, dY, add=one), one)


@pytest.mark.parametrize("T,m,n", [(1, 65, 300), (2, 64, 512), (4, 33, 1000), (5, 96, 777), (16, 40, 2048)])
def test_apply_tokens_of_any_range(hsl, T, m, n):
    """Tokens whose values span far more binades than one scaled 16-bit operand holds, with the
    small ones alone deciding the outputs of half the rows; all zeros; a single value."""
    rng = np.random.default_rng(T + m)
    d0 = weights(m, n, 3)
    x = rng.standard_normal((T, n)) * np.exp2(rng.integers(-100, 40, size=(T, n)))
    big = rng.random(n) < 0.1
    x[:, big] *= 2.0 ** 70
    d0[::2, big] = 0.0               # these rows see only the small values
    if T > 1:
        x[1] = 0.0
    if T > 2:
        x[2] = 0.0
        x[2, n // 2] = 2.0 ** -130    # a bf16 subnormal
    D, d = blocks(hsl, d0, "e2m1")
    t = tensor(x, "bf16")
    want, mag = mx.apply(d, f64(t)), mx.apply(np.abs(d), np.abs(f64(t)))
    # (fp32 products below 2^-126 may lose bits: 2^-149 for each of the n terms)
    close(hsl.mx4_apply(D, t), want, mag, n, "bf16", n * 2.0 ** -140)
    hsl.mx_check()


@pytest.mark.parametrize("T,m,n", [(1, 40, 28672), (2, 2400, 28672), (3, 17, 30001), (4, 48, 16384), (8, 40, 11008),
                                   (7, 33, 28672)])
def test_apply_long_tokens_of_any_range(hsl, T, m, n):
    """The same where the columns of all tokens, or two per token, do not fit a CTA's shared memory."""
    test_apply_tokens_of_any_range(hsl, T, m, n)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T", [7, 8, 9, 16, 31, 32, 33, 65])
@pytest.mark.parametrize("m,n", [(70, 1500), (1000, 4200)])
def test_apply_where_kernels_change(hsl, T, m, n, dtype):
    D, d = blocks(hsl, weights(m, n, T), "e2m1")
    t, add = tensor(tokens(T, n, T + 1), dtype), tensor(tokens(T, m, T + 2), dtype)
    want, mag = mx.apply(d, f64(t)) + f64(add), mx.apply(np.abs(d), np.abs(f64(t))) + np.abs(f64(add))
    close(hsl.mx4_apply(D, t, add=add), want, mag, n, dtype)
    close(hsl.mx4_apply(D, t, Y=add, add=add), want, mag, n, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,m,n", [(256, 65, 96), (300, 257, 130), (513, 1023, 64), (270, 520, 300)])
def test_matmul_rows_off_sixteen_bytes(hsl, T, m, n, dtype):
    A, a = blocks(hsl, tokens(T, n, 5), "e2m1")
    B, b = blocks(hsl, weights(m, n, 6), "e2m1")
    add = tensor(tokens(T, m, 7), dtype)
    want, mag = a @ b.T + f64(add), np.abs(a) @ np.abs(b).T + np.abs(f64(add))
    close(hsl.mx4_matmul(A, B, dtype=dtype, add=add), want, mag, n, dtype)
    close(hsl.mx4_matmul(A, B, dtype=dtype), want - f64(add), mag, n, dtype)
    close(hsl.mx4_matmul(A, B, Y=add, dtype=dtype, add=add), want, mag, n, dtype)


@pytest.mark.parametrize("T", [1, 3, 17, 70])
def test_apply_infinities_and_nan(hsl, T):
    """An infinity or a NaN in a token reaches its outputs and no other token's; a NaN block
    of D reaches its row."""
    m, n = 130, 352
    D, d = blocks(hsl, weights(m, n, 1), "e2m1")
    x = tokens(T, n, 2)
    x[0, 5], x[T - 1, 7] = np.inf, (np.nan if T > 1 else 1.0)
    t = tensor(x, "bf16")
    with np.errstate(invalid="ignore"):
        want = mx.apply(d, f64(t))
    got = f64(hsl.mx4_apply(D, t))
    assert np.array_equal(np.isnan(got), np.isnan(want))
    assert np.array_equal(np.isinf(got), np.isinf(want))
    both = np.isinf(want)
    assert np.array_equal(got[both], want[both])
    w = weights(m, n, 1)
    w[3, 40] = np.nan
    q = hsl.mx_quantize(tensor(w, "bf16"))
    y = f64(hsl.mx4_apply(q, tensor(tokens(T, n, 2), "bf16")))
    assert np.isnan(y[:, 3]).all() and np.isfinite(np.delete(y, 3, axis=1)).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,m,n,r", [(1, 24, 40, 8), (70, 136, 200, 24)])
def test_factor_grad_infinities(hsl, T, m, n, r, dtype):
    """Infinities in U, V and dY: exactly those gradients are not finite that are not by the
    formulas (where the formula has a NaN or an infinity, either may come out), and those of
    V alone, which Z alone carries to dU, come out as they are."""
    X, x = blocks(hsl, 1 + np.abs(tokens(T, n, 1)), "int8")
    rng = np.random.default_rng(2)
    base = [1 + rng.random(s) for s in ((T, m), (m, r), (n, r))]
    for at in ((0, (T - 1, 5)), (1, (7, 3)), (2, (4, 2))):
        arrays = [a.copy() for a in base]
        arrays[at[0]][at[1]] = -np.inf
        dY, U, V = (tensor(a, dtype) for a in arrays)
        with np.errstate(invalid="ignore"):
            want = mx.factor_grad(x, f64(dY), f64(U), f64(V), None)
        got = [f64(g) for g in hsl.mx8_factor_grad(X, dY, U, V, dx=True)]
        for g, w in zip(got, want):
            assert np.array_equal(np.isfinite(g), np.isfinite(w))
        if at[0] == 2:
            assert np.array_equal(np.isinf(got[0]), np.isinf(want[0])) and (got[0][:, 2] == -np.inf).all()
    hsl.mx_check()


def test_f32_product_with_millions_of_columns(hsl):
    """More 64-column tiles than one grid dimension of 65535 holds."""
    m, n, T = 65536 * 64 + 70, 32, 65
    g = torch.Generator(device="cuda").manual_seed(3)
    W = torch.randn(m, n, generator=g, device="cuda")
    D = hsl.mx_quantize(W)
    x = torch.randn(T, n, generator=g, device="cuda")
    y = hsl.mx4_apply(D, x)
    d = f64(hsl.mx_dequantize(D, "f32")[-5000:])
    want, mag = mx.apply(d, f64(x)), mx.apply(np.abs(d), np.abs(f64(x)))
    close(y[:, -5000:], want, mag, n, "f32")


@pytest.mark.parametrize("T", [1, 6, 40])
def test_apply_scales_at_the_ends(hsl, T):
    """Blocks whose power of two is very small or very large."""
    m, n = 48, 320
    w = weights(m, n, 4)
    w[::3] *= 2.0 ** -121
    w[1::3] *= 2.0 ** 60
    w[5, :32] = 0.0
    D, d = blocks(hsl, w, "e2m1")
    t = tensor(tokens(T, n, 5), "bf16")
    want, mag = mx.apply(d, f64(t)), mx.apply(np.abs(d), np.abs(f64(t)))
    close(hsl.mx4_apply(D, t), want, mag, n, "bf16", n * 2.0 ** -140)


@pytest.mark.parametrize("op,T,m,n,r", [
    ("apply", 1, 4096, 4096, 0), ("apply", 16, 4096, 4096, 0), ("apply", 64, 11008, 4096, 0),
    ("apply", 200, 11008, 4096, 0), ("apply", 2048, 11008, 4096, 0), ("apply_t", 64, 4096, 11008, 0),
    ("apply_t", 200, 4096, 11008, 0), ("apply_t", 2048, 4096, 11008, 0), ("matmul", 64, 4096, 8192, 0),
    ("matmul", 2048, 11008, 8192, 0), ("factor_grad", 500, 4096, 4096, 128),
    ("factor_grad", 2048, 11008, 4096, 256)])
def test_every_call_gives_the_same_bits(hsl, op, T, m, n, r):
    """Calls one behind the other at sizes that fill the device: sums are in a fixed order, so a
    copy that overtakes a reader, or a tile that starts too early, shows as another bit."""
    g = torch.Generator(device="cuda").manual_seed(T + m)
    rand = lambda a, b: torch.randn(a, b, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    if op == "matmul":
        A, B = hsl.mx_quantize(rand(T, n)), hsl.mx_quantize(rand(m, n))
        call = lambda: (hsl.mx4_matmul(A, B),)  # noqa: E731
    elif op == "factor_grad":
        X, dY, U, V, add = hsl.mx_quantize(rand(T, n), "int8"), rand(T, m), rand(m, r), rand(n, r), rand(T, n)
        call = lambda: hsl.mx8_factor_grad(X, dY, U, V, dx=True, add=add)  # noqa: E731
    else:
        D = hsl.mx_quantize(rand(m, n))
        x = rand(T, n if op == "apply" else m)
        call = lambda: (getattr(hsl, "mx4_" + op)(D, x),)  # noqa: E731
    first = call()
    torch.cuda.synchronize()
    differ = torch.zeros((), dtype=torch.int64, device="cuda")
    for _ in range(40):
        for a, b in zip(call(), first):
            differ += (a != b).sum()
    assert int(differ) == 0
    hsl.mx_check()
