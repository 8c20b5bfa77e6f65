"""Calls whose kernels hand over to one another, again and again at sizes that fill the device: sums are in
a fixed order, so a kernel that reads before the one ahead of it has written, or a copy
that overtakes a reader, shows as another bit.  Every operand gets new contents half way, so
that what a call leaves in its scratch is never right for the next."""
import pytest
import torch

pytestmark = pytest.mark.gpu

TDT = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def hsl():
    from sparse_rank_linear_03_b200 import hsl as mod
    return mod


def repeat(hsl, op, dtype, T, m, n, r, off=0):
    g = torch.Generator(device="cuda").manual_seed(T + m + n)

    def rand(a, b):
        buf = torch.empty(a * b + off, dtype=TDT[dtype], device="cuda")
        x = buf[off:].view(a, b)
        x.copy_(torch.randn(a, b, generator=g, device="cuda"))
        return x

    def make():
        if op == "matmul":
            A, B, add = hsl.mx_quantize(rand(T, n)), hsl.mx_quantize(rand(m, n)), rand(T, m)
            return lambda: (hsl.mx4_matmul(A, B, dtype=dtype, add=add),)
        if op == "factor_grad":
            X, dY, U, V, add = hsl.mx_quantize(rand(T, n), "int8"), rand(T, m), rand(m, r), rand(n, r), rand(T, n)
            return lambda: hsl.mx8_factor_grad(X, dY, U, V, dx=True, add=add)
        D, x = hsl.mx_quantize(rand(m, n)), rand(T, n if op == "apply" else m)
        return lambda: (getattr(hsl, "mx4_" + op)(D, x),)

    calls = [make(), make()]
    first = []
    for call in calls:
        first.append(call())
        torch.cuda.synchronize()
    assert any(not torch.equal(a, b) for a, b in zip(*first))
    differ = torch.zeros((), dtype=torch.int64, device="cuda")
    for k in range(40):
        for a, b in zip(calls[k & 1](), first[k & 1]):
            differ += (a != b).sum()
    assert int(differ) == 0
    hsl.mx_check()


@pytest.mark.parametrize("T,m,n,r", [(64, 4096, 4096, 64), (500, 1000, 777, 40), (33, 1001, 2048, 17)])
def test_f32_factor_gradients(hsl, T, m, n, r):
    """Five products, each with its sum of K ranges: Z and G go from kernel to kernel."""
    repeat(hsl, "factor_grad", "f32", T, m, n, r)


def test_bf16_factor_gradients_off_sixteen_bytes(hsl):
    repeat(hsl, "factor_grad", "bf16", 300, 520, 1000, 24, off=1)


@pytest.mark.parametrize("op,T,m,n", [("apply", 8, 4096, 4096), ("apply", 64, 4096, 4096), ("apply_t", 64, 4096, 4096),
                                      ("apply_t", 7, 1001, 777)])
def test_f32_products_in_ranges(hsl, op, T, m, n):
    repeat(hsl, op, "f32", T, m, n, 0)


@pytest.mark.parametrize("op,T,m,n", [
    ("apply", 1, 4096, 11008), ("apply", 2, 28672, 8192), ("apply", 8, 28672, 8192),   # columns, then the product
    ("apply", 8, 333, 28672), ("apply", 33, 1001, 777), ("apply_t", 33, 1001, 777),    # padded rows, K ranges, sum
    ("apply", 300, 11008, 4095), ("apply_t", 300, 4095, 11008)])
def test_bf16_products_handed_on(hsl, op, T, m, n):
    repeat(hsl, op, "bf16", T, m, n, 0)


@pytest.mark.parametrize("T,m,n,r", [(500, 4097, 4096, 100), (300, 1001, 777, 17), (2048, 4100, 1030, 256), (1, 4099, 513, 8)])
def test_bf16_factor_gradients_of_odd_sizes(hsl, T, m, n, r):
    """Up to three paddings, Z and G with their sum, three products with theirs."""
    repeat(hsl, "factor_grad", "bf16", T, m, n, r)


@pytest.mark.parametrize("T,m,n,dtype", [(300, 4097, 2048, "bf16"), (513, 11007, 4100, "bf16"), (300, 4096, 2048, "f32"),
                                         (40, 4096, 8192, "bf16"), (200, 1001, 777, "f32")])
def test_matmul_of_odd_rows(hsl, T, m, n, dtype):
    repeat(hsl, "matmul", dtype, T, m, n, 0)
