"""Matrices that do not start on a whole element are refused on the host: their loads would fault."""
import ctypes

import pytest

hsl = pytest.importorskip("sparse_rank_linear_03_b200.hsl")
lib = hsl.lib
INVALID = 1
K = 1 << 20
F32, BF16 = 0, 1


def ref(elem, codes=4 * K, scales=8 * K):
    v = hsl._MXView(codes, scales, 8, 64, elem)
    _kept.append(v)
    return ctypes.addressof(v)


_kept = []


def refused(status):
    assert status == INVALID and b"start on a whole element" in lib.hsl_last_message()


@pytest.mark.parametrize("dtype,off", [(BF16, 1), (F32, 1), (F32, 2)])
def test_pointers_inside_an_element(dtype, off):
    assert (hsl.DTYPE["f32"], hsl.DTYPE["bf16"]) == (F32, BF16)
    refused(lib.hsl_mx_quantize(16 * K + off, dtype, 8, 64, 0, 4 * K, 8 * K, None))
    refused(lib.hsl_mx_dequantize(ref(0), 16 * K + off, dtype, None))
    for fn in (lib.hsl_mx4_apply, lib.hsl_mx4_apply_t):
        for bad in range(3):
            p = [16 * K, 24 * K, 32 * K]
            p[bad] += off
            refused(fn(ref(0), *p, 2, dtype, 64 * K, 1 << 40, None))
    for add, Y in ((24 * K + off, 32 * K), (None, 32 * K + off)):
        refused(lib.hsl_mx4_matmul(ref(0), ref(0, 5 * K, 9 * K), add, Y, dtype, 64 * K, 1 << 40, None))
    for bad in range(7):
        p = [16 * K, 20 * K, 24 * K, 28 * K, 32 * K, 36 * K, 40 * K]   # dY U V add dU dV dX
        p[bad] += off
        dY, U, V, add, dU, dV, dX = p
        refused(lib.hsl_mx8_factor_grad(ref(1), dY, 8, U, V, 4, add, dU, dV, dX, dtype, 64 * K, 1 << 40, None))
