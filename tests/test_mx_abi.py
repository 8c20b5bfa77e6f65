"""Host-side checks of the microscaled operators: pitches, workspace sizes and every refusal
(no device call is reached on these paths)."""
import ctypes

import pytest
import torch

hsl = pytest.importorskip("sparse_rank_linear_03_b200.hsl")
lib = hsl.lib
OK, INVALID, UNSUPPORTED = 0, 1, 2
P = 4096   # a non-NULL, 16-byte aligned address that no call reaches


def view(codes=P, scales=P, rows=8, cols=64, elem=0):
    return hsl._MXView(codes, scales, rows, cols, elem)


_kept = []   # views stay alive behind their addresses


def ref(v):
    _kept.append(v)
    return ctypes.addressof(v) if v is not None else None


@pytest.mark.parametrize("cols,elem,want", [(1, "e2m1", (16, 16)), (32, "int8", (32, 16)),
                                            (33, "e2m1", (32, 16)), (512, "int8", (512, 16)),
                                            (513, "e2m1", (272, 32)), (8192, "e2m1", (4096, 256))])
def test_pitches(cols, elem, want):
    assert hsl.mx_pitch(cols, elem) == want


def test_pitch_refusals():
    c, s = ctypes.c_int64(), ctypes.c_int64()
    assert lib.hsl_mx_pitch(0, 0, ctypes.byref(c), ctypes.byref(s)) == INVALID
    assert lib.hsl_mx_pitch(1 << 31, 0, ctypes.byref(c), ctypes.byref(s)) == INVALID
    assert lib.hsl_mx_pitch(8, 2, ctypes.byref(c), ctypes.byref(s)) == INVALID
    assert lib.hsl_mx_pitch(8, 0, None, ctypes.byref(s)) == INVALID
    assert lib.hsl_last_message()


def test_workspace_refusals():
    b = ctypes.c_size_t()
    ok = [0, 4, 64, 64, 8, 1]
    assert lib.hsl_mx_workspace(*ok, ctypes.byref(b)) == OK
    for at, bad in ((0, -1), (0, 4), (1, -1), (1, 1 << 31), (2, -1), (3, 0), (4, 257), (4, -1), (5, 2)):
        args = list(ok)
        args[at] = bad
        assert lib.hsl_mx_workspace(*args, ctypes.byref(b)) == INVALID, (at, bad)
    assert lib.hsl_mx_workspace(*ok, None) == INVALID


def test_quantize_refusals():
    q = lambda X=P, dt=1, rows=4, cols=64, el=0, c=P, s=P: lib.hsl_mx_quantize(  # noqa: E731
        X, dt, rows, cols, el, c, s, None)
    assert q(X=None) == INVALID
    assert q(dt=2) == INVALID
    assert q(rows=-1) == INVALID
    assert q(cols=0) == INVALID
    assert q(el=2) == INVALID
    assert q(c=None) == INVALID
    assert q(s=None) == INVALID
    assert q(c=P + 8) == INVALID
    assert q(s=P + 1) == INVALID
    assert q(rows=0, X=None, c=None, s=None) == OK      # nothing to do


def test_dequantize_refusals():
    f = lambda v, X=P, dt=1: lib.hsl_mx_dequantize(ref(v), X, dt, None)  # noqa: E731
    assert f(None) == INVALID
    assert f(view(), X=None) == INVALID
    assert f(view(), dt=7) == INVALID
    assert f(view(elem=3)) == INVALID
    assert f(view(codes=None)) == INVALID
    assert f(view(rows=0, codes=None, scales=None), X=None) == OK


@pytest.mark.parametrize("name", ["hsl_mx4_apply", "hsl_mx4_apply_t"])
def test_apply_refusals(name):
    fn = getattr(lib, name)
    f = lambda v, X=P, Y=P, b=2, dt=1, ws=P, wb=1 << 40: fn(  # noqa: E731
        ref(v), X, None, Y, b, dt, ws, wb, None)
    assert f(None) == INVALID
    assert f(view(elem=1)) == UNSUPPORTED                # int8 weights
    assert f(view(cols=0)) == INVALID
    assert f(view(scales=P + 2)) == INVALID
    assert f(view(), X=None) == INVALID
    assert f(view(), Y=None) == INVALID
    assert f(view(), b=-1) == INVALID
    assert f(view(), b=1 << 31) == INVALID
    assert f(view(), dt=5) == INVALID
    assert f(view(), b=0, X=None, Y=None) == OK
    assert lib.hsl_last_message() == b""


def test_matmul_refusals():
    f = lambda a, b, Y=P, dt=1: lib.hsl_mx4_matmul(  # noqa: E731
        ref(a), ref(b), None, Y, dt, P, 1 << 40, None)
    assert f(None, view()) == INVALID
    assert f(view(), None) == INVALID
    assert f(view(elem=1), view()) == UNSUPPORTED
    assert f(view(), view(elem=1)) == UNSUPPORTED
    assert f(view(), view(cols=96)) == INVALID
    assert f(view(), view(), Y=None) == INVALID
    assert f(view(), view(), dt=3) == INVALID
    assert f(view(rows=0), view(), Y=None) == OK
    assert f(view(), view(rows=0), Y=None) == OK


def test_factor_grad_refusals():
    def f(x=view(elem=1), dY=P, m=8, U=P, V=P, r=4, add=None, dU=P, dV=P, dX=None, dt=1, ws=P,
          wb=1 << 40):
        return lib.hsl_mx8_factor_grad(ref(x), dY, m, U, V, r, add, dU, dV, dX, dt, ws, wb, None)
    assert f(x=None) == INVALID
    assert f(x=view(elem=0)) == UNSUPPORTED
    assert f(dY=None) == INVALID
    assert f(m=0) == INVALID
    assert f(U=None) == INVALID
    assert f(V=None) == INVALID
    assert f(r=0) == UNSUPPORTED
    assert f(r=257) == UNSUPPORTED
    assert f(dU=None) == INVALID
    assert f(dV=None) == INVALID
    assert f(add=P) == INVALID                           # add without dX
    assert f(dt=9) == INVALID
    assert f(ws=None) == INVALID
    assert f(wb=16) == INVALID
    assert f(ws=P + 4) == INVALID
    assert b"workspace" in lib.hsl_last_message()


def test_overlaps_are_refused():
    """Spans that touch are fine, a shared byte is not; `add` may be the output itself."""
    K = 1 << 20                                          # far apart
    d = lambda **k: view(codes=4 * K, scales=8 * K, **k)  # noqa: E731   8 rows x 64: 256 + 128 bytes
    b = ctypes.c_size_t()

    def apart(status):
        # (spans that are apart end in a launch that finds no device, or no tensor map: not here)
        assert status == INVALID and b"overlap" in lib.hsl_last_message()

    # 2 x 64 bf16 in, 2 x 8 out
    assert lib.hsl_mx_workspace(0, 2, 8, 64, 0, 1, ctypes.byref(b)) == OK
    for fn, xb, yb in ((lib.hsl_mx4_apply, 256, 32), (lib.hsl_mx4_apply_t, 32, 256)):
        f = lambda X=16 * K, add=None, Y=32 * K, ws=64 * K: fn(  # noqa: E731
            ref(d()), X, add, Y, 2, 1, ws, 1 << 40, None)
        apart(f(Y=16 * K))
        apart(f(Y=16 * K + xb - 2))
        apart(f(Y=16 * K - yb + 2))
        apart(f(add=32 * K + 2))                         # neither the output nor apart from it
        apart(f(Y=4 * K + 16))
        apart(f(Y=8 * K + 126))
    f = lambda Y=32 * K, add=None: lib.hsl_mx4_matmul(  # noqa: E731
        ref(d()), ref(view(codes=5 * K, scales=9 * K)), add, Y, 1, 64 * K, 1 << 40, None)
    apart(f(Y=5 * K))
    apart(f(Y=9 * K - 126))
    apart(f(add=32 * K + 16))
    apart(lib.hsl_mx_quantize(4 * K - 16, 1, 8, 64, 0, 4 * K, 8 * K, None))
    apart(lib.hsl_mx_quantize(16 * K, 1, 8, 64, 0, 4 * K, 4 * K + 240, None))
    apart(lib.hsl_mx_dequantize(ref(d()), 8 * K, 1, None))

    def g(dY=16 * K, U=20 * K, V=24 * K, add=None, dU=32 * K, dV=36 * K, dX=None, ws=64 * K):
        return lib.hsl_mx8_factor_grad(ref(d(elem=1)), dY, 8, U, V, 4, add, dU, dV, dX, 1, ws, 1 << 40, None)
    apart(g(dU=20 * K))                                  # the factor itself
    apart(g(dV=24 * K + 16))
    apart(g(dU=36 * K))                                  # both gradients in one place
    apart(g(dX=16 * K))
    apart(g(dX=40 * K, add=40 * K + 4))
    apart(g(ws=20 * K))
    apart(g(ws=32 * K - 256))


def test_binding_refuses_before_the_library():
    cpu = torch.zeros(4, 16, dtype=torch.uint8)
    with pytest.raises(ValueError):
        hsl.MX(cpu, cpu, 32)                             # not on a CUDA device
    with pytest.raises(ValueError):
        hsl.MX(cpu, cpu, 32, "e4m3")
    with pytest.raises(ValueError):
        hsl.MX(cpu, cpu, 64)                             # too few bytes per row
    with pytest.raises(ValueError):
        hsl.MX(cpu, cpu[:3], 32)
    with pytest.raises(ValueError):
        hsl.MX(cpu.float(), cpu, 32)
    with pytest.raises(ValueError):
        hsl.mx_quantize(torch.zeros(4, 32))              # CPU tensor
    with pytest.raises(hsl.HslError) as e:
        hsl.mx_pitch(0, "e2m1")
    assert e.value.name == "HSL_ERR_INVALID_ARG"
