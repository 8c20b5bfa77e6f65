"""The microscaled operators as a program uses them: together with a layer's sparse and low-rank
part, on other streams, captured into graphs, at odd addresses, over matrices past 4 GB, and
the calls that the binding refuses.  Bounds as in test_mx_gpu."""
import numpy as np
import pytest
import torch

import oracle
from oracle import mx
from sparse_rank_linear_03_b200 import synth

from test_mx_gpu import blocks, chain, close, f64, tensor, tokens, weights

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def hsl():
    from sparse_rank_linear_03_b200 import hsl as mod
    return mod


@pytest.mark.parametrize("T", [1, 12, 150])
def test_a_layer_served_and_tuned(hsl, T):
    """W ≈ S + D + U Vᵀ: S the largest weights, D the rest in 4 bits, U Vᵀ a factor pair on top.
    Forward with the layer's own apply plus D; gradients of U, V and the input from the input
    kept in 8 bits.  Each step is held to its own bound, from what it was given."""
    m, n, r = 384, 512, 16
    a = np.abs
    W = tensor(weights(m, n, 11), "bf16")
    L = hsl.Layer(m, n, r, "csr", "bf16")
    R = torch.empty_like(W)
    L.split(W, 0.02, R)
    D = hsl.mx_quantize(R)
    d = mx.values(D.codes.cpu().numpy(), D.scales.cpu().numpy(), n, "e2m1")
    c, s = mx.quantize(f64(R), "e2m1")
    assert np.array_equal(d, mx.values(c, s, n, "e2m1"))
    Uf, Vf = synth.stand_in_factors(m, n, r, 3)
    U, V = tensor(Uf, "bf16"), tensor(Vf, "bf16")
    L.pack(U, V)
    X = tensor(tokens(T, n, T), "bf16")
    Y0 = L.apply(X)
    Y = hsl.mx4_apply(D, X, add=Y0)
    L.check()
    close(Y, mx.apply(d, f64(X)) + f64(Y0), mx.apply(a(d), a(f64(X))) + a(f64(Y0)), n, "bf16")
    S = f64(W) - f64(R)
    whole = f64(X) @ (S + d + f64(U) @ f64(V).T).T
    assert oracle.rel_err(f64(Y), whole) <= 1e-2          # the layer's own tolerance
    # what 4 bits cost the weights: an element is off by at most half a step, half of the
    # largest held value's distance to the next (2 of 6, or saturation from 8 to 6)
    assert np.max(a(d - f64(R)) / np.maximum(a(f64(R)).reshape(m, -1, 32).max(2).repeat(32, 1), 1e-30)) <= 0.25

    Xq = hsl.mx_quantize(X, "int8")
    xq = mx.values(Xq.codes.cpu().numpy(), Xq.scales.cpu().numpy(), n, "int8")
    # an int8 block is off by at most 2^-6 of its largest value (half a step, or 128 held as 127)
    assert np.max(a(xq - f64(X)) - a(f64(X)).reshape(T, -1, 32).max(2).repeat(32, 1) * 2.0 ** -6) <= 0
    dY = tensor(0.01 * np.random.default_rng(5).standard_normal((T, m)), "bf16")
    dXd = hsl.mx4_apply_t(D, dY)
    dU, dV, dX = hsl.mx8_factor_grad(Xq, dY, U, V, dx=True, add=dXd)
    y, u, v = f64(dY), f64(U), f64(V)
    wU, wV, wX = mx.factor_grad(xq, y, u, v, f64(dXd))
    eZ = chain(n) * (a(xq) @ a(v)) + 2.0 ** -16 * a(xq @ v)
    eG = chain(m) * (a(y) @ a(u)) + 2.0 ** -16 * a(y @ u)
    close(dU, wU, a(y).T @ a(xq @ v), T, "bf16", a(y).T @ eZ * 1.01)
    close(dV, wV, a(xq).T @ a(y @ u), T, "bf16", a(xq).T @ eG * 1.01)
    close(dX, wX, a(y @ u) @ a(v).T + a(f64(dXd)), r, "bf16", eG @ a(v).T * 1.01)
    # the 4-bit product with the tokens in 4 bits as well
    Xf = hsl.mx_quantize(X)
    xf = mx.values(Xf.codes.cpu().numpy(), Xf.scales.cpu().numpy(), n, "e2m1")
    close(hsl.mx4_matmul(Xf, D), mx.apply(d, xf), mx.apply(a(d), a(xf)), n, "bf16")
    hsl.mx_check()


def _set(hsl, T, m, n, r, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda a, b: torch.randn(a, b, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    return dict(W=rand(m, n), X=rand(T, n), dY=rand(T, m), U=rand(m, r), V=rand(n, r))


def _step(hsl, t, stream=None):
    D = hsl.mx_quantize(t["W"], stream=stream)
    Y = hsl.mx4_apply(D, t["X"], stream=stream)
    dXd = hsl.mx4_apply_t(D, t["dY"], stream=stream)
    Xq = hsl.mx_quantize(t["X"], "int8", stream=stream)
    dU, dV, dX = hsl.mx8_factor_grad(Xq, t["dY"], t["U"], t["V"], dx=True, add=dXd, stream=stream)
    Z = hsl.mx4_matmul(hsl.mx_quantize(t["X"], stream=stream), D, stream=stream)
    return [Y, dX, dU, dV, Z, hsl.mx_dequantize(Xq, "f32", stream=stream)]


@pytest.mark.parametrize("T", [1, 9, 100])
def test_other_streams(hsl, T):
    """The same calls on torch's current stream, on one passed as an object, and on one passed as
    a pointer; two streams at once."""
    t = _set(hsl, T, 520, 1000, 24, T)
    want = _step(hsl, t)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    both = [_step(hsl, t, s1), _step(hsl, t, s2.cuda_stream)]
    with torch.cuda.stream(s2):
        both.append(_step(hsl, t))
    torch.cuda.synchronize()
    for got in both:
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("T", [1, 9, 100])
def test_two_captured_graphs(hsl, T):
    """Two graphs captured one after the other (each with its own scratch), replayed at once on two
    streams with new contents of their inputs, with eager calls in between."""
    ts = [_set(hsl, T, 520, 1000, 24, T + k) for k in (0, 1)]
    for t in ts:
        _step(hsl, t)                                    # (first calls outside of the capture)
    graphs, outs = [], []
    for t in ts:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(_step(hsl, t))
        graphs.append(graph)
    for k, t in enumerate(ts):
        new = _set(hsl, T, 520, 1000, 24, 50 + T + k)
        for name in t:
            t[name].copy_(new[name])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        for graph, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                graph.replay()
        eager = [_step(hsl, t) for t in ts]
    torch.cuda.synchronize()
    for got, want in zip(outs, eager):
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def _off(t):
    """The same values two (bf16) or four (f32) bytes past a 16-byte boundary."""
    base = torch.empty(t.numel() + 1, dtype=t.dtype, device=t.device)
    v = base[1:].view(t.shape)
    v.copy_(t)
    assert v.data_ptr() % 16 != 0 and v.is_contiguous()
    return v


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,m,n", [(3, 130, 256), (40, 136, 264)])
def test_pointers_off_sixteen_bytes(hsl, T, m, n, dtype):
    D, d = blocks(hsl, weights(m, n, 1), "e2m1")
    x, dy = _off(tensor(tokens(T, n, 2), dtype)), _off(tensor(tokens(T, m, 3), dtype))
    ay, ax = _off(tensor(tokens(T, m, 4), dtype)), _off(tensor(tokens(T, n, 5), dtype))
    a = np.abs
    y = _off(torch.empty_like(ay))
    hsl.mx4_apply(D, x, Y=y, add=ay)
    close(y, mx.apply(d, f64(x)) + f64(ay), mx.apply(a(d), a(f64(x))) + a(f64(ay)), n, dtype)
    al = tensor(tokens(T, m, 4), dtype)                  # aligned input, everything else off
    close(hsl.mx4_apply(D, tensor(tokens(T, n, 2), dtype), Y=y, add=ay), mx.apply(d, f64(x)) + f64(ay),
          mx.apply(a(d), a(f64(x))) + a(f64(ay)), n, dtype)
    close(hsl.mx4_apply(D, tensor(tokens(T, n, 2), dtype), add=ay), mx.apply(d, f64(x)) + f64(al),
          mx.apply(a(d), a(f64(x))) + a(f64(al)), n, dtype)
    g = _off(torch.empty_like(ax))
    hsl.mx4_apply_t(D, dy, dX=g, add=ax)
    close(g, mx.apply_t(d, f64(dy)) + f64(ax), mx.apply_t(a(d), a(f64(dy))) + a(f64(ax)), m, dtype)
    A, av = blocks(hsl, tokens(T, n, 6), "e2m1")
    hsl.mx4_matmul(A, D, Y=y, dtype=dtype, add=ay)
    close(y, mx.apply(d, av) + f64(ay), mx.apply(a(d), a(av)) + a(f64(ay)), n, dtype)
    X, xv = blocks(hsl, tokens(T, n, 7), "int8")
    U, V = _off(tensor(weights(m, 12, 8), dtype)), _off(tensor(weights(n, 12, 9), dtype))
    dU, dV, dX = hsl.mx8_factor_grad(X, dy, U, V, dx=True, add=ax)
    gy, u, v = f64(dy), f64(U), f64(V)
    wU, wV, wX = mx.factor_grad(xv, gy, u, v, f64(ax))
    eZ = chain(n) * (a(xv) @ a(v)) + 2.0 ** -16 * a(xv @ v)
    eG = chain(m) * (a(gy) @ a(u)) + 2.0 ** -16 * a(gy @ u)
    close(dU, wU, a(gy).T @ a(xv @ v), T, dtype, a(gy).T @ eZ * 1.01)
    close(dV, wV, a(xv).T @ a(gy @ u), T, dtype, a(xv).T @ eG * 1.01)
    close(dX, wX, a(gy @ u) @ a(v).T + a(f64(ax)), 12, dtype, eG @ a(v).T * 1.01)


@pytest.mark.parametrize("T", [2, 70])
def test_a_nan_block_stays_in_its_row(hsl, T):
    m, n, r = 150, 320, 8
    w, x = weights(m, n, 1), tokens(T, n, 2)
    w[7, 100], x[1, 300] = np.nan, np.inf
    D, A = hsl.mx_quantize(tensor(w, "bf16")), hsl.mx_quantize(tensor(x, "bf16"))
    y = f64(hsl.mx4_matmul(A, D))
    assert np.isnan(y[:, 7]).all() and np.isnan(y[1]).all()
    assert np.isfinite(np.delete(np.delete(y, 7, axis=1), 1, axis=0)).all()
    g = f64(hsl.mx4_apply_t(D, tensor(tokens(T, m, 3), "bf16")))
    assert np.isnan(g[:, 96:128]).all()
    assert np.isfinite(np.delete(g, np.s_[96:128], axis=1)).all()
    X = hsl.mx_quantize(tensor(x, "bf16"), "int8")
    dY, U, V = (tensor(weights(*s, 4), "bf16") for s in ((T, m), (m, r), (n, r)))
    dU, dV, dX = hsl.mx8_factor_grad(X, dY, U, V, dx=True)
    assert torch.isnan(dU).all()                         # Z of that token is NaN
    assert torch.isnan(dV[288:]).all() and torch.isfinite(dV[:288]).all()
    assert torch.isfinite(dX).all()                      # dX does not read X


def test_matrices_past_four_gigabytes(hsl):
    """5 GB of codes: every row repeats the first ones, so every output does too."""
    m, n, k = 600000, 16384, 5
    few = tensor(weights(k, n, 1), "bf16")
    reps = m // k
    D0 = hsl.mx_quantize(few)
    D = hsl.MX(D0.codes.repeat(reps, 1), D0.scales.repeat(reps, 1), n, "e2m1")
    for T in (1, 3, 40):
        x = tensor(tokens(T, n, T), "bf16")
        y = hsl.mx4_apply(D, x).view(T, reps, k)
        assert torch.equal(y, y[:, :1].expand(T, reps, k))
        close(y[:, -1], mx.apply(mx.values(D0.codes.cpu().numpy(), D0.scales.cpu().numpy(), n, "e2m1"), f64(x)),
              mx.apply(np.abs(f64(hsl.mx_dequantize(D0, "f32"))), np.abs(f64(x))), n, "bf16")
    x = few.repeat(140000, 1)                            # 11.5 G values in, 5.7 GB of codes out
    q = hsl.mx_quantize(x)
    assert torch.equal(q.codes.view(140000, k, -1), D0.codes.expand(140000, k, n // 2))
    assert torch.equal(q.scales.view(140000, k, -1), D0.scales.expand(140000, k, n // 32))
    assert torch.equal(hsl.mx_dequantize(q, "bf16")[-k:], hsl.mx_dequantize(D0, "bf16"))


def test_refusals(hsl):
    D, _ = blocks(hsl, weights(16, 64, 1), "e2m1")
    I8, _ = blocks(hsl, weights(16, 64, 1), "int8")
    x = torch.zeros(4, 64, dtype=torch.bfloat16, device="cuda")
    bad = [
        lambda: hsl.mx_quantize(x.t()),                               # not contiguous
        lambda: hsl.mx_quantize(x.half()),                            # no such dtype
        lambda: hsl.mx_quantize(x, "e4m3"),
        lambda: hsl.mx_quantize(x[0]),
        lambda: hsl.mx_quantize(x[:, :0]),
        lambda: hsl.mx_dequantize(D, "f16"),
        lambda: hsl.mx4_apply(D, x[:, :32]),                          # wrong width
        lambda: hsl.mx4_apply(D, x.cpu()),
        lambda: hsl.mx4_apply(D, x.half()),
        lambda: hsl.mx4_apply(D, x, add=x),                           # add of the wrong shape
        lambda: hsl.mx4_apply(D, x, add=torch.zeros(4, 16, device="cuda")),   # of another dtype
        lambda: hsl.mx4_apply(D, x, Y=torch.zeros(16, 4, dtype=torch.bfloat16, device="cuda").t()),
        lambda: hsl.mx4_apply(D, x[0]),
        lambda: hsl.mx4_apply_t(D, x),
        lambda: hsl.mx4_matmul(D, D, dtype="f16"),
        lambda: hsl.mx8_factor_grad(I8, x, x, x),
        lambda: hsl.mx8_factor_grad(I8, torch.zeros(16, 4, dtype=torch.bfloat16, device="cuda"),
                                    torch.zeros(4, 2, dtype=torch.bfloat16, device="cuda"),
                                    torch.zeros(64, 2, dtype=torch.bfloat16, device="cuda"), add=x),
        lambda: hsl.MX(D.codes[:, :16].contiguous(), D.scales, 64),
        lambda: hsl.MX(D.codes.t().contiguous().t(), D.scales, 64),   # not contiguous
        lambda: hsl.MX(D.codes, D.scales.cpu(), 64),
    ]
    for k, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
            pytest.fail(f"call {k} was not refused")
    for f in (lambda: hsl.mx4_apply(I8, x),                           # int8 where 4 bits are wanted
              lambda: hsl.mx4_matmul(I8, D), lambda: hsl.mx4_matmul(D, I8),
              lambda: hsl.mx4_matmul(D, hsl.mx_quantize(x[:, :32].contiguous())),
              lambda: hsl.mx8_factor_grad(D, torch.zeros(16, 4, dtype=torch.bfloat16, device="cuda"),
                                          torch.zeros(4, 2, dtype=torch.bfloat16, device="cuda"),
                                          torch.zeros(64, 2, dtype=torch.bfloat16, device="cuda"))):
        with pytest.raises(hsl.HslError):
            f()
    base = torch.zeros(16 * 32 + 8, dtype=torch.uint8, device="cuda")
    with pytest.raises(hsl.HslError):                                 # codes off 16 bytes
        hsl.mx4_apply(hsl.MX(base[8:].view(16, 32), D.scales, 64), x)
