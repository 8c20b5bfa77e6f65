"""Timed cases of the microscaled operators: block quantisation, products with a 4-bit matrix, gradients of the factors.

A microscaled matrix holds blocks of 32 consecutive values of a row that share one power of two.  ``e2m1`` blocks hold
4-bit floats (0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives), ``int8`` blocks hold integers in units of 1/64.  The
shared power is 2^floor(log2 max|x|), divided by 4 for e2m1, so that the largest value of a block lands in [4, 8) of
e2m1 (6 is the largest held) or in [64, 128) integer units (127 is the largest held).

Operators (``op`` of a case):

* ``quant``    x -> codes and scales -> the values they stand for, in x's type
* ``apply``    Y = X Dᵀ (+ add): a layer's forward with its dense part D [m][n] held in e2m1 blocks
* ``apply_t``  dX = dY D: the gradient of that layer's input
* ``matmul``   Y = A Bᵀ with both matrices in e2m1 blocks: tokens quantised too
* ``grads``    the backward pass of x -> U (Vᵀ x) from X kept in int8 blocks:
               Z = X V, G = dY U, dU = dYᵀ Z, dV = Xᵀ G and, where asked for, dX = add + G Vᵀ
"""
from __future__ import annotations

import math

import torch

own = False

BLOCK = 32
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "bf16": 2}
MAX_FLOPS = 2 * 4096 * 28672 * 8192
MAX_ELEMS = 28672 * 8192


def listed():
    return [
        # the residual of the 70B MLP up-projection going to 4 bits, and its values back (a layer being compressed)
        dict(name="quant_mlp70b_e2m1", op="quant", rows=28672, cols=8192, elem="e2m1", dtype="bf16"),
        # a small f32 activation of odd sizes into an 8-bit checkpoint: a call whose time is its launches
        dict(name="quant_odd_int8", op="quant", rows=77, cols=1001, elem="int8", dtype="f32"),
        # the smallest layer of the package, one f32 token
        dict(name="apply_1024_1tok_f32", op="apply", m=1024, n=1024, t=1, dtype="f32", add=False),
        # decoding one token through the 70B MLP up-projection: every byte of the layer is read once
        dict(name="apply_mlp70b_1tok", op="apply", m=28672, n=8192, t=1, dtype="bf16", add=False),
        # 16 sequences decoding through the 7B MLP up-projection, added to the sparse part's output
        dict(name="apply_mlp11008_16tok", op="apply", m=11008, n=4096, t=16, dtype="bf16", add=True),
        # a prompt through the same layer
        dict(name="apply_mlp11008_2048tok", op="apply", m=11008, n=4096, t=2048, dtype="bf16", add=False),
        # the gradient of the 7B MLP down-projection's input in a training step
        dict(name="apply_t_down11008_2048tok", op="apply_t", m=4096, n=11008, t=2048, dtype="bf16", add=False),
        # the same for a short ragged batch of a layer of odd sizes
        dict(name="apply_t_odd_33tok", op="apply_t", m=1001, n=777, t=33, dtype="bf16", add=True),
        # a long prompt through the 70B MLP up-projection with tokens in 4 bits as well: the largest case
        dict(name="matmul_mlp70b_4096tok", op="matmul", m=28672, n=8192, t=4096, dtype="bf16"),
        # a short prompt, odd sizes
        dict(name="matmul_odd_300tok", op="matmul", m=1000, n=1023, t=300, dtype="bf16"),
        # tuning the factors of the 70B MLP up-projection: 4096 tokens, rank 256, with the gradient passed on
        dict(name="grads_mlp70b_4096tok", op="grads", m=28672, n=8192, r=256, t=4096, dtype="bf16", dx=True),
        # tuning the factors of the attention projection on a short ragged batch
        dict(name="grads_attn4096_500tok", op="grads", m=4096, n=4096, r=128, t=500, dtype="bf16", dx=False),
    ]


def _size(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high + 0.5)))))))


def draw(rng):
    op = rng.choice(["quant", "apply", "apply", "apply_t", "matmul", "grads"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    if op == "quant":
        rows, cols = _size(rng, 1, 28672), _size(rng, 16, 11008)
        rows = max(1, min(rows, MAX_ELEMS // cols // (2 if dtype == "f32" else 1)))
        return dict(op=op, rows=rows, cols=cols, elem=rng.choice(["e2m1", "int8"]), dtype=dtype)
    # f32 layers of the package are small ones (up to 4096 wide) at small batches
    top = 4096 if dtype == "f32" else 28672
    m, n = _size(rng, 64, top), _size(rng, 64, min(top, 11008))
    if rng.random() < 0.5:  # layers are mostly multiples of 64
        m, n = m // 64 * 64, n // 64 * 64
    t = _size(rng, 1, 64 if dtype == "f32" else 4096)
    t = max(1, min(t, MAX_FLOPS // (4 * m * n)))
    if op == "grads":
        r = min(rng.choice([8, 16, 40, 64, 100, 128, 256]), m, n)
        return dict(op=op, m=m, n=n, r=r, t=t, dtype=dtype, dx=rng.random() < 0.5)
    if op == "matmul":
        return dict(op=op, m=m, n=n, t=t, dtype=dtype)
    return dict(op=op, m=m, n=n, t=t, dtype=dtype, add=rng.random() < 0.5)


# ---- inputs ------------------------------------------------------------------------------------------------------


def _gen(seed, device):
    return torch.Generator(device=device).manual_seed(seed)


def _weights(m, n, g, device):
    """0.02 t3, the heavy-tailed stand-in for LLM weights."""
    chi2 = torch.zeros(m, n, device=device)
    for _ in range(3):
        chi2 += torch.randn(m, n, generator=g, device=device).square_()
    return chi2.div_(3.0).rsqrt_().mul_(torch.randn(m, n, generator=g, device=device)).mul_(0.02)


def _tokens(t, n, g, device):
    """N(0, 1) with one channel in a hundred eight times as large, as activations have."""
    wide = torch.where(torch.rand(n, generator=g, device=device) < 0.01, 8.0, 1.0)
    return torch.randn(t, n, generator=g, device=device) * wide


def prepare(case, seed):
    device = torch.device("cuda")
    g = _gen(seed, device)
    op, dt = case["op"], TYPES[case["dtype"]]
    if op == "quant":
        rows, cols = case["rows"], case["cols"]
        make = _weights if case["elem"] == "e2m1" else _tokens
        return dict(case=case, x=make(rows, cols, g, device).to(dt))
    m, n, t = case["m"], case["n"], case["t"]
    if op == "grads":
        s = (0.01**2 / case["r"]) ** 0.25
        st = dict(case=case, x=_quantize(_tokens(t, n, g, device), "int8"),
                  dy=(0.01 * torch.randn(t, m, generator=g, device=device)).to(dt),
                  u=(s * torch.randn(m, case["r"], generator=g, device=device)).to(dt),
                  v=(s * torch.randn(n, case["r"], generator=g, device=device)).to(dt))
        if case["dx"]:
            st["add"] = (0.001 * torch.randn(t, n, generator=g, device=device)).to(dt)
        return st
    st = dict(case=case, d=_quantize(_weights(m, n, g, device), "e2m1"))
    if op == "matmul":
        st["a"] = _quantize(_tokens(t, n, g, device), "e2m1")
        return st
    k, f = (n, m) if op == "apply" else (m, n)
    st["x"] = _tokens(t, k, g, device).to(dt)
    if case["add"]:
        st["add"] = torch.randn(t, f, generator=g, device=device).to(dt)
    return st


# ---- plain forms -------------------------------------------------------------------------------------------------


def _blocks(x):
    rows, cols = x.shape
    nb = (cols + BLOCK - 1) // BLOCK
    p = torch.zeros(rows, nb * BLOCK, dtype=torch.float32, device=x.device)
    p[:, :cols] = x
    return p.view(rows, nb, BLOCK)


def _pow2(e):
    """2^e in fp32, e in -127 .. 127, from its bits: torch.ldexp and powers round on some devices."""
    return torch.where(e > -127, (e + 127) << 23, 1 << 22).to(torch.int32).view(torch.float32)


def _quantize(x, elem):
    """Codes (two 4-bit codes a byte, the even element in the low half; or one int8) and scale bytes, as held in memory:
    whole blocks a row, scale rows padded with zeros to a multiple of 16."""
    b = _blocks(x)
    rows, nb, _ = b.shape
    amax = b.abs().amax(2)
    emax = 2 if elem == "e2m1" else 0
    e = torch.where(amax > 0, torch.frexp(amax)[1] - 1 - emax, -127).clamp(-127, 127)
    bad = ~torch.isfinite(b).all(2)
    v = b * _pow2(-e)[..., None]
    v = torch.where(bad[..., None], torch.zeros_like(v), v)
    if elem == "e2m1":
        a = v.abs()
        step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
        a = (torch.round(a / step) * step).clamp(max=6.0)
        code = torch.where(a < 2, 2 * a, torch.where(a < 4, a + 2, 0.5 * a + 4)).to(torch.uint8)
        code = torch.where(torch.signbit(v), code + 8, code).view(rows, nb * BLOCK)
        codes = code[:, 0::2] | (code[:, 1::2] << 4)
    else:
        codes = torch.round(v * 64.0).clamp(-127, 127).to(torch.int8).view(rows, nb * BLOCK)
    scales = torch.zeros(rows, (nb + 15) // 16 * 16, dtype=torch.uint8, device=x.device)
    scales[:, :nb] = torch.where(bad, 255, e + 127).to(torch.uint8)
    return codes.contiguous(), scales


def _values(q, cols, elem):
    """The fp32 values that codes and scales stand for."""
    codes, scales = q
    rows = codes.shape[0]
    nb = (cols + BLOCK - 1) // BLOCK
    if elem == "e2m1":
        code = torch.stack([codes & 15, codes >> 4], 2).view(rows, nb * BLOCK).to(torch.int64)
        held = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], device=codes.device)
        v = held[code]
    else:
        v = codes.to(torch.float32) / 64.0
    e = scales[:, :nb].to(torch.int32)
    v = v.view(rows, nb, BLOCK) * _pow2((e - 127).clamp(max=127))[..., None]
    v = torch.where((e == 255)[..., None], torch.full_like(v, float("nan")), v)
    return v.view(rows, nb * BLOCK)[:, :cols]


def _plain(st):
    case = st["case"]
    op, dt = case["op"], TYPES[case["dtype"]]
    if op == "quant":
        return _values(_quantize(st["x"], case["elem"]), case["cols"], case["elem"]).to(dt)
    n = case["n"]
    if op == "grads":
        x, dy, u, v = _values(st["x"], n, "int8"), st["dy"].float(), st["u"].float(), st["v"].float()
        z, g = x @ v, dy @ u
        out = [(dy.T @ z).to(dt), (x.T @ g).to(dt)]
        if case["dx"]:
            out.append((st["add"].float() + g @ v.T).to(dt))
        return out
    d = _values(st["d"], n, "e2m1")
    if op == "matmul":
        return (_values(st["a"], n, "e2m1") @ d.T).to(dt)
    y = st["x"].float() @ (d.T if op == "apply" else d)
    if case["add"]:
        y = y + st["add"].float()
    return y.to(dt)


# ---- the framework's calls ---------------------------------------------------------------------------------------


def _framework(st):
    from sparse_rank_linear_03_b200 import hsl

    case = st["case"]
    op, dt = case["op"], case["dtype"]
    if op == "quant":
        return hsl.mx_dequantize(hsl.mx_quantize(st["x"], case["elem"]), dt)
    if op == "grads":
        x = hsl.MX(*st["x"], case["n"], "int8")
        return list(hsl.mx8_factor_grad(x, st["dy"], st["u"], st["v"], dx=case["dx"], add=st.get("add")))
    d = hsl.MX(*st["d"], case["n"], "e2m1")
    if op == "matmul":
        return hsl.mx4_matmul(hsl.MX(*st["a"], case["n"], "e2m1"), d, dtype=dt)
    if op == "apply":
        return hsl.mx4_apply(d, st["x"], add=st.get("add"))
    return hsl.mx4_apply_t(d, st["x"], add=st.get("add"))


def run(state):
    return _framework(state) if own else _plain(state)


# ---- what a pass cannot do without -------------------------------------------------------------------------------


def _held(rows, cols, elem):
    """Bytes of codes and scales."""
    nb = (cols + BLOCK - 1) // BLOCK
    return rows * nb * ((16 if elem == "e2m1" else 32) + 1)


def work(case):
    op, b = case["op"], SIZE[case["dtype"]]
    if op == "quant":
        e = case["rows"] * case["cols"]
        return {"bytes": 2 * e * b, "flops": 4 * e}
    m, n, t = case["m"], case["n"], case["t"]
    if op == "grads":
        r, dx = case["r"], 1 if case["dx"] else 0
        return {"bytes": _held(t, n, "int8") + t * m * b + 2 * (m + n) * r * b + 2 * dx * t * n * b,
                "flops": 4 * t * r * (m + n) + 2 * dx * t * n * r}
    if op == "matmul":
        return {"bytes": _held(m, n, "e2m1") + _held(t, n, "e2m1") + t * m * b, "flops": 2 * t * m * n}
    f = m if op == "apply" else n
    return {"bytes": _held(m, n, "e2m1") + t * (m + n) * b + (t * f * b if case["add"] else 0), "flops": 2 * t * m * n}


# ---- the definition in 64 bits -----------------------------------------------------------------------------------

_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
# between neighbours of the list above; at a border itself the value with the even code is taken
_BORDERS = (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)


def _exact_pow2(e):
    return ((e.long() + 1023) << 52).view(torch.float64)


def _exact_quant(x, elem):
    rows, cols = x.shape
    pad = -cols % BLOCK
    b = torch.nn.functional.pad(x.double(), (0, pad)).reshape(rows, -1, BLOCK)
    top = b.abs().amax(2, keepdim=True)
    power = (top.view(torch.int64) >> 52) - 1023  # top is an fp32 value or 0: never subnormal in fp64
    power = power - (2 if elem == "e2m1" else 0)
    scale = _exact_pow2(power.clamp(-127, 127))
    v = b / scale
    if elem == "e2m1":
        held = torch.tensor(_E2M1, dtype=torch.float64, device=x.device)
        index = torch.zeros(v.shape, dtype=torch.int64, device=x.device)
        for k, border in enumerate(_BORDERS):
            index += (v.abs() > border) if k % 2 == 0 else (v.abs() >= border)
        v = held[index] * torch.sign(v)
    else:
        low = torch.floor(v * 64.0)
        part = v * 64.0 - low
        up = (part > 0.5) | ((part == 0.5) & (low % 2 == 1))
        v = (low + up.double()).clamp(-127, 127) / 64.0
    return (v * scale).reshape(rows, -1)[:, :cols]


def _exact_values(q, cols, elem):
    codes, scales = q
    rows = codes.shape[0]
    if elem == "e2m1":
        held = torch.tensor(_E2M1, dtype=torch.float64, device=codes.device)
        v = torch.empty(rows, 2 * codes.shape[1], dtype=torch.float64, device=codes.device)
        for half in (0, 1):
            c = (codes >> (4 * half)) & 15
            v[:, half::2] = held[(c & 7).long()] * (1.0 - 2.0 * (c >> 3).double())
    else:
        v = codes.double() / 64.0
    power = _exact_pow2(scales.long() - 127)
    return v[:, :cols] * power.repeat_interleave(BLOCK, 1)[:, :cols]


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "quant":
        return _exact_quant(st["x"], case["elem"])
    n = case["n"]
    if op == "grads":
        x, dy, u, v = _exact_values(st["x"], n, "int8"), st["dy"].double(), st["u"].double(), st["v"].double()
        g = torch.einsum("ti,ik->tk", dy, u)
        out = [torch.einsum("ti,tk->ik", dy, torch.einsum("tj,jk->tk", x, v)), torch.einsum("tj,tk->jk", x, g)]
        if case["dx"]:
            out.append(torch.einsum("tk,jk->tj", g, v) + st["add"].double())
        return out
    d = _exact_values(st["d"], n, "e2m1")
    if op == "matmul":
        return torch.einsum("tj,ij->ti", _exact_values(st["a"], n, "e2m1"), d)
    y = torch.einsum("tj,ij->ti" if op == "apply" else "ti,ij->tj", st["x"].double(), d)
    return y + st["add"].double() if case["add"] else y
