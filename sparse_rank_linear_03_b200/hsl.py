"""ctypes binding of libhsl (include/hsl.h).

Argument marshalling only: every step of the split, pack and apply runs in
libhsl's CUDA kernels.  torch tensors supply device memory and the current
stream.  Importing this module loads ``libhsl.so`` and raises ImportError if
it has not been built (``python -m sparse_rank_linear_03_b200.build``); there
is no fallback path.
"""
from __future__ import annotations

import ctypes
import functools
import os

import torch

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libhsl.so")

FMT = {"csr": 0, "nm24": 1}
DTYPE = {"f32": 0, "bf16": 1}
TORCH_DTYPE = {"f32": torch.float32, "bf16": torch.bfloat16}
STATUS = {0: "HSL_OK", 1: "HSL_ERR_INVALID_ARG", 2: "HSL_ERR_UNSUPPORTED", 3: "HSL_ERR_NOT_READY",
          4: "HSL_ERR_OOM", 5: "HSL_ERR_CUDA", 6: "HSL_ERR_NAN_INPUT", 7: "HSL_ERR_TIMEOUT"}

# every symbol include/hsl.h declares
EXPORTS = (
    "hsl_create", "hsl_destroy", "hsl_split_topk", "hsl_get_nnz", "hsl_get_sparse",
    "hsl_set_sparse_csr", "hsl_set_sparse_nm24", "hsl_pack", "hsl_apply",
    "hsl_group_create", "hsl_group_apply", "hsl_group_destroy", "hsl_check",
    "hsl_status_str", "hsl_last_message", "hsl_launch_count", "hsl_split_topk_noalloc",
    "hsl_concentration", "hsl_rcm_order", "hsl_permute", "hsl_set_permutation", "hsl_factor",
    "hsl_set_index_bits", "hsl_mx_pitch", "hsl_mx_workspace", "hsl_mx_quantize",
    "hsl_mx_dequantize", "hsl_mx4_apply", "hsl_mx4_apply_t", "hsl_mx4_matmul",
    "hsl_mx8_factor_grad", "hsl_mx_check",
)


class _MXView(ctypes.Structure):
    """hsl_mx."""
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("rows", ctypes.c_int64),
                ("cols", ctypes.c_int64), ("elem", ctypes.c_int)]


class HslError(RuntimeError):
    def __init__(self, status: int, where: str, message: str):
        self.status = status
        self.name = STATUS.get(status, str(status))
        super().__init__(f"{where}: {self.name}: {message}")


def _load() -> ctypes.CDLL:
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it with "
                          "`python -m sparse_rank_linear_03_b200.build`")
    lib = ctypes.CDLL(LIB_PATH)
    P, I32, I64, D = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_double
    sig = {
        "hsl_create": [I64, I64, I32, ctypes.c_int, ctypes.c_int, ctypes.POINTER(P)],
        "hsl_destroy": [P],
        "hsl_split_topk": [P, P, ctypes.c_int, D, P, P],
        "hsl_get_nnz": [P, ctypes.POINTER(I64)],
        "hsl_get_sparse": [P, P, P, P, P, P],
        "hsl_set_sparse_csr": [P, I64, P, P, P, P],
        "hsl_set_sparse_nm24": [P, P, P, P],
        "hsl_pack": [P, P, P, P],
        "hsl_apply": [P, P, P, I64, P],
        "hsl_group_create": [P, I32, ctypes.POINTER(P), P],
        "hsl_group_apply": [P, P, P, I64, P],
        "hsl_group_destroy": [P],
        "hsl_check": [P, P],
        "hsl_status_str": [ctypes.c_int],
        "hsl_last_message": [],
        "hsl_launch_count": [],
        "hsl_split_topk_noalloc": [P, I64, I64, ctypes.c_int, D, P, P, P, ctypes.c_int, P, P, P],
        "hsl_concentration": [P, I64, I64, ctypes.c_int, ctypes.POINTER(D), P],
        "hsl_rcm_order": [I64, I64, P, P, P, P],
        "hsl_permute": [P, I64, I64, ctypes.c_int, P, P, P, P],
        "hsl_set_permutation": [P, P, P, P],
        "hsl_factor": [P, P, ctypes.c_int, P, I32, I32, P, P, P, P],
        "hsl_set_index_bits": [P, I32],
        "hsl_mx_pitch": [I64, I32, ctypes.POINTER(I64), ctypes.POINTER(I64)],
        "hsl_mx_workspace": [I32, I64, I64, I64, I64, I32, ctypes.POINTER(ctypes.c_size_t)],
        "hsl_mx_quantize": [P, I32, I64, I64, I32, P, P, P],
        "hsl_mx_dequantize": [P, P, I32, P],
        "hsl_mx4_apply": [P, P, P, P, I64, I32, P, ctypes.c_size_t, P],
        "hsl_mx4_apply_t": [P, P, P, P, I64, I32, P, ctypes.c_size_t, P],
        "hsl_mx4_matmul": [P, P, P, P, I32, P, ctypes.c_size_t, P],
        "hsl_mx_check": [P],
        "hsl_mx8_factor_grad": [P, P, I64, P, P, I32, P, P, P, P, I32, P, ctypes.c_size_t, P],
    }
    for name, args in sig.items():
        f = getattr(lib, name)
        f.argtypes = args
        f.restype = ctypes.c_int
    lib.hsl_status_str.restype = ctypes.c_char_p
    lib.hsl_last_message.restype = ctypes.c_char_p
    lib.hsl_launch_count.restype = ctypes.c_uint64
    return lib


lib = _load()


def _ok(status: int, where: str) -> None:
    if status != 0:
        raise HslError(status, where, lib.hsl_last_message().decode(errors="replace"))


def _stream(stream) -> int:
    if stream is not None:
        return int(getattr(stream, "cuda_stream", stream))
    return torch.cuda.current_stream().cuda_stream


def _ptr(t) -> int | None:
    if t is None:
        return None
    if isinstance(t, torch.Tensor):
        if not t.is_contiguous():
            raise ValueError("tensor must be contiguous")
        return t.data_ptr()
    return int(t)


def _need(t, numel: int, what: str) -> None:
    if t is not None and isinstance(t, torch.Tensor) and t.numel() != numel:
        raise ValueError(f"{what} has {t.numel()} elements, expected {numel}")


def _dtype_of(t, want: str, what: str) -> None:
    if isinstance(t, torch.Tensor) and t.dtype != TORCH_DTYPE[want]:
        raise ValueError(f"{what} is {t.dtype}, the layer stores {want}")


def _wdtype(t: torch.Tensor) -> str:
    return {torch.float32: "f32", torch.bfloat16: "bf16"}[t.dtype]


def concentration(W: torch.Tensor, stream=None) -> float:
    """ρ of a device matrix W (hsl_concentration)."""
    m, n = W.shape
    rho = ctypes.c_double()
    _ok(lib.hsl_concentration(_ptr(W), m, n, DTYPE[_wdtype(W)], ctypes.byref(rho), _stream(stream)),
        "hsl_concentration")
    return rho.value


def rcm_order(m: int, n: int, row_ptr, col):
    """RCM row and column orders of a CSR pattern (hsl_rcm_order; host arrays)."""
    import numpy as np
    rp = np.ascontiguousarray(np.asarray(row_ptr, dtype=np.int32))
    cl = np.ascontiguousarray(np.asarray(col, dtype=np.int32))
    ro = np.empty(m, np.int32)
    co = np.empty(n, np.int32)
    _ok(lib.hsl_rcm_order(m, n, rp.ctypes.data, cl.ctypes.data if cl.size else None,
                          ro.ctypes.data, co.ctypes.data), "hsl_rcm_order")
    return ro, co


def permute(W: torch.Tensor, row_order: torch.Tensor, col_order: torch.Tensor,
            out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """out[k][l] = W[row_order[k]][col_order[l]] on the device (hsl_permute)."""
    m, n = W.shape
    _need(row_order, m, "row_order")
    _need(col_order, n, "col_order")
    if out is None:
        out = torch.empty_like(W)
    _ok(lib.hsl_permute(_ptr(W), m, n, DTYPE[_wdtype(W)], _ptr(row_order), _ptr(col_order),
                        _ptr(out), _stream(stream)), "hsl_permute")
    return out


def launch_count() -> int:
    """Kernels libhsl has launched in this process."""
    return int(lib.hsl_launch_count())


class Layer:
    """One compressed layer: W ≈ S + U Vᵀ held on the device (an hsl_handle)."""

    def __init__(self, m: int, n: int, r: int, fmt: str = "csr", dtype: str = "bf16"):
        self.m, self.n, self.r, self.fmt, self.dtype = m, n, r, fmt, dtype
        h = ctypes.c_void_p()
        _ok(lib.hsl_create(m, n, r, FMT[fmt], DTYPE[dtype], ctypes.byref(h)), "hsl_create")
        self._h = h

    @property
    def handle(self) -> ctypes.c_void_p:
        return self._h

    def close(self) -> None:
        if getattr(self, "_h", None) is not None and self._h.value:
            lib.hsl_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    # -- stage 1 ------------------------------------------------------------
    def split(self, W: torch.Tensor, frac: float, residual: torch.Tensor | None = None,
              stream=None) -> None:
        wdt = {torch.float32: "f32", torch.bfloat16: "bf16"}[W.dtype]
        _need(W, self.m * self.n, "W")
        if residual is not None and (residual.dtype != W.dtype or residual.numel() != W.numel()):
            raise ValueError("residual must match W")
        _ok(lib.hsl_split_topk(self._h, _ptr(W), DTYPE[wdt], float(frac), _ptr(residual),
                               _stream(stream)), "hsl_split_topk")

    def nnz(self) -> int:
        v = ctypes.c_int64()
        _ok(lib.hsl_get_nnz(self._h, ctypes.byref(v)), "hsl_get_nnz")
        return v.value

    def get_sparse(self, stream=None) -> dict:
        dev = torch.device("cuda")
        vt = TORCH_DTYPE[self.dtype]
        if self.fmt == "csr":
            k = self.nnz()
            rp = torch.empty(self.m + 1, dtype=torch.int32, device=dev)
            col = torch.empty(max(k, 1), dtype=torch.int32, device=dev)
            val = torch.empty(max(k, 1), dtype=vt, device=dev)
            _ok(lib.hsl_get_sparse(self._h, _ptr(rp), _ptr(col), _ptr(val), None, _stream(stream)),
                "hsl_get_sparse")
            return {"row_ptr": rp, "col": col[:k], "val": val[:k]}
        val = torch.empty(self.m, self.n // 2, dtype=vt, device=dev)
        idx = torch.empty(self.m, self.n // 4, dtype=torch.uint8, device=dev)
        _ok(lib.hsl_get_sparse(self._h, None, None, _ptr(val), _ptr(idx), _stream(stream)),
            "hsl_get_sparse")
        return {"val": val, "idx": idx}

    def set_sparse_csr(self, row_ptr, col, val, stream=None) -> None:
        _need(row_ptr, self.m + 1, "row_ptr")
        _need(val, col.numel(), "val")
        _dtype_of(val, self.dtype, "val")
        _ok(lib.hsl_set_sparse_csr(self._h, int(col.numel()), _ptr(row_ptr), _ptr(col), _ptr(val),
                                   _stream(stream)), "hsl_set_sparse_csr")

    def set_sparse_nm24(self, val, idx, stream=None) -> None:
        _need(val, self.m * (self.n // 2), "val")
        _need(idx, self.m * (self.n // 4), "idx")
        _dtype_of(val, self.dtype, "val")
        _ok(lib.hsl_set_sparse_nm24(self._h, _ptr(val), _ptr(idx), _stream(stream)),
            "hsl_set_sparse_nm24")

    def set_index_bits(self, bits: int) -> None:
        """Column width of the packed CSR S (8, 16, 32; 0 = default) from the next pack."""
        _ok(lib.hsl_set_index_bits(self._h, int(bits)), "hsl_set_index_bits")

    # -- pack + apply -------------------------------------------------------
    def pack(self, U, V, stream=None) -> None:
        _need(U, self.m * self.r, "U")
        _need(V, self.n * self.r, "V")
        _dtype_of(U, self.dtype, "U")
        _dtype_of(V, self.dtype, "V")
        _ok(lib.hsl_pack(self._h, _ptr(U), _ptr(V), _stream(stream)), "hsl_pack")

    def apply(self, X: torch.Tensor, Y: torch.Tensor | None = None, stream=None) -> torch.Tensor:
        batch = X.shape[0] if X.dim() == 2 else 1
        _need(X, batch * self.n, "X")
        _dtype_of(X, self.dtype, "X")
        if Y is not None:
            _need(Y, batch * self.m, "Y")
            _dtype_of(Y, self.dtype, "Y")
        if Y is None:
            Y = torch.empty(batch, self.m, dtype=X.dtype, device=X.device,
                            pin_memory=(X.device.type == "cpu"))
        _ok(lib.hsl_apply(self._h, _ptr(X), _ptr(Y), batch, _stream(stream)), "hsl_apply")
        return Y

    def factor(self, R: torch.Tensor, omega: torch.Tensor, power_iters: int = 2, stream=None):
        """Stage 2: U [m][r], V [n][r] (layer dtype) and σ [r] of the residual R
        by the randomized truncated SVD with test matrix omega [n][k] (fp32)."""
        _need(R, self.m * self.n, "R")
        if omega.dtype != torch.float32 or omega.dim() != 2 or omega.shape[0] != self.n:
            raise ValueError("omega must be fp32 [n][k]")
        dev = R.device
        U = torch.empty(self.m, self.r, dtype=TORCH_DTYPE[self.dtype], device=dev)
        V = torch.empty(self.n, self.r, dtype=TORCH_DTYPE[self.dtype], device=dev)
        sig = torch.empty(self.r, dtype=torch.float32, device=dev)
        _ok(lib.hsl_factor(self._h, _ptr(R), DTYPE[_wdtype(R)], _ptr(omega), int(omega.shape[1]),
                           int(power_iters), _ptr(U), _ptr(V), _ptr(sig), _stream(stream)),
            "hsl_factor")
        return U, V, sig

    def set_permutation(self, row_order, col_order, stream=None) -> None:
        """The layer holds W[row_order][:, col_order]; apply in the original order."""
        if row_order is not None:
            _need(row_order, self.m, "row_order")
            _need(col_order, self.n, "col_order")
        _ok(lib.hsl_set_permutation(self._h, _ptr(row_order), _ptr(col_order), _stream(stream)),
            "hsl_set_permutation")

    def check(self, stream=None) -> None:
        _ok(lib.hsl_check(self._h, _stream(stream)), "hsl_check")


class Group:
    """Several packed layers applied in one pass (hsl_group)."""

    def __init__(self, layers: list[Layer], stream=None):
        self.layers = list(layers)
        arr = (ctypes.c_void_p * len(layers))(*[l.handle.value for l in layers])
        g = ctypes.c_void_p()
        _ok(lib.hsl_group_create(arr, len(layers), ctypes.byref(g), _stream(stream)),
            "hsl_group_create")
        self._g = g
        self._tabs = None

    def apply(self, Xs: list[torch.Tensor], Ys: list[torch.Tensor], stream=None) -> None:
        batch = Xs[0].shape[0]
        if len(Xs) != len(self.layers) or len(Ys) != len(self.layers):
            raise ValueError("one X and one Y per layer")
        for l, x, y in zip(self.layers, Xs, Ys):
            _need(x, batch * l.n, "X")
            _need(y, batch * l.m, "Y")
        xa = (ctypes.c_void_p * len(Xs))(*[_ptr(x) for x in Xs])
        ya = (ctypes.c_void_p * len(Ys))(*[_ptr(y) for y in Ys])
        _ok(lib.hsl_group_apply(self._g, xa, ya, batch, _stream(stream)), "hsl_group_apply")

    def close(self) -> None:
        if getattr(self, "_g", None) is not None and self._g.value:
            lib.hsl_group_destroy(self._g)
            self._g = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


# ---- microscaled blocks -------------------------------------------------------

MX_ELEM = {"e2m1": 0, "int8": 1}
_DTYPE_NAME = {torch.float32: "f32", torch.bfloat16: "bf16"}


def mx_pitch(cols: int, elem: str) -> tuple[int, int]:
    """Bytes per row of the codes and of the scales (hsl_mx_pitch)."""
    c, s = ctypes.c_int64(), ctypes.c_int64()
    _ok(lib.hsl_mx_pitch(cols, MX_ELEM[elem], ctypes.byref(c), ctypes.byref(s)), "hsl_mx_pitch")
    return c.value, s.value


@functools.lru_cache(maxsize=4096)
def _mx_workspace_bytes(op: int, batch: int, m: int, n: int, r: int, dtype: int) -> int:
    b = ctypes.c_size_t()
    _ok(lib.hsl_mx_workspace(op, batch, m, n, r, dtype, ctypes.byref(b)), "hsl_mx_workspace")
    return b.value


# the pointer of torch's current stream on a device, without the Stream object around it
_raw_stream = torch._C._cuda_getCurrentRawStream


class MX:
    """A matrix in microscaled blocks: codes and scales in the layout of hsl_mx.

    ``codes`` is [rows][code pitch] (uint8 for e2m1; int8 or uint8 for int8),
    ``scales`` [rows][scale pitch] uint8; both contiguous, on one CUDA device."""

    __slots__ = ("_codes", "_scales", "_buf", "rows", "cols", "elem", "device", "_view", "_ref")

    def __init__(self, codes: torch.Tensor, scales: torch.Tensor, cols: int, elem: str = "e2m1"):
        code = MX_ELEM.get(elem)
        if code is None:
            raise ValueError(f"unknown element type {elem!r}")
        if cols < 1 or codes.dim() != 2 or scales.dim() != 2:
            raise ValueError("codes and scales are 2-D and cols >= 1")
        rows, cp = codes.shape
        want_c, want_s = _pitches(cols, code)
        if cp != want_c:
            raise ValueError(f"codes have {cp} bytes per row, expected {want_c}")
        if scales.shape != (rows, want_s):
            raise ValueError(f"scales must be [{rows}][{want_s}]")
        if codes.dtype not in (torch.uint8, torch.int8) or scales.dtype != torch.uint8:
            raise ValueError("codes are uint8 (int8 for int8 blocks), scales uint8")
        if not codes.is_cuda or scales.device != codes.device:
            raise ValueError("codes and scales must be on one CUDA device")
        self._codes, self._scales, self._buf = codes, scales, None
        self._set(_ptr(codes), _ptr(scales), rows, cols, elem, code, codes.device)

    def _set(self, cptr, sptr, rows, cols, elem, code, device):
        self.rows, self.cols, self.elem, self.device = rows, cols, elem, device
        self._view = _MXView(cptr, sptr, rows, cols, code)
        self._ref = ctypes.addressof(self._view)

    @classmethod
    def empty(cls, rows: int, cols: int, elem: str, device) -> "MX":
        """Room for a matrix, codes and scales in one allocation of torch's current stream."""
        q = cls.__new__(cls)
        code = MX_ELEM[elem]
        cp, sp = _pitches(cols, code)
        q._codes = q._scales = None
        q._buf = buf = torch.empty(rows * (cp + sp), dtype=torch.uint8, device=device)
        p = buf.data_ptr()
        q._set(p, p + rows * cp, rows, cols, elem, code, buf.device)
        return q

    @property
    def codes(self) -> torch.Tensor:
        if self._codes is None:
            cp, _ = _pitches(self.cols, MX_ELEM[self.elem])
            c = self._buf[:self.rows * cp].view(self.rows, cp)
            self._codes = c.view(torch.int8) if self.elem == "int8" else c
        return self._codes

    @property
    def scales(self) -> torch.Tensor:
        if self._scales is None:
            cp, sp = _pitches(self.cols, MX_ELEM[self.elem])
            self._scales = self._buf[self.rows * cp:].view(self.rows, sp)
        return self._scales


def _pitches(cols: int, code: int) -> tuple[int, int]:
    nb = (cols + 31) >> 5
    return nb << (5 if code else 4), (nb + 15) & ~15


class _Using:
    """Makes a stream (and its device) torch's current one for the allocations and the launch of a
    call."""

    __slots__ = ("_ctx", "ptr")

    def __init__(self, device: torch.device, stream):
        if stream is None:
            self._ctx = torch.cuda.device(device)
            self.ptr = torch.cuda.current_stream(device).cuda_stream
            return
        if not isinstance(stream, torch.cuda.Stream):
            stream = torch.cuda.ExternalStream(int(getattr(stream, "cuda_stream", stream)),
                                               device=device)
        elif stream.device != device:
            raise ValueError(f"the stream is on {stream.device}, the data on {device}")
        self._ctx = torch.cuda.stream(stream)
        self.ptr = stream.cuda_stream

    def __enter__(self):
        self._ctx.__enter__()
        return self.ptr

    def __exit__(self, *exc):
        self._ctx.__exit__(*exc)


def _mx_call(device: torch.device, stream, fn, *args):
    """fn(stream pointer, *args) with the data's device current, and torch's current stream the
    given one (None: the device's current stream)."""
    if stream is None and device.index == torch.cuda.current_device():
        return fn(_raw_stream(device.index), *args)
    with _Using(device, stream) as s:
        return fn(s, *args)


def _operand(t: torch.Tensor, shape: tuple, dtype: torch.dtype, device: torch.device, what: str) -> int:
    """The pointer of a contiguous tensor of this shape, type and device."""
    if t.shape != shape:
        raise ValueError(f"{what} is {tuple(t.shape)}, expected {shape}")
    if t.dtype != dtype:
        raise ValueError(f"{what} is {t.dtype}, expected {dtype}")
    if t.device != device:
        raise ValueError(f"{what} is on {t.device}, expected {device}")
    if not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous")
    return t.data_ptr()


def _mx_dtype(t: torch.Tensor) -> int:
    name = _DTYPE_NAME.get(t.dtype)
    if name is None:
        raise ValueError(f"{t.dtype} is not supported: f32 or bf16")
    return DTYPE[name]


def _scratch(op: int, batch: int, m: int, n: int, r: int, dtype: int, device: torch.device):
    """Scratch memory of a call: the tensor that holds it (or None), its pointer and size."""
    b = _mx_workspace_bytes(op, batch, m, n, r, dtype)
    if b == 0:
        return None, None, 0
    t = torch.empty(b, dtype=torch.uint8, device=device)
    return t, t.data_ptr(), b


def _quantize(s, X, xp, dt, rows, cols, elem):
    q = MX.empty(rows, cols, elem, X.device)
    v = q._view
    st = lib.hsl_mx_quantize(xp, dt, rows, cols, v.elem, v.codes, v.scales, s)
    if st:
        _ok(st, "hsl_mx_quantize")
    return q


def mx_quantize(X: torch.Tensor, elem: str = "e2m1", stream=None) -> MX:
    """X [rows][cols] in blocks of 32 along its rows (hsl_mx_quantize)."""
    if X.dim() != 2 or not X.is_cuda:
        raise ValueError("X must be a 2-D CUDA tensor")
    if elem not in MX_ELEM:
        raise ValueError(f"unknown element type {elem!r}")
    rows, cols = X.shape
    if cols < 1:
        raise ValueError("X must have a column")
    dt = _mx_dtype(X)
    if not X.is_contiguous():
        raise ValueError("X must be contiguous")
    return _mx_call(X.device, stream, _quantize, X, X.data_ptr(), dt, rows, cols, elem)


def _dequantize(s, q, dtype):
    X = torch.empty(q.rows, q.cols, dtype=TORCH_DTYPE[dtype], device=q.device)
    st = lib.hsl_mx_dequantize(q._ref, X.data_ptr(), DTYPE[dtype], s)
    if st:
        _ok(st, "hsl_mx_dequantize")
    return X


def mx_dequantize(q: MX, dtype: str = "bf16", stream=None) -> torch.Tensor:
    """The values that the blocks stand for, [rows][cols] (hsl_mx_dequantize)."""
    if dtype not in DTYPE:
        raise ValueError(f"unknown dtype {dtype!r}")
    return _mx_call(q.device, stream, _dequantize, q, dtype)


def _apply(s, trans, D, X, xp, ap, add, Y, batch, f, dt):
    dev = D.device
    if Y is None:
        Y = X.new_empty(batch, f)
        yp = Y.data_ptr()
    else:
        yp = _operand(Y, (batch, f), X.dtype, dev, "the output")
    keep, wp, wb = _scratch(trans, batch, D.rows, D.cols, 0, dt, dev)
    fn = lib.hsl_mx4_apply_t if trans else lib.hsl_mx4_apply
    st = fn(D._ref, xp, ap, yp, batch, dt, wp, wb, s)
    if st:
        _ok(st, "hsl_mx4_apply_t" if trans else "hsl_mx4_apply")
    return Y


def _mx4_product(trans: int, D: MX, X: torch.Tensor, add, Y, stream):
    if X.dim() != 2:
        raise ValueError("the input must be 2-D [batch][features]")
    k, f = (D.rows, D.cols) if trans else (D.cols, D.rows)
    dt = _mx_dtype(X)
    batch = X.shape[0]
    xp = _operand(X, (batch, k), X.dtype, D.device, "the input")
    ap = None if add is None else _operand(add, (batch, f), X.dtype, D.device, "add")
    return _mx_call(D.device, stream, _apply, trans, D, X, xp, ap, add, Y, batch, f, dt)


def mx4_apply(D: MX, X: torch.Tensor, Y: torch.Tensor | None = None,
              add: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Y [batch][m] = X [batch][n] Dᵀ (+ add), D [m][n] in e2m1 blocks (hsl_mx4_apply).
    ``add`` may be Y, e.g. the output of the layer's sparse and low-rank part."""
    return _mx4_product(0, D, X, add, Y, stream)


def mx4_apply_t(D: MX, dY: torch.Tensor, dX: torch.Tensor | None = None,
                add: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """dX [batch][n] = dY [batch][m] D (+ add): the gradient of mx4_apply's input
    (hsl_mx4_apply_t)."""
    return _mx4_product(1, D, dY, add, dX, stream)


def _matmul(s, A, B, Y, ap, add, tdt, dt):
    if Y is None:
        Y = torch.empty(A.rows, B.rows, dtype=tdt, device=A.device)
        yp = Y.data_ptr()
    else:
        yp = _operand(Y, (A.rows, B.rows), tdt, A.device, "Y")
    keep, wp, wb = _scratch(2, A.rows, B.rows, A.cols, 0, dt, A.device)
    st = lib.hsl_mx4_matmul(A._ref, B._ref, ap, yp, dt, wp, wb, s)
    if st:
        _ok(st, "hsl_mx4_matmul")
    return Y


def mx4_matmul(A: MX, B: MX, Y: torch.Tensor | None = None, dtype: str = "bf16",
               add: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Y [A.rows][B.rows] = A Bᵀ (+ add), both in e2m1 blocks (hsl_mx4_matmul)."""
    if dtype not in DTYPE:
        raise ValueError(f"unknown dtype {dtype!r}")
    if B.device != A.device:
        raise ValueError(f"B is on {B.device}, expected {A.device}")
    tdt = TORCH_DTYPE[dtype]
    ap = None if add is None else _operand(add, (A.rows, B.rows), tdt, A.device, "add")
    return _mx_call(A.device, stream, _matmul, A, B, Y, ap, add, tdt, DTYPE[dtype])


def _factor_grad(s, X, dY, U, V, gp, up, vp, ap, add, dx, dt):
    dev = X.device
    m, r = U.shape
    dU, dV = torch.empty_like(U), torch.empty_like(V)
    dX = dY.new_empty(X.rows, X.cols) if dx else None
    keep, wp, wb = _scratch(3, X.rows, m, X.cols, r, dt, dev)
    st = lib.hsl_mx8_factor_grad(X._ref, gp, m, up, vp, r, ap, dU.data_ptr(), dV.data_ptr(),
                                 dX.data_ptr() if dx else None, dt, wp, wb, s)
    if st:
        _ok(st, "hsl_mx8_factor_grad")
    return (dU, dV, dX) if dx else (dU, dV)


def mx8_factor_grad(X: MX, dY: torch.Tensor, U: torch.Tensor, V: torch.Tensor, dx: bool = False,
                    add: torch.Tensor | None = None, stream=None):
    """Backward pass of x → U (Vᵀ x) from its input kept in int8 blocks (hsl_mx8_factor_grad):
    dU [m][r] and dV [n][r], and with ``dx`` also dX [T][n] = dY U Vᵀ (+ add)."""
    if dY.dim() != 2 or U.dim() != 2:
        raise ValueError("dY and U must be 2-D")
    if add is not None and not dx:
        raise ValueError("add is for dX: pass dx=True")
    dev, dt, tdt = X.device, _mx_dtype(dY), dY.dtype
    m, r = U.shape
    gp = _operand(dY, (X.rows, m), tdt, dev, "dY")
    up = _operand(U, (m, r), tdt, dev, "U")
    vp = _operand(V, (X.cols, r), tdt, dev, "V")
    ap = None if add is None else _operand(add, (X.rows, X.cols), tdt, dev, "add")
    return _mx_call(dev, stream, _factor_grad, X, dY, U, V, gp, up, vp, ap, add, dx, dt)


def mx_check(device=None, stream=None) -> None:
    """Synchronise the stream and raise if a device wait of the microscaled operators gave up
    on the device, on whatever stream, since the last check (hsl_mx_check)."""
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    _ok(_mx_call(dev, stream, lib.hsl_mx_check), "hsl_mx_check")
