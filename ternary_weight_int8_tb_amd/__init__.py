"""Python binding of libtb.so: ternary-weight int8 FFN decode on MI355X (gfx950).

Argument marshalling only. Every step of the path runs in the HIP kernels of
``csrc/tb.hip`` behind the C ABI in ``include/tb.h``. The functions take the
ABI's names; torch tensors supply device memory and the stream. There is no
CPU fallback: if libtb.so is missing or cannot be loaded, every call raises.

Importing this package loads nothing. ``synth`` (the input generator) works
without a GPU.
"""

from __future__ import annotations

import ctypes
import functools
import os

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libtb.so")

TB_OK, TB_EINVAL, TB_EALIGN, TB_EUNSUPPORTED, TB_EHIP, TB_ESCRATCH = 0, -1, -2, -3, -4, -5
TB_FMT_TERNARY2, TB_FMT_SIGN1, TB_FMT_SIGN1_RI4 = 0, 1, 2
BLOCK = 128
MAX_ROWS = 8
MAX_BATCH_ROWS = 32
ABI_VERSION = 7
TB_F32, TB_BF16, TB_F16 = 0, 1, 2

# every symbol include/tb.h declares
ABI_SYMBOLS = ("tb_rotate_quant_i8", "tb_gemv_ternary", "tb_gemv_ternary_x", "tb_ffn_gateup_silu",
               "tb_ffn_gateup_silu_x",
               "tb_ffn_down",
               "tb_gemv_block_sums", "tb_rotate_quant_i8_batch", "tb_gemv_ternary_batch",
               "tb_ffn_gateup_silu_batch", "tb_ffn_down_batch", "tb_gemv_block_sums_batch",
               "tb_ffn_down_noalloc", "tb_sign_interleave",
               "tb_ffn_down_split", "tb_ffn_down_split_workspace_bytes",
               "tb_ffn_down_split_batch", "tb_ffn_down_split_batch_workspace_bytes",
               "tb_ffn_workspace_bytes", "tb_ffn_workspace_init",
               "tb_ffn_layers", "tb_ffn_workspace_error",
               "tb_add_rmsnorm_quant_i8",
               "tb_mxfp4_quant", "tb_mxfp4_dequant", "tb_mxfp4_gemm", "tb_mxfp4_gemm_workspace_bytes",
               "tb_moe_plan", "tb_moe_gateup_silu", "tb_moe_down", "tb_moe_combine",
               "tb_status_str", "tb_abi_version")
TB_FFN_CHAIN = 1


class TbError(RuntimeError):
    def __init__(self, fn: str, status: int, why: str = ""):
        self.status = status
        super().__init__(f"{fn} failed: {status} ({tb_status_str(status)})" + (f": {why}" if why else ""))


class CMatrix(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("n", ctypes.c_int32),
                ("k", ctypes.c_int32), ("fmt", ctypes.c_int32)]


class CFfnWeights(ctypes.Structure):
    _fields_ = [("gate", CMatrix), ("up", CMatrix), ("down", CMatrix)]


class CMxfp4(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("n", ctypes.c_int32),
                ("k", ctypes.c_int32)]


class CExperts(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("experts", ctypes.c_int32),
                ("n", ctypes.c_int32), ("k", ctypes.c_int32), ("fmt", ctypes.c_int32)]


_P = ctypes.c_void_p
_I = ctypes.c_int
_XP = ctypes.POINTER(CMxfp4)
_EP = ctypes.POINTER(CExperts)
_MP = ctypes.POINTER(CMatrix)
_SIGS = {
    "tb_rotate_quant_i8": ([_P, _I, _I, _P, _P, _P], _I),
    "tb_gemv_ternary": ([_MP, _P, _P, _I, _P, _P], _I),
    "tb_ffn_gateup_silu": ([_MP, _MP, _P, _P, _I, _P, _P], _I),
    "tb_ffn_gateup_silu_x": ([_MP, _MP, _P, _I, _P, _P, _P, _P], _I),
    "tb_gemv_ternary_x": ([_MP, _P, _I, _P, _P, _P, _P], _I),
    "tb_ffn_down": ([_MP, _P, _I, _P, _P, _P, _P], _I),
    "tb_gemv_block_sums": ([_MP, _P, _I, _P, _P], _I),
    "tb_rotate_quant_i8_batch": ([_P, _I, _I, _P, _P, _P], _I),
    "tb_gemv_ternary_batch": ([_MP, _P, _P, _I, _P, _P], _I),
    "tb_ffn_gateup_silu_batch": ([_MP, _MP, _P, _P, _I, _P, _P], _I),
    "tb_ffn_down_batch": ([_MP, _P, _I, _P, _P, _P, _P], _I),
    "tb_gemv_block_sums_batch": ([_MP, _P, _I, _P, _P], _I),
    "tb_ffn_down_noalloc": ([_MP, _P, _I, _P, _P], _I),
    "tb_sign_interleave": ([_MP, _P, _P, _P], _I),
    "tb_ffn_down_split": ([_MP, _P, _I, _P, _P, _P, _P, ctypes.c_size_t, _P], _I),
    "tb_ffn_down_split_workspace_bytes": ([_MP, _I], ctypes.c_size_t),
    "tb_ffn_down_split_batch": ([_MP, _P, _I, _P, _P, _P, _P, ctypes.c_size_t, _P], _I),
    "tb_ffn_down_split_batch_workspace_bytes": ([_MP, _I], ctypes.c_size_t),
    "tb_ffn_workspace_bytes": ([_I, _I, _I], ctypes.c_size_t),
    "tb_ffn_workspace_init": ([_P, ctypes.c_size_t, ctypes.c_uint32, _P], _I),
    "tb_ffn_layers": ([ctypes.POINTER(CFfnWeights), _I, _P, _I, ctypes.c_uint, _P, ctypes.c_size_t,
                       _P, _P], _I),
    "tb_ffn_workspace_error": ([_P, ctypes.POINTER(_I)], _I),
    "tb_add_rmsnorm_quant_i8": ([_P, _P, _P, _I, _I, _I, ctypes.c_float, _P, _P, _P, _P, _P], _I),
    "tb_mxfp4_quant": ([_P, _I, _I, _I, _I, _P, _P, _P], _I),
    "tb_mxfp4_dequant": ([_P, _P, _I, _I, _P, _I, _P], _I),
    "tb_mxfp4_gemm": ([_XP, _P, _P, _I, _P, _I, _P, ctypes.c_size_t, _P], _I),
    "tb_mxfp4_gemm_workspace_bytes": ([_XP, _I], ctypes.c_size_t),
    "tb_moe_plan": ([_P, _I, _I, _I, _P, _P, _P], _I),
    "tb_moe_gateup_silu": ([_EP, _EP, _P, _P, _I, _I, _P, _P, _P, _P, _P, _P], _I),
    "tb_moe_down": ([_EP, _P, _P, _I, _P, _P, _P, _P], _I),
    "tb_moe_combine": ([_P, _P, _P, _I, _I, _I, _I, _P, _I, _P], _I),
    "tb_status_str": ([_I], ctypes.c_char_p),
    "tb_abi_version": ([], _I),
}

_lib: ctypes.CDLL | None = None


def lib() -> ctypes.CDLL:
    """Load libtb.so (once). Raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -c 'import __graft_entry__ as g; g.build()'`")
        L = ctypes.CDLL(LIB_PATH)
        for name, (args, res) in _SIGS.items():
            fn = getattr(L, name)
            fn.argtypes = args
            fn.restype = res
        _lib = L
    return _lib


def tb_status_str(status: int) -> str:
    return lib().tb_status_str(int(status)).decode()


def tb_abi_version() -> int:
    return lib().tb_abi_version()


class Matrix:
    """A weight matrix on the device: codes and scales tensors plus its shape and format."""

    def __init__(self, codes, scales, n: int, k: int, fmt: int):
        self.codes, self.scales = codes, scales
        self.n, self.k, self.fmt = int(n), int(k), int(fmt)
        self._c = CMatrix(codes.data_ptr(), scales.data_ptr(), self.n, self.k, self.fmt)

    @property
    def c(self) -> CMatrix:
        return self._c

    @property
    def nbytes(self) -> int:
        return self.codes.numel() * self.codes.element_size() + \
            self.scales.numel() * self.scales.element_size()

    @classmethod
    def upload(cls, packed, device="cuda") -> "Matrix":
        """Copy a host matrix (synth.PackedMatrix) to the device."""
        import torch
        codes = torch.from_numpy(packed.codes).to(device)
        scales = torch.from_numpy(packed.scales.view("int16")).to(device)
        return cls(codes, scales, packed.n, packed.k, packed.fmt)


def _stream(stream):
    if stream is None:
        import torch
        # the handle alone: building a Stream object costs 2.7 us of a call's 11
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _rows(t) -> int:
    return int(t.shape[0]) if t.dim() > 1 else 1


def _call(name: str, *args):
    rc = getattr(lib(), name)(*args)
    if rc != TB_OK:
        raise TbError(name, rc)


def tb_rotate_quant_i8(x, q, dq, stream=None) -> None:
    """x float32 [m][k] -> q int8 [m][k], dq float32 [m][k/128] (device tensors)."""
    m, k = _rows(x), int(x.shape[-1])
    _call("tb_rotate_quant_i8", x.data_ptr(), m, k, q.data_ptr(), dq.data_ptr(), _stream(stream))


def tb_gemv_ternary(w: Matrix, q, dq, y, stream=None) -> None:
    """y float32 [m][w.n] = GEMV of w against the int8 rows q with scales dq."""
    _call("tb_gemv_ternary", ctypes.byref(w.c), q.data_ptr(), dq.data_ptr(), _rows(q),
          y.data_ptr(), _stream(stream))


def tb_gemv_ternary_x(w: Matrix, x, qx, dqx, y, stream=None) -> None:
    """y = GEMV of w against rotquant(x), written to qx, dqx; one call."""
    _call("tb_gemv_ternary_x", ctypes.byref(w.c), x.data_ptr(), _rows(x), qx.data_ptr(),
          dqx.data_ptr(), y.data_ptr(), _stream(stream))


def tb_ffn_gateup_silu(wg: Matrix, wu: Matrix, q, dq, h, stream=None) -> None:
    """h float32 [m][wg.n] = silu(wg q) * (wu q), from one shared int8 copy."""
    _call("tb_ffn_gateup_silu", ctypes.byref(wg.c), ctypes.byref(wu.c), q.data_ptr(),
          dq.data_ptr(), _rows(q), h.data_ptr(), _stream(stream))


def tb_ffn_gateup_silu_x(wg: Matrix, wu: Matrix, x, qx, dqx, h, stream=None) -> None:
    """h = silu(wg q) * (wu q) with (q, dq) = rotquant(x), written to qx, dqx; one call."""
    _call("tb_ffn_gateup_silu_x", ctypes.byref(wg.c), ctypes.byref(wu.c), x.data_ptr(), _rows(x),
          qx.data_ptr(), dqx.data_ptr(), h.data_ptr(), _stream(stream))


def tb_ffn_down(wd: Matrix, h, qh_ws, dqh_ws, y, stream=None) -> None:
    """y float32 [m][wd.n] = down GEMV of rotquant(h); qh_ws/dqh_ws are the workspace."""
    _call("tb_ffn_down", ctypes.byref(wd.c), h.data_ptr(), _rows(h), qh_ws.data_ptr(),
          dqh_ws.data_ptr(), y.data_ptr(), _stream(stream))


def tb_gemv_block_sums(w: Matrix, q, isum, stream=None) -> None:
    """isum int32 [m][w.n][w.k/128]: the integer block sums before the scale fold."""
    _call("tb_gemv_block_sums", ctypes.byref(w.c), q.data_ptr(), _rows(q), isum.data_ptr(),
          _stream(stream))


def tb_rotate_quant_i8_batch(x, q, dq, stream=None) -> None:
    """tb_rotate_quant_i8 for up to 32 rows."""
    m, k = _rows(x), int(x.shape[-1])
    _call("tb_rotate_quant_i8_batch", x.data_ptr(), m, k, q.data_ptr(), dq.data_ptr(),
          _stream(stream))


def tb_gemv_ternary_batch(w: Matrix, q, dq, y, stream=None) -> None:
    """tb_gemv_ternary for up to 32 rows."""
    _call("tb_gemv_ternary_batch", ctypes.byref(w.c), q.data_ptr(), dq.data_ptr(), _rows(q),
          y.data_ptr(), _stream(stream))


def tb_ffn_gateup_silu_batch(wg: Matrix, wu: Matrix, q, dq, h, stream=None) -> None:
    """tb_ffn_gateup_silu for up to 32 rows."""
    _call("tb_ffn_gateup_silu_batch", ctypes.byref(wg.c), ctypes.byref(wu.c), q.data_ptr(),
          dq.data_ptr(), _rows(q), h.data_ptr(), _stream(stream))


def tb_ffn_down_batch(wd: Matrix, h, qh_ws, dqh_ws, y, stream=None) -> None:
    """tb_ffn_down for up to 32 rows."""
    _call("tb_ffn_down_batch", ctypes.byref(wd.c), h.data_ptr(), _rows(h), qh_ws.data_ptr(),
          dqh_ws.data_ptr(), y.data_ptr(), _stream(stream))


def tb_gemv_block_sums_batch(w: Matrix, q, isum, stream=None) -> None:
    """tb_gemv_block_sums for up to 32 rows."""
    _call("tb_gemv_block_sums_batch", ctypes.byref(w.c), q.data_ptr(), _rows(q), isum.data_ptr(),
          _stream(stream))


def tb_sign_interleave(w: Matrix, stream=None) -> Matrix:
    """The TB_FMT_SIGN1_RI4 copy of a sign matrix (rows interleaved by four), in new device
    tensors, for the lookup-table GEMV."""
    import torch
    with _owned_by(stream, w.codes.device):
        codes = torch.empty_like(w.codes)
        scales = torch.empty_like(w.scales)
    _call("tb_sign_interleave", ctypes.byref(w.c), codes.data_ptr(), scales.data_ptr(),
          _stream(stream))
    return Matrix(codes, scales, w.n, w.k, TB_FMT_SIGN1_RI4)


def tb_ffn_down_noalloc(wd: Matrix, h, y, stream=None) -> None:
    """tb_ffn_down with the library's static scratch instead of a caller workspace."""
    _call("tb_ffn_down_noalloc", ctypes.byref(wd.c), h.data_ptr(), _rows(h), y.data_ptr(),
          _stream(stream))


def tb_ffn_down_split_workspace_bytes(wd: Matrix, m: int) -> int:
    """Bytes of device workspace tb_ffn_down_split needs for m rows (0 for bad arguments)."""
    return int(lib().tb_ffn_down_split_workspace_bytes(ctypes.byref(wd.c), int(m)))


def tb_ffn_down_split_batch_workspace_bytes(wd: Matrix, m: int) -> int:
    """Bytes of device workspace tb_ffn_down_split_batch needs for m rows (0 for bad arguments)."""
    return int(lib().tb_ffn_down_split_batch_workspace_bytes(ctypes.byref(wd.c), int(m)))


def tb_ffn_down_split_workspace(wd: Matrix, m: int, batch: bool = False):
    """A new tb_ffn_down_split (batch: tb_ffn_down_split_batch) workspace for m rows
    (uint8 device tensor; no initialisation)."""
    import torch
    name = "tb_ffn_down_split_batch_workspace_bytes" if batch else "tb_ffn_down_split_workspace_bytes"
    nbytes = int(getattr(lib(), name)(ctypes.byref(wd.c), int(m)))
    if nbytes == 0:
        raise TbError(name, TB_EINVAL)
    return torch.empty(nbytes, dtype=torch.uint8, device=wd.codes.device)


def tb_ffn_down_split(wd: Matrix, h, qh, dqh, y, ws, stream=None) -> None:
    """tb_ffn_down with a workspace for the split over k; y, qh, dqh are bit-identical."""
    _call("tb_ffn_down_split", ctypes.byref(wd.c), h.data_ptr(), _rows(h), qh.data_ptr(),
          dqh.data_ptr(), y.data_ptr(), ws.data_ptr(), ws.numel() * ws.element_size(),
          _stream(stream))


def tb_ffn_down_split_batch(wd: Matrix, h, qh, dqh, y, ws, stream=None) -> None:
    """tb_ffn_down_split for 1 ... 32 rows; each row bit-identical to tb_ffn_down alone."""
    _call("tb_ffn_down_split_batch", ctypes.byref(wd.c), h.data_ptr(), _rows(h), qh.data_ptr(),
          dqh.data_ptr(), y.data_ptr(), ws.data_ptr(), ws.numel() * ws.element_size(),
          _stream(stream))


def tb_ffn_workspace_bytes(m: int, hidden: int, inter: int) -> int:
    """Bytes of device workspace tb_ffn_layers needs for m rows (0 for bad arguments)."""
    return int(lib().tb_ffn_workspace_bytes(int(m), int(hidden), int(inter)))


def tb_ffn_workspace_init(ws, spin_ticks: int = 0, stream=None) -> None:
    """Initialise a workspace (uint8 device tensor); spin_ticks 0 = the default limit."""
    _call("tb_ffn_workspace_init", ws.data_ptr(), ws.numel() * ws.element_size(),
          int(spin_ticks), _stream(stream))


def tb_ffn_workspace_error(ws) -> int:
    """The sticky error word of a workspace (synchronises with the device)."""
    err = _I(0)
    _call("tb_ffn_workspace_error", ws.data_ptr(), ctypes.byref(err))
    return int(err.value)


class FfnLayers:
    """A host array of tb_ffn_weights for tb_ffn_layers, built once from (gate, up, down)."""

    def __init__(self, layers):
        self.layers = list(layers)
        self.arr = (CFfnWeights * len(self.layers))()
        for i, (g, u, d) in enumerate(self.layers):
            self.arr[i].gate, self.arr[i].up, self.arr[i].down = g.c, u.c, d.c

    def __len__(self) -> int:
        return len(self.layers)


def tb_ffn_layers(layers: FfnLayers, x, ws, y, chain: bool = False, stream=None) -> None:
    """Run len(layers) whole FFN layers (one launch per 32 layers).

    x float32 [L][m][hidden] (or [m][hidden] with chain=True: layer l+1 takes layer l's y),
    y float32 [L][m][hidden], ws an initialised uint8 workspace tensor."""
    if y.dim() != 3:
        raise ValueError("y must be [layers][m][hidden]")
    m = int(y.shape[1])
    _call("tb_ffn_layers", layers.arr, len(layers), x.data_ptr(), m,
          TB_FFN_CHAIN if chain else 0, ws.data_ptr(), ws.numel() * ws.element_size(),
          y.data_ptr(), _stream(stream))


# ---- row operators, microscaled 4-bit products, experts ----------------------------------
# These check their tensors here (type, shape, contiguity, device) and run on the tensors'
# device, on its current stream unless one is given.
# A call costs the host about as much as a launch does, so that they look torch up once and ask for
# the current device once.
@functools.lru_cache(maxsize=None)
def _torch():
    import torch
    return torch


def _bad(fn: str, why: str):
    raise TbError(fn, TB_EINVAL, why)


_DTYPES: dict = {}


def _dtype(fn: str, t) -> int:
    if not _DTYPES:
        import torch
        _DTYPES.update({torch.float32: TB_F32, torch.bfloat16: TB_BF16, torch.float16: TB_F16})
    code = _DTYPES.get(t.dtype)
    if code is None:
        _bad(fn, f"{t.dtype} rows: float32, bfloat16 or float16 are wanted")
    return code


def _check(fn: str, device, *arrays) -> None:
    """Each of arrays is (name, tensor, dtype, shape): contiguous, on `device`."""
    index = device.index
    for name, t, dtype, shape in arrays:
        if t.dtype is not dtype or t.shape != shape or t.get_device() != index or not t.is_contiguous():
            _bad(fn, f"{name} has to be a contiguous {dtype} tensor of shape {tuple(shape)} on {device}")


def _matrix_rows(fn: str, name: str, t):
    if t.dim() != 2 or not t.is_cuda or not t.is_contiguous():
        _bad(fn, f"{name} has to be a contiguous matrix on the GPU")
    return t.shape


def _launch(fn: str, device, stream, *args) -> None:
    torch = _torch()
    index = torch._C._cuda_getDevice()   # the tensors are there, so the device is initialised
    if device.index != index:
        with torch.cuda.device(device):
            _call(fn, *args, _stream(stream))
    elif stream is None:
        _call(fn, *args, torch._C._cuda_getCurrentRawStream(index))
    else:
        _call(fn, *args, _stream(stream))


def _ptr(t):
    return None if t is None else t.data_ptr()


def _owned_by(stream, device):
    """Within it new tensors on `device` belong to `stream`, as the call's stream argument names it: memory
    that another stream has freed, and may still be using, is not handed to them."""
    torch = _torch()
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream, device) if stream else torch.cuda.default_stream(device)
    return torch.cuda.stream(stream)   # None: as it is


def tb_add_rmsnorm_quant_i8(x, res, gamma, eps: float, res_out, y, q, dq, stream=None) -> None:
    """s = x + res; q int8 [m][k], dq float32 [m][k/128] = rotated int8 copy of the normed rows.

    x, res (or None) [m][k] of one type (float32, bfloat16, float16); gamma float32 [k]. res_out
    (or None; may be x or res) takes s, y (or None) the normed rows, both in that type."""
    torch = _torch()
    fn = "tb_add_rmsnorm_quant_i8"
    m, k = _matrix_rows(fn, "x", x)
    dev, dt = x.device, x.dtype
    code = _dtype(fn, x)
    _check(fn, dev, ("gamma", gamma, torch.float32, (k,)), ("q", q, torch.int8, (m, k)), ("dq", dq, torch.float32, (m, k // BLOCK)))
    if res is not None:
        _check(fn, dev, ("res", res, dt, (m, k)))
    if res_out is not None:
        _check(fn, dev, ("res_out", res_out, dt, (m, k)))
    if y is not None:
        _check(fn, dev, ("y", y, dt, (m, k)))
    _launch(fn, dev, stream, x.data_ptr(), _ptr(res), gamma.data_ptr(), code, m, k, eps, _ptr(res_out), _ptr(y),
            q.data_ptr(), dq.data_ptr())


class Mxfp4:
    """Weights in microscaled 4-bit floating point: codes uint8 [n][k/2], scales uint8 [n][k/32]."""

    def __init__(self, codes, scales):
        import torch
        n, half = _matrix_rows("Mxfp4", "codes", codes)
        _check("Mxfp4", codes.device, ("codes", codes, torch.uint8, (n, half)), ("scales", scales, torch.uint8, (n, half // 16)))
        self.codes, self.scales, self.n, self.k, self.device = codes, scales, int(n), 2 * int(half), codes.device
        self.c = CMxfp4(codes.data_ptr(), scales.data_ptr(), self.n, self.k)

    @classmethod
    def quantise(cls, x, rotate: bool = False, stream=None) -> "Mxfp4":
        """The rows of x, quantised into new tensors, which belong to `stream`: another stream waits for it
        before it reads them."""
        import torch
        m, k = _matrix_rows("Mxfp4.quantise", "x", x)
        with _owned_by(stream, x.device):
            codes = torch.empty(m, k // 2, dtype=torch.uint8, device=x.device)
            scales = torch.empty(m, k // 32, dtype=torch.uint8, device=x.device)
        tb_mxfp4_quant(x, codes, scales, rotate, stream)
        return cls(codes, scales)


def tb_mxfp4_quant(x, codes, scales, rotate: bool = False, stream=None) -> None:
    """codes uint8 [m][k/2], scales uint8 [m][k/32] of the rows x [m][k] (rotated first, if asked)."""
    torch = _torch()
    fn = "tb_mxfp4_quant"
    m, k = _matrix_rows(fn, "x", x)
    code = _dtype(fn, x)
    _check(fn, x.device, ("codes", codes, torch.uint8, (m, k // 2)), ("scales", scales, torch.uint8, (m, k // 32)))
    _launch(fn, x.device, stream, x.data_ptr(), code, m, k, int(bool(rotate)), codes.data_ptr(), scales.data_ptr())


def tb_mxfp4_dequant(codes, scales, y, stream=None) -> None:
    """y [m][k] (float32, bfloat16 or float16) = the values that the codes stand for."""
    torch = _torch()
    fn = "tb_mxfp4_dequant"
    m, k = _matrix_rows(fn, "y", y)
    code = _dtype(fn, y)
    _check(fn, y.device, ("codes", codes, torch.uint8, (m, k // 2)), ("scales", scales, torch.uint8, (m, k // 32)))
    _launch(fn, y.device, stream, codes.data_ptr(), scales.data_ptr(), m, k, y.data_ptr(), code)


def tb_mxfp4_gemm_workspace_bytes(w: Mxfp4, m: int) -> int:
    """Bytes of device workspace tb_mxfp4_gemm needs for m rows."""
    return int(lib().tb_mxfp4_gemm_workspace_bytes(ctypes.byref(w.c), int(m)))


def tb_mxfp4_gemm(w: Mxfp4, codes, scales, y, ws=None, stream=None) -> None:
    """y [m][w.n] (float32, bfloat16 or float16) = the rows (codes, scales) times w's rows.

    ws: a uint8 workspace of tb_mxfp4_gemm_workspace_bytes(w, m) bytes, or None where that is 0."""
    torch = _torch()
    fn = "tb_mxfp4_gemm"
    m, n = _matrix_rows(fn, "y", y)
    code, dev = _dtype(fn, y), y.device
    if n != w.n or w.device != dev:
        _bad(fn, f"y has to have {w.n} columns, on {w.device}")
    _check(fn, dev, ("codes", codes, torch.uint8, (m, w.k // 2)), ("scales", scales, torch.uint8, (m, w.k // 32)))
    if ws is not None:
        _check(fn, dev, ("ws", ws, torch.uint8, (ws.numel(),)))
    _launch(fn, dev, stream, ctypes.byref(w.c), codes.data_ptr(), scales.data_ptr(), m, y.data_ptr(), code, _ptr(ws),
            0 if ws is None else ws.numel())


class Experts:
    """One projection of all experts of a layer: codes uint8 [experts][n][k/128][32 or 16], scales
    fp16 (or their bits as int16) [experts][n][k/128], fmt TB_FMT_TERNARY2 or TB_FMT_SIGN1."""

    def __init__(self, codes, scales, fmt: int):
        import torch
        fn = "Experts"
        if scales.dim() != 3 or not scales.is_cuda or scales.dtype not in (torch.float16, torch.int16):
            _bad(fn, "scales has to be a float16 (or int16) tensor [experts][n][k/128] on the GPU")
        if fmt not in (TB_FMT_TERNARY2, TB_FMT_SIGN1):
            _bad(fn, f"format {fmt}")
        e, n, nb = scales.shape
        _check(fn, scales.device, ("codes", codes, torch.uint8, (e, n, nb, 32 if fmt == TB_FMT_TERNARY2 else 16)),
               ("scales", scales, scales.dtype, (e, n, nb)))
        self.codes, self.scales, self.device = codes, scales, scales.device
        self.experts, self.n, self.k, self.fmt = int(e), int(n), int(nb) * BLOCK, int(fmt)
        self.c = CExperts(codes.data_ptr(), scales.data_ptr(), self.experts, self.n, self.k, self.fmt)

    @classmethod
    def upload(cls, packed, device="cuda") -> "Experts":
        """Copy host matrices (a list of synth.PackedMatrix of one shape and format) to the device."""
        import numpy as np
        import torch
        first = packed[0]
        nb = first.k // BLOCK
        codes = np.stack([p.codes.reshape(first.n, nb, -1) for p in packed])
        scales = np.stack([p.scales.reshape(first.n, nb) for p in packed])
        return cls(torch.from_numpy(codes).to(device), torch.from_numpy(scales.view("int16")).to(device), first.fmt)


def tb_moe_plan(ids, experts: int, offsets, order, stream=None) -> None:
    """Sort the pairs of ids int32 [tokens][topk] by expert: offsets int32 [experts + 1], order
    int32 [tokens * topk]. An id outside [0, experts) belongs to no expert."""
    torch = _torch()
    fn = "tb_moe_plan"
    t, topk = _matrix_rows(fn, "ids", ids)
    _check(fn, ids.device, ("ids", ids, torch.int32, (t, topk)), ("offsets", offsets, torch.int32, (experts + 1,)),
           ("order", order, torch.int32, (t * topk,)))
    _launch(fn, ids.device, stream, ids.data_ptr(), t, topk, experts, offsets.data_ptr(), order.data_ptr())


def tb_moe_gateup_silu(wg: Experts, wu: Experts, q, dq, topk: int, offsets, order, h, qh, dqh, stream=None) -> None:
    """qh, dqh = rotated int8 copy of silu(gate q) * (up q), a row per slot of the plan.

    q int8 [tokens][k], dq float32 [tokens][k/128]; h float32 [tokens * topk][n] is workspace; qh int8
    [tokens * topk][n], dqh float32 [tokens * topk][n/128]."""
    torch = _torch()
    fn = "tb_moe_gateup_silu"
    t, k = _matrix_rows(fn, "q", q)
    n, dev, p = wg.n, q.device, t * topk
    if k != wg.k or wg.device != dev or wu.device != dev:
        _bad(fn, f"q has to have {wg.k} columns, on {wg.device}")
    i32, f32 = torch.int32, torch.float32
    _check(fn, dev, ("q", q, torch.int8, (t, k)), ("dq", dq, f32, (t, k // BLOCK)), ("offsets", offsets, i32, (wg.experts + 1,)),
           ("order", order, i32, (p,)), ("h", h, f32, (p, n)), ("qh", qh, torch.int8, (p, n)), ("dqh", dqh, f32, (p, n // BLOCK)))
    _launch(fn, dev, stream, ctypes.byref(wg.c), ctypes.byref(wu.c), q.data_ptr(), dq.data_ptr(), t, topk,
            offsets.data_ptr(), order.data_ptr(), h.data_ptr(), qh.data_ptr(), dqh.data_ptr())


def tb_moe_down(wd: Experts, qh, dqh, offsets, order, y, stream=None) -> None:
    """y float32 [tokens * topk][n] = down product of the plan's slots, a row per pair."""
    torch = _torch()
    fn = "tb_moe_down"
    p, k = _matrix_rows(fn, "qh", qh)
    dev = qh.device
    if k != wd.k or wd.device != dev:
        _bad(fn, f"qh has to have {wd.k} columns, on {wd.device}")
    i32, f32 = torch.int32, torch.float32
    _check(fn, dev, ("qh", qh, torch.int8, (p, k)), ("dqh", dqh, f32, (p, k // BLOCK)), ("offsets", offsets, i32, (wd.experts + 1,)),
           ("order", order, i32, (p,)), ("y", y, f32, (p, wd.n)))
    _launch(fn, dev, stream, ctypes.byref(wd.c), qh.data_ptr(), dqh.data_ptr(), p, offsets.data_ptr(), order.data_ptr(),
            y.data_ptr())


def tb_moe_combine(y, weights, ids, experts: int, out, stream=None) -> None:
    """out [tokens][n] (float32, bfloat16 or float16) = each token's pairs, weighted and summed."""
    torch = _torch()
    fn = "tb_moe_combine"
    t, topk = _matrix_rows(fn, "ids", ids)
    code, n, dev = _dtype(fn, out), int(out.shape[-1]), ids.device
    _check(fn, dev, ("y", y, torch.float32, (t * topk, n)), ("weights", weights, torch.float32, (t, topk)),
           ("ids", ids, torch.int32, (t, topk)), ("out", out, out.dtype, (t, n)))
    _launch(fn, dev, stream, y.data_ptr(), weights.data_ptr(), ids.data_ptr(), t, topk, experts, n, out.data_ptr(), code)
