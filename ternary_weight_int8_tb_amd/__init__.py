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
ABI_VERSION = 8
TB_F32, TB_BF16, TB_F16 = 0, 1, 2
TB_ROPE_HALF, TB_ROPE_INTERLEAVED = 0, 1

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
               "tb_kv_plan", "tb_rope_kv", "tb_attn_paged", "tb_attn_paged_workspace_bytes",
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


class CKvCache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("pages", ctypes.c_int32), ("kv_heads", ctypes.c_int32),
                ("page", ctypes.c_int32), ("dim", ctypes.c_int32), ("dtype", ctypes.c_int32)]


class CHeads(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("row_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64),
                ("heads", ctypes.c_int32), ("dtype", ctypes.c_int32)]


class CRope(ctypes.Structure):
    _fields_ = [("freq", ctypes.c_void_p), ("rot", ctypes.c_int32), ("layout", ctypes.c_int32), ("factor", ctypes.c_float)]


_P = ctypes.c_void_p
_I = ctypes.c_int
_XP = ctypes.POINTER(CMxfp4)
_EP = ctypes.POINTER(CExperts)
_MP = ctypes.POINTER(CMatrix)
_CP = ctypes.POINTER(CKvCache)
_HP = ctypes.POINTER(CHeads)
_RP = ctypes.POINTER(CRope)
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
    "tb_kv_plan": ([_P, _P, _I, _I, _I, _I, _P, _I, _P, _P, _P, _P, _P, _P, _P, _P, _P], _I),
    "tb_rope_kv": ([_HP, _HP, _HP, _I, _I, _RP, _P, _P, _CP, _P, _I, _P], _I),
    "tb_attn_paged": ([_HP, _HP, _CP, _P, _I, _P, _P, _I, _I, ctypes.c_float, _I, _P, _P, ctypes.c_size_t, _P], _I),
    "tb_attn_paged_workspace_bytes": ([_CP, _I, _I, _I, _I], ctypes.c_size_t),
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


def _int32(fn: str, name: str, v: int) -> int:
    """v, refused where 32 bits do not hold it: ctypes would cut it off."""
    if not -1 << 31 <= v < 1 << 31:
        _bad(fn, f"{name} = {v}")
    return v


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
    _launch(fn, dev, stream, y.data_ptr(), weights.data_ptr(), ids.data_ptr(), t, topk, _int32(fn, "experts", experts), n, out.data_ptr(), code)


# ---- attention over a paged cache ---------------------------------------------------------
class KvCache:
    """A paged cache of one layer: k, v bfloat16 or float16 [pages][kv_heads][page][dim]; page is 16, 32, 64, 128 or 256."""

    def __init__(self, k, v):
        fn = "KvCache"
        if k.dim() != 4 or not k.is_cuda or not k.is_contiguous() or k.dtype not in (_torch().bfloat16, _torch().float16):
            _bad(fn, "k has to be a contiguous bfloat16 or float16 tensor [pages][kv_heads][page][dim] on the GPU")
        _check(fn, k.device, ("v", v, k.dtype, k.shape))
        self.k, self.v, self.device = k, v, k.device
        self.pages, self.kv_heads, self.page, self.dim = (int(n) for n in k.shape)
        self.dtype = _dtype(fn, k)
        self.c = CKvCache(k.data_ptr(), v.data_ptr(), self.pages, self.kv_heads, self.page, self.dim, self.dtype)
        self.ref = ctypes.byref(self.c)


class Rope:
    """Rotary positions: freq float64 [rot/2], radians per position of each pair, on the GPU; layout TB_ROPE_HALF or
    TB_ROPE_INTERLEAVED; factor multiplies what is turned."""

    def __init__(self, freq, layout: int = TB_ROPE_HALF, factor: float = 1.0):
        fn = "Rope"
        if freq.dim() != 1 or not freq.is_cuda:
            _bad(fn, "freq has to be a float64 vector on the GPU")
        _check(fn, freq.device, ("freq", freq, _torch().float64, freq.shape))
        self.freq, self.device, self.rot, self.layout, self.factor = freq, freq.device, 2 * int(freq.shape[0]), _int32(fn, "layout", int(layout)), float(factor)
        self.c = CRope(freq.data_ptr(), self.rot, self.layout, self.factor)
        self.ref = ctypes.byref(self.c)

    @staticmethod
    def frequencies(rot: int, base: float = 10000.0, scaling: str = "none", stretch: float = 1.0, trained: float = 0.0,
                    slow: float = 1.0, fast: float = 32.0):
        """(freq float64 [rot/2] on the CPU, factor) of base^(-2i/rot), scaled for contexts `stretch` times as long as the
        trained length:

        "none"    not at all
        "linear"  every pair is slowed by stretch
        "base"    the base is raised, so that the slowest pair is slowed by stretch and the fastest is kept
        "parts"   pairs that turn less than `slow` times over the trained length are slowed by stretch, those that turn more
                  than `fast` times are kept, those between are mixed in proportion to their turns; factor = 0.1 ln(stretch) + 1

        A checkpoint may want another rule: pairs mixed in proportion to their index between the two bounds (the middle pair of
        128 elements then differs by a factor of 1.7 at base 1e6 and stretch 4), or a factor of 1. Its frequencies and factor go
        to Rope(freq, layout, factor) as they are."""
        import math
        import torch
        fn = "Rope.frequencies"
        if rot < 2 or rot % 2 or not base > 0 or not stretch > 0:
            _bad(fn, f"rot {rot}, base {base}, stretch {stretch}")
        if scaling == "base":
            base *= stretch ** (rot / (rot - 2)) if rot > 2 else 1.0
        f = base ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
        if scaling in ("none", "base"):
            return f, 1.0
        if scaling == "linear":
            return f / stretch, 1.0
        if scaling != "parts" or not trained > 0 or not fast > slow:
            _bad(fn, f"scaling {scaling!r}, trained {trained}, slow {slow}, fast {fast}")
        keep = ((trained * f / (2 * math.pi) - slow) / (fast - slow)).clamp(0, 1)
        return f * (keep + (1 - keep) / stretch), 0.1 * math.log(stretch) + 1 if stretch > 1 else 1.0

    @classmethod
    def make(cls, rot: int, layout: int = TB_ROPE_HALF, device="cuda", **scaling) -> "Rope":
        """frequencies(rot, **scaling) on the device."""
        freq, factor = cls.frequencies(rot, **scaling)
        return cls(freq.to(device), layout, factor)


def _heads(fn: str, name: str, t, device, rows: int, dim: int):
    """A view [rows][heads][dim] of wider rows as a tb_heads."""
    shape, stride = t.shape, t.stride()
    if len(shape) != 3 or shape[0] != rows or shape[2] != dim or stride[2] != 1 or t.get_device() != device.index:
        _bad(fn, f"{name} has to be a tensor [{rows}][heads][{dim}] on {device} with consecutive elements of a head")
    return CHeads(t.data_ptr(), stride[0], stride[1], shape[1], _dtype(fn, t))


def tb_kv_plan(context, fresh, page: int, pages: int, table, free_list, count, lengths, offsets, positions, slots, left, missing,
               stream=None) -> None:
    """Block tables and slots of a step (int32 tensors).

    context, fresh [requests] (fresh -1: the request has ended), table [requests][width] and free_list [pages] updated,
    count [1] -> lengths [requests] (may be context), offsets [requests + 1], positions, slots [rows], left [1] (may be
    count), missing [1]. Where missing > 0, put a request's length back to the position of its first row with slot -1, and
    bring the tokens from there on again when there are pages."""
    fn = "tb_kv_plan"
    n, width = _matrix_rows(fn, "table", table)
    dev, i32 = table.device, _torch().int32
    if positions.dim() != 1:
        _bad(fn, "positions has to be a vector")
    rows = positions.shape[0]
    _check(fn, dev, ("table", table, i32, (n, width)), ("context", context, i32, (n,)), ("fresh", fresh, i32, (n,)),
           ("free_list", free_list, i32, (pages,)), ("count", count, i32, (1,)), ("lengths", lengths, i32, (n,)),
           ("offsets", offsets, i32, (n + 1,)), ("positions", positions, i32, (rows,)), ("slots", slots, i32, (rows,)),
           ("left", left, i32, (1,)), ("missing", missing, i32, (1,)))
    _launch(fn, dev, stream, context.data_ptr(), fresh.data_ptr(), n, rows, _int32(fn, "page", page), pages, table.data_ptr(), width, free_list.data_ptr(),
            count.data_ptr(), lengths.data_ptr(), offsets.data_ptr(), positions.data_ptr(), slots.data_ptr(), left.data_ptr(),
            missing.data_ptr())


def tb_rope_kv(q, k, v, rope: Rope | None, positions, slots, cache: KvCache | None, q_out, stream=None) -> None:
    """q_out [tokens][heads][dim] = the rotated rows of q; those of k, and v as they are, into the cache's slots.

    q, k, v [tokens][heads][dim] of one type (float32, bfloat16, float16), views of wider rows as they come; positions,
    slots int32 [tokens] from tb_kv_plan. q and q_out, or k, v, slots and cache, may be None; rope None: nothing is turned."""
    fn = "tb_rope_kv"
    x = q if q is not None else k
    if x is None or x.dim() != 3 or (q is None) != (q_out is None):
        _bad(fn, "q has to be a tensor [tokens][heads][dim], with q_out, or None in both places")
    dev, i32 = x.device, _torch().int32
    t, dim = x.shape[0], x.shape[2]
    _check(fn, dev, ("positions", positions, i32, (t,)))
    hq = hk = hv = None
    code = 0
    if q is not None:
        hq, code = ctypes.byref(_heads(fn, "q", q, dev, t, dim)), _dtype(fn, q_out)
        _check(fn, dev, ("q_out", q_out, q_out.dtype, q.shape))
    if k is not None or v is not None or slots is not None or cache is not None:
        if k is None or v is None or slots is None or cache is None:
            _bad(fn, "k, v, slots and cache come together")
        if cache.device != dev:
            _bad(fn, f"the cache is on {cache.device}, the rows on {dev}")
        hk, hv = ctypes.byref(_heads(fn, "k", k, dev, t, dim)), ctypes.byref(_heads(fn, "v", v, dev, t, dim))
        _check(fn, dev, ("slots", slots, i32, (t,)))
    if rope is not None and rope.device != dev:
        _bad(fn, f"freq is on {rope.device}, the rows on {dev}")
    _launch(fn, dev, stream, hq, hk, hv, t, dim, None if rope is None else rope.ref, positions.data_ptr(), _ptr(slots),
            None if cache is None else cache.ref, _ptr(q_out), code)


def tb_attn_paged_workspace_bytes(cache: KvCache, heads: int, dtype, requests: int, tokens: int) -> int:
    """Bytes of device workspace tb_attn_paged needs for q rows of a torch dtype, with at most these requests and tokens."""
    torch = _torch()
    code = {torch.float32: TB_F32, torch.bfloat16: TB_BF16, torch.float16: TB_F16}.get(dtype, -1)
    sizes = (int(heads), code, int(requests), int(tokens))
    return int(lib().tb_attn_paged_workspace_bytes(cache.ref, *sizes)) if max(sizes) < 1 << 31 else 0


def tb_attn_paged(q, cache: KvCache, table, offsets, lengths, scale: float, out, ws, gate=None, window: int = 0, stream=None) -> None:
    """out [tokens][heads][dim] = attention of each request's rows (offsets[s] .. offsets[s+1] - 1, the last of its lengths[s]
    tokens) over its pages, times sigmoid(gate).

    q [tokens][heads][dim], float32 or the cache's type (a view of wider rows as it comes), and gate alike, of any type; table
    int32 [requests][width], offsets int32 [requests + 1], lengths int32 [requests]; ws a uint8 workspace of
    tb_attn_paged_workspace_bytes bytes."""
    torch = _torch()
    fn = "tb_attn_paged"
    n, width = _matrix_rows(fn, "table", table)
    if q.dim() != 3:
        _bad(fn, "q has to be a tensor [tokens][heads][dim]")
    dev, i32, dim = cache.device, torch.int32, cache.dim
    t, heads = q.shape[0], q.shape[1]
    _check(fn, dev, ("table", table, i32, (n, width)), ("offsets", offsets, i32, (n + 1,)), ("lengths", lengths, i32, (n,)),
           ("out", out, q.dtype, (t, heads, dim)), ("ws", ws, torch.uint8, (ws.numel(),)))
    hq = _heads(fn, "q", q, dev, t, dim)
    hg = None
    if gate is not None:
        hg = ctypes.byref(_heads(fn, "gate", gate, dev, t, dim))
    _launch(fn, dev, stream, ctypes.byref(hq), hg, cache.ref, table.data_ptr(), width, offsets.data_ptr(), lengths.data_ptr(), n, t, scale,
            _int32(fn, "window", window), out.data_ptr(), ws.data_ptr(), ws.numel())
