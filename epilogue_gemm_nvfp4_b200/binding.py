"""ctypes binding of libnvfp4 (the C ABI in include/nvfp4.h): argument marshalling only.

Every step of the NVFP4 path runs in the library's CUDA kernels; this module
turns torch tensors into the C structs (device pointers, sizes, the current
CUDA stream) and raises when the library reports an error.  There is no CPU
fallback: if the shared library is missing, ``load()`` raises.
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libnvfp4.so")

#: every function the header declares
EXPORTS = ("nvfp4_quantize", "nvfp4_linear", "nvfp4_dequantize", "nvfp4_amax", "nvfp4_scale_bytes",
           "nvfp4_scale_offset", "nvfp4_get_device_error", "nvfp4_linear_tile_n", "nvfp4_linear_split_k",
           "nvfp4_status_string", "nvfp4_version", "nvfp4_linear_noalloc", "nvfp4_linear_noalloc_scratch_bytes",
           "nvfp4_fake_quantize", "nvfp4_adaln_quantize", "nvfp4_int8_quantize", "nvfp4_int8_linear",
           "nvfp4_w4a16_linear", "nvfp4_w4a16_workspace_bytes", "nvfp4_qk_norm_rope",
           "nvfp4_cross_attention")

OK, ERR_INVALID_ARG, ERR_UNSUPPORTED_SHAPE, ERR_MISALIGNED, ERR_CUDA, ERR_DEVICE_TIMEOUT, ERR_SCRATCH_LIMIT = range(7)
EPI_BIAS, EPI_QKNORM, EPI_GATED_SILU, EPI_RESID_GATE = range(4)
EPI_KINDS = {"bias": EPI_BIAS, "qknorm": EPI_QKNORM, "gated_silu": EPI_GATED_SILU, "resid_gate": EPI_RESID_GATE}


class CTensor(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("tensor_scale", ctypes.c_void_p),
                ("rows", ctypes.c_int64), ("cols", ctypes.c_int64), ("ld_codes", ctypes.c_int64)]


class CEpilogue(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int32), ("bias", ctypes.c_void_p), ("gamma_q", ctypes.c_void_p),
                ("gamma_k", ctypes.c_void_p), ("eps", ctypes.c_float), ("head_dim", ctypes.c_int32),
                ("q_col0", ctypes.c_int64), ("k_col0", ctypes.c_int64), ("qk_cols", ctypes.c_int64),
                ("residual", ctypes.c_void_p), ("ld_residual", ctypes.c_int64), ("gate", ctypes.c_void_p),
                ("out_nvfp4", ctypes.c_int32), ("out_amax", ctypes.c_void_p)]


class CAdaln(ctypes.Structure):
    _fields_ = [("shift", ctypes.c_void_p), ("scale", ctypes.c_void_p), ("ld_mod", ctypes.c_int64),
                ("rows_per_sample", ctypes.c_int64), ("eps", ctypes.c_float), ("rstd", ctypes.c_void_p),
                ("u_out", ctypes.c_void_p), ("ld_u", ctypes.c_int64)]


class CInt8Tensor(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("scale", ctypes.c_void_p), ("rows", ctypes.c_int64), ("cols", ctypes.c_int64),
                ("ld", ctypes.c_int64)]


class CHeads(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p), ("row_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64),
                ("out", ctypes.c_void_p), ("out_row_stride", ctypes.c_int64), ("out_head_stride", ctypes.c_int64),
                ("heads", ctypes.c_int32), ("gamma", ctypes.c_void_p)]


class CRope(ctypes.Structure):
    _fields_ = [("cos", ctypes.c_void_p), ("sin", ctypes.c_void_p), ("table_rows", ctypes.c_int64),
                ("ld_table", ctypes.c_int64), ("rot_dim", ctypes.c_int32), ("interleaved", ctypes.c_int32),
                ("positions", ctypes.c_void_p), ("eps", ctypes.c_float)]


class CAttention(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("out", ctypes.c_void_p),
                ("batch", ctypes.c_int64), ("q_len", ctypes.c_int64), ("kv_len", ctypes.c_int64),
                ("heads", ctypes.c_int32), ("kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("scale", ctypes.c_float)] + [
                    (f"{t}_{what}_stride", ctypes.c_int64) for t in ("q", "k", "v", "out")
                    for what in ("batch", "row", "head")] + [("kv_lens", ctypes.c_void_p), ("lse", ctypes.c_void_p)]


class NvFp4Error(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {status_string(status)} (status {status})")


_lib = None


def load() -> ctypes.CDLL:
    """Load libnvfp4.so (in-tree).  Raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is missing: build it with `python -m epilogue_gemm_nvfp4_b200.build`")
    lib = ctypes.CDLL(LIB_PATH)
    P, I64, I32, SZ = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_size_t
    TP = ctypes.POINTER(CTensor)
    EP = ctypes.POINTER(CEpilogue)
    AP = ctypes.POINTER(CAdaln)
    IP = ctypes.POINTER(CInt8Tensor)
    HP = ctypes.POINTER(CHeads)
    RP = ctypes.POINTER(CRope)
    sig = {
        "nvfp4_quantize": (I32, [P, I64, I64, I64, I32, TP, P]),
        "nvfp4_linear": (I32, [TP, TP, EP, P, I64, TP, P]),
        "nvfp4_linear_noalloc": (I32, [TP, TP, EP, P, I64, TP, P]),
        "nvfp4_linear_noalloc_scratch_bytes": (SZ, []),
        "nvfp4_dequantize": (I32, [TP, P, I64, P]),
        "nvfp4_fake_quantize": (I32, [P, I64, I64, I64, I32, P, P, I64, P]),
        "nvfp4_adaln_quantize": (I32, [P, I64, I64, I64, AP, I32, TP, P]),
        "nvfp4_int8_quantize": (I32, [P, I64, I64, I64, P, IP, P]),
        "nvfp4_int8_linear": (I32, [IP, IP, EP, P, I64, TP, P]),
        "nvfp4_w4a16_linear": (I32, [P, I64, I64, I32, TP, EP, P, I64, P, SZ, P]),
        "nvfp4_w4a16_workspace_bytes": (SZ, [I64, I64, I64]),
        "nvfp4_cross_attention": (I32, [ctypes.POINTER(CAttention), P]),
        "nvfp4_qk_norm_rope": (I32, [HP, HP, I64, I32, RP, P]),
        "nvfp4_amax": (I32, [P, I64, I64, I64, P, P]),
        "nvfp4_scale_bytes": (SZ, [I64, I64]),
        "nvfp4_scale_offset": (I64, [I64, I64, I64]),
        "nvfp4_get_device_error": (I32, [P]),
        "nvfp4_linear_tile_n": (I32, [I64, I64, I32]),
        "nvfp4_linear_split_k": (I32, [I64, I64, I32]),
        "nvfp4_status_string": (ctypes.c_char_p, [I32]),
        "nvfp4_version": (I32, []),
    }
    for name, (res, args) in sig.items():
        f = getattr(lib, name)
        f.restype, f.argtypes = res, args
    _lib = lib
    return lib


def status_string(status: int) -> str:
    return load().nvfp4_status_string(status).decode()


def _check(status: int, what: str):
    if status != OK:
        raise NvFp4Error(status, what)


def _stream(stream=None):
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


# ------------------------------------------------------------------------------------------
# NVFP4 tensor held in torch device memory
# ------------------------------------------------------------------------------------------

@dataclass
class QTensor:
    """An NVFP4 tensor: packed codes uint8 [rows, cols/2], padded scale bytes, fp32 decode scale [1]."""
    codes: torch.Tensor
    scales: torch.Tensor
    g: torch.Tensor
    rows: int
    cols: int

    @classmethod
    def empty(cls, rows: int, cols: int, device="cuda") -> "QTensor":
        lib = load()
        nbytes = int(lib.nvfp4_scale_bytes(rows, cols))
        return cls(torch.empty((rows, cols // 2), dtype=torch.uint8, device=device),
                   torch.empty(nbytes, dtype=torch.uint8, device=device),
                   torch.empty(1, dtype=torch.float32, device=device), rows, cols)

    def c(self) -> CTensor:
        return CTensor(self.codes.data_ptr(), self.scales.data_ptr(), self.g.data_ptr(), self.rows, self.cols,
                       self.codes.stride(0))


def scale_bytes(rows: int, cols: int) -> int:
    return int(load().nvfp4_scale_bytes(rows, cols))


def scale_offset(r: int, kb: int, cols: int) -> int:
    return int(load().nvfp4_scale_offset(r, kb, cols))


def tile_n(N: int, K: int, kind: str) -> int:
    return int(load().nvfp4_linear_tile_n(N, K, EPI_KINDS[kind]))


def split_k(N: int, K: int, kind: str) -> int:
    return int(load().nvfp4_linear_split_k(N, K, EPI_KINDS[kind]))


def quantize(x: torch.Tensor, out: QTensor | None = None, g: float | torch.Tensor | None = None,
             static: bool = False, stream=None) -> QTensor:
    """bf16 [rows, cols] (CUDA) -> NVFP4.  By default the tensor scale is computed on the device.
    With ``g`` the given decode scale is stored in out.g and used; with ``static=True`` the scale
    already held in out.g is used."""
    assert x.is_cuda and x.dtype == torch.bfloat16 and x.dim() == 2 and x.stride(1) == 1
    rows, cols = x.shape
    out = QTensor.empty(rows, cols, x.device) if out is None else out
    if g is not None:
        out.g.copy_(torch.as_tensor(g, dtype=torch.float32).reshape(1))
    compute = g is None and not static
    ct = out.c()
    _check(load().nvfp4_quantize(_ptr(x), rows, cols, x.stride(0), int(compute), ctypes.byref(ct),
                                 _stream(stream)), "nvfp4_quantize")
    return out


def fake_quantize(x: torch.Tensor, y: torch.Tensor | None = None, g: float | torch.Tensor | None = None,
                  scale: torch.Tensor | None = None, static: bool = False,
                  stream=None) -> tuple[torch.Tensor, torch.Tensor]:
    """y = dequantize(quantize(x)) in bf16, one pass.  By default g is computed on the device and
    returned in ``scale`` (one fp32 element); with ``g`` the given decode scale is stored there and
    used; with ``static=True`` the value already in ``scale`` is used."""
    assert x.is_cuda and x.dtype == torch.bfloat16 and x.dim() == 2 and x.stride(1) == 1
    rows, cols = x.shape
    y = torch.empty((rows, cols), dtype=torch.bfloat16, device=x.device) if y is None else y
    scale = torch.empty(1, dtype=torch.float32, device=x.device) if scale is None else scale
    if g is not None:
        scale.copy_(torch.as_tensor(g, dtype=torch.float32).reshape(1))
    compute = g is None and not static
    _check(load().nvfp4_fake_quantize(_ptr(x), rows, cols, x.stride(0), int(compute), _ptr(scale), _ptr(y),
                                      y.stride(0), _stream(stream)), "nvfp4_fake_quantize")
    return y, scale


def adaln_quantize(x: torch.Tensor, shift: torch.Tensor | None = None, scale: torch.Tensor | None = None,
                   eps: float = 1e-6, rows_per_sample: int = 0, out: QTensor | None = None,
                   g: float | torch.Tensor | None = None, static: bool = False, rstd: torch.Tensor | None = None,
                   u_out: torch.Tensor | None = None, stream=None) -> QTensor:
    """NVFP4 of u = bf16(RMSNorm(x) * (1 + scale) + shift) through nvfp4_adaln_quantize.  shift / scale are
    bf16 [cols] or [samples, cols] (row r uses sample r // rows_per_sample).  The tensor scale follows
    ``quantize``: computed on the device by default, ``g`` given, or ``static`` (out.g as it is).
    ``rstd`` (fp32 [rows]) and ``u_out`` (bf16 [rows, cols]) receive the per-row 1/rms and u when given."""
    assert x.is_cuda and x.dtype == torch.bfloat16 and x.dim() == 2 and x.stride(1) == 1
    rows, cols = x.shape
    out = QTensor.empty(rows, cols, x.device) if out is None else out
    if g is not None:
        out.g.copy_(torch.as_tensor(g, dtype=torch.float32).reshape(1))
    compute = g is None and not static
    mods = [m for m in (shift, scale) if m is not None]
    for m in mods:
        assert m.is_cuda and m.dtype == torch.bfloat16 and m.stride(-1) == 1 and m.shape[-1] == cols
    samples = 1 if rows_per_sample <= 0 or rows_per_sample >= rows else -(-rows // rows_per_sample)
    ld_mod = cols
    if mods:
        dims = {m.dim() for m in mods}
        assert dims in ({1}, {2}), "shift and scale are both [cols] or both [samples, cols]"
        if dims == {2}:
            ld_mod = mods[0].stride(0)
            assert all(m.stride(0) == ld_mod and m.shape[0] >= samples for m in mods), \
                "shift and scale need the same sample stride and one row per sample"
        else:
            assert samples == 1, "per-sample modulation needs [samples, cols] vectors"
    desc = CAdaln(_ptr(shift), _ptr(scale), int(ld_mod), int(rows_per_sample), float(eps), _ptr(rstd),
                  _ptr(u_out), u_out.stride(0) if u_out is not None else 0)
    ct = out.c()
    _check(load().nvfp4_adaln_quantize(_ptr(x), rows, cols, x.stride(0), ctypes.byref(desc), int(compute),
                                       ctypes.byref(ct), _stream(stream)), "nvfp4_adaln_quantize")
    return out


def dequantize(q: QTensor, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    out = torch.empty((q.rows, q.cols), dtype=torch.bfloat16, device=q.codes.device) if out is None else out
    ct = q.c()
    _check(load().nvfp4_dequantize(ctypes.byref(ct), _ptr(out), out.stride(0), _stream(stream)), "nvfp4_dequantize")
    return out


def amax(x: torch.Tensor, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    out = torch.empty(1, dtype=torch.float32, device=x.device) if out is None else out
    rows, cols = x.shape
    _check(load().nvfp4_amax(_ptr(x), rows, cols, x.stride(0), _ptr(out), _stream(stream)), "nvfp4_amax")
    return out


def make_epilogue(kind: str = "bias", bias=None, gamma_q=None, gamma_k=None, eps=1e-6, q_col0=0, k_col0=0,
                  qk_cols=0, head_dim=256, residual=None, gate=None, out_nvfp4=False, out_amax=None) -> CEpilogue:
    """``out_amax``: fp32 device tensor of one element (zeroed by the caller) that the kernel raises to
    max |bf16 output|."""
    return CEpilogue(EPI_KINDS[kind], _ptr(bias), _ptr(gamma_q), _ptr(gamma_k), float(eps), int(head_dim),
                     int(q_col0), int(k_col0), int(qk_cols), _ptr(residual),
                     residual.stride(0) if residual is not None else 0, _ptr(gate), int(bool(out_nvfp4)),
                     _ptr(out_amax))


def linear(a: QTensor, w: QTensor, kind: str = "bias", bias=None, out: torch.Tensor | None = None,
           out_fp4: QTensor | None = None, want_bf16: bool = True, stream=None, **epi) -> torch.Tensor | None:
    """Fused NVFP4 linear through nvfp4_linear.  ``out_fp4`` (with its g set) turns on the NVFP4
    re-quantisation of the output; ``want_bf16=False`` skips the bf16 output then."""
    n_out = w.rows // 2 if kind == "gated_silu" else w.rows
    if out is None and want_bf16:
        out = torch.empty((a.rows, n_out), dtype=torch.bfloat16, device=a.codes.device)
    desc = make_epilogue(kind, bias=bias, out_nvfp4=out_fp4 is not None, **epi)
    ca, cw = a.c(), w.c()
    cq = out_fp4.c() if out_fp4 is not None else None
    _check(load().nvfp4_linear(ctypes.byref(ca), ctypes.byref(cw), ctypes.byref(desc), _ptr(out),
                               out.stride(0) if out is not None else 0,
                               ctypes.byref(cq) if cq is not None else None, _stream(stream)), "nvfp4_linear")
    return out


# ------------------------------------------------------------------------------------------
# W8A8 INT8 path
# ------------------------------------------------------------------------------------------

@dataclass
class Int8Tensor:
    """Per-row INT8: codes int8 [rows, cols] and the fp32 decode scale of each row [rows]."""
    q: torch.Tensor
    scale: torch.Tensor
    rows: int
    cols: int

    @classmethod
    def empty(cls, rows: int, cols: int, device="cuda") -> "Int8Tensor":
        return cls(torch.empty((rows, cols), dtype=torch.int8, device=device),
                   torch.empty(max(rows, 1), dtype=torch.float32, device=device), rows, cols)

    def c(self) -> CInt8Tensor:
        return CInt8Tensor(self.q.data_ptr(), self.scale.data_ptr(), self.rows, self.cols, self.q.stride(0))


def int8_quantize(x: torch.Tensor, col_mult: torch.Tensor | None = None, out: Int8Tensor | None = None,
                  stream=None) -> Int8Tensor:
    """bf16 [rows, cols] -> per-row INT8 through nvfp4_int8_quantize; ``col_mult`` (fp32 [cols]) multiplies
    each column first (1 / lambda for activations, lambda for a weight under SmoothQuant)."""
    assert x.is_cuda and x.dtype == torch.bfloat16 and x.dim() == 2 and x.stride(1) == 1
    rows, cols = x.shape
    if col_mult is not None:
        assert col_mult.is_cuda and col_mult.dtype == torch.float32 and col_mult.numel() == cols
    out = Int8Tensor.empty(rows, cols, x.device) if out is None else out
    ct = out.c()
    _check(load().nvfp4_int8_quantize(_ptr(x), rows, cols, x.stride(0), _ptr(col_mult), ctypes.byref(ct),
                                      _stream(stream)), "nvfp4_int8_quantize")
    return out


def int8_linear(a: Int8Tensor, w: Int8Tensor, kind: str = "bias", bias=None, out: torch.Tensor | None = None,
                out_fp4: QTensor | None = None, want_bf16: bool = True, stream=None, **epi) -> torch.Tensor | None:
    """Fused W8A8 linear through nvfp4_int8_linear (the epilogue arguments of ``linear``)."""
    n_out = w.rows // 2 if kind == "gated_silu" else w.rows
    if out is None and want_bf16:
        out = torch.empty((a.rows, n_out), dtype=torch.bfloat16, device=a.q.device)
    desc = make_epilogue(kind, bias=bias, out_nvfp4=out_fp4 is not None, **epi)
    ca, cw = a.c(), w.c()
    cq = out_fp4.c() if out_fp4 is not None else None
    _check(load().nvfp4_int8_linear(ctypes.byref(ca), ctypes.byref(cw), ctypes.byref(desc), _ptr(out),
                                    out.stride(0) if out is not None else 0,
                                    ctypes.byref(cq) if cq is not None else None, _stream(stream)),
           "nvfp4_int8_linear")
    return out


# ------------------------------------------------------------------------------------------
# around the linears of a block: few-row products, head norm + rotation
# ------------------------------------------------------------------------------------------

# These calls take a few microseconds on the device, so their marshalling is kept to what it needs.

def _here(stream, t: torch.Tensor):
    """The context of a call on t's device when it needs one: that device current, and ``stream`` (when one is
    given) the current stream, so that what the call allocates belongs to the stream it runs on."""
    if not t.is_cuda:
        raise ValueError("the call's tensors are CUDA tensors")
    if stream is not None:
        if stream.device.index != t.get_device():
            raise ValueError(f"stream: of {stream.device}, the call's tensors are on cuda:{t.get_device()}")
        return torch.cuda.stream(stream)
    if t.get_device() != _current_device():
        return torch.cuda.device(t.device)
    return None


_current_device = torch._C._cuda_getDevice if hasattr(torch._C, "_cuda_getDevice") else torch.cuda.current_device


def _raw_stream(t: torch.Tensor) -> int:
    return torch._C._cuda_getCurrentRawStream(t.get_device())


def _require(t, what, dtype, device, shape=None):
    """Argument check: ``dtype``, on CUDA device number ``device``, unit stride along the last dimension, ``shape``."""
    if t is None or t.dtype is not dtype or t.get_device() != device or (t.dim() and t.stride(-1) != 1 and t.shape[-1] > 1) or (
            shape is not None and t.shape != shape):
        raise ValueError(f"{what}: {dtype} on one CUDA device with the call's other tensors"
                         + (f", shape {tuple(shape)}" if shape is not None else "")
                         + ", unit stride along the last dimension")


def w4a16_linear(x: torch.Tensor, w: QTensor, kind: str = "bias", bias=None, silu_input: bool = False,
                 out: torch.Tensor | None = None, residual=None, gate=None, stream=None) -> torch.Tensor:
    """Linear of up to 32 bf16 rows on an NVFP4 weight through nvfp4_w4a16_linear: x (or silu(x) with
    ``silu_input``) is rounded to 2^-17 of the largest of each 16 elements, not to NVFP4.  ``kind`` is "bias",
    "gated_silu" or "resid_gate"."""
    here = _here(stream, x)
    if here is not None:
        with here:
            return w4a16_linear(x, w, kind, bias, silu_input, out, residual, gate)
    dev = x.get_device()
    N, K = w.rows, w.cols
    if x.dim() != 2 or x.shape[1] != K:
        raise ValueError("x: [rows, K] with the weight's K")
    _require(x, "x", torch.bfloat16, dev)
    _require(w.codes, "w.codes", torch.uint8, dev)
    _require(w.scales, "w.scales", torch.uint8, dev)
    _require(w.g, "w.g", torch.float32, dev)
    if w.codes.dim() != 2 or w.codes.shape[0] < N or w.codes.shape[1] < K // 2 or (N > 1 and w.codes.stride(0) < K // 2) or (
            w.scales.numel() < 512 * (-(-N // 128) * -(-K // 64)) or not w.scales.is_contiguous()):
        raise ValueError("w: codes [rows, cols / 2] whose rows do not overlap, and the scale bytes of its rows and columns")
    M = x.shape[0]
    n_out = N // 2 if kind == "gated_silu" else N
    if kind not in ("bias", "gated_silu", "resid_gate"):
        raise ValueError(f"kind {kind!r}: bias, gated_silu or resid_gate")
    if kind != "resid_gate" and (residual is not None or gate is not None):
        raise ValueError("residual and gate belong to kind resid_gate")
    desc = CEpilogue(EPI_KINDS[kind])
    if bias is not None:
        _require(bias, "bias", torch.bfloat16, dev, (N,))
        desc.bias = bias.data_ptr()
    if kind == "resid_gate":
        _require(residual, "residual", torch.bfloat16, dev, (M, n_out))
        _require(gate, "gate", torch.float32, dev, (n_out,))
        desc.residual, desc.ld_residual, desc.gate = residual.data_ptr(), _ld(residual), gate.data_ptr()
    if out is None:
        out = x.new_empty((M, n_out))
    else:
        _require(out, "out", torch.bfloat16, dev, (M, n_out))
    lib = load()
    nbytes = lib.nvfp4_w4a16_workspace_bytes(M, N, K)
    ws = w.codes.new_empty(nbytes)
    status = lib.nvfp4_w4a16_linear(x.data_ptr(), M, _ld(x), silu_input, w.c(), desc, out.data_ptr(), _ld(out),
                                    ws.data_ptr(), nbytes, _raw_stream(x))
    if status != OK:
        raise NvFp4Error(status, "nvfp4_w4a16_linear")
    return out


def _ld(t: torch.Tensor) -> int:
    """Row stride of a matrix; its width where there is one row, whose stride says nothing."""
    return t.stride(0) if t.shape[0] > 1 else t.shape[1]


def _heads(x: torch.Tensor, out: torch.Tensor, gamma) -> CHeads:
    row, head, _ = x.stride()
    out_row, out_head, _ = out.stride()
    return CHeads(x.data_ptr(), row, head, out.data_ptr(), out_row, out_head, x.shape[1],
                  None if gamma is None else gamma.data_ptr())


def qk_norm_rope(q: torch.Tensor, k: torch.Tensor | None, cos: torch.Tensor | None, sin: torch.Tensor | None,
                 positions: torch.Tensor | None = None, gamma_q: torch.Tensor | None = None,
                 gamma_k: torch.Tensor | None = None, eps: float = 1e-6, interleaved: bool = False,
                 q_out: torch.Tensor | None = None, k_out: torch.Tensor | None = None, stream=None):
    """Head RMSNorm (with gamma_q / gamma_k) and position rotation of q and k [rows, heads, head_dim] (bf16
    views, e.g. column ranges of a QKV product) through nvfp4_qk_norm_rope.  cos / sin: fp32 [table_rows,
    rot_dim / 2] (None: no rotation); ``positions`` int32 [rows] picks the table row, outside the table = not
    rotated; without it row r uses table row r % table_rows.  ``q_out`` / ``k_out`` may be q / k (in place).
    Returns (q_out, k_out)."""
    here = _here(stream, q)
    if here is not None:
        with here:
            return qk_norm_rope(q, k, cos, sin, positions, gamma_q, gamma_k, eps, interleaved, q_out, k_out)
    dev = q.get_device()
    rows, _, D = q.shape
    _require(q, "q", torch.bfloat16, dev)
    if gamma_q is not None:
        _require(gamma_q, "gamma_q", torch.bfloat16, dev, (D,))
    if q_out is None:
        q_out = torch.empty_like(q)
    else:
        _require(q_out, "q_out", torch.bfloat16, dev, q.shape)
    hk = None
    if k is None:
        if k_out is not None or gamma_k is not None:
            raise ValueError("k_out and gamma_k belong to k")
    else:
        if k.dim() != 3 or k.shape[0] != rows or k.shape[2] != D:
            raise ValueError("q and k: [rows, heads, head_dim] with the same rows and head_dim")
        _require(k, "k", torch.bfloat16, dev)
        if gamma_k is not None:
            _require(gamma_k, "gamma_k", torch.bfloat16, dev, (D,))
        if k_out is None:
            k_out = torch.empty_like(k)
        else:
            _require(k_out, "k_out", torch.bfloat16, dev, k.shape)
        hk = _heads(k, k_out, gamma_k)
    if (cos is None) != (sin is None):
        raise ValueError("cos and sin come together")
    if cos is None:
        if positions is not None:
            raise ValueError("positions belong to cos and sin")
        rope = CRope(None, None, 0, 0, 0, 0, None, eps)
    else:
        _require(cos, "cos", torch.float32, dev)
        _require(sin, "sin", torch.float32, dev, cos.shape)
        P, half = cos.shape
        if _ld(cos) != _ld(sin):
            raise ValueError("cos and sin: the same row stride")
        if positions is not None:
            _require(positions, "positions", torch.int32, dev, (rows,))
        rope = CRope(cos.data_ptr(), sin.data_ptr(), P, _ld(cos), 2 * half, interleaved,
                     None if positions is None else positions.data_ptr(), eps)
    status = load().nvfp4_qk_norm_rope(_heads(q, q_out, gamma_q), hk, rows, D, rope, _raw_stream(q))
    if status != OK:
        raise NvFp4Error(status, "nvfp4_qk_norm_rope")
    return q_out, k_out


def cross_attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, kv_lens: torch.Tensor | None = None,
                    scale: float | None = None, out: torch.Tensor | None = None, want_lse: bool = False, stream=None):
    """Attention of q [batch, q_len, heads, head_dim] to k and v [batch, kv_len, kv_heads, head_dim] (bf16, any
    strides with unit stride along head_dim) through nvfp4_cross_attention.  ``kv_lens`` int32 [batch]: keys of
    each sample that count.  ``scale`` defaults to head_dim ** -0.5.  Returns out, or (out, lse) with
    ``want_lse``, lse fp32 [batch, heads, q_len]."""
    here = _here(stream, q)
    if here is not None:
        with here:
            return cross_attention(q, k, v, kv_lens, scale, out, want_lse)
    dev = q.get_device()
    batch, q_len, heads, D = q.shape
    _require(q, "q", torch.bfloat16, dev)
    _require(k, "k", torch.bfloat16, dev)
    if k.dim() != 4 or k.shape[0] != batch or k.shape[3] != D:
        raise ValueError("k and v: [batch, kv_len, kv_heads, head_dim] with q's batch and head_dim")
    _require(v, "v", torch.bfloat16, dev, k.shape)
    if kv_lens is not None:
        _require(kv_lens, "kv_lens", torch.int32, dev, (batch,))
    if out is None:
        out = torch.empty_like(q)
    else:
        _require(out, "out", torch.bfloat16, dev, q.shape)
    lse = torch.empty((batch, heads, q_len), dtype=torch.float32, device=q.device) if want_lse else None
    desc = CAttention(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), batch, q_len, k.shape[1], heads,
                      k.shape[2], D, D ** -0.5 if scale is None else scale, *q.stride()[:3], *k.stride()[:3],
                      *v.stride()[:3], *out.stride()[:3], None if kv_lens is None else kv_lens.data_ptr(),
                      None if lse is None else lse.data_ptr())
    status = load().nvfp4_cross_attention(desc, _raw_stream(q))
    if status != OK:
        raise NvFp4Error(status, "nvfp4_cross_attention")
    return (out, lse) if want_lse else out


def get_device_error(stream=None) -> int:
    return int(load().nvfp4_get_device_error(_stream(stream)))


def check_device_error(stream=None):
    _check(get_device_error(stream), "device")
