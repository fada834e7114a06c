"""Python binding of libqmm (include/qmm.h): argument marshalling only.

Every step of the computation runs in the library's HIP kernels; PyTorch is used
only to hold device memory and to name the stream.  If libqmm.so has not been
built, importing this package raises immediately -- there is no other path.

    import quant_q8_gemm_amd as qmm
    w = qmm.register_weights(qmm.Q6_K, od, id, raw_bytes)      # numpy uint8
    qact = qmm.quantize_activations(x)                          # x: cuda f32 [T][id]
    out = qmm.mmq(w, qact, n_tok)                               # cuda f32 [T][od]

and what stands between the products of a layer:

    r = qmm.norm_quantize(h, weight, y=out)                     # r.h = h + out, r.qact = q8(norm(r.h))
    out = qmm.mmq_epilogue(w, r.qact, n_tok, act="silu", dtype=torch.float16)
    out = qmm.mmv(w_rows, x, residual=h)                        # up to 16 tokens, w_rows: a rows-form handle
"""
from __future__ import annotations

import ctypes
import os
from typing import NamedTuple

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libqmm.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"{LIB_PATH} is missing: build it first (python quant_q8_gemm_amd/_build.py or "
        "__graft_entry__.build()); there is no fallback implementation")

# One HIP runtime per process: PyTorch ships its own libamdhip64 under the same
# soname.  Loading torch first makes libqmm bind to that runtime; loading libqmm
# first would pull in a second runtime that cannot see the device.
import torch  # noqa: E402

_lib = ctypes.CDLL(LIB_PATH)

# keep in step with include/qmm.h
Q4_K = 4
Q6_K = 6
Q4_K_PACKED = 14  # q4_K blocks, codes kept two per byte on the device
OK = 0
EINVAL = -1
ESHAPE = -2
ENOMEM = -3
EHIP = -4
TOKEN_PAD = 128
Q4_K_ROWS = 24  # the rows forms, for mmv
Q6_K_ROWS = 26
MV_MAX_TOKENS = 16
BLOCK_BYTES = {Q4_K: 144, Q4_K_PACKED: 144, Q6_K: 210, Q4_K_ROWS: 144, Q6_K_ROWS: 210}

# The full list of entry points include/qmm.h declares.
EXPORTS = ("qmm_register_weights", "qmm_weights_info", "qmm_weights_export", "qmm_release_weights",
           "qmm_set_memory_cap", "qmm_qact_bytes", "qmm_quantize_activations", "qmm_mmq",
           "qmm_mmq_noalloc", "qmm_stream_release", "qmm_mmq_plan", "qmm_mmq_plan_work", "qmm_last_error",
           "qmm_dequantize_activations", "qmm_norm_quantize", "qmm_mmq_epilogue", "qmm_mmv")
MAX_CUS = 65536
# element types of activation tensors
F32, F16, BF16 = 0, 1, 2
ELEM_TYPES = {torch.float32: F32, torch.float16: F16, torch.bfloat16: BF16}
NORM_KINDS = {"rms": 0, "layer": 1}
Q8 = 3  # as the output of a product: q8 blocks
ACTS = {"none": 0, "relu": 1, "silu": 2, "gelu": 3, "gelu_tanh": 4}


class Info(ctypes.Structure):
    _fields_ = [("type", ctypes.c_int), ("od", ctypes.c_int64), ("id", ctypes.c_int64),
                ("od_pad", ctypes.c_int64), ("raw_bytes", ctypes.c_size_t),
                ("plane_bytes", ctypes.c_size_t), ("wd_offset", ctypes.c_size_t),
                ("sm_offset", ctypes.c_size_t)]


class Plan(ctypes.Structure):
    _fields_ = [("work_groups", ctypes.c_int64), ("scratch_bytes", ctypes.c_size_t),
                ("threads", ctypes.c_int32), ("many", ctypes.c_int32), ("tile_rows", ctypes.c_int32),
                ("tile_tokens", ctypes.c_int32), ("k_groups", ctypes.c_int32), ("per_cu", ctypes.c_int32),
                ("row_tiles", ctypes.c_int32), ("tok_tiles", ctypes.c_int32), ("dp_row_tiles", ctypes.c_int32),
                ("n_tail", ctypes.c_int32), ("split", ctypes.c_int32), ("nsb", ctypes.c_int32)]


class Norm(ctypes.Structure):
    _fields_ = [("type", ctypes.c_int32), ("kind", ctypes.c_int32), ("eps", ctypes.c_float),
                ("residual_scale", ctypes.c_float), ("block_scale", ctypes.c_float),
                ("h", ctypes.c_void_p), ("h_stride", ctypes.c_int64), ("y", ctypes.c_void_p),
                ("y_stride", ctypes.c_int64), ("post_weight", ctypes.c_void_p), ("post_bias", ctypes.c_void_p),
                ("gate", ctypes.c_void_p), ("gate_stride", ctypes.c_int64), ("weight", ctypes.c_void_p),
                ("bias", ctypes.c_void_p), ("h_out", ctypes.c_void_p), ("h_out_stride", ctypes.c_int64),
                ("normed", ctypes.c_void_p), ("normed_stride", ctypes.c_int64), ("qact", ctypes.c_void_p),
                ("qact_bytes", ctypes.c_size_t)]


class Epilogue(ctypes.Structure):
    _fields_ = [("bias", ctypes.c_void_p), ("act", ctypes.c_int32), ("type", ctypes.c_int32),
                ("scale", ctypes.c_float), ("residual_scale", ctypes.c_float), ("mul", ctypes.c_void_p),
                ("mul_stride", ctypes.c_int64), ("residual", ctypes.c_void_p), ("residual_stride", ctypes.c_int64)]


_P = ctypes.c_void_p
_I64 = ctypes.c_int64
_SZ = ctypes.c_size_t
_lib.qmm_register_weights.argtypes = [ctypes.c_int, _I64, _I64, _P, _SZ, _P, ctypes.POINTER(_P)]
_lib.qmm_register_weights.restype = ctypes.c_int
_lib.qmm_weights_info.argtypes = [_P, ctypes.POINTER(Info)]
_lib.qmm_weights_info.restype = ctypes.c_int
_lib.qmm_weights_export.argtypes = [_P, _P, _SZ]
_lib.qmm_weights_export.restype = ctypes.c_int
_lib.qmm_release_weights.argtypes = [_P]
_lib.qmm_release_weights.restype = None
_lib.qmm_set_memory_cap.argtypes = [_SZ]
_lib.qmm_set_memory_cap.restype = None
_lib.qmm_qact_bytes.argtypes = [_I64, _I64]
_lib.qmm_qact_bytes.restype = _SZ
_lib.qmm_quantize_activations.argtypes = [_P, _I64, _I64, _P, _SZ, _P]
_lib.qmm_quantize_activations.restype = ctypes.c_int
_lib.qmm_mmq.argtypes = [_P, _P, _SZ, _I64, _P, _P]
_lib.qmm_mmq.restype = ctypes.c_int
_lib.qmm_mmq_noalloc.argtypes = [_P, _P, _SZ, _I64, _P, _P]
_lib.qmm_mmq_noalloc.restype = ctypes.c_int
_lib.qmm_stream_release.argtypes = [_P, ctypes.POINTER(_SZ)]
_lib.qmm_stream_release.restype = ctypes.c_int
_lib.qmm_mmq_plan.argtypes = [ctypes.c_int, _I64, _I64, _I64, ctypes.c_int, ctypes.POINTER(Plan)]
_lib.qmm_mmq_plan.restype = ctypes.c_int
_I32P = ctypes.POINTER(ctypes.c_int32)
_lib.qmm_mmq_plan_work.argtypes = [ctypes.POINTER(Plan), _I64, _I32P, _I32P, _I32P, _I32P]
_lib.qmm_mmq_plan_work.restype = ctypes.c_int
_lib.qmm_dequantize_activations.argtypes = [_P, _SZ, _I64, _I64, ctypes.c_int, _P, _I64, _P]
_lib.qmm_dequantize_activations.restype = ctypes.c_int
_lib.qmm_norm_quantize.argtypes = [ctypes.POINTER(Norm), _I64, _I64, _P]
_lib.qmm_norm_quantize.restype = ctypes.c_int
_lib.qmm_mmq_epilogue.argtypes = [_P, _P, _SZ, _I64, ctypes.POINTER(Epilogue), ctypes.c_int, _P, _I64, _P, _SZ, _P]
_lib.qmm_mmq_epilogue.restype = ctypes.c_int
_lib.qmm_mmv.argtypes = [_P, _P, ctypes.c_int, _I64, _I64, ctypes.POINTER(Epilogue), ctypes.c_int, _P, _I64, _P]
_lib.qmm_mmv.restype = ctypes.c_int
_lib.qmm_last_error.argtypes = []
_lib.qmm_last_error.restype = ctypes.c_char_p


class QmmError(RuntimeError):
    def __init__(self, code: int, message: str):
        super().__init__(f"qmm error {code}: {message}")
        self.code = code


def last_error() -> str:
    return _lib.qmm_last_error().decode()


def _check(rc: int) -> None:
    if rc != OK:
        raise QmmError(rc, last_error())


def _check_qact(qact) -> None:
    if qact.dtype != torch.uint8 or not qact.is_cuda or qact.dim() != 1 or not qact.is_contiguous():
        raise QmmError(EINVAL, "qact must be a contiguous one-dimensional cuda uint8 tensor")


def _stream(stream):
    if stream is None:
        return ctypes.c_void_p(torch._C._cuda_getCurrentRawStream(torch.cuda.current_device()))
    if isinstance(stream, int):
        return ctypes.c_void_p(stream)
    return ctypes.c_void_p(stream.cuda_stream)


def set_memory_cap(nbytes: int) -> None:
    _lib.qmm_set_memory_cap(int(nbytes))


def qact_bytes(n_tok: int, id_: int) -> int:
    return int(_lib.qmm_qact_bytes(int(n_tok), int(id_)))


class Weights:
    """A registered weight matrix (device planes owned by the library)."""

    def __init__(self, handle: int):
        self._h = handle
        info = Info()
        _check(_lib.qmm_weights_info(ctypes.c_void_p(handle), ctypes.byref(info)))
        self.type = info.type
        self.od = info.od
        self.id = info.id
        self.od_pad = info.od_pad
        self.raw_bytes = info.raw_bytes
        self.plane_bytes = info.plane_bytes
        self.wd_offset = info.wd_offset
        self.sm_offset = info.sm_offset

    @property
    def handle(self) -> int:
        if self._h is None:
            raise QmmError(EINVAL, "weights already released")
        return self._h

    def export(self) -> np.ndarray:
        """Host copy of the device planes (layout: include/qmm.h, qmm_weights_export)."""
        buf = np.empty(self.plane_bytes, np.uint8)
        _check(_lib.qmm_weights_export(ctypes.c_void_p(self.handle),
                                       buf.ctypes.data_as(ctypes.c_void_p), buf.nbytes))
        return buf

    def release(self) -> None:
        if self._h is not None:
            _lib.qmm_release_weights(ctypes.c_void_p(self._h))
            self._h = None

    def __del__(self):
        try:
            self.release()
        except Exception:
            pass


def register_weights(type_: int, od: int, id_: int, raw, stream=None) -> Weights:
    """Copy k-quant bytes (host numpy/bytes, od x (id/256) blocks) to the device and
    expand them into the library's planes."""
    buf = np.ascontiguousarray(np.frombuffer(raw, np.uint8) if isinstance(raw, (bytes, bytearray))
                               else np.asarray(raw, np.uint8).reshape(-1))
    h = ctypes.c_void_p()
    _check(_lib.qmm_register_weights(int(type_), int(od), int(id_),
                                     buf.ctypes.data_as(ctypes.c_void_p), buf.nbytes,
                                     _stream(stream), ctypes.byref(h)))
    return Weights(h.value)


def quantize_activations(x, qact=None, stream=None):
    """x: cuda float32 [n_tok][id] contiguous -> qact (cuda uint8, qact_bytes)."""
    if x.dtype != torch.float32 or not x.is_cuda or x.dim() != 2 or not x.is_contiguous():
        raise QmmError(EINVAL, "x must be a contiguous cuda float32 [n_tok][id] tensor")
    n_tok, id_ = x.shape
    if qact is None:
        nb = qact_bytes(n_tok, id_)
        if nb == 0 and n_tok != 0:
            raise QmmError(EINVAL, f"bad shape n_tok={n_tok} id={id_}")
        qact = torch.empty_strided((nb,), (1,), dtype=torch.uint8, device=x.device)
    _check_qact(qact)
    _check(_lib.qmm_quantize_activations(x.data_ptr(), n_tok, id_, qact.data_ptr(), qact.numel(), _stream(stream)))
    return qact


def _mmq_args(w: Weights, qact, n_tok: int, out):
    _check_qact(qact)
    if out is None:
        out = torch.empty((n_tok, w.od), dtype=torch.float32, device=qact.device)
    elif (out.dtype != torch.float32 or not out.is_cuda or not out.is_contiguous()
          or tuple(out.shape) != (n_tok, w.od)):
        raise QmmError(EINVAL, "out must be a contiguous cuda float32 [n_tok][od] tensor")
    return out


def mmq(w: Weights, qact, n_tok: int, out=None, stream=None):
    """out[t][j] (cuda float32 [n_tok][od]) from a handle and a qact buffer."""
    out = _mmq_args(w, qact, n_tok, out)
    _check(_lib.qmm_mmq(ctypes.c_void_p(w.handle), ctypes.c_void_p(qact.data_ptr()), qact.numel(),
                        int(n_tok), ctypes.c_void_p(out.data_ptr()), _stream(stream)))
    return out


def mmq_noalloc(w: Weights, qact, n_tok: int, out, stream=None):
    """mmq through the allocation-free entry point (the caller passes out)."""
    out = _mmq_args(w, qact, n_tok, out)
    _check(_lib.qmm_mmq_noalloc(ctypes.c_void_p(w.handle), ctypes.c_void_p(qact.data_ptr()), qact.numel(),
                                int(n_tok), ctypes.c_void_p(out.data_ptr()), _stream(stream)))
    return out


def stream_release(stream=None) -> int:
    """Free the MMQ scratch the library keeps for `stream` (torch's current
    stream if None); synchronizes the stream first.  Returns the bytes freed."""
    freed = _SZ(0)
    _check(_lib.qmm_stream_release(_stream(stream), ctypes.byref(freed)))
    return int(freed.value)


def mmq_plan(type_: int, od: int, id_: int, n_tok: int, num_cus: int) -> Plan:
    """The launch plan qmm_mmq follows for this shape on a GPU with num_cus
    compute units (host arithmetic only; no device needed)."""
    plan = Plan()
    _check(_lib.qmm_mmq_plan(int(type_), int(od), int(id_), int(n_tok), int(num_cus), ctypes.byref(plan)))
    return plan


def mmq_plan_work(plan: Plan, wg: int):
    """(row tile, token tile, first super-block, end super-block) that
    work-group wg of the plan's launch computes."""
    out = [ctypes.c_int32() for _ in range(4)]
    _check(_lib.qmm_mmq_plan_work(ctypes.byref(plan), int(wg), *[ctypes.byref(o) for o in out]))
    return tuple(o.value for o in out)


# ---- what stands between the products ----

def _elem(dtype, what: str = "dtype") -> int:
    t = ELEM_TYPES.get(dtype)
    if t is None:
        raise QmmError(EINVAL, f"{what} must be float32, float16 or bfloat16, got {dtype}")
    return t


def _current(t, what: str) -> int:
    """The index of t's device, which has to be the current one."""
    device = t.get_device()
    if device < 0:
        raise QmmError(EINVAL, f"{what} must be a cuda tensor")
    if device != torch._C._cuda_getDevice():  # torch.cuda.current_device without its detours: t is a cuda tensor
        raise QmmError(EINVAL, f"{what} is on device {device} but device {torch.cuda.current_device()} is current")
    return device


def _rows(t, what: str, shape, device: int, dtype=None):
    """(address, stride) of a tensor of rows with adjacent elements; the library checks the rest."""
    if t.get_device() == device and t.shape == shape and (dtype is None or t.dtype == dtype):
        strides = t.stride()
        if strides[1] == 1 or shape[1] == 1:
            return t.data_ptr(), strides[0] if shape[0] > 1 else shape[1]
        raise QmmError(EINVAL, f"{what} must have adjacent elements in a row")
    raise QmmError(EINVAL, f"{what} must be {list(shape)} {dtype or ''} on device {device}, got {list(t.shape)} "
                           f"{t.dtype} on {t.device}")


def _vector(t, what: str, n: int, device: int):
    if t.get_device() != device or t.dtype != torch.float32 or t.shape != (n,) or not t.is_contiguous():
        raise QmmError(EINVAL, f"{what} must be a contiguous float32 [{n}] tensor on device {device}")
    return t.data_ptr()


def _bytes(t, what: str, device: int):
    """(address, size) of a flat byte tensor."""
    if t.get_device() != device or t.dtype != torch.uint8 or t.dim() != 1 or not t.is_contiguous():
        raise QmmError(EINVAL, f"{what} must be a contiguous one-dimensional uint8 tensor on device {device}")
    return t.data_ptr(), t.numel()


def _empty(like, shape, dtype, stream):
    """A new contiguous tensor on like's device that belongs to the stream it is written on."""
    strides = (shape[1], 1) if len(shape) == 2 else (1,)
    if stream is None:
        return torch.empty_strided(shape, strides, dtype=dtype, device=like.device)
    if isinstance(stream, int):  # 0 is the null stream, which ExternalStream does not know
        stream = torch.cuda.ExternalStream(stream, device=like.device) if stream else torch.cuda.default_stream(like.device)
    with torch.cuda.stream(stream):
        return torch.empty_strided(shape, strides, dtype=dtype, device=like.device)


def _raw_stream(stream, device: int):
    """The hipStream_t of `stream` (None: torch's current one), as _stream without its detours."""
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(device)
    return stream if isinstance(stream, int) else stream.cuda_stream


def dequantize_activations(qact, n_tok: int, id_: int, dtype=torch.float32, out=None, stream=None):
    """The numbers a qact buffer stands for: [n_tok][id] of dtype (float32, float16 or bfloat16)."""
    device = _current(qact, "qact")
    q_ptr, q_bytes = _bytes(qact, "qact", device)
    if out is None:
        _elem(dtype)
        out = _empty(qact, (n_tok, id_), dtype, stream)
    ptr, stride = _rows(out, "out", (n_tok, id_), device)
    _check(_lib.qmm_dequantize_activations(q_ptr, q_bytes, n_tok, id_, _elem(out.dtype, "out"), ptr, stride,
                                           _raw_stream(stream, device)))
    return out


class NormResult(NamedTuple):
    h: object       # the sum, or None
    normed: object  # its norm as numbers, or None
    qact: object    # its norm as q8 blocks, or None


def norm_quantize(h, weight, *, y=None, bias=None, post_weight=None, post_bias=None, gate=None,
                  residual_scale: float = 1.0, block_scale: float = 1.0, kind: str = "rms", eps: float = 1e-5,
                  h_out=True, normed=False, qact=True, stream=None) -> NormResult:
    """Norm after a block, gate, scaled residual sum, norm before the next block and its q8 blocks in one pass:

        s = residual_scale * h + block_scale * gate * norm(y; post_weight, post_bias),  n = norm(s; weight, bias)

    h, y: cuda [n_tok][id] of float32, float16 or bfloat16 (rows may be strided); gate: [id] or [n_tok][id] of the
    same type; weights and biases float32 [id]; kind "rms" or "layer".  h_out (s), normed (n) and qact (n quantized):
    True for a new tensor, a tensor to write into, or False.  h_out may be h or y itself."""
    if h.dim() != 2:
        raise QmmError(EINVAL, "h must be [n_tok][id]")
    shape, dtype = h.shape, h.dtype
    n_tok, id_ = shape
    elem = _elem(dtype, "h")
    if kind not in NORM_KINDS:
        raise QmmError(EINVAL, f"kind must be 'rms' or 'layer', got {kind!r}")
    device = _current(h, "h")
    a = Norm(elem, NORM_KINDS[kind], eps, residual_scale, block_scale, *_rows(h, "h", shape, device))
    if y is not None:
        a.y, a.y_stride = _rows(y, "y", shape, device, dtype)
    a.weight = _vector(weight, "weight", id_, device)
    if bias is not None:
        a.bias = _vector(bias, "bias", id_, device)
    if post_weight is not None:
        a.post_weight = _vector(post_weight, "post_weight", id_, device)
    if post_bias is not None:
        a.post_bias = _vector(post_bias, "post_bias", id_, device)
    if gate is not None:
        if gate.dim() == 1:
            a.gate, a.gate_stride = _rows(gate.unsqueeze(0), "gate", (1, id_), device, dtype)[0], 0
        else:
            a.gate, a.gate_stride = _rows(gate, "gate", shape, device, dtype)
    if h_out is True:
        h_out = _empty(h, shape, dtype, stream)
        a.h_out, a.h_out_stride = h_out.data_ptr(), id_
    elif h_out is False:
        h_out = None
    else:
        a.h_out, a.h_out_stride = _rows(h_out, "h_out", shape, device, dtype)
    if normed is True:
        normed = _empty(h, shape, dtype, stream)
        a.normed, a.normed_stride = normed.data_ptr(), id_
    elif normed is False:
        normed = None
    else:
        a.normed, a.normed_stride = _rows(normed, "normed", shape, device, dtype)
    if qact is True:
        qact = _empty(h, (qact_bytes(n_tok, id_),), torch.uint8, stream)
    if qact is False:
        qact = None
    else:
        a.qact, a.qact_bytes = _bytes(qact, "qact", device)
    _check(_lib.qmm_norm_quantize(a, n_tok, id_, _raw_stream(stream, device)))
    return NormResult(h_out, normed, qact)


def _epilogue(shape, device: int, bias, act: str, mul, residual, scale: float, residual_scale: float) -> Epilogue:
    ep = Epilogue(None, ACTS.get(act, -1), F32, scale, residual_scale)
    if ep.act < 0:
        raise QmmError(EINVAL, f"act must be one of {sorted(ACTS)}, got {act!r}")
    if bias is not None:
        ep.bias = _vector(bias, "bias", shape[1], device)
    if mul is not None:
        ep.type = _elem(mul.dtype, "mul")
        ep.mul, ep.mul_stride = _rows(mul, "mul", shape, device)
    if residual is not None:
        if mul is not None and residual.dtype != mul.dtype:
            raise QmmError(EINVAL, f"mul is {mul.dtype} but residual is {residual.dtype}")
        ep.type = _elem(residual.dtype, "residual")
        ep.residual, ep.residual_stride = _rows(residual, "residual", shape, device)
    return ep


def mmq_epilogue(w: Weights, qact, n_tok: int, *, bias=None, act: str = "none", mul=None, residual=None,
                 scale: float = 1.0, residual_scale: float = 1.0, dtype=torch.float32, out=None, work=None,
                 stream=None):
    """The product of mmq with an epilogue, in one kernel:

        scale * mul * act(x @ W^T + bias) + residual_scale * residual

    bias: float32 [od]; mul, residual: [n_tok][od] of one type (rows may be strided); act: "none", "relu", "silu",
    "gelu" or "gelu_tanh".  The result is [n_tok][od] of `dtype`, or with dtype "q8" the qact buffer of the values
    (the next product's input; od % 256 == 0).  out: a tensor to write into; it may be mul or residual itself.
    work: a uint8 tensor for the split tails (mmq_plan(...).scratch_bytes), for graph capture; the stream's own
    scratch without it."""
    device = _current(qact, "qact")
    q_ptr, q_bytes = _bytes(qact, "qact", device)
    shape = (n_tok, w.od)
    ep = _epilogue(shape, device, bias, act, mul, residual, scale, residual_scale)
    if dtype == "q8":
        if out is None:
            out = _empty(qact, (qact_bytes(n_tok, w.od),), torch.uint8, stream)
        out_type, (ptr, stride) = Q8, _bytes(out, "out", device)
    else:
        if out is None:
            _elem(dtype)  # before the allocation
            out = _empty(qact, shape, dtype, stream)
        out_type, (ptr, stride) = _elem(out.dtype, "out"), _rows(out, "out", shape, device)
    work_ptr, work_bytes = _bytes(work, "work", device) if work is not None and work.numel() else (None, 0)
    _check(_lib.qmm_mmq_epilogue(w.handle, q_ptr, q_bytes, n_tok, ep, out_type, ptr, stride, work_ptr, work_bytes,
                                 _raw_stream(stream, device)))
    return out


def mmv(w: Weights, x, n_tok: int = None, *, bias=None, act: str = "none", mul=None, residual=None, scale: float = 1.0,
        residual_scale: float = 1.0, dtype=torch.float32, out=None, stream=None):
    """The product for up to MV_MAX_TOKENS tokens straight from the activations, with mmq_epilogue's epilogue:

        scale * mul * act(x @ W^T + bias) + residual_scale * residual

    w: a handle of Q4_K_ROWS or Q6_K_ROWS; x: [n_tok][id] of float32, float16 or bfloat16 (rows may be strided), or
    the qact buffer of n_tok tokens.  The result is [n_tok][od] of `dtype`, or its qact buffer with dtype "q8" (od %
    256 == 0), or `out`."""
    device = _current(x, "x")
    if n_tok is not None:
        x_type, (x_ptr, x_stride) = Q8, _bytes(x, "x", device)
    elif x.dim() == 2:
        n_tok, x_type = x.shape[0], _elem(x.dtype, "x")
        x_ptr, x_stride = _rows(x, "x", (n_tok, w.id), device)
    else:
        raise QmmError(EINVAL, "x must be [n_tok][id], or a qact buffer with n_tok")
    shape = (n_tok, w.od)
    ep = _epilogue(shape, device, bias, act, mul, residual, scale, residual_scale)
    if dtype == "q8":
        if out is None:
            out = _empty(x, (qact_bytes(n_tok, w.od),), torch.uint8, stream)
        out_type, (out_ptr, out_stride) = Q8, _bytes(out, "out", device)
    elif out is None:
        out_type = _elem(dtype)
        out = _empty(x, shape, dtype, stream)
        out_ptr, out_stride = out.data_ptr(), w.od
    else:
        out_type, (out_ptr, out_stride) = _elem(out.dtype, "out"), _rows(out, "out", shape, device)
    _check(_lib.qmm_mmv(w.handle, x_ptr, x_type, x_stride, n_tok, ep, out_type, out_ptr, out_stride,
                        _raw_stream(stream, device)))
    return out
