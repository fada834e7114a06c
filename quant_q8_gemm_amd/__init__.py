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

and between the q, k, v products and the output product:

    q = qmm.rope_cache(cache, batch, q=q, k=k, v=v, frequencies=f)          # cache: Cache(...), batch: Batch(...)
    qact = qmm.attention(q, cache, batch, dtype="q8")
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
           "qmm_dequantize_activations", "qmm_norm_quantize", "qmm_mmq_epilogue", "qmm_mmv",
           "qmm_cache_page_bytes", "qmm_rope_frequencies", "qmm_rope_cache", "qmm_cache_read", "qmm_attention",
           "qmm_attention_plan")
MAX_CUS = 65536
# element types of activation tensors
F32, F16, BF16 = 0, 1, 2
ELEM_TYPES = {torch.float32: F32, torch.float16: F16, torch.bfloat16: BF16}
NORM_KINDS = {"rms": 0, "layer": 1}
Q8 = 3  # as the output of a product: q8 blocks
MAX_TOKENS = 1 << 20
MAX_SLOTS = 1 << 30
ROPE_SCALINGS = {"none": 0, "linear": 1, "base": 2, "yarn": 3, "turns": 4}
ROPE_LAYOUTS = {"half": 0, "interleaved": 1}
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


class CacheStruct(ctypes.Structure):
    _fields_ = [("type", ctypes.c_int32), ("heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("page", ctypes.c_int32), ("n_pages", ctypes.c_int64), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p)]


class BatchStruct(ctypes.Structure):
    _fields_ = [("n_seq", ctypes.c_int32), ("columns", ctypes.c_int32), ("starts", ctypes.c_void_p),
                ("lengths", ctypes.c_void_p), ("table", ctypes.c_void_p), ("table_stride", ctypes.c_int64),
                ("max_new", ctypes.c_int64), ("max_length", ctypes.c_int64)]


class Rope(ctypes.Structure):
    _fields_ = [("type", ctypes.c_int32), ("out_type", ctypes.c_int32), ("q_heads", ctypes.c_int32),
                ("layout", ctypes.c_int32), ("n_rot", ctypes.c_int32), ("magnitude", ctypes.c_float),
                ("frequencies", ctypes.c_void_p), ("positions", ctypes.c_void_p),
                ("q", ctypes.c_void_p), ("q_stride", ctypes.c_int64), ("q_head_stride", ctypes.c_int64),
                ("q_out", ctypes.c_void_p), ("q_out_stride", ctypes.c_int64), ("q_out_head_stride", ctypes.c_int64),
                ("k", ctypes.c_void_p), ("k_stride", ctypes.c_int64), ("k_head_stride", ctypes.c_int64),
                ("v", ctypes.c_void_p), ("v_stride", ctypes.c_int64), ("v_head_stride", ctypes.c_int64)]


class Attn(ctypes.Structure):
    _fields_ = [("heads", ctypes.c_int32), ("causal", ctypes.c_int32), ("out_type", ctypes.c_int32),
                ("scale", ctypes.c_float), ("window", ctypes.c_int64), ("q", ctypes.c_void_p),
                ("q_stride", ctypes.c_int64), ("q_head_stride", ctypes.c_int64), ("out", ctypes.c_void_p),
                ("out_stride", ctypes.c_int64)]


class AttnPlan(ctypes.Structure):
    _fields_ = [("work_bytes", ctypes.c_size_t), ("work_groups", ctypes.c_int64), ("few", ctypes.c_int32),
                ("columns", ctypes.c_int32), ("tiles", ctypes.c_int32), ("splits", ctypes.c_int32),
                ("share", ctypes.c_int32)]


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
_D = ctypes.c_double
_lib.qmm_cache_page_bytes.argtypes = [ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_int]
_lib.qmm_cache_page_bytes.restype = _SZ
_lib.qmm_rope_frequencies.argtypes = [_I64, _D, ctypes.c_int, _D, _D, _D, _D, _P, _P]
_lib.qmm_rope_frequencies.restype = ctypes.c_int
_CB = [ctypes.POINTER(CacheStruct), ctypes.POINTER(BatchStruct)]
_lib.qmm_rope_cache.argtypes = [ctypes.POINTER(Rope), *_CB, _I64, _P]
_lib.qmm_rope_cache.restype = ctypes.c_int
_lib.qmm_cache_read.argtypes = [*_CB, _I64, ctypes.c_int, _P, _P, _P]
_lib.qmm_cache_read.restype = ctypes.c_int
_lib.qmm_attention.argtypes = [ctypes.POINTER(Attn), *_CB, _I64, _P, _SZ, _P]
_lib.qmm_attention.restype = ctypes.c_int
_lib.qmm_attention_plan.argtypes = [*_CB, ctypes.c_int, _I64, _I64, ctypes.c_int, ctypes.POINTER(AttnPlan)]
_lib.qmm_attention_plan.restype = ctypes.c_int
# the same two with their structs as addresses, for the calls below: a decode step makes them for every layer
_rope_cache, _attention = _lib["qmm_rope_cache"], _lib["qmm_attention"]
_rope_cache.argtypes, _rope_cache.restype = [_P, _P, _P, _I64, _P], ctypes.c_int
_attention.argtypes, _attention.restype = [_P, _P, _P, _I64, _P, _SZ, _P], ctypes.c_int
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
    strides = (shape[1], 1) if len(shape) == 2 else (1,) if len(shape) == 1 else (shape[1] * shape[2], shape[2], 1)
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


# ---- between the q, k, v products and the output product: positions, a paged cache, attention ----

def rope_frequencies(n_rot: int, base: float = 10000.0, *, scaling: str = "none", factor: float = 1.0,
                     original: float = 4096.0, fast: float = 32.0, slow: float = 1.0, device=None):
    """(frequencies, magnitude) of rope_cache: the angle per position of each of the n_rot/2 pairs (float64, on the
    device) and the factor of what is rotated.  scaling: "none", "linear", "base", "yarn" or "turns" (include/qmm.h)."""
    if scaling not in ROPE_SCALINGS:
        raise QmmError(EINVAL, f"scaling must be one of {sorted(ROPE_SCALINGS)}, got {scaling!r}")
    f = (ctypes.c_double * max(1, n_rot // 2))()
    magnitude = ctypes.c_float()
    _check(_lib.qmm_rope_frequencies(n_rot, base, ROPE_SCALINGS[scaling], factor, original, fast, slow, f,
                                     ctypes.byref(magnitude)))
    return torch.tensor(list(f), dtype=torch.float64).to("cuda" if device is None else device), magnitude.value


class Cache:
    """A paged cache of keys and values: n_pages pages of `page` slots (a power of two from 32 on) of `heads` heads of
    head_dim channels, held as float16, bfloat16 or "q8" (blocks of 32 channels).  k and v are the pools, flat uint8
    tensors, zero at first; give both to use memory of your own."""

    def __init__(self, n_pages: int, heads: int, head_dim: int, *, page: int = 64, dtype=torch.float16, k=None, v=None,
                 device=None):
        type_ = Q8 if dtype == "q8" else ELEM_TYPES.get(dtype, -1)
        nbytes = n_pages * int(_lib.qmm_cache_page_bytes(type_, heads, head_dim, page)) if n_pages > 0 else 0
        if nbytes == 0:
            raise QmmError(EINVAL, f"no cache of {n_pages} pages of {page} slots, {heads} heads of {head_dim}, {dtype}")
        if (k is None) != (v is None):
            raise QmmError(EINVAL, "k and v come together")
        if k is None:
            device = "cuda" if device is None else device
            k, v = (torch.zeros(nbytes, dtype=torch.uint8, device=device) for _ in range(2))
        for t in (k, v):
            if t.dtype != torch.uint8 or t.shape != (nbytes,) or not t.is_contiguous() or t.get_device() != k.get_device():
                raise QmmError(EINVAL, f"k and v must be contiguous uint8 tensors of {nbytes} bytes on one device")
        self.k, self.v, self.dtype = k, v, dtype
        self.kind = torch.float16 if dtype == "q8" else dtype  # of the queries that read it
        self.n_pages, self.heads, self.head_dim, self.page = n_pages, heads, head_dim, page
        self.device, self._views = k.get_device(), None
        self.struct = CacheStruct(type_, heads, head_dim, page, n_pages, k.data_ptr(), v.data_ptr())
        self.address = ctypes.addressof(self.struct)

    def views(self):
        """What a float16 or bfloat16 cache holds, as strided views of its pools with the slots' and channels' indexes
        split: k [n_pages][heads][page/32][2][2][2][4][head_dim/16][2][8], v [n_pages][heads][page/32][2][2][8]
        [head_dim/32][32]; reshape(n_pages, heads, page, head_dim) of either is a copy in plain order."""
        if self._views is None:
            if self.dtype == "q8":
                raise QmmError(EINVAL, "a q8 cache holds codes and scales: cache_read gives their numbers")
            tiles, d = (self.n_pages, self.heads, self.page // 32), self.head_dim
            self._views = (self.k.view(self.dtype).view(*tiles, d // 16, 2, 2, 2, 2, 4, 8).permute(0, 1, 2, 5, 7, 6, 8, 3, 4, 9),
                           self.v.view(self.dtype).view(*tiles, d // 32, 2, 2, 32, 8).permute(0, 1, 2, 4, 5, 7, 3, 6))
        return self._views


class Batch:
    """The sequences of a call: starts int32 [n_seq + 1] (sequence s has rows starts[s] .. starts[s + 1] - 1), lengths
    int32 [n_seq] (slots in use, the call's tokens the last of them), table int32 [n_seq][columns] (page numbers), all
    on the device and read there, so that a captured graph takes what they hold when it is replayed.  max_new and
    max_length: the most tokens and slots of any sequence (None: what a sequence can have at most); they size
    the launch, and change a result in its roundings at most.  Sequences that pass them take longer, and so does attention over ones far shorter than
    max_length, None among them: give the longest length where it is known."""

    def __init__(self, starts, lengths, table, *, max_new: int = None, max_length: int = None):
        for hint, what, most in ((max_new, "max_new", MAX_TOKENS), (max_length, "max_length", MAX_SLOTS)):
            if hint is not None and not 0 <= hint <= most:
                raise QmmError(EINVAL, f"{what} must be None or in [0, {most}], got {hint}")
        device = starts.get_device()
        for t, what, dims in ((starts, "starts", 1), (lengths, "lengths", 1), (table, "table", 2)):
            if t.get_device() != device or device < 0 or t.dtype != torch.int32 or t.dim() != dims or (
                    t.numel() > 1 and t.stride(-1) != 1):
                raise QmmError(EINVAL, f"{what} must be int32 with {dims} dimension(s) and adjacent elements, on starts' cuda device")
        n = lengths.shape[0]
        if starts.shape[0] != n + 1 or table.shape[0] != n:
            raise QmmError(EINVAL, f"starts, lengths and table are of {starts.shape[0] - 1}, {n} and {table.shape[0]} sequences")
        self.starts, self.lengths, self.table, self.device = starts, lengths, table, device
        self.max_new = -1 if max_new is None else max_new
        columns = table.shape[1]
        self.max_length = -1 if max_length is None else max_length
        self.work = {}  # bytes of work memory by a call's sizes
        self.struct = BatchStruct(n, columns, starts.data_ptr(), lengths.data_ptr(), table.data_ptr(),
                                  table.stride(0) if n > 1 else columns, max(self.max_new, 0), max(self.max_length, 0))

    def _for(self, cache: Cache, n_tok: int) -> BatchStruct:
        if self.max_new >= 0 and self.max_length >= 0:
            return self.struct
        b = BatchStruct()  # of this call alone: other threads' may have other sizes
        ctypes.pointer(b)[0] = self.struct
        if self.max_new < 0:
            b.max_new = min(n_tok, MAX_TOKENS)
        if self.max_length < 0:
            b.max_length = min(b.columns * cache.page, MAX_SLOTS)
        return b


def _heads(t, what: str, n_tok: int, heads: int, dim: int, device: int, dtype=None):
    """(address, token stride, head stride) of a tensor [n_tok][heads][dim]; the library checks the rest."""
    if t.get_device() == device and t.shape == (n_tok, heads, dim) and (dtype is None or t.dtype == dtype):
        row, head, one = t.stride()
        if one == 1:
            return t.data_ptr(), row, head
        raise QmmError(EINVAL, f"{what} must have adjacent channels")
    raise QmmError(EINVAL, f"{what} must be {[n_tok, heads, dim]} {dtype or ''} on device {device}, got {list(t.shape)} "
                           f"{t.dtype} on {t.device}")


def _same_device(cache: Cache, batch: Batch, device: int) -> None:
    if cache.device != device or batch.device != device:  # the tensors that they hold
        raise QmmError(EINVAL, f"the tensors are on device {device}, the cache on {cache.device} and the batch on {batch.device}")


def rope_cache(cache: Cache, batch: Batch, *, q=None, k=None, v=None, frequencies=None, magnitude: float = 1.0,
               layout: str = "half", positions=None, dtype=None, out=None, stream=None):
    """The new tokens' queries and keys turned by their positions, and keys and values kept in their slots of the cache,
    in one kernel.  q [n_tok][heads][head_dim], k and v [n_tok][cache.heads][head_dim] of one type, any of them; channels
    adjacent, other strides free.  frequencies: float64 [n_rot/2] on the device (rope_frequencies); the first n_rot
    channels of a head are rotated, "half" (i with i + n_rot/2) or "interleaved" (2i with 2i + 1), and times magnitude;
    None: nothing turns.  positions: int32 [n_tok], or the tokens' slots.  Returns the queries, of `dtype` (None: that of
    the cache where q is float32, else q's) or in `out` (which may be q), or None without q.  Rows of tokens of no
    sequence are not set."""
    x = q if q is not None else k if k is not None else v
    if x is None:
        raise QmmError(EINVAL, "rope_cache needs q, k or v")
    if x.dim() != 3:
        raise QmmError(EINVAL, "q, k and v must be [n_tok][heads][head_dim]")
    device = _current(x, "q, k and v")
    _same_device(cache, batch, device)
    if layout not in ROPE_LAYOUTS:
        raise QmmError(EINVAL, f"layout must be 'half' or 'interleaved', got {layout!r}")
    n_tok, dim, kind = x.shape[0], cache.head_dim, x.dtype
    a = Rope(_elem(kind, "q, k and v"), F16, 1, ROPE_LAYOUTS[layout], 0, magnitude)
    if frequencies is not None:
        if (frequencies.get_device() != device or frequencies.dtype != torch.float64 or frequencies.dim() != 1
                or not frequencies.is_contiguous()):
            raise QmmError(EINVAL, f"frequencies must be a contiguous float64 vector on device {device}")
        a.n_rot, a.frequencies = 2 * frequencies.shape[0], frequencies.data_ptr()
    if positions is not None:
        if (positions.get_device() != device or positions.dtype != torch.int32 or positions.shape != (n_tok,)
                or not positions.is_contiguous()):
            raise QmmError(EINVAL, f"positions must be a contiguous int32 [{n_tok}] tensor on device {device}")
        a.positions = positions.data_ptr()
    if q is not None:
        a.q_heads = x.shape[1]
        a.q, a.q_stride, a.q_head_stride = _heads(q, "q", n_tok, a.q_heads, dim, device)
        if out is None:
            if dtype is None:
                dtype = kind if kind != torch.float32 else cache.kind
            a.out_type = _elem(dtype)
            out = _empty(q, (n_tok, a.q_heads, dim), dtype, stream)
            a.q_out, a.q_out_stride, a.q_out_head_stride = out.data_ptr(), a.q_heads * dim, dim
        else:
            a.out_type = _elem(out.dtype, "out")
            a.q_out, a.q_out_stride, a.q_out_head_stride = _heads(out, "out", n_tok, a.q_heads, dim, device)
    elif out is not None:
        raise QmmError(EINVAL, "out is where the queries go: it needs q")
    if k is not None:
        a.k, a.k_stride, a.k_head_stride = _heads(k, "k", n_tok, cache.heads, dim, device, kind)
    if v is not None:
        a.v, a.v_stride, a.v_head_stride = _heads(v, "v", n_tok, cache.heads, dim, device, kind)
    b = batch._for(cache, n_tok)
    rc = _rope_cache(ctypes.addressof(a), cache.address, ctypes.addressof(b), n_tok, _raw_stream(stream, device))
    if rc:
        _check(rc)
    return out


def cache_read(cache: Cache, batch: Batch, n_tok: int, *, dtype=torch.float32, stream=None):
    """(k, v), each [n_tok][cache.heads][head_dim] of dtype: what the cache holds for the batch's tokens.  Rows of
    tokens of no sequence are not set."""
    device = _current(cache.k, "the cache")
    _same_device(cache, batch, device)
    elem = _elem(dtype)
    shape = (n_tok, cache.heads, cache.head_dim)
    k, v = (_empty(cache.k, shape, dtype, stream) for _ in range(2))
    _check(_lib.qmm_cache_read(cache.struct, batch._for(cache, n_tok), n_tok, elem, k.data_ptr(), v.data_ptr(),
                               _raw_stream(stream, device)))
    return k, v


def _window(window: int) -> int:
    if not 0 <= window < 1 << 63:  # ctypes would take other numbers modulo 2^64
        raise QmmError(EINVAL, f"window must be in [0, 2^63), got {window}")
    return window


def attention_plan(cache: Cache, batch: Batch, heads: int, n_tok: int, num_cus: int, window: int = 0) -> AttnPlan:
    """How attention of these sizes is launched, and the work memory it needs (host arithmetic only)."""
    plan = AttnPlan()
    window = _window(window)
    _check(_lib.qmm_attention_plan(cache.struct, batch._for(cache, n_tok), heads, window, n_tok, num_cus, plan))
    return plan


_cus = {}  # device -> its compute units


def attention(q, cache: Cache, batch: Batch, *, scale: float = None, causal: bool = True, window: int = 0, dtype=None,
              out=None, work=None, stream=None):
    """Attention of the batch's tokens over the cache: softmax(scale * q k^T) v for each head, keys and values those of
    cache head h // (heads // cache.heads).

    q: [n_tok][heads][head_dim] of the cache's type (float16 with a q8 cache), channels adjacent, other strides free.
    causal: a token sees the slots up to its own, with window only the last `window` of them; else all in use (an
    encoder's states).  scale: head_dim ** -0.5 if None.  The result is [n_tok][heads][head_dim] of q's type, or with
    dtype "q8" the qact buffer of its rows (the output product's input), or `out`: [n_tok][heads * head_dim], rows may be
    strided, or a qact buffer with dtype "q8".  A token that sees nothing gets zeros; rows of tokens of no sequence are not
    set.  work: a uint8 tensor of attention_plan's work_bytes; new memory without it."""
    shape = q.shape
    if len(shape) != 3:
        raise QmmError(EINVAL, "q must be [n_tok][heads][head_dim]")
    n_tok, heads, dim = shape
    device = _current(q, "q")
    _same_device(cache, batch, device)
    kind = cache.kind
    if dtype is not None and dtype != "q8" and dtype != kind:
        raise QmmError(EINVAL, f"dtype must be None, 'q8' or {kind}, got {dtype}")
    a = Attn(heads, 1 if causal else 0, Q8 if dtype == "q8" else ELEM_TYPES[kind], dim ** -0.5 if scale is None else scale,
             _window(window), *_heads(q, "q", n_tok, heads, cache.head_dim, device, kind))
    result = out
    if dtype == "q8":
        if out is None:
            result = out = _empty(q, (qact_bytes(n_tok, heads * dim),), torch.uint8, stream)
        a.out, a.out_stride = _bytes(out, "out", device)
    elif out is None:
        result = out = _empty(q, shape, kind, stream)
        a.out, a.out_stride = out.data_ptr(), heads * dim
    else:
        a.out, a.out_stride = _rows(out, "out", (n_tok, heads * dim), device, kind)
    b = batch._for(cache, n_tok)
    if work is None:
        sizes = (n_tok, heads, cache.heads, dim, cache.dtype, b.max_new, b.max_length, window)  # what the plan goes by
        need = batch.work.get(sizes)
        if need is None:
            if device not in _cus:
                _cus[device] = torch.cuda.get_device_properties(device).multi_processor_count
            need = batch.work[sizes] = attention_plan(cache, batch, heads, n_tok, _cus[device], window).work_bytes
        work = _empty(q, (need,), torch.uint8, stream) if need else None
    work_ptr, work_bytes = (None, 0) if work is None or work.numel() == 0 else _bytes(work, "work", device)
    rc = _attention(ctypes.addressof(a), cache.address, ctypes.addressof(b), n_tok, work_ptr, work_bytes,
                    _raw_stream(stream, device))
    if rc:
        _check(rc)
    return result
