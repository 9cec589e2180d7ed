"""Python binding of libft.so (argument marshalling only).

Every step of the path runs in the gfx950 kernels behind the C ABI declared in
include/ft.h; this module turns torch tensors (device memory, current stream)
into pointers and sizes and raises on a non-OK status.  There is no CPU
fallback: if libft.so is missing or cannot load, every call raises.

A call with `stream` does all of its work on that stream, as under torch.cuda.stream(stream): the tensors that
it makes are the stream's, and the caller orders the stream after the work that its inputs come from.
"""
from __future__ import annotations

import ctypes
import math
import os

import torch  # loaded first so libft.so binds to the same HIP runtime as torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libft.so")

TYPES = {"Q4_0": 0, "Q8_0": 1, "Q4_K": 2, "Q5_K": 3, "Q6_K": 4, "MXFP4": 5, "Q8_1": 6, "Q8_K": 7,
         "Q2_K": 8, "Q3_K": 9, "Q4_1": 10, "Q5_0": 11, "Q5_1": 12}
OPS = {"quantize": 0, "dequant": 1, "mmvq": 2, "moe_vec": 3, "grouped": 4, "block_dots": 5, "kv_cache": 6}
FLOATS = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}
ACTS = ("Q8_1", "Q8_0", "Q8_K")  # the formats of activations
STATUS = {0: "FT_OK", 1: "FT_ERR_INVALID_ARG", 2: "FT_ERR_UNSUPPORTED", 3: "FT_ERR_SHAPE",
          4: "FT_ERR_ALIGNMENT", 5: "FT_ERR_NO_SCRATCH", 6: "FT_ERR_HIP"}


class FtError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {STATUS.get(status, status)} ({lib().ft_status_str(status).decode()})")


class _MoeOpts(ctypes.Structure):
    _fields_ = [("route", ctypes.c_int), ("direct_max_t", ctypes.c_int),
                ("tap_g", ctypes.c_void_p), ("tap_u", ctypes.c_void_p), ("tap_h", ctypes.c_void_p),
                ("tap_hq", ctypes.c_void_p), ("tap_down", ctypes.c_void_p), ("in_hq", ctypes.c_void_p),
                ("logits", ctypes.c_void_p), ("ids_out", ctypes.c_void_p), ("w_out", ctypes.c_void_p)]


class _RouteOpts(ctypes.Structure):
    _fields_ = [("sigmoid", ctypes.c_int), ("bias", ctypes.c_void_p), ("n_group", ctypes.c_int),
                ("topk_group", ctypes.c_int), ("group_top", ctypes.c_int), ("no_renorm", ctypes.c_int),
                ("scale", ctypes.c_double)]


class _KvCache(ctypes.Structure):
    _fields_ = [("k_type", ctypes.c_int), ("v_type", ctypes.c_int), ("k_pages", ctypes.c_void_p),
                ("v_pages", ctypes.c_void_p), ("n_pages", ctypes.c_int64), ("page_size", ctypes.c_int64),
                ("n_kv_head", ctypes.c_int64), ("head_dim", ctypes.c_int64)]


class _AttnOpts(ctypes.Structure):
    _fields_ = [("scale", ctypes.c_float), ("softcap", ctypes.c_float), ("bidirectional", ctypes.c_int),
                ("window", ctypes.c_int64), ("slopes", ctypes.c_void_p), ("prefix_len", ctypes.c_void_p),
                ("n_shared", ctypes.c_int64), ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t)]


_P, _I64 = ctypes.c_void_p, ctypes.c_int64

EXPORTS = {
    "ft_block_elems": (ctypes.c_int, [ctypes.c_int]),
    "ft_block_bytes": (ctypes.c_size_t, [ctypes.c_int]),
    "ft_supported": (ctypes.c_int, [ctypes.c_int, ctypes.c_int, ctypes.c_int]),
    "ft_status_str": (ctypes.c_char_p, [ctypes.c_int]),
    "ft_version": (ctypes.c_char_p, []),
    "ft_quantize_act": (ctypes.c_int, [ctypes.c_int, ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64,
                                       ctypes.c_int64, ctypes.c_void_p, ctypes.c_void_p]),
    "ft_dequant": (ctypes.c_int, [ctypes.c_int, ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64,
                                  ctypes.c_void_p, ctypes.c_void_p]),
    "ft_mul_mat_vec_q": (ctypes.c_int, [ctypes.c_int, ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64,
                                        ctypes.c_int, ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p,
                                        ctypes.c_int64, ctypes.c_void_p]),
    "ft_moe_route": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64, ctypes.c_int,
                                    ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p]),
    "ft_moe_sort": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_int64,
                                   ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p]),
    "ft_moe_q_vec": (ctypes.c_int, [ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                    ctypes.c_int64, ctypes.c_int64, ctypes.c_int64, ctypes.c_int,
                                    ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p, ctypes.c_void_p,
                                    ctypes.c_int, ctypes.c_void_p, ctypes.POINTER(_MoeOpts), ctypes.c_void_p]),
    "ft_moe_q_vec_noalloc": (ctypes.c_int, [ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                            ctypes.c_int64, ctypes.c_int64, ctypes.c_int64, ctypes.c_int,
                                            ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p, ctypes.c_void_p,
                                            ctypes.c_int, ctypes.c_void_p, ctypes.POINTER(_MoeOpts),
                                            ctypes.c_void_p]),
    "ft_grouped_gemm_q": (ctypes.c_int, [ctypes.c_int, ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64,
                                         ctypes.c_int64, ctypes.c_int, ctypes.c_void_p, ctypes.c_int,
                                         ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_void_p,
                                         ctypes.c_void_p]),
    "ft_debug_block_dots": (ctypes.c_int, [ctypes.c_int, ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64,
                                           ctypes.c_int, ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p,
                                           ctypes.c_void_p]),
    "ft_debug_ceiling": (ctypes.c_int, [ctypes.c_int, ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64,
                                        ctypes.c_void_p, ctypes.c_void_p]),
    "ft_moe_route_ex": (ctypes.c_int, [_P, ctypes.c_int, _I64, _I64, _I64, ctypes.c_int, ctypes.POINTER(_RouteOpts),
                                       _P, _P, _P]),
    "ft_kv_page_bytes": (ctypes.c_size_t, [ctypes.c_int, _I64, _I64, _I64]),
    "ft_kv_store": (ctypes.c_int, [ctypes.POINTER(_KvCache), ctypes.c_int, _P, _I64, _I64, _P, _I64, _I64, _P, _I64,
                                   _P]),
    "ft_kv_load": (ctypes.c_int, [ctypes.POINTER(_KvCache), _P, _I64, ctypes.c_int, _P, _I64, _I64, _P, _I64, _I64,
                                  _P]),
    "ft_attn_kv": (ctypes.c_int, [ctypes.POINTER(_KvCache), ctypes.c_int, _P, _I64, _I64, _I64, _I64, _P, _P, _P, _I64,
                                  _I64, _I64, _I64, _P, _I64, _I64, ctypes.POINTER(_AttnOpts), _P]),
    "ft_attn_kv_scratch_bytes": (ctypes.c_size_t, [ctypes.POINTER(_KvCache), _I64, _I64, _I64, _I64,
                                                   ctypes.POINTER(_AttnOpts)]),
    "ft_rope_table": (ctypes.c_int, [_P, _I64, _I64, ctypes.c_double, _P, _P]),
    "ft_rope": (ctypes.c_int, [_P, ctypes.c_int, _P, _I64, _I64, _I64, _I64, _I64, _P, ctypes.c_double, _P,
                               _I64, _I64, _P]),
    "ft_kv_store_rope": (ctypes.c_int, [ctypes.POINTER(_KvCache), _P, ctypes.c_int, _P, _P, _I64, _P]),
    "ft_norm": (ctypes.c_int, [ctypes.c_int, _P, _I64, _I64, _I64, _P, _P]),
    "ft_lora": (ctypes.c_int, [ctypes.c_int, _P, _I64, _I64, _I64, ctypes.c_int, _P, _P, _I64, _I64, _I64, _P, _P, _I64, _P, _I64,
                               _P, _P]),
    "ft_lora_scratch_bytes": (ctypes.c_size_t, [_I64, _I64, _I64, _I64]),
    "ft_scratch_reserve": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_size_t]),
    "ft_moe_scratch_bytes": (ctypes.c_size_t, [ctypes.c_int, ctypes.c_int, ctypes.c_int64, ctypes.c_int64,
                                               ctypes.c_int64, ctypes.c_int64, ctypes.c_int]),
    "ft_grouped_scratch_bytes": (ctypes.c_size_t, [ctypes.c_int, ctypes.c_int64, ctypes.c_int64, ctypes.c_int64,
                                                    ctypes.c_int, ctypes.c_int]),
    "ft_shutdown": (None, []),
}

_lib = None


def lib() -> ctypes.CDLL:
    """Load libft.so (raises if it was not built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is not built: run `python -m block_quantized_matvec_amd.build`")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in EXPORTS.items():
            f = getattr(L, name)
            f.restype = res
            f.argtypes = args
        _lib = L
    return _lib


_ext = None
# the entry points that the compiled marshalling calls, in its order
_MARSHALLED = ("ft_rope", "ft_kv_store_rope", "ft_kv_load", "ft_norm", "ft_lora", "ft_block_elems", "ft_block_bytes")


def _marshalling():
    """The marshalling of the calls of a decoder layer's step, compiled against torch, or the ImportError where it does
    not load."""
    global _ext
    if _ext is None:
        L = lib()
        try:
            from . import _ft_bind
        except ImportError as e:
            _ext = e
        else:
            _ft_bind.setup(FtError, *(ctypes.cast(getattr(L, f), _P).value for f in _MARSHALLED))
            _ext = _ft_bind
    return _ext


def _bind():
    """The compiled marshalling (raises if it was not built)."""
    ext = _ext or _marshalling()
    if isinstance(ext, ImportError):
        raise RuntimeError(f"{_PKG}/_ft_bind.so does not load: run `python -m block_quantized_matvec_amd.build`") from ext
    return ext


def _check(status: int, what: str) -> None:
    if status != 0:
        raise FtError(status, what)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _on(stream):
    """torch.cuda.stream of a call's stream (nothing for None)."""
    if stream is not None and not isinstance(stream, torch.cuda.Stream):  # its handle is enough
        stream = torch.cuda.ExternalStream(stream.cuda_stream, device=getattr(stream, "device", None))
    return torch.cuda.stream(stream)


def _new(shape, dtype, device, stream) -> torch.Tensor:
    """A new tensor of the call's stream.  (Memory that the current stream gave back may still be in use there; the
    allocator hands it out to tensors of that stream only.)"""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with _on(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _dev(t: torch.Tensor, name: str) -> torch.Tensor:
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


def block_elems(ty: str) -> int:
    return lib().ft_block_elems(TYPES[ty])


def block_bytes(ty: str) -> int:
    return lib().ft_block_bytes(TYPES[ty])


def row_bytes(ty: str, k: int) -> int:
    return k // block_elems(ty) * block_bytes(ty)


def supported(op: str, w: str, act: str) -> bool:
    return bool(lib().ft_supported(OPS[op], TYPES[w], TYPES[act]))


def version() -> str:
    return lib().ft_version().decode()


def quantize_act(act: str, x: torch.Tensor, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """x: (rows, k) fp32 on the device; rows may be strided (row stride -> ldx)."""
    if not x.is_cuda:
        raise ValueError("x must be a device tensor")
    rows, k = x.shape
    if x.stride(1) != 1 or (rows > 1 and x.stride(0) < k):
        raise ValueError("x must have unit element stride and rows at least k apart")
    ldx = x.stride(0) if rows > 1 else k
    if out is None:
        out = _new((rows, row_bytes(act, k)), torch.uint8, x.device, stream)
    _check(lib().ft_quantize_act(TYPES[act], _ptr(x), rows, k, ldx, _ptr(out), _stream(stream)), "ft_quantize_act")
    return out


def dequant(w: str, blocks: torch.Tensor, rows: int, k: int, out: torch.Tensor | None = None,
            stream=None) -> torch.Tensor:
    _dev(blocks, "blocks")
    if out is None:
        out = _new((rows, k), torch.float32, blocks.device, stream)
    _check(lib().ft_dequant(TYPES[w], _ptr(blocks), rows, k, _ptr(out), _stream(stream)), "ft_dequant")
    return out


def mul_mat_vec_q(w: str, W: torch.Tensor, n: int, k: int, act: str, xq: torch.Tensor, t: int,
                  out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    _dev(W, "W")
    _dev(xq, "xq")
    if out is None:
        out = _new((t, n), torch.float32, W.device, stream)
    _check(lib().ft_mul_mat_vec_q(TYPES[w], _ptr(W), n, k, TYPES[act], _ptr(xq), t, _ptr(out), out.shape[-1],
                                  _stream(stream)), "ft_mul_mat_vec_q")
    return out


def moe_route(logits: torch.Tensor, topk: int, ids: torch.Tensor | None = None, w: torch.Tensor | None = None,
              stream=None):
    _dev(logits, "logits")
    t, e = logits.shape
    if ids is None:
        ids = _new((t, topk), torch.int32, logits.device, stream)
    if w is None:
        w = _new((t, topk), torch.float32, logits.device, stream)
    _check(lib().ft_moe_route(_ptr(logits), t, e, topk, _ptr(ids), _ptr(w), _stream(stream)), "ft_moe_route")
    return ids, w


def _float_type(t: torch.Tensor, name: str) -> int:
    ty = FLOATS.get(t.dtype)
    if ty is None:
        raise ValueError(f"{name} must be float32, float16 or bfloat16, not {t.dtype}")
    return ty


def _plain(t: torch.Tensor, name: str, dtype, shape: tuple, device) -> int:
    """Pointer of a contiguous tensor of this type, shape and device."""
    if t.dtype is not dtype or t.shape != shape or t.device != device or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {shape} on {device}, "
                         f"not {t.dtype} {tuple(t.shape)} on {t.device}")
    return t.data_ptr()


def _call(name: str, device, stream, *args) -> None:
    """The entry point `name` on the caller's stream, or the current one of `device`, which the library then sees as
    its current device (torch's own handles of both: its Stream objects cost more than the rest of a small call)."""
    f = getattr(lib(), name)
    if stream is None and device.index == torch._C._cuda_getDevice():
        status = f(*args, torch._C._cuda_getCurrentRawStream(device.index))
    else:
        if stream is not None and stream.device != device:
            raise ValueError(f"the stream is on {stream.device}, the tensors on {device}")
        with torch.cuda.device(device):
            s = stream if stream is not None else torch.cuda.current_stream(device)
            status = f(*args, s.cuda_stream)
    _check(status, name)


def moe_route_ex(logits: torch.Tensor, topk: int, score: str = "softmax", bias: torch.Tensor | None = None,
                 n_group: int = 1, topk_group: int | None = None, group_top: int = 1, renorm: bool = True,
                 scale: float = 1.0, ids: torch.Tensor | None = None, w: torch.Tensor | None = None, stream=None):
    """ids, w of the topk experts per row of logits ((t, n_expert), rows may be strided): score "softmax" (over all
    experts) or "sigmoid"; the choice by score + bias among the topk_group best of n_group groups (a group's value:
    the sum of its group_top largest choices); w the scores, over their sum with renorm, times scale."""
    if not logits.is_cuda:
        raise ValueError("logits must be a device tensor")
    ty = _float_type(logits, "logits")
    if score not in ("softmax", "sigmoid"):
        raise ValueError(f"score must be softmax or sigmoid, not {score}")
    t, e = logits.shape
    ld, step = logits.stride()
    if e > 1 and step != 1 or (t > 1 and ld < e):
        raise ValueError("logits must have unit element stride and rows at least n_expert apart")
    if not scale:
        raise ValueError("scale must not be 0")
    if n_group < 1 or topk_group is not None and topk_group < 1 or group_top < 1 or topk < 1:
        raise ValueError("topk, n_group, topk_group and group_top start at 1")
    dev = logits.device
    if ids is None:
        ids = _new((t, topk), torch.int32, dev, stream)
    if w is None:
        w = _new((t, topk), torch.float32, dev, stream)
    o = _RouteOpts(score == "sigmoid", None if bias is None else _plain(bias, "bias", torch.float32, (e,), dev), n_group,
                   topk_group or 0, group_top, not renorm, scale)
    _call("ft_moe_route_ex", dev, stream, logits.data_ptr(), ty, t, e, ld if t > 1 else e, topk, ctypes.byref(o),
          _plain(ids, "ids", torch.int32, (t, topk), dev), _plain(w, "w", torch.float32, (t, topk), dev))
    return ids, w


def moe_sort(ids: torch.Tensor, n_expert: int, stream=None):
    _dev(ids, "ids")
    t, topk = ids.shape
    counts = _new(n_expert, torch.int32, ids.device, stream)
    offsets = _new(n_expert + 1, torch.int32, ids.device, stream)
    pairs = _new(t * topk, torch.int32, ids.device, stream)
    _check(lib().ft_moe_sort(_ptr(ids), t, topk, n_expert, _ptr(counts), _ptr(offsets), _ptr(pairs),
                             _stream(stream)), "ft_moe_sort")
    return counts, offsets, pairs


def _moe(entry: str, w: str, w_gate, w_up, w_down, n_expert: int, hidden: int, inter: int, act: str,
         x: torch.Tensor, ids, expert_w, out, route: int, taps, in_hq, direct_max_t: int, stream,
         logits=None, topk=None, ids_out=None, w_out=None) -> torch.Tensor:
    for nm, tt in (("w_gate", w_gate), ("w_up", w_up), ("w_down", w_down), ("x", x), ("ids", ids),
                   ("expert_w", expert_w), ("logits", logits), ("ids_out", ids_out), ("w_out", w_out)):
        if tt is not None:
            _dev(tt, nm)
    t = x.shape[0]
    if topk is None:
        topk = ids.shape[1]
    if out is None:
        out = _new((t, hidden), torch.float32, x.device, stream)
    taps = taps or {}
    opts = _MoeOpts(route, direct_max_t, *(_ptr(taps.get(k)) for k in ("g", "u", "h", "hq", "down")), _ptr(in_hq),
                    _ptr(logits), _ptr(ids_out), _ptr(w_out))
    _check(getattr(lib(), entry)(TYPES[w], _ptr(w_gate), _ptr(w_up), _ptr(w_down), n_expert, hidden, inter,
                                 TYPES[act], _ptr(x), t, _ptr(ids), _ptr(expert_w), topk, _ptr(out),
                                 ctypes.byref(opts), _stream(stream)), entry)
    return out


def moe_q_vec(w: str, w_gate, w_up, w_down, n_expert: int, hidden: int, inter: int, act: str,
              x: torch.Tensor, ids, expert_w, out: torch.Tensor | None = None,
              route: int = 0, taps: dict | None = None, in_hq: torch.Tensor | None = None,
              direct_max_t: int = 0, stream=None, logits=None, topk=None, ids_out=None,
              w_out=None) -> torch.Tensor:
    """taps: optional dict of preallocated device tensors g, u, h, hq, down.  With
    logits ([t][n_expert]) the layer routes itself (ids / expert_w may be None;
    topk is then required) and ids_out / w_out receive the routing."""
    return _moe("ft_moe_q_vec", w, w_gate, w_up, w_down, n_expert, hidden, inter, act, x, ids, expert_w, out,
                route, taps, in_hq, direct_max_t, stream, logits, topk, ids_out, w_out)


def moe_q_vec_noalloc(w: str, w_gate, w_up, w_down, n_expert: int, hidden: int, inter: int, act: str,
                      x: torch.Tensor, ids: torch.Tensor, expert_w: torch.Tensor, out: torch.Tensor | None = None,
                      route: int = 0, taps: dict | None = None, in_hq: torch.Tensor | None = None,
                      direct_max_t: int = 0, stream=None) -> torch.Tensor:
    """As moe_q_vec, with the library's fixed per-GPU scratch instead of the stream's pool."""
    return _moe("ft_moe_q_vec_noalloc", w, w_gate, w_up, w_down, n_expert, hidden, inter, act, x, ids, expert_w,
                out, route, taps, in_hq, direct_max_t, stream)


def grouped_gemm_q(w: str, W: torch.Tensor, n_expert: int, n: int, k: int, act: str, xq: torch.Tensor,
                   x_per_pair: bool, ids: torch.Tensor, out: torch.Tensor | None = None,
                   stream=None) -> torch.Tensor:
    _dev(W, "W")
    _dev(xq, "xq")
    _dev(ids, "ids")
    t, topk = ids.shape
    if out is None:
        out = _new((t * topk, n), torch.float32, W.device, stream)
    _check(lib().ft_grouped_gemm_q(TYPES[w], _ptr(W), n_expert, n, k, TYPES[act], _ptr(xq),
                                   1 if x_per_pair else 0, _ptr(ids), t, topk, _ptr(out), _stream(stream)),
           "ft_grouped_gemm_q")
    return out


def debug_block_dots(w: str, W: torch.Tensor, n: int, k: int, act: str, xq: torch.Tensor, t: int,
                     stream=None) -> torch.Tensor:
    _dev(W, "W")
    _dev(xq, "xq")
    sub = 16 if w in ("Q6_K", "Q2_K", "Q3_K") else 32
    out = _new((t, n, k // sub), torch.int32, W.device, stream)
    _check(lib().ft_debug_block_dots(TYPES[w], _ptr(W), n, k, TYPES[act], _ptr(xq), t, _ptr(out),
                                     _stream(stream)), "ft_debug_block_dots")
    return out


def debug_ceiling(which: str, buf: torch.Tensor | None = None, iters: int = 0, out: torch.Tensor | None = None,
                  stream=None) -> None:
    """Enqueue one measurement microkernel: "stream_read" over buf, "mfma_i8"
    (K = 32), "mfma_i8_k64" or "dot4" for iters rounds.  out: a device int32 scalar
    (allocated if None)."""
    code = {"stream_read": 0, "mfma_i8": 1, "dot4": 2, "mfma_i8_k64": 3}[which]
    dev = buf.device if buf is not None else torch.device("cuda")
    if out is None:
        with _on(stream):
            out = torch.zeros(1, dtype=torch.int32, device=dev)
    nbytes = 0
    if buf is not None:
        _dev(buf, "buf")
        nbytes = buf.numel() * buf.element_size()
    _check(lib().ft_debug_ceiling(code, _ptr(buf) if buf is not None else None, nbytes, iters, _ptr(out),
                                  _stream(stream)), "ft_debug_ceiling")


def scratch_reserve(nbytes: int, stream=None) -> None:
    _check(lib().ft_scratch_reserve(_stream(stream), nbytes), "ft_scratch_reserve")


def moe_scratch_bytes(w: str, act: str, n_expert: int, hidden: int, inter: int, t: int, topk: int) -> int:
    return lib().ft_moe_scratch_bytes(TYPES[w], TYPES[act], n_expert, hidden, inter, t, topk)


# ---------------------------------------------------------------------------
# paged, block-quantized key/value cache and the attention over it
# ---------------------------------------------------------------------------
def kv_page_bytes(ty: str, page_size: int, n_kv_head: int, head_dim: int) -> int:
    """Bytes of one page of one side (keys or values) of a cache."""
    n = lib().ft_kv_page_bytes(TYPES[ty], page_size, n_kv_head, head_dim)
    if not n:
        raise FtError(3, f"no cache pages of {ty}, {page_size} tokens, {n_kv_head} heads of {head_dim}")
    return n


class KvCache:
    """A paged key/value cache: the caller's two page pools (uint8, n_pages * kv_page_bytes each, any shape) and what
    they hold.  Slot s is token s % page_size of page s // page_size."""

    def __init__(self, k_pages: torch.Tensor, v_pages: torch.Tensor, page_size: int, n_kv_head: int, head_dim: int,
                 k: str = "Q8_0", v: str = "Q8_0"):
        kb, vb = (kv_page_bytes(ty, page_size, n_kv_head, head_dim) for ty in (k, v))
        for t, name in ((k_pages, "k_pages"), (v_pages, "v_pages")):
            _dev(t, name)
            if t.dtype != torch.uint8:
                raise ValueError(f"{name} must be uint8")
        n = k_pages.numel() // kb
        if not n or k_pages.numel() != n * kb or v_pages.numel() != n * vb:
            raise ValueError(f"the pools hold {k_pages.numel()} and {v_pages.numel()} bytes: want a whole number of "
                             f"pages, the same for both, of {kb} and {vb} bytes")
        if v_pages.device != k_pages.device:
            raise ValueError(f"k_pages are on {k_pages.device}, v_pages on {v_pages.device}")
        self.k_pages, self.v_pages, self.device = k_pages, v_pages, k_pages.device
        self.k, self.v = k, v
        self.n_pages, self.page_size, self.n_kv_head, self.head_dim = n, page_size, n_kv_head, head_dim
        self._c = _KvCache(TYPES[k], TYPES[v], k_pages.data_ptr(), v_pages.data_ptr(), n, page_size, n_kv_head, head_dim)
        self._ref, self._at = ctypes.byref(self._c), ctypes.addressof(self._c)

    @classmethod
    def empty(cls, n_pages: int, page_size: int, n_kv_head: int, head_dim: int, k: str = "Q8_0", v: str = "Q8_0",
              device="cuda") -> "KvCache":
        """A cache with pools of its own (not cleared: a slot is read only after it was written)."""
        pools = [torch.empty((n_pages, kv_page_bytes(ty, page_size, n_kv_head, head_dim)), dtype=torch.uint8,
                             device=device) for ty in (k, v)]
        return cls(*pools, page_size, n_kv_head, head_dim, k, v)


def _rows(t: torch.Tensor, name: str, shape: tuple, dtype, device) -> tuple:
    """Strides of a (tokens, heads, dim) tensor."""
    st = t.stride()
    if t.shape != shape or t.dtype is not dtype or t.device != device or st[2] != 1:
        raise ValueError(f"{name} must be {shape} {dtype} on {device} with unit element stride, "
                         f"not {tuple(t.shape)} {t.dtype} on {t.device} with strides {st}")
    return st


def kv_store(cache: KvCache, k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor, stream=None) -> None:
    """Quantize k, v ((t, n_kv_head, head_dim), float32, float16 or bfloat16, strided tokens and heads) into the slots
    (int64 (t,), distinct; a negative one is skipped)."""
    t, dev = k.shape[0], cache.device
    ty, shape = _float_type(k, "k"), (t, cache.n_kv_head, cache.head_dim)
    ks, vs = _rows(k, "k", shape, k.dtype, dev), _rows(v, "v", shape, k.dtype, dev)
    _call("ft_kv_store", dev, stream, cache._ref, ty, k.data_ptr(), ks[0], ks[1], v.data_ptr(), vs[0], vs[1],
          _plain(slots, "slots", torch.int64, (t,), dev), t)


def kv_load(cache: KvCache, slots: torch.Tensor, dtype=torch.float32, k: torch.Tensor | None = None,
            v: torch.Tensor | None = None, stream=None):
    """The slots' rows as plain numbers: (k, v), each (t, n_kv_head, head_dim) of dtype, into the given tensors where
    there are any (whose type then counts).  A negative slot gives zeros."""
    ext = _ext or _marshalling()
    if not isinstance(ext, ImportError):
        return ext.kv_load(cache._at, cache.k_pages, slots, dtype, k, v, stream)
    # with the library alone: the same from here, 2 us a call longer
    t, dev = slots.shape[0], cache.device
    shape = (t, cache.n_kv_head, cache.head_dim)
    if k is not None or v is not None:
        dtype = (k if k is not None else v).dtype
    if dtype not in FLOATS:
        raise ValueError(f"dtype must be float32, float16 or bfloat16, not {dtype}")
    k, v = (_new(shape, dtype, dev, stream) if x is None else x for x in (k, v))
    ks, vs = _rows(k, "k", shape, dtype, dev), _rows(v, "v", shape, dtype, dev)
    _call("ft_kv_load", dev, stream, cache._ref, _plain(slots, "slots", torch.int64, (t,), dev), t, FLOATS[dtype],
          k.data_ptr(), ks[0], ks[1], v.data_ptr(), vs[0], vs[1])
    return k, v


def attn_kv_scratch_bytes(cache: KvCache, n_tok: int, n_head: int, n_seq: int, max_kv: int, causal: bool = True,
                          window: int = 0, prefix: bool = False, n_shared: int = 0) -> int:
    """Bytes of a workspace that is enough for attn_kv at these sizes and any smaller max_kv (prefix: a prefix_len will
    be given).  A smaller batch can take more: a workspace for several takes the largest of their sizes."""
    o = _AttnOpts(0.0, 0.0, not causal, window, None, 1 if prefix else None, n_shared, None, 0)
    return lib().ft_attn_kv_scratch_bytes(cache._ref, n_tok, n_head, n_seq, max_kv, ctypes.byref(o))


def attn_kv(cache: KvCache, q: torch.Tensor, table: torch.Tensor, kv_len: torch.Tensor, q_start: torch.Tensor,
            max_kv: int | None = None, out: torch.Tensor | None = None, scale: float | None = None,
            causal: bool = True, window: int = 0, softcap: float = 0.0, slopes: torch.Tensor | None = None,
            prefix_len: torch.Tensor | None = None, n_shared: int = 0, workspace: torch.Tensor | None = None,
            stream=None) -> torch.Tensor:
    """Attention of q ((n_tok, n_head, head_dim), strided tokens and heads) over the cache.  table: int32 (n_seq,
    pages) page ids; kv_len: int32 (n_seq,); q_start: int32 (n_seq + 1,), sequence i's query tokens are
    q_start[i] .. q_start[i+1] - 1, the newest of its kv_len keys.  max_kv: a bound of kv_len (default: what the table
    holds).  window: a token sees its last `window` keys; prefix_len (int32 (n_seq,)): leading keys that all tokens
    see; slopes (float32 (n_head,)): a bias of -slope * distance; n_shared: leading keys that all sequences share
    (pages of table row 0).  workspace: uint8, attn_kv_scratch_bytes (default: the stream's pool)."""
    if q.dim() != 3:
        raise ValueError("q must be (n_tok, n_head, head_dim)")
    ty, dev, shape = _float_type(q, "q"), cache.device, q.shape
    n_tok, n_head, dim = shape
    if dim != cache.head_dim:
        raise ValueError(f"q has rows of {dim}, the cache of {cache.head_dim}")
    qs = _rows(q, "q", shape, q.dtype, dev)
    n_seq = kv_len.shape[0]
    ld, step = table.stride() if table.dim() == 2 else (0, 0)
    if step != 1 or table.shape[0] != n_seq or table.dtype is not torch.int32 or table.device != dev:
        raise ValueError(f"table must be int32 (n_seq, pages) on {dev} with unit element stride")
    cols = table.shape[1]
    if scale is not None and not scale:
        raise ValueError("scale must not be 0")
    if out is None:
        out = _new(shape, q.dtype, dev, stream)
    os_ = _rows(out, "out", shape, q.dtype, dev)
    o = _AttnOpts(scale or 0.0, softcap, not causal, window,
                  None if slopes is None else _plain(slopes, "slopes", torch.float32, (n_head,), dev),
                  None if prefix_len is None else _plain(prefix_len, "prefix_len", torch.int32, (n_seq,), dev), n_shared,
                  None, 0)
    if workspace is not None:
        if workspace.device != dev or not workspace.is_contiguous():
            raise ValueError(f"workspace must be contiguous on {dev}")
        o.workspace, o.workspace_bytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    _call("ft_attn_kv", dev, stream, cache._ref, ty, q.data_ptr(), qs[0], qs[1], n_tok, n_head,
          _plain(q_start, "q_start", torch.int32, (n_seq + 1,), dev), _plain(kv_len, "kv_len", torch.int32, (n_seq,), dev),
          table.data_ptr(), ld if n_seq > 1 else cols, cols, n_seq,
          cols * cache.page_size if max_kv is None else max_kv, out.data_ptr(), os_[0], os_[1], ctypes.byref(o))
    return out


# ---------------------------------------------------------------------------
# rotary positions
# ---------------------------------------------------------------------------
def rope_freqs(rot_dim: int, base: float = 10000.0, scaling: str | None = None, factor: float = 1.0,
               original: int = 8192, low: float = 1.0, high: float | None = None):
    """(freqs, scale) for rope_table: the angles per position of rot_dim / 2 pairs, a list of floats, and the factor of
    their cosines and sines.  scaling stretches positions past the `original` ones that a model was trained on by
    `factor`: "linear" (all pairs alike), "ntk" (by the base, NTK-aware), "blend" (pairs that turn fewer than `low` times over
    the original positions stretch, those of more than `high` (default: 4) times do not, linear between: by turns; model
    configurations call this form "llama3"), "ramp" (the same, `high` 32 by default, linear by the pair's number, with the
    cosines and sines scaled by 0.1 ln(factor) + 1: YaRN, Peng et al. 2023)."""
    if high is None:
        high = 4.0 if scaling == "blend" else 32.0
    if rot_dim < 2 or rot_dim % 2:
        raise ValueError("rot_dim must be even")
    if not base > 1 or not factor > 0:
        raise ValueError("base must be above 1 and factor above 0")
    half = rot_dim // 2
    if scaling == "ntk" and half > 1:
        base *= factor ** (half / (half - 1))
    f = [base ** (-j / half) for j in range(half)]
    if scaling in (None, "ntk"):
        return f, 1.0
    if scaling == "linear":
        return [x / factor for x in f], 1.0
    if scaling not in ("blend", "ramp"):
        raise ValueError(f"scaling must be linear, ntk, blend or ramp, not {scaling}")
    if not 0 < low < high:
        raise ValueError("low must be above 0 and below high")
    if scaling == "blend":
        keep = [(x * original / (2 * math.pi) - low) / (high - low) for x in f]
    else:  # the pair's number at which a pair turns so many times
        first, last = (half * math.log(original / (n * 2 * math.pi)) / math.log(base) for n in (high, low))
        first, last = max(math.floor(first), 0), min(math.ceil(last), rot_dim - 1)
        keep = [1 - (j - first) / (max(last - first, 0.001)) for j in range(half)]
    keep = [min(1.0, max(0.0, x)) for x in keep]
    scale = 0.1 * math.log(factor) + 1.0 if scaling == "ramp" and factor > 1 else 1.0
    return [x * k + x / factor * (1 - k) for x, k in zip(f, keep)], scale


def rope_table(n_pos: int, freqs, scale: float = 1.0, device="cuda", out: torch.Tensor | None = None,
               stream=None) -> torch.Tensor:
    """The table of rope and kv_store_rope, float32 (n_pos, 2 * len(freqs)): row p the cosines, then the sines of
    p * freqs, times scale, computed in 64 bits.  freqs: a list, or a float64 tensor on the device."""
    if not isinstance(freqs, torch.Tensor):
        with _on(stream):  # this call's own: nobody else can keep it until the stream has read it
            freqs = torch.tensor(freqs, dtype=torch.float64, device=device)
    dev, half = freqs.device, freqs.numel()
    if not freqs.is_cuda:
        raise ValueError("freqs must be a list or a device tensor")
    if out is None:
        out = _new((n_pos, 2 * half), torch.float32, dev, stream)
    _call("ft_rope_table", dev, stream, _plain(freqs, "freqs", torch.float64, (half,), dev), half, n_pos, scale,
          _plain(out, "out", torch.float32, (n_pos, 2 * half), dev))
    return out


def rope(x: torch.Tensor, positions: torch.Tensor, table: torch.Tensor, interleaved: bool = False,
         weight: torch.Tensor | None = None, eps: float = 1e-6, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """The rows of x ((t, heads, dim), strided tokens and heads) turned by their token's position (int32 (t,)): pairs
    (j, j + rot_dim / 2), or neighbours with interleaved; elements from the table's width on stay.  weight (float32
    (dim,)): each row is first divided by its root mean square (with eps) and multiplied by weight.  out may be x."""
    return _bind().rope(x, positions, table, interleaved, weight, eps, out, stream)


def kv_store_rope(cache: KvCache, q: torch.Tensor | None, k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor,
                  positions: torch.Tensor, table: torch.Tensor, interleaved: bool = False, q_weight: torch.Tensor | None = None,
                  k_weight: torch.Tensor | None = None, eps: float = 1e-6, q_out: torch.Tensor | None = None, stream=None):
    """kv_store with the keys turned (and normed, with k_weight) on the way, and the queries q ((t, heads, head_dim),
    any number of heads, or None) turned in the same launch, as rope does: returns them (in q_out, which may be q)."""
    return _bind().kv_store_rope(cache._at, cache.k_pages, q, k, v, slots, positions, table, interleaved, q_weight, k_weight, eps,
                                 q_out, stream)


# ---------------------------------------------------------------------------
# the norm around a block
# ---------------------------------------------------------------------------
def norm(x: torch.Tensor, weight: torch.Tensor | None = None, bias: torch.Tensor | None = None,
         residual: torch.Tensor | None = None, post_weight: torch.Tensor | None = None, post_bias: torch.Tensor | None = None,
         post: bool | None = None, gate: torch.Tensor | None = None, scale: float = 1.0, kind: str = "rms", eps: float = 1e-6,
         act: str | None = None, rows: bool | None = None, r: torch.Tensor | None = None, out: torch.Tensor | None = None,
         xq: torch.Tensor | None = None, stream=None):
    """(r, n, xq) of x ((t, width), rows may be strided, as those of all others): r = residual + scale * gate * x, x first
    normed with `post` (by default where there is a post_weight); n = norm(r) * weight + bias.  gate: (t, width), or
    (1, width) or (width,) for all rows.  kind: "rms" or "layer".  act ("Q8_1", "Q8_0", "Q8_K"): n as quantized blocks,
    xq, and as rows only with rows=True; without act n is rows.  r is x where nothing is done to it.  What is not
    computed is None.  r and out may be x or residual."""
    if kind not in ("rms", "layer"):
        raise ValueError(f"kind must be rms or layer, not {kind}")
    if act is not None and act not in ACTS:
        raise ValueError(f"act must be Q8_1, Q8_0 or Q8_K, not {act}")
    return _bind().norm(x, weight, bias, residual, post_weight, post_bias, post, gate, scale, kind == "layer", eps,
                        -1 if act is None else TYPES[act], rows, r, out, xq, stream)


# ---------------------------------------------------------------------------
# low-rank adapters
# ---------------------------------------------------------------------------
def lora_scratch_bytes(t: int, k: int, n_adapter: int, rank: int) -> int:
    """Bytes of a workspace that is enough for lora at these sizes and any smaller t."""
    n = lib().ft_lora_scratch_bytes(t, k, n_adapter, rank)
    if not n:
        raise FtError(3, f"no adapters for {t} rows of {k}, {n_adapter} of rank {rank}")
    return n


def lora(x: torch.Tensor, a: torch.Tensor, b: torch.Tensor, ids: torch.Tensor, y: torch.Tensor | None = None,
         scales: torch.Tensor | None = None, ranks: torch.Tensor | None = None, out: torch.Tensor | None = None,
         workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """y + scales[i] * b[i] (a[i] x) for every row of x ((t, k), rows may be strided) with the adapter i = ids (int32
    (t,)) of a (n_adapter, rank, k) and b (n_adapter, n, rank), which share a type; an id outside them leaves y's row.  y
    (default: zeros) and out are float32 (t, n); out may be y.  scales float32, ranks int32 (n_adapter,): an
    adapter's own rank, what a and b hold beyond is not used.  workspace: uint8, lora_scratch_bytes (default: the
    stream's pool)."""
    return _bind().lora(x, a, b, ids, y, scales, ranks, out, workspace, stream)
