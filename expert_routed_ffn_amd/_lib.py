"""ctypes binding of libmoe.so.

Argument marshalling only: every step of the layer runs in the HIP kernels of
libmoe.so.  PyTorch supplies device memory and the current stream.  If the
library is not built, importing this module raises ImportError; there is no
fallback.
"""
from __future__ import annotations

import ctypes
import functools
import os
import re

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libmoe.so")
HEADER = os.path.join(os.path.dirname(_PKG), "include", "moe.h")

MOE_OK, MOE_EINVAL, MOE_EUNSUPPORTED, MOE_EWORKSPACE, MOE_EHIP, MOE_ENOTPINNED, MOE_ECAPACITY = range(7)
MOE_F32, MOE_BF16, MOE_I8 = 0, 1, 2
PATHS = {"auto": 0, "gemv": 1, "mfma": 2}


class MoeError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{message} (status {status})")
        self.status = status


class QLayer(ctypes.Structure):
    _fields_ = [("E", ctypes.c_int), ("H", ctypes.c_int), ("I", ctypes.c_int), ("bits", ctypes.c_int),
                ("base", ctypes.c_void_p), ("stride", ctypes.c_int64), ("slot_map", ctypes.c_void_p)]


class SlotStats(ctypes.Structure):
    _fields_ = [("hits", ctypes.c_uint64), ("misses", ctypes.c_uint64), ("bytes_h2d", ctypes.c_uint64),
                ("resolves", ctypes.c_uint64), ("evictions", ctypes.c_uint64)]


COPY_FN = ctypes.CFUNCTYPE(None, ctypes.c_void_p, ctypes.c_int, ctypes.c_int, ctypes.c_int)


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is not built: run `python -m expert_routed_ffn_amd.build` "
                          "(or __graft_entry__.build()) first")
    L = ctypes.CDLL(LIB_PATH)
    i32, i64, vp, sz = ctypes.c_int, ctypes.c_int64, ctypes.c_void_p, ctypes.c_size_t
    st = ctypes.c_int
    L.moe_abi_version.restype = i32
    L.moe_last_error.restype = ctypes.c_char_p
    L.moe_status_string.restype = ctypes.c_char_p
    L.moe_status_string.argtypes = [st]
    L.moe_expert_bytes.restype = sz
    L.moe_expert_bytes.argtypes = [i32, i32, i32]
    L.moe_route_topk.restype = st
    L.moe_route_topk.argtypes = [vp, i32, i32, i32, vp, vp, vp]
    L.moe_router_logits.restype = st
    L.moe_router_logits.argtypes = [vp, i32, vp, i32, i32, i32, vp, vp]
    L.moe_router_topk.restype = st
    L.moe_router_topk.argtypes = [vp, i32, vp, i32, i32, i32, i32, vp, vp, vp, vp]
    L.moe_dispatch_workspace_bytes.restype = sz
    L.moe_dispatch_workspace_bytes.argtypes = [i32, i32, i32]
    L.moe_dispatch.restype = st
    L.moe_dispatch.argtypes = [vp, i32, i32, i32, vp, vp, vp, vp, vp, vp, sz, vp]
    L.moe_expert_ffn_workspace_bytes.restype = sz
    L.moe_expert_ffn_workspace_bytes.argtypes = [ctypes.POINTER(QLayer), i32, i32, i32]
    L.moe_expert_ffn_q.restype = st
    L.moe_expert_ffn_q.argtypes = [ctypes.POINTER(QLayer), vp, i32, i32, i32, vp, vp, vp, vp, vp, i32, i32, vp, sz,
                                   vp]
    L.moe_combine.restype = st
    L.moe_combine.argtypes = [vp, i32, vp, i32, i32, i32, vp, i32, vp, vp, vp]
    L.moe_slot_table_create.restype = st
    L.moe_slot_table_create.argtypes = [i32, i32, i32, sz, vp, vp, vp, vp, ctypes.POINTER(vp)]
    L.moe_slot_table_preload.restype = st
    L.moe_slot_table_preload.argtypes = [vp, vp, i32, vp]
    L.moe_slot_table_resolve.restype = st
    L.moe_slot_table_resolve.argtypes = [vp, i32, vp, vp, vp]
    L.moe_slot_table_stats.restype = st
    L.moe_slot_table_stats.argtypes = [vp, ctypes.POINTER(SlotStats)]
    L.moe_slot_table_map_host.restype = st
    L.moe_slot_table_map_host.argtypes = [vp, vp]
    L.moe_slot_table_device_bytes.restype = sz
    L.moe_slot_table_device_bytes.argtypes = [i32, i32, i32]
    L.moe_slot_table_enable_device.restype = st
    L.moe_slot_table_enable_device.argtypes = [vp, vp, sz, vp]
    L.moe_slot_table_resolve_device.restype = st
    L.moe_slot_table_resolve_device.argtypes = [vp, i32, vp, vp, i32, vp]
    L.moe_slot_table_destroy.restype = None
    L.moe_slot_table_destroy.argtypes = [vp]
    L.moe_slot_table_create_host.restype = st
    L.moe_slot_table_create_host.argtypes = [i32, i32, i32, COPY_FN, vp, ctypes.POINTER(vp)]
    L.moe_slot_table_resolve_host.restype = st
    L.moe_slot_table_resolve_host.argtypes = [vp, i32, vp, i32]
    L.moe_layer_decode_workspace_bytes.restype = sz
    L.moe_layer_decode_workspace_bytes.argtypes = [ctypes.POINTER(QLayer), i32, i32]
    L.moe_layer_decode.restype = st
    L.moe_layer_decode.argtypes = [ctypes.POINTER(QLayer), vp, vp, i32, i32, i32, vp, i32, vp, vp, vp, vp, vp, vp, vp,
                                   vp, i32, vp, vp, vp, sz, vp]
    L.moe_layer_decode_noalloc_max_bytes.restype = sz
    L.moe_layer_decode_noalloc_max_bytes.argtypes = []
    L.moe_layer_decode_noalloc.restype = st
    L.moe_layer_decode_noalloc.argtypes = [ctypes.POINTER(QLayer), vp, vp, i32, i32, i32, vp, i32, vp, vp, vp, vp, vp,
                                           vp, vp, vp, i32, vp, vp, vp]
    L.moe_layer_decode_slots.restype = st
    L.moe_layer_decode_slots.argtypes = [ctypes.POINTER(QLayer), vp, i32, vp, vp, i32, i32, i32, vp, i32, vp, vp, vp,
                                         vp, vp, vp, vp, vp, i32, vp, vp, vp, sz, vp]
    L.moe_balance_loss_workspace_bytes.restype = sz
    L.moe_balance_loss_workspace_bytes.argtypes = [i32, i32]
    L.moe_balance_loss.restype = st
    L.moe_balance_loss.argtypes = [vp, vp, vp, i32, i32, i32, vp, vp, vp, vp, sz, vp]
    L.moe_route_backward.restype = st
    L.moe_route_backward.argtypes = [vp, vp, vp, vp, vp, vp, vp, i32, i32, i32, vp, vp]
    L.moe_combine_backward.restype = st
    L.moe_combine_backward.argtypes = [vp, i32, vp, vp, i32, i32, i32, i32, vp, vp, vp]
    L.moe_linear_workspace_bytes.restype = sz
    L.moe_linear_workspace_bytes.argtypes = [i32, i32, i32, i32, i32, i32]
    L.moe_linear.restype = st
    L.moe_linear.argtypes = [vp, i32, vp, vp, i32, vp, i32, i32, i32, i32, vp, i32, vp, vp, sz, vp]
    L.moe_linear_backward_workspace_bytes.restype = sz
    L.moe_linear_backward_workspace_bytes.argtypes = [i32, i32, i32, i32, i32, i32, i32, i32, i32]
    L.moe_linear_backward.restype = st
    L.moe_linear_backward.argtypes = [vp, i32, vp, vp, i32, vp, i32, i32, i32, i32, vp, i32, vp, i32, vp, vp, sz, vp]
    L.moe_linear_form.restype = st
    L.moe_linear_form.argtypes = [i32, i32, i32, i32, i32, i32, ctypes.POINTER(i32)]
    L.moe_linear_backward_form.restype = st
    L.moe_linear_backward_form.argtypes = [i32, i32, i32, i32, i32, i32, i32, i32, i32, ctypes.POINTER(i32)]
    f64 = ctypes.c_double
    L.moe_orthogonalize_workspace_bytes.restype = sz
    L.moe_orthogonalize_workspace_bytes.argtypes = [i32, i32, i32, i32]
    L.moe_orthogonalize.restype = st
    L.moe_orthogonalize.argtypes = [vp, i32, vp, f64, i32, i32, i32, i32, i32, vp, f64, vp, i32, vp, sz, vp]
    L.moe_orthogonalize_form.restype = st
    L.moe_orthogonalize_form.argtypes = [i32, i32, i32, i32, ctypes.POINTER(i32)]
    L.moe_quantize_rows.restype = st
    L.moe_quantize_rows.argtypes = [vp, i32, i32, i32, vp, vp, vp]
    L.moe_linear_q8_workspace_bytes.restype = sz
    L.moe_linear_q8_workspace_bytes.argtypes = [i32, i32, i32, i32, i32]
    L.moe_linear_q8.restype = st
    L.moe_linear_q8.argtypes = [vp, i32, vp, vp, vp, vp, i32, vp, i32, i32, i32, i32, vp, i32, vp, sz, vp]
    L.moe_linear_q8_form.restype = st
    L.moe_linear_q8_form.argtypes = [i32, i32, i32, i32, i32, ctypes.POINTER(i32)]
    L.moe_profile_next_launch.restype = st
    L.moe_profile_next_launch.argtypes = [i32, vp, vp]
    return L


lib = _load()


def header_functions() -> list[str]:
    """Names of the functions include/moe.h declares."""
    src = open(HEADER).read()
    src = re.sub(r"/\*.*?\*/", "", src, flags=re.S)
    return sorted(set(re.findall(r"\b(moe_[a-z0-9_]+)\s*\(", src)) - {"moe_copy_fn"})


def _check(status: int):
    if status != MOE_OK:
        raise MoeError(status, lib.moe_last_error().decode())


def _ptr(t: torch.Tensor | None):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream, device=None):
    if stream is None:
        return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)
    if isinstance(stream, torch.cuda.Stream):
        return ctypes.c_void_p(stream.cuda_stream)
    return ctypes.c_void_p(int(stream))


def _on(stream, device):
    """Context in which the binding allocates outputs and workspaces: the stream the kernels run on, so the
    caching allocator does not hand their memory to other work while the kernels are still queued."""
    import contextlib
    if stream is None:
        return contextlib.nullcontext()
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream), device=device)
    return torch.cuda.stream(stream)


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return MOE_F32
    if t.dtype == torch.bfloat16:
        return MOE_BF16
    raise TypeError(f"unsupported dtype {t.dtype} (float32 or bfloat16)")


def _need(t: torch.Tensor, name: str):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA (HIP) tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


KERNELS = {"route": 0, "dispatch": 1, "gemv_gateup": 2, "gemv_down": 3, "mfma_gateup": 4, "mfma_down": 5,
           "combine": 6, "decode_prep": 7, "router": 8, "balance": 9, "route_backward": 10, "combine_backward": 11,
           "linear": 12, "linear_backward": 13, "quantize": 14, "linear_q8": 15,
           "orthogonalize": 16}
ACTS = {"none": 0, "gelu": 1, "silu": 2, "swiglu": 3}


def profile_next_launch(kernel: str, start, stop):
    """Attach HIP events (raw hipEvent_t handles) to the next launch of `kernel` on this thread."""
    _check(lib.moe_profile_next_launch(KERNELS[kernel], ctypes.c_void_p(int(getattr(start, "value", start))),
                                       ctypes.c_void_p(int(getattr(stop, "value", stop)))))


def abi_version() -> int:
    return int(lib.moe_abi_version())


def expert_bytes(H: int, I: int, bits: int) -> int:
    return int(lib.moe_expert_bytes(H, I, bits))


# ---- moe_route_topk --------------------------------------------------------------

def route_topk(logits: torch.Tensor, k: int, ids: torch.Tensor | None = None, w: torch.Tensor | None = None,
               stream=None):
    _need(logits, "logits")
    T, E = logits.shape
    with _on(stream, logits.device):
        if ids is None:
            ids = torch.empty((T, k), dtype=torch.int32, device=logits.device)
        if w is None:
            w = torch.empty((T, k), dtype=torch.float32, device=logits.device)
    _check(lib.moe_route_topk(_ptr(logits), T, E, k, _ptr(ids), _ptr(w), _stream(stream, logits.device)))
    return ids, w


# ---- router projection ----------------------------------------------------------------

def router_logits(x: torch.Tensor, w_r: torch.Tensor, logits: torch.Tensor | None = None, stream=None):
    """logits [T, E] fp32 = x [T, H] (fp32 or bf16) . w_r [E, H] (bf16)^T."""
    _need(x, "x")
    _need(w_r, "w_r")
    if w_r.dtype != torch.bfloat16:
        raise TypeError("w_r must be bfloat16")
    T, H = x.shape
    E = w_r.shape[0]
    with _on(stream, x.device):
        if logits is None:
            logits = torch.empty((T, E), dtype=torch.float32, device=x.device)
    _check(lib.moe_router_logits(_ptr(x), _dtype_code(x), _ptr(w_r), T, H, E, _ptr(logits),
                                 _stream(stream, x.device)))
    return logits


def router_topk(x: torch.Tensor, w_r: torch.Tensor, k: int, logits: torch.Tensor | None = None,
                ids: torch.Tensor | None = None, w: torch.Tensor | None = None, stream=None):
    """Router projection then top-k: (logits, ids, w)."""
    _need(x, "x")
    _need(w_r, "w_r")
    T, H = x.shape
    E = w_r.shape[0]
    dev = x.device
    with _on(stream, dev):
        if logits is None:
            logits = torch.empty((T, E), dtype=torch.float32, device=dev)
        if ids is None:
            ids = torch.empty((T, k), dtype=torch.int32, device=dev)
        if w is None:
            w = torch.empty((T, k), dtype=torch.float32, device=dev)
    _check(lib.moe_router_topk(_ptr(x), _dtype_code(x), _ptr(w_r), T, H, E, k, _ptr(logits), _ptr(ids), _ptr(w),
                               _stream(stream, dev)))
    return logits, ids, w


# ---- moe_dispatch ------------------------------------------------------------------

class Dispatch:
    """Device outputs of moe_dispatch."""

    def __init__(self, T: int, k: int, E: int, device):
        n = T * k
        self.T, self.k, self.E = T, k, E
        self.offsets = torch.empty(E + 1, dtype=torch.int32, device=device)
        self.sorted_assign = torch.empty(max(n, 1), dtype=torch.int32, device=device)
        self.assign_pos = torch.empty(max(n, 1), dtype=torch.int32, device=device)
        self.active = torch.empty(max(min(E, n), 1), dtype=torch.int32, device=device)
        self.n_active = torch.empty(1, dtype=torch.int32, device=device)
        nb = int(lib.moe_dispatch_workspace_bytes(T, k, E))
        self.ws = torch.empty(max(nb, 1), dtype=torch.uint8, device=device)


def dispatch(ids: torch.Tensor, E: int, out: Dispatch | None = None, stream=None) -> Dispatch:
    _need(ids, "ids")
    T, k = ids.shape
    with _on(stream, ids.device):
        d = out if out is not None else Dispatch(T, k, E, ids.device)
    _check(lib.moe_dispatch(_ptr(ids), T, k, E, _ptr(d.offsets), _ptr(d.sorted_assign), _ptr(d.assign_pos),
                            _ptr(d.active), _ptr(d.n_active), _ptr(d.ws), d.ws.numel(), _stream(stream, ids.device)))
    return d


# ---- moe_expert_ffn_q ------------------------------------------------------------

class ExpertLayer:
    """One layer's quantized experts in device memory: expert e's blob at base + idx(e) * stride."""

    def __init__(self, E: int, H: int, I: int, bits: int, base: torch.Tensor, stride: int | None = None,
                 slot_map: torch.Tensor | None = None, base_offset: int = 0):
        _need(base, "base")
        self.E, self.H, self.I, self.bits = E, H, I, bits
        self.base = base  # keeps the storage alive
        self.stride = stride if stride is not None else expert_bytes(H, I, bits)
        self.slot_map = slot_map
        self.q = QLayer(E, H, I, bits, base.data_ptr() + base_offset, self.stride,
                        None if slot_map is None else slot_map.data_ptr())

    def workspace_bytes(self, T: int, k: int, path: str = "auto") -> int:
        return int(lib.moe_expert_ffn_workspace_bytes(ctypes.byref(self.q), T, k, PATHS[path]))


def expert_ffn_q(layer: ExpertLayer, x: torch.Tensor, k: int, d: Dispatch, y: torch.Tensor | None = None,
                 y_dtype=torch.float32, path: str = "auto", ws: torch.Tensor | None = None, stream=None):
    _need(x, "x")
    T, H = x.shape
    with _on(stream, x.device):
        if y is None:
            y = torch.empty((T, k, H), dtype=y_dtype, device=x.device)
        if ws is None:
            ws = torch.empty(max(layer.workspace_bytes(T, k, path), 1), dtype=torch.uint8, device=x.device)
    _need(y, "y")
    _check(lib.moe_expert_ffn_q(ctypes.byref(layer.q), _ptr(x), _dtype_code(x), T, k, _ptr(d.offsets),
                                _ptr(d.sorted_assign), _ptr(d.active), _ptr(d.n_active), _ptr(y), _dtype_code(y),
                                PATHS[path], _ptr(ws), ws.numel(), _stream(stream, x.device)))
    return y


# ---- moe_combine -------------------------------------------------------------------

def combine(y: torch.Tensor, w: torch.Tensor, residual: torch.Tensor | None = None, out: torch.Tensor | None = None,
            out_bf16: torch.Tensor | None = None, stream=None):
    _need(y, "y")
    _need(w, "w")
    T, k, H = y.shape
    with _on(stream, y.device):
        if out is None:
            out = torch.empty((T, H), dtype=torch.float32, device=y.device)
    r_t = MOE_F32 if residual is None else _dtype_code(residual)
    _check(lib.moe_combine(_ptr(y), _dtype_code(y), _ptr(w), T, k, H, _ptr(residual), r_t, _ptr(out),
                           _ptr(out_bf16), _stream(stream, y.device)))
    return out


# ---- whole layer (four calls in order) ---------------------------------------------

def layer_forward(layer: ExpertLayer, x: torch.Tensor, logits: torch.Tensor, k: int, residual=None,
                  y_dtype=torch.float32, path: str = "auto", out_bf16: torch.Tensor | None = None, bufs=None,
                  stream=None):
    """route -> dispatch -> expert FFN -> combine.  Returns (ids, w, dispatch, y, out)."""
    T = x.shape[0]
    if bufs is None:
        bufs = {}
    ids, w = route_topk(logits, k, bufs.get("ids"), bufs.get("w"), stream)
    d = dispatch(ids, layer.E, bufs.get("dispatch"), stream)
    y = expert_ffn_q(layer, x, k, d, bufs.get("y"), y_dtype, path, bufs.get("ws"), stream)
    out = combine(y, w, residual, bufs.get("out"), out_bf16, stream)
    return ids, w, d, y, out


# ---- fused decode step ------------------------------------------------------------

def _decode_buffers(layer, T, k, H, y_dtype, b, stream, dev):
    """Outputs and workspace of a decode step: the caller's from `b`, the rest allocated on `stream`."""
    with _on(stream, dev):
        ids = b.get("ids")
        if ids is None:
            ids = torch.empty((T, k), dtype=torch.int32, device=dev)
        w = b.get("w")
        if w is None:
            w = torch.empty((T, k), dtype=torch.float32, device=dev)
        d = b.get("dispatch") or Dispatch(T, k, layer.E, dev)
        y = b.get("y")
        if y is None:
            y = torch.empty((T, k, H), dtype=y_dtype, device=dev)
        out = b.get("out")
        if out is None:
            out = torch.empty((T, H), dtype=torch.float32, device=dev)
        ws = b.get("dws")
        if ws is None:
            ws = torch.empty(max(int(lib.moe_layer_decode_workspace_bytes(ctypes.byref(layer.q), T, k)), 1),
                             dtype=torch.uint8, device=dev)
    return ids, w, d, y, out, ws


def layer_decode(layer: ExpertLayer, x: torch.Tensor, logits: torch.Tensor, k: int, residual=None,
                 y_dtype=torch.float32, out_bf16: torch.Tensor | None = None, bufs=None, stream=None):
    """moe_layer_decode: the whole layer step (two launches for the decode shapes, else four).  Returns (ids, w, dispatch, y, out)."""
    _need(x, "x")
    _need(logits, "logits")
    T, H = x.shape
    dev = x.device
    ids, w, d, y, out, ws = _decode_buffers(layer, T, k, H, y_dtype, bufs or {}, stream, dev)
    r_t = MOE_F32 if residual is None else _dtype_code(residual)
    _check(lib.moe_layer_decode(ctypes.byref(layer.q), _ptr(logits), _ptr(x), _dtype_code(x), T, k, _ptr(residual),
                                r_t, _ptr(ids), _ptr(w), _ptr(d.offsets), _ptr(d.sorted_assign), _ptr(d.assign_pos),
                                _ptr(d.active), _ptr(d.n_active), _ptr(y), _dtype_code(y), _ptr(out), _ptr(out_bf16),
                                _ptr(ws), ws.numel(), _stream(stream, dev)))
    return ids, w, d, y, out


def layer_decode_noalloc(layer: ExpertLayer, x: torch.Tensor, logits: torch.Tensor, k: int, residual=None,
                         y_dtype=torch.float32, out_bf16: torch.Tensor | None = None, bufs=None, stream=None):
    """moe_layer_decode_noalloc: moe_layer_decode with the library's fixed device scratch as its workspace (no
    workspace argument; outputs from `bufs` or allocated here).  Returns (ids, w, dispatch, y, out)."""
    _need(x, "x")
    _need(logits, "logits")
    T, H = x.shape
    dev = x.device
    b = dict(bufs or {})
    b["dws"] = torch.empty(0, dtype=torch.uint8, device=dev)  # unused: the call takes no workspace
    ids, w, d, y, out, _ = _decode_buffers(layer, T, k, H, y_dtype, b, stream, dev)
    r_t = MOE_F32 if residual is None else _dtype_code(residual)
    _check(lib.moe_layer_decode_noalloc(ctypes.byref(layer.q), _ptr(logits), _ptr(x), _dtype_code(x), T, k,
                                        _ptr(residual), r_t, _ptr(ids), _ptr(w), _ptr(d.offsets),
                                        _ptr(d.sorted_assign), _ptr(d.assign_pos), _ptr(d.active), _ptr(d.n_active),
                                        _ptr(y), _dtype_code(y), _ptr(out), _ptr(out_bf16), _stream(stream, dev)))
    return ids, w, d, y, out


def noalloc_max_bytes() -> int:
    return int(lib.moe_layer_decode_noalloc_max_bytes())


def layer_decode_slots(table, l: int, layer: ExpertLayer, x: torch.Tensor, logits: torch.Tensor, k: int,
                       residual=None, y_dtype=torch.float32, out_bf16: torch.Tensor | None = None, bufs=None,
                       stream=None):
    """moe_layer_decode_slots: the layer step through `table` (device mode); `layer` is table.layer(l, ...)."""
    _need(x, "x")
    _need(logits, "logits")
    T, H = x.shape
    dev = x.device
    ids, w, d, y, out, ws = _decode_buffers(layer, T, k, H, y_dtype, bufs or {}, stream, dev)
    r_t = MOE_F32 if residual is None else _dtype_code(residual)
    _check(lib.moe_layer_decode_slots(ctypes.byref(layer.q), table.h, l, _ptr(logits), _ptr(x), _dtype_code(x), T, k,
                                      _ptr(residual), r_t, _ptr(ids), _ptr(w), _ptr(d.offsets), _ptr(d.sorted_assign),
                                      _ptr(d.assign_pos), _ptr(d.active), _ptr(d.n_active), _ptr(y), _dtype_code(y),
                                      _ptr(out), _ptr(out_bf16), _ptr(ws), ws.numel(), _stream(stream, dev)))
    return ids, w, d, y, out


def decode_workspace_bytes(layer: ExpertLayer, T: int, k: int) -> int:
    return int(lib.moe_layer_decode_workspace_bytes(ctypes.byref(layer.q), T, k))


# ---- training the router and the dense parts beside the experts ------------------------
#
# There is no autograd here: what these calls return is detached, whatever their inputs require, and each has its gradient
# as a call of its own.

_F32, _BF16, _I32 = torch.float32, torch.bfloat16, torch.int32


# What a call costs on the host decides how fast small steps run (a decode-size product's kernel takes 3 to 5 us), so
# the checks below are plain comparisons, and the current stream and device are asked for without their wrappers.
_current_stream = torch._C._cuda_getCurrentRawStream if hasattr(torch._C, "_cuda_getCurrentRawStream") else \
    (lambda index: torch.cuda.current_stream(index).cuda_stream)
_current_device = torch._C._cuda_getDevice if hasattr(torch._C, "_cuda_getDevice") else torch.cuda.current_device


def _arg(t: torch.Tensor, name: str, shape: tuple, dtypes: tuple, index: int | None = None):
    """Checks an argument's shape, type, layout and device; returns its address."""
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be {' or '.join(str(d) for d in dtypes)}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA (HIP) tensor")
    if index is not None and t.get_device() != index:
        raise ValueError(f"{name} is on {t.device}, the other tensors are on cuda:{index}")
    return t.data_ptr()


def _rows(t: torch.Tensor, name: str, dims: int):
    if t.dim() != dims:
        raise ValueError(f"{name} must have {dims} dimensions, got {t.dim()}")
    if max(t.shape) > 0x7FFFFFFF:  # (the library's sizes are 32-bit)
        raise ValueError(f"{name} must have less than 2^31 rows and columns, got {tuple(t.shape)}")
    return t.shape


def _ws(ws: torch.Tensor | None, need: int, like: torch.Tensor, index: int, stream):
    """The caller's workspace, or a new one of `need` bytes on like's device: (tensor to keep, address, bytes)."""
    if ws is None:
        if need == 0:
            return None, None, 0
        ws = _new(like, need, torch.uint8, stream)
    else:
        _arg(ws, "ws", ws.shape, (torch.uint8,), index)
    return ws, ws.data_ptr(), ws.numel()


def _launch(fn, index: int, stream, *args):
    """One library call on `stream` (or device `index`'s current stream) with that device current."""
    s = _current_stream(index) if stream is None else _stream(stream, index)
    if index != _current_device():
        with torch.cuda.device(index):
            status = fn(*args, s)
    else:
        status = fn(*args, s)
    if status != MOE_OK:
        _check(status)


def _new(like: torch.Tensor, shape, dtype, stream):
    """An uninitialised tensor on like's device, belonging to the stream that will write it."""
    if stream is None:
        return like.new_empty(shape, dtype=dtype)
    with _on(stream, like.device):
        return like.new_empty(shape, dtype=dtype)


def balance_loss(logits: torch.Tensor, ids: torch.Tensor, mask: torch.Tensor | None = None,
                 loss: torch.Tensor | None = None, counts: torch.Tensor | None = None,
                 lse: torch.Tensor | None = None, ws: torch.Tensor | None = None, stream=None):
    """moe_balance_loss: (loss [2] fp32, counts [E + 1] int32, lse [T] fp32) of logits [T, E] fp32 routed to ids
    [T, k]; loss[0] is the balance loss, loss[1] the mean squared log-sum-exp, counts[E] the number of tokens that
    take part.  mask [T] (bool or uint8) leaves padding out.  The losses are detached; their gradient is
    route_backward."""
    T, E = _rows(logits, "logits", 2)
    k = _rows(ids, "ids", 2)[1]
    a_logits = _arg(logits, "logits", (T, E), (_F32,))
    at = logits.get_device()
    a_ids = _arg(ids, "ids", (T, k), (_I32,), at)
    a_mask = None if mask is None else _arg(mask, "mask", (T,), (torch.bool, torch.uint8), at)
    if loss is None:
        loss = _new(logits, 2, _F32, stream)
    if counts is None:
        counts = _new(logits, E + 1, _I32, stream)
    if lse is None:
        lse = _new(logits, T, _F32, stream)
    ws, a_ws, n_ws = _ws(ws, lib.moe_balance_loss_workspace_bytes(T, E), logits, at, stream)
    _launch(lib.moe_balance_loss, at, stream, a_logits, a_ids, a_mask, T, E, k,
            _arg(loss, "loss", (2,), (_F32,), at), _arg(counts, "counts", (E + 1,), (_I32,), at),
            _arg(lse, "lse", (T,), (_F32,), at), a_ws, n_ws)
    return loss, counts, lse


def route_backward(logits: torch.Tensor, ids: torch.Tensor, w: torch.Tensor | None = None,
                   dw: torch.Tensor | None = None, lse: torch.Tensor | None = None,
                   counts: torch.Tensor | None = None, dloss: torch.Tensor | None = None,
                   dlogits: torch.Tensor | None = None, stream=None):
    """moe_route_backward: dlogits [T, E] fp32.  w and dw [T, k]: route_topk's gate weights and their gradient
    (combine_backward).  lse, counts: balance_loss's outputs, dloss [2] fp32 the gradients of its two losses.  Either
    part may be left out."""
    T, E = _rows(logits, "logits", 2)
    k = _rows(ids, "ids", 2)[1]
    if (w is None) != (dw is None):
        raise ValueError("w and dw go together")
    if (lse is None) != (counts is None) or (lse is None) != (dloss is None):
        raise ValueError("lse, counts and dloss go together")
    if w is None and lse is None:
        raise ValueError("neither gate weights (w, dw) nor losses (lse, counts, dloss)")
    a_logits = _arg(logits, "logits", (T, E), (_F32,))
    at = logits.get_device()
    a_ids = _arg(ids, "ids", (T, k), (_I32,), at)
    a_w = a_dw = a_lse = a_counts = a_dloss = None
    if w is not None:
        a_w, a_dw = _arg(w, "w", (T, k), (_F32,), at), _arg(dw, "dw", (T, k), (_F32,), at)
    if lse is not None:
        a_lse, a_counts = _arg(lse, "lse", (T,), (_F32,), at), _arg(counts, "counts", (E + 1,), (_I32,), at)
        a_dloss = _arg(dloss, "dloss", (2,), (_F32,), at)
    if dlogits is None:
        dlogits = _new(logits, (T, E), _F32, stream)
    _launch(lib.moe_route_backward, at, stream, a_logits, a_ids, a_w, a_dw, a_lse, a_counts, a_dloss, T, E, k,
            _arg(dlogits, "dlogits", (T, E), (_F32,), at))
    return dlogits


def _needs(need, names: tuple):
    if not need or any(n not in names for n in need):
        raise ValueError("need holds some of " + ", ".join(f'"{n}"' for n in names))


def combine_backward(y: torch.Tensor, w: torch.Tensor, dout: torch.Tensor, dw: torch.Tensor | None = None,
                     dy: torch.Tensor | None = None, need=("dw", "dy"), stream=None):
    """moe_combine_backward: (dw [T, k] fp32, dy [T, k, H] of y's type) from dout [T, H]; None for what `need` leaves
    out.  The gradient of combine's residual is dout itself."""
    T, k, H = _rows(y, "y", 3)
    _needs(need, ("dw", "dy"))
    a_y = _arg(y, "y", (T, k, H), (_F32, _BF16))
    at = y.get_device()
    a_w, a_dout = _arg(w, "w", (T, k), (_F32,), at), _arg(dout, "dout", (T, H), (_F32, _BF16), at)
    a_dw = a_dy = None
    if "dw" in need:
        if dw is None:
            dw = _new(y, (T, k), _F32, stream)
        a_dw = _arg(dw, "dw", (T, k), (_F32,), at)
    else:
        dw = None
    if "dy" in need:
        if dy is None:
            dy = _new(y, (T, k, H), y.dtype, stream)
        a_dy = _arg(dy, "dy", (T, k, H), (y.dtype,), at)
    else:
        dy = None
    _launch(lib.moe_combine_backward, at, stream, a_y, _dtype_code(y), a_w, a_dout, _dtype_code(dout), T, k, H, a_dw,
            a_dy)
    return dw, dy


def _act_rows(w: torch.Tensor, act: str):
    """(activation code, output columns) of weight rows w."""
    code = ACTS.get(act)
    if code is None:
        raise ValueError(f"act must be one of {', '.join(ACTS)}, got {act!r}")
    R = w.shape[0]
    if code != 3:
        return code, R
    if R % 2:
        raise ValueError("swiglu needs an even number of weight rows (gate rows, then up rows)")
    return code, R // 2


def linear(x: torch.Tensor, w: torch.Tensor, bias: torch.Tensor | None = None, act: str = "none",
           residual: torch.Tensor | None = None, y: torch.Tensor | None = None, y_dtype=None,
           pre: torch.Tensor | None = None, ws: torch.Tensor | None = None, stream=None):
    """moe_linear: y [T, N] = act(x [T, K] . w [R, K]^T + bias [R]) + residual [T, N].

    w is bf16, x and residual fp32 or bf16, bias fp32, y of y_dtype (x's by default).  act is "none", "gelu" (tanh
    form), "silu" or "swiglu", whose w holds N gate rows, then N up rows (R = 2 N; else R = N).  `pre` [T, R], of y's
    type, receives the values before the activation, which linear_backward needs.  y may be the residual itself.
    y is detached; its gradient is linear_backward."""
    T, K = _rows(x, "x", 2)
    R = _rows(w, "w", 2)[0]
    code, N = _act_rows(w, act)
    a_x = _arg(x, "x", (T, K), (_F32, _BF16))
    at = x.get_device()
    a_w = _arg(w, "w", (R, K), (_BF16,), at)
    a_bias = None if bias is None else _arg(bias, "bias", (R,), (_F32,), at)
    a_res, r_t = None, MOE_F32
    if residual is not None:
        a_res, r_t = _arg(residual, "residual", (T, N), (_F32, _BF16), at), _dtype_code(residual)
    x_t = _dtype_code(x)
    if y is None:
        y = _new(x, (T, N), x.dtype if y_dtype is None else y_dtype, stream)
    a_y, y_t = _arg(y, "y", (T, N), (_F32, _BF16), at), _dtype_code(y)
    a_pre = None if pre is None else _arg(pre, "pre", (T, R), (y.dtype,), at)
    ws, a_ws, n_ws = _ws(ws, lib.moe_linear_workspace_bytes(T, K, N, code, x_t, y_t), x, at, stream)
    _launch(lib.moe_linear, at, stream, a_x, x_t, a_w, a_bias, code, a_res, r_t, T, K, N, a_y, y_t, a_pre, a_ws, n_ws)
    return y


def _size_codes(act: str, *dtypes):
    if act not in ACTS:
        raise ValueError(f"act must be one of {', '.join(ACTS)}, got {act!r}")
    for d in dtypes:
        if d not in (_F32, _BF16):
            raise TypeError(f"unsupported dtype {d} (float32 or bfloat16)")
    return ACTS[act], [MOE_F32 if d == _F32 else MOE_BF16 for d in dtypes]


def linear_workspace_bytes(T: int, K: int, N: int, act: str = "none", x_dtype=torch.bfloat16,
                           y_dtype=torch.bfloat16) -> int:
    """Bytes of linear's workspace for N output columns."""
    code, t = _size_codes(act, x_dtype, y_dtype)
    return int(lib.moe_linear_workspace_bytes(T, K, N, code, *t))


_NEED = {"dx": 1, "dw": 2, "db": 4}


def linear_backward(dy: torch.Tensor, x: torch.Tensor, w: torch.Tensor, act: str = "none",
                    pre: torch.Tensor | None = None, need=("dx", "dw", "db"), dx: torch.Tensor | None = None,
                    dw: torch.Tensor | None = None, db: torch.Tensor | None = None, dx_dtype=None,
                    dw_dtype=torch.float32, ws: torch.Tensor | None = None, stream=None):
    """moe_linear_backward: (dx [T, K], dw [R, K], db [R] fp32) of linear(x, w, bias, act), None for what `need`
    leaves out.  dx is of dx_dtype (x's by default), dw of dw_dtype.  `pre` is what linear wrote there, of dy's type
    (not needed for act "none").  The residual's gradient is dy itself."""
    T, K = _rows(x, "x", 2)
    R = _rows(w, "w", 2)[0]
    code, N = _act_rows(w, act)
    _needs(need, ("dx", "dw", "db"))
    if code and pre is None:
        raise ValueError(f"act {act!r} needs pre")
    a_dy = _arg(dy, "dy", (T, N), (_F32, _BF16))
    at = dy.get_device()
    a_x, a_w = _arg(x, "x", (T, K), (_F32, _BF16), at), _arg(w, "w", (R, K), (_BF16,), at)
    a_pre = _arg(pre, "pre", (T, R), (dy.dtype,), at) if code else None
    bits = 0
    a_dx = a_dw = a_db = None
    dx_t = dw_t = MOE_BF16
    if "dx" in need:
        if dx is None:
            dx = _new(x, (T, K), x.dtype if dx_dtype is None else dx_dtype, stream)
        a_dx, dx_t, bits = _arg(dx, "dx", (T, K), (_F32, _BF16), at), _dtype_code(dx), 1
    else:
        dx = None
    if "dw" in need:
        if dw is None:
            dw = _new(x, (R, K), dw_dtype, stream)
        a_dw, dw_t, bits = _arg(dw, "dw", (R, K), (_F32, _BF16), at), _dtype_code(dw), bits | 2
    else:
        dw = None
    if "db" in need:
        if db is None:
            db = _new(x, R, _F32, stream)
        a_db, bits = _arg(db, "db", (R,), (_F32,), at), bits | 4
    else:
        db = None
    x_t, dy_t = _dtype_code(x), _dtype_code(dy)
    ws, a_ws, n_ws = _ws(ws, lib.moe_linear_backward_workspace_bytes(T, K, N, code, dy_t, x_t, dx_t, dw_t, bits), x, at,
                         stream)
    _launch(lib.moe_linear_backward, at, stream, a_dy, dy_t, a_pre, a_x, x_t, a_w, code, T, K, N, a_dx, dx_t, a_dw,
            dw_t, a_db, a_ws, n_ws)
    return dx, dw, db


def linear_backward_workspace_bytes(T: int, K: int, N: int, act: str = "none", dy_dtype=torch.bfloat16,
                                    x_dtype=torch.bfloat16, dx_dtype=torch.bfloat16, dw_dtype=torch.float32,
                                    need=("dx", "dw", "db")) -> int:
    """Bytes of linear_backward's workspace for N output columns."""
    code, t = _size_codes(act, dy_dtype, x_dtype, dx_dtype, dw_dtype)
    _needs(need, ("dx", "dw", "db"))
    return int(lib.moe_linear_backward_workspace_bytes(T, K, N, code, *t, sum(_NEED[n] for n in set(need))))


def linear_form(T: int, K: int, N: int, act: str = "none", x_dtype=torch.bfloat16, y_dtype=torch.bfloat16) -> dict:
    """How linear cuts its work at these sizes, for tests and measurements (moe_linear_form)."""
    code, t = _size_codes(act, x_dtype, y_dtype)
    form = (ctypes.c_int32 * 4)()
    _check(lib.moe_linear_form(T, K, N, code, *t, form))
    return dict(zip(("tile", "parts", "terms", "planes"), form))


def linear_backward_form(T: int, K: int, N: int, act: str = "none", dy_dtype=torch.bfloat16, x_dtype=torch.bfloat16,
                         dx_dtype=torch.bfloat16, dw_dtype=torch.float32, need=("dx", "dw", "db")) -> dict:
    """How linear_backward cuts its work at these sizes, for tests and measurements (moe_linear_backward_form)."""
    code, t = _size_codes(act, dy_dtype, x_dtype, dx_dtype, dw_dtype)
    _needs(need, ("dx", "dw", "db"))
    form = (ctypes.c_int32 * 4)()
    _check(lib.moe_linear_backward_form(T, K, N, code, *t, sum(_NEED[n] for n in set(need)), form))
    return dict(zip(("tile", "dw_parts", "dx_parts", "terms"), form))


def _newton_coefs(coef, steps: int) -> list:
    """The coefficients of all steps in a row."""
    rows = coef.tolist() if hasattr(coef, "tolist") else list(coef)
    if rows and not hasattr(rows[0], "__len__"):
        rows = [rows] * max(0, min(steps, 16))  # (the call refuses more steps)
    elif len(rows) != steps:
        rows = [()]
    if any(not hasattr(c, "__len__") or len(c) != 3 for c in rows):
        raise ValueError(f"coef holds one (a, b, c), or one for each of {steps} steps")
    return [float(v) for c in rows for v in c]


def orthogonalize(g: torch.Tensor, momentum: torch.Tensor | None = None, beta: float = 0.95, nesterov: bool = True,
                  steps: int = 5, coef=None, eps: float = 1e-7, o: torch.Tensor | None = None, o_dtype=None,
                  ws: torch.Tensor | None = None, stream=None):
    """moe_orthogonalize: o, the gradient g [R, K] or [B, R, K] (fp32 or bf16; linear_backward's dw) with every singular
    value brought near 1, as the Muon optimiser applies it: w -= lr * scale * o.

    momentum (fp32, g's shape) is updated in place to beta * momentum + (1 - beta) * g and used instead of g, with
    `nesterov` mixed with g once more.  coef: (a, b, c) of every step, or one triple per step; None takes the usual
    quintic.  o is bf16 by default, fp32 with o_dtype (three times the work).  The matrices of a batch share every launch."""
    if g.dim() not in (2, 3):
        raise ValueError(f"g must have 2 or 3 dimensions, got {g.dim()}")
    shape = _rows(g, "g", g.dim())
    B, R, K = shape if len(shape) == 3 else (1, *shape)
    a_g = _arg(g, "g", shape, (_F32, _BF16))
    at = g.get_device()
    a_m = None if momentum is None else _arg(momentum, "momentum", shape, (_F32,), at)
    a_coef = None
    if coef is not None:
        flat = _newton_coefs(coef, steps)
        a_coef = (ctypes.c_float * len(flat))(*flat)
    if o is None:
        o = _new(g, shape, o_dtype or _BF16, stream)
    a_o, o_t = _arg(o, "o", shape, (_F32, _BF16), at), _dtype_code(o)
    ws, a_ws, n_ws = _ws(ws, lib.moe_orthogonalize_workspace_bytes(B, R, K, o_t), g, at, stream)
    _launch(lib.moe_orthogonalize, at, stream, a_g, _dtype_code(g), a_m, beta, bool(nesterov), B, R, K, steps, a_coef, eps, a_o,
            o_t, a_ws, n_ws)
    return o


def orthogonalize_workspace_bytes(B: int, R: int, K: int, o_dtype=torch.bfloat16) -> int:
    """Bytes of orthogonalize's workspace for B matrices."""
    return int(lib.moe_orthogonalize_workspace_bytes(B, R, K, *_size_codes("none", o_dtype)[1]))


def orthogonalize_form(B: int, R: int, K: int, o_dtype=torch.bfloat16) -> dict:
    """How orthogonalize cuts its work at these sizes, for tests and measurements (moe_orthogonalize_form)."""
    form = (ctypes.c_int32 * 4)()
    _check(lib.moe_orthogonalize_form(B, R, K, *_size_codes("none", o_dtype)[1], form))
    return dict(zip(("gram", "apply", "gram_paired", "apply_paired"), form))


# ---- the dense parts in 8 bits ----------------------------------------------------------

_I8 = torch.int8


# These two calls are short enough on the GPU for the host to decide how fast decode steps run, so what is usual is
# tested in place, and _arg is asked for the error when a test fails (linear_q8 of one token: 9.3 -> 7.6 us on the host).

def quantize_rows(x: torch.Tensor, q: torch.Tensor | None = None, scale: torch.Tensor | None = None, stream=None):
    """moe_quantize_rows: (q [T, K] int8, scale [T] fp32) of x [T, K] (fp32 or bf16): x is about q * scale[:, None], with
    scale a 127th of the row's largest magnitude.  Rows are a weight's output channels or tokens."""
    shape = x.shape
    if len(shape) != 2 or max(shape) > 0x7FFFFFFF:
        _rows(x, "x", 2)
    T, K = shape
    at, dtype = x.get_device(), x.dtype
    if at < 0 or not x.is_contiguous() or (dtype is not _BF16 and dtype is not _F32):
        _arg(x, "x", shape, (_F32, _BF16))
    a_q = a_scale = None
    if q is not None:
        a_q = _arg(q, "q", (T, K), (_I8,), at)
    if scale is not None:
        a_scale = _arg(scale, "scale", (T,), (_F32,), at)
    if q is None:
        q = _new(x, shape, _I8, stream)
        a_q = q.data_ptr()
    if scale is None:
        scale = _new(x, T, _F32, stream)
        a_scale = scale.data_ptr()
    _launch(lib.moe_quantize_rows, at, stream, x.data_ptr(), MOE_BF16 if dtype is _BF16 else MOE_F32, T, K, a_q, a_scale)
    return q, scale


_Q8_CODE = {_F32: MOE_F32, _BF16: MOE_BF16, _I8: MOE_I8}


def linear_q8(x: torch.Tensor, w: torch.Tensor, w_scale: torch.Tensor, x_scale: torch.Tensor | None = None,
              bias: torch.Tensor | None = None, act: str = "none", residual: torch.Tensor | None = None,
              y: torch.Tensor | None = None, y_dtype=None, ws: torch.Tensor | None = None, stream=None):
    """moe_linear_q8: y [T, N] = act((x [T, K] . w [R, K]^T) * scales + bias [R]) + residual [T, N] in 8-bit integers.

    w int8 and w_scale [R] fp32 come from quantize_rows.  x is int8 with x_scale [T] fp32 (quantize_rows of the
    activations), or fp32 or bf16, which the call codes the same way.  bias is fp32, residual fp32 or bf16, y of y_dtype
    (x's by default, bf16 for int8 x).  act as for linear: "swiglu" takes N gate rows, then N up rows.  y may be the
    residual itself."""
    shape, w_shape = x.shape, w.shape
    if len(shape) != 2 or max(shape) > 0x7FFFFFFF:
        _rows(x, "x", 2)
    if len(w_shape) != 2 or max(w_shape) > 0x7FFFFFFF:
        _rows(w, "w", 2)
    T, K = shape
    R = w_shape[0]
    code, N = (0, R) if act == "none" else _act_rows(w, act)
    at, x_t = x.get_device(), _Q8_CODE.get(x.dtype)
    if at < 0 or x_t is None or not x.is_contiguous():
        _arg(x, "x", shape, (_F32, _BF16, _I8))
    a_xs = a_bias = a_res = None
    r_t = MOE_F32
    if x_scale is not None:
        if x_t != MOE_I8:
            raise ValueError("x_scale goes with int8 x")
        a_xs = _arg(x_scale, "x_scale", (T,), (_F32,), at)
    elif x_t == MOE_I8:
        raise ValueError("x_scale goes with int8 x")
    if w.dtype is not _I8 or w_shape[1] != K or not w.is_contiguous() or w.get_device() != at:
        _arg(w, "w", (R, K), (_I8,), at)
    if w_scale.dtype is not _F32 or w_scale.shape != (R,) or not w_scale.is_contiguous() or w_scale.get_device() != at:
        _arg(w_scale, "w_scale", (R,), (_F32,), at)
    if bias is not None:
        a_bias = _arg(bias, "bias", (R,), (_F32,), at)
    if residual is not None:
        a_res, r_t = _arg(residual, "residual", (T, N), (_F32, _BF16), at), _dtype_code(residual)
    if y is None:
        if y_dtype is None:
            y_dtype = _BF16 if x_t == MOE_I8 else x.dtype
        elif y_dtype is not _BF16 and y_dtype is not _F32:
            raise TypeError(f"y_dtype must be {_F32} or {_BF16}, got {y_dtype}")
        y = _new(x, (T, N), y_dtype, stream)
        a_y, y_t = y.data_ptr(), MOE_BF16 if y_dtype is _BF16 else MOE_F32
    else:
        a_y, y_t = _arg(y, "y", (T, N), (_F32, _BF16), at), _dtype_code(y)
    need, a_ws, n_ws = _q8_need(T, K, N, code, x_t), None, 0
    if need or ws is not None:
        ws, a_ws, n_ws = _ws(ws, need, x, at, stream)
    _launch(lib.moe_linear_q8, at, stream, x.data_ptr(), x_t, a_xs, w.data_ptr(), w_scale.data_ptr(), a_bias, code, a_res, r_t, T,
            K, N, a_y, y_t, a_ws, n_ws)
    return y


@functools.lru_cache(maxsize=4096)
def _q8_need(T, K, N, code, x_t):
    """The workspace query's answer, which depends on these numbers alone."""
    return int(lib.moe_linear_q8_workspace_bytes(T, K, N, code, x_t))


def _q8_codes(act: str, x_dtype):
    if act not in ACTS:
        raise ValueError(f"act must be one of {', '.join(ACTS)}, got {act!r}")
    if x_dtype not in _Q8_CODE:
        raise TypeError(f"unsupported dtype {x_dtype} (float32, bfloat16 or int8)")
    return ACTS[act], _Q8_CODE[x_dtype]


def linear_q8_workspace_bytes(T: int, K: int, N: int, act: str = "none", x_dtype=torch.bfloat16) -> int:
    """Bytes of linear_q8's workspace for N output columns."""
    return int(lib.moe_linear_q8_workspace_bytes(T, K, N, *_q8_codes(act, x_dtype)))


def linear_q8_form(T: int, K: int, N: int, act: str = "none", x_dtype=torch.bfloat16) -> dict:
    """How linear_q8 cuts its work at these sizes, for tests and measurements (moe_linear_q8_form)."""
    form = (ctypes.c_int32 * 3)()
    _check(lib.moe_linear_q8_form(T, K, N, *_q8_codes(act, x_dtype), form))
    return dict(zip(("tile", "parts", "coded_before"), form))


# ---- slot table -------------------------------------------------------------------------

class SlotTable:
    """Resident-expert slot table over L*E page-locked host blobs (see moe.h)."""

    def __init__(self, L: int, E: int, n_slots: int, expert_bytes_: int, host_experts: torch.Tensor,
                 slots: torch.Tensor, slot_map: torch.Tensor, stream=None):
        self.L, self.E, self.n_slots, self.expert_bytes = L, E, n_slots, expert_bytes_
        self.host_experts, self.slots, self.slot_map = host_experts, slots, slot_map
        h = ctypes.c_void_p()
        _check(lib.moe_slot_table_create(L, E, n_slots, expert_bytes_, ctypes.c_void_p(host_experts.data_ptr()),
                                         _ptr(slots), _ptr(slot_map), _stream(stream, slots.device),
                                         ctypes.byref(h)))
        self.h = h

    def preload(self, pairs, stream=None):
        import numpy as np
        arr = np.ascontiguousarray(np.asarray(pairs, np.int32).reshape(-1))
        _check(lib.moe_slot_table_preload(self.h, ctypes.c_void_p(arr.ctypes.data), arr.size // 2,
                                          _stream(stream, self.slots.device)))

    def resolve(self, layer: int, d: Dispatch, stream=None):
        _check(lib.moe_slot_table_resolve(self.h, layer, _ptr(d.active), _ptr(d.n_active),
                                          _stream(stream, self.slots.device)))

    def enable_device(self, stream=None):
        """Switch to device mode: the policy runs on the GPU (state in a device buffer this object keeps)."""
        nb = int(lib.moe_slot_table_device_bytes(self.L, self.E, self.n_slots))
        self.state = torch.empty(nb, dtype=torch.uint8, device=self.slots.device)
        _check(lib.moe_slot_table_enable_device(self.h, _ptr(self.state), nb, _stream(stream, self.slots.device)))

    def resolve_device(self, layer: int, d: Dispatch, max_active: int | None = None, stream=None):
        m = max_active if max_active is not None else min(self.E, d.T * d.k)
        _check(lib.moe_slot_table_resolve_device(self.h, layer, _ptr(d.active), _ptr(d.n_active), m,
                                                 _stream(stream, self.slots.device)))

    def layer(self, l: int, H: int, I: int, bits: int) -> ExpertLayer:
        return ExpertLayer(self.E, H, I, bits, self.slots, self.expert_bytes, self.slot_map[l * self.E:(l + 1) * self.E])

    def stats(self) -> dict:
        s = SlotStats()
        _check(lib.moe_slot_table_stats(self.h, ctypes.byref(s)))
        return {f: int(getattr(s, f)) for f, _ in SlotStats._fields_}

    def map_host(self):
        import numpy as np
        out = np.empty(self.L * self.E, np.int32)
        _check(lib.moe_slot_table_map_host(self.h, ctypes.c_void_p(out.ctypes.data)))
        return out

    def close(self):
        if self.h:
            lib.moe_slot_table_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class HostSlotTable:
    """Host-only slot table (no GPU): copies are reported to a Python callback."""

    def __init__(self, L: int, E: int, n_slots: int):
        self.copies = []

        def cb(user, slot, layer, expert):
            self.copies.append((slot, layer, expert))

        self._cb = COPY_FN(cb)
        h = ctypes.c_void_p()
        _check(lib.moe_slot_table_create_host(L, E, n_slots, self._cb, None, ctypes.byref(h)))
        self.h = h
        self.L, self.E = L, E

    def preload(self, pairs):
        import numpy as np
        arr = np.ascontiguousarray(np.asarray(pairs, np.int32).reshape(-1))
        _check(lib.moe_slot_table_preload(self.h, ctypes.c_void_p(arr.ctypes.data), arr.size // 2, None))

    def resolve(self, layer: int, active):
        import numpy as np
        arr = np.ascontiguousarray(np.asarray(active, np.int32))
        _check(lib.moe_slot_table_resolve_host(self.h, layer, ctypes.c_void_p(arr.ctypes.data), arr.size))

    def stats(self) -> dict:
        s = SlotStats()
        _check(lib.moe_slot_table_stats(self.h, ctypes.byref(s)))
        return {f: int(getattr(s, f)) for f, _ in SlotStats._fields_}

    def map_host(self):
        import numpy as np
        out = np.empty(self.L * self.E, np.int32)
        _check(lib.moe_slot_table_map_host(self.h, ctypes.c_void_p(out.ctypes.data)))
        return out

    def close(self):
        if self.h:
            lib.moe_slot_table_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
