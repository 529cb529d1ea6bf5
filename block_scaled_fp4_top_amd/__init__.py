"""Block-scaled (NVFP4 / MXFP8) MoE layer forward for MI355X: Python binding.

Argument marshalling only: tensors are checked (dtype, contiguity, shape,
device) and their device pointers handed to the C ABI in include/moe_fp4.h;
every step of the layer runs in the HIP library libmoe_fp4.so. There is no
fallback: if the library is missing, importing the binding fails.
"""
from __future__ import annotations

import ctypes
import functools
import os
from dataclasses import dataclass

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_PKG, "libmoe_fp4.so")

MODES = {"w4a4_tensor": 0, "w4a4_token": 1, "w4a16": 2, "mxfp8": 3, "w4a4_token_4o6": 4,
         "w4a4_token_mxfp4": 5}
ACTS = {"swiglu": 0, "relu2": 1}
WFMTS = {"nvfp4": 0, "mxfp8": 1, "mxfp4": 2}
VIEWS = {"topk_ids": 0, "topk_w": 1, "counts": 2, "offsets": 3, "row_to_route": 4,
         "route_to_row": 5, "x_codes": 6, "x_scales": 7, "x_g": 8, "a2_pre": 9,
         "a2_codes": 10, "a2_scales": 11, "a2_g": 12, "o": 13, "x_mx_codes": 14,
         "x_mx_scales": 15, "a2_mx_codes": 16, "a2_mx_scales": 17}
STAGES = ["route", "permute", "quantize_x", "fc1", "quantize_fc2_input", "fc2", "finalize"]


class MoeError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"moe_fp4 error {code}: {msg}")
        self.code = code


class _Dims(ctypes.Structure):
    _fields_ = [("E", ctypes.c_int32), ("H", ctypes.c_int32), ("I", ctypes.c_int32),
                ("act", ctypes.c_int32), ("wfmt", ctypes.c_int32)]


def _load():
    if not os.path.exists(_LIB_PATH):
        raise ImportError(
            f"{_LIB_PATH} is not built; run `python -c 'import __graft_entry__ as g; g.build()'` "
            "(hipcc --offload-arch=gfx950)")
    L = ctypes.CDLL(_LIB_PATH)
    P, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
    D = ctypes.POINTER(_Dims)
    sig = {
        "moe_prepared_bytes": (sz, [D]),
        "moe_prepare_weights": (ctypes.c_int, [D, P, P, P, sz, P]),
        "moe_check_prepared": (ctypes.c_int, [D, P, P]),
        "moe_workspace_bytes": (sz, [D, i32, i32, i32]),
        "moe_forward": (ctypes.c_int, [D, P, sz, P, P, i32, i32, i32, i32, i32, i32, P, sz, P, P]),
        "moe_forward_status": (ctypes.c_int, [P, ctypes.POINTER(i32), P]),
        "moe_forward_noalloc": (ctypes.c_int, [D, P, sz, P, P, i32, i32, i32, i32, i32, i32, P, P]),
        "moe_finalize": (ctypes.c_int, [P, i32, P, P, i32, i32, i32, P, P]),
        "moe_quantize": (ctypes.c_int, [P, i32, i32, i32, P, P, P, P, P]),
        "moe_workspace_view": (ctypes.c_int, [D, i32, i32, i32, i32, ctypes.POINTER(sz),
                                              ctypes.POINTER(sz)]),
        "moe_stage_timing": (ctypes.c_int, [i32]),
        "moe_stage_times": (ctypes.c_int, [ctypes.POINTER(ctypes.c_float), i32,
                                           ctypes.POINTER(i32)]),
        "moe_last_error": (ctypes.c_char_p, []),
        "moe_sort_workspace_bytes": (sz, [i32, i32, i32]),
        "moe_sort_routes": (ctypes.c_int, [P, i32, i32, i32, i32, P, sz, P, P, P, P]),
        "moe_dispatch": (ctypes.c_int, [P, i64, i32, P, P, i32, i32, i32, P, i64, P]),
        "moe_dispatch_grad": (ctypes.c_int, [P, i64, i32, P, P, P, i64, i32, i32, i32, P, i64, P, P]),
        "moe_combine": (ctypes.c_int, [P, i64, i32, P, P, i32, i32, i32, P, i64, P]),
        "moe_combine_grad": (ctypes.c_int, [P, i64, i32, P, P, P, i64, i32, i32, i32, P, i64, P, P]),
        "moe_int_quantize": (ctypes.c_int, [P, i64, i32, i32, i32, P, i64, P, P]),
        "moe_int_matmul": (ctypes.c_int, [P, i64, P, P, i64, P, P, i32, i32, i32, i32, P, i64, P]),
        "moe_int_grouped_matmul": (ctypes.c_int, [P, i64, P, i32, P, i64, i64, P, P, P, P, i32, i32,
                                                  i32, i32, i32, i32, P, i64, P]),
    }
    for name, (res, args) in sig.items():
        f = getattr(L, name)
        f.restype, f.argtypes = res, args
    return L


_lib = _load()
EXPORTS = ["moe_prepared_bytes", "moe_prepare_weights", "moe_check_prepared",
           "moe_workspace_bytes", "moe_forward", "moe_forward_noalloc", "moe_forward_status",
           "moe_finalize", "moe_quantize",
           "moe_workspace_view", "moe_stage_timing", "moe_stage_times", "moe_last_error",
           "moe_sort_workspace_bytes", "moe_sort_routes", "moe_dispatch", "moe_dispatch_grad",
           "moe_combine", "moe_combine_grad", "moe_int_quantize", "moe_int_matmul",
           "moe_int_grouped_matmul"]


def lib_path() -> str:
    return _LIB_PATH


def _check(rc: int):
    if rc != 0:
        raise MoeError(rc, _lib.moe_last_error().decode())


def _stream(stream) -> int:
    s = torch.cuda.current_stream() if stream is None else stream
    return s.cuda_stream


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else None


def _need(t, name, dtype, shape=None, device=None):
    if t is None:
        raise ValueError(f"{name} is required")
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a GPU")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")


@dataclass(frozen=True)
class Dims:
    E: int
    H: int
    I: int
    act: str = "swiglu"
    wfmt: str = "nvfp4"

    @property
    def N1(self) -> int:
        return 2 * self.I if self.act == "swiglu" else self.I

    def c(self) -> _Dims:
        return _Dims(self.E, self.H, self.I, ACTS[self.act], WFMTS[self.wfmt])


def prepared_bytes(d: Dims) -> int:
    n = _lib.moe_prepared_bytes(ctypes.byref(d.c()))
    if n == 0:
        raise MoeError(1, _lib.moe_last_error().decode())
    return n


def prepare_weights(d: Dims, w1: torch.Tensor, w2: torch.Tensor, out=None, stream=None):
    """Quantize and reorder checkpoint-layout weights W1 [E, N1, H], W2 [E, H, I]
    (fp32, on the GPU) into a prepared blob (uint8 tensor on the same GPU)."""
    _need(w1, "w1", torch.float32, (d.E, d.N1, d.H))
    _need(w2, "w2", torch.float32, (d.E, d.H, d.I), w1.device)
    n = prepared_bytes(d)
    if out is None:
        out = torch.empty(n, dtype=torch.uint8, device=w1.device)
    _need(out, "out", torch.uint8, device=w1.device)
    _check(_lib.moe_prepare_weights(ctypes.byref(d.c()), _ptr(w1), _ptr(w2), _ptr(out),
                                    out.numel(), ctypes.c_void_p(_stream(stream))))
    return out


def check_prepared(d: Dims, blob: torch.Tensor, stream=None):
    _check(_lib.moe_check_prepared(ctypes.byref(d.c()), _ptr(blob),
                                   ctypes.c_void_p(_stream(stream))))


def workspace_bytes(d: Dims, T: int, K: int, mode: str) -> int:
    n = _lib.moe_workspace_bytes(ctypes.byref(d.c()), T, K, MODES[mode])
    if n == 0:
        raise MoeError(1, _lib.moe_last_error().decode())
    return n


def forward(d: Dims, blob: torch.Tensor, x: torch.Tensor, logits: torch.Tensor, K: int,
            mode: str, router_weight_on_input: bool = False, deterministic: bool = True,
            workspace=None, out=None, stream=None) -> torch.Tensor:
    """One MoE layer forward. x [T, H] bf16, logits [T, E] fp32; returns y [T, H]
    bf16. The workspace (uint8, see workspace_bytes) may be passed in to be
    reused and inspected with workspace_view."""
    _need(x, "x", torch.bfloat16)
    if x.dim() != 2 or x.shape[1] != d.H:
        raise ValueError(f"x must be [T, {d.H}], got {tuple(x.shape)}")
    T = x.shape[0]
    _need(logits, "router_logits", torch.float32, (T, d.E), x.device)
    _need(blob, "prepared", torch.uint8, device=x.device)
    if blob.numel() < prepared_bytes(d):
        raise MoeError(3, f"prepared blob has {blob.numel()} bytes, {prepared_bytes(d)} needed "
                          "for these dimensions")
    if workspace is None:
        workspace = torch.empty(workspace_bytes(d, T, K, mode), dtype=torch.uint8,
                                device=x.device)
    _need(workspace, "workspace", torch.uint8, device=x.device)
    if out is None:
        out = torch.empty((T, d.H), dtype=torch.bfloat16, device=x.device)
    _need(out, "out", torch.bfloat16, (T, d.H), x.device)
    _check(_lib.moe_forward(ctypes.byref(d.c()), _ptr(blob), blob.numel(), _ptr(x), _ptr(logits), T, K,
                            MODES[mode], ACTS[d.act], int(bool(router_weight_on_input)),
                            int(bool(deterministic)), _ptr(workspace), workspace.numel(),
                            _ptr(out), ctypes.c_void_p(_stream(stream))))
    return out


def forward_noalloc(d: Dims, blob: torch.Tensor, x: torch.Tensor, logits: torch.Tensor, K: int,
                    mode: str, router_weight_on_input: bool = False, deterministic: bool = True,
                    out=None, stream=None) -> torch.Tensor:
    """forward() on the library's built-in workspace (moe_forward_noalloc): no
    workspace argument and no device allocation by the library. Forwards that
    overlap in time on one GPU share that workspace and must not be run
    concurrently. `out` (y, [T, H] bf16) is allocated here when not given."""
    _need(x, "x", torch.bfloat16)
    if x.dim() != 2 or x.shape[1] != d.H:
        raise ValueError(f"x must be [T, {d.H}], got {tuple(x.shape)}")
    T = x.shape[0]
    _need(logits, "router_logits", torch.float32, (T, d.E), x.device)
    _need(blob, "prepared", torch.uint8, device=x.device)
    if out is None:
        out = torch.empty((T, d.H), dtype=torch.bfloat16, device=x.device)
    _need(out, "out", torch.bfloat16, (T, d.H), x.device)
    _check(_lib.moe_forward_noalloc(ctypes.byref(d.c()), _ptr(blob), blob.numel(), _ptr(x),
                                    _ptr(logits), T, K, MODES[mode], ACTS[d.act],
                                    int(bool(router_weight_on_input)), int(bool(deterministic)),
                                    _ptr(out), ctypes.c_void_p(_stream(stream))))
    return out


def forward_status(workspace: torch.Tensor, stream=None) -> int:
    """Status word of the last forward on `workspace` (synchronises): 0, or
    MOE_ERR_INVALID (1) when the blob's header did not match the call."""
    _need(workspace, "workspace", torch.uint8)
    st = ctypes.c_int32(-1)
    _check(_lib.moe_forward_status(_ptr(workspace), ctypes.byref(st),
                                   ctypes.c_void_p(_stream(stream))))
    return st.value


def finalize(permuted_out: torch.Tensor, route_to_row: torch.Tensor, weights, T: int, K: int,
             out=None, stream=None) -> torch.Tensor:
    """Unfused finalize: y[t] = sum_k w[t, k] * permuted_out[route_to_row[t*K + k]]."""
    if permuted_out.dtype not in (torch.float32, torch.bfloat16):
        raise TypeError("permuted_out must be float32 or bfloat16")
    _need(permuted_out, "permuted_out", permuted_out.dtype)
    R, H = permuted_out.shape
    if R != T * K:
        raise ValueError(f"permuted_out has {R} rows, expected T*K = {T * K}")
    _need(route_to_row, "route_to_row", torch.int32, (T * K,), permuted_out.device)
    if weights is not None:
        _need(weights, "weights", torch.float32, (T, K), permuted_out.device)
    if out is None:
        out = torch.empty((T, H), dtype=torch.bfloat16, device=permuted_out.device)
    _need(out, "out", torch.bfloat16, (T, H), permuted_out.device)
    _check(_lib.moe_finalize(_ptr(permuted_out), int(permuted_out.dtype == torch.bfloat16),
                             _ptr(route_to_row), _ptr(weights), T, K, H, _ptr(out),
                             ctypes.c_void_p(_stream(stream))))
    return out


def quantize(v: torch.Tensor, kind: str, stream=None):
    """Block-quantize an fp32 [rows, cols] matrix. kind: "nvfp4_tensor",
    "nvfp4_row", "mxfp8" or "nvfp4_row_4o6". Returns (codes, scales, g) as uint8/uint8/fp32
    tensors (g is None for MXFP8)."""
    _need(v, "v", torch.float32)
    rows, cols = v.shape
    k = {"nvfp4_tensor": 0, "nvfp4_row": 1, "mxfp8": 2, "nvfp4_row_4o6": 3}[kind]
    dev = v.device
    if k == 2:
        codes = torch.empty((rows, cols), dtype=torch.uint8, device=dev)
        scales = torch.empty((rows, cols // 32), dtype=torch.uint8, device=dev)
        g = None
    else:
        codes = torch.empty((rows, cols // 2), dtype=torch.uint8, device=dev)
        scales = torch.empty((rows, cols // 16), dtype=torch.uint8, device=dev)
        g = torch.empty((1 if k == 0 else rows,), dtype=torch.float32, device=dev)
    scratch = torch.empty(256, dtype=torch.uint8, device=dev)
    _check(_lib.moe_quantize(_ptr(v), rows, cols, k, _ptr(codes), _ptr(scales), _ptr(g),
                             _ptr(scratch), ctypes.c_void_p(_stream(stream))))
    return codes, scales, g


_VIEW_DTYPES = {0: torch.int32, 1: torch.float32, 2: torch.int32, 3: torch.int32,
                4: torch.int32, 5: torch.int32, 6: torch.uint8, 7: torch.uint8,
                8: torch.float32, 10: torch.uint8, 11: torch.uint8, 12: torch.float32,
                13: torch.float32, 14: torch.uint8, 15: torch.uint8, 16: torch.uint8, 17: torch.uint8}


def workspace_view(d: Dims, workspace: torch.Tensor, T: int, K: int, mode: str, view: str):
    """A typed, flat view into the workspace after a forward (no copy)."""
    vid = VIEWS[view]
    off, nbytes = ctypes.c_size_t(0), ctypes.c_size_t(0)
    _check(_lib.moe_workspace_view(ctypes.byref(d.c()), T, K, MODES[mode], vid,
                                   ctypes.byref(off), ctypes.byref(nbytes)))
    raw = workspace[off.value: off.value + nbytes.value]
    if vid == 9:
        dt = torch.bfloat16 if mode == "w4a16" else torch.float32
    else:
        dt = _VIEW_DTYPES[vid]
    return raw.view(dt)


def stage_timing(enable: bool):
    _check(_lib.moe_stage_timing(int(enable)))


def stage_times():
    """(dict stage -> summed ms, number of forwards) since the last call."""
    ms = (ctypes.c_float * len(STAGES))()
    n = ctypes.c_int32(0)
    _check(_lib.moe_stage_times(ms, len(STAGES), ctypes.byref(n)))
    return {s: ms[i] for i, s in enumerate(STAGES)}, n.value


# ---------------------------------------------------------------------------
# Operators around the experts: routes sorted by expert, dispatch, combine, their
# gradients, and 8-bit integer products. They run on the tensors' device, on
# `stream` or that device's current stream; what they allocate belongs to that
# stream. Matrices may have any row stride; the elements of a row are
# contiguous. Gradients are functions of their own (autograd records nothing).
# ---------------------------------------------------------------------------
DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}


def _on_stream(f):
    """Runs f on the device of its first argument and on the stream it is given,
    with both current, so that f itself only uses the current ones."""
    @functools.wraps(f)
    def call(*args, stream=None, **kw):
        first = args[0] if args else next(iter(kw.values()), None)
        if not isinstance(first, torch.Tensor):
            raise TypeError("the first argument must be a torch.Tensor")
        if not first.is_cuda:
            raise ValueError("the tensors must be on a GPU")
        dev = first.device
        if stream is None:
            if dev.index == torch._C._cuda_getDevice():
                return f(*args, **kw)
            with torch.cuda.device(dev):
                return f(*args, **kw)
        if stream.device != dev:
            raise ValueError(f"the stream is on {stream.device}, the tensors on {dev}")
        with torch.cuda.stream(stream):
            got = f(*args, **kw)
            if not torch.cuda.is_current_stream_capturing():
                for t in (*args, *kw.values()):  # may be freed while the stream still reads them
                    for u in t.tensors() if isinstance(t, RouteOrder) else (t,):
                        if isinstance(u, torch.Tensor):
                            u.record_stream(stream)
        return got
    return call


def _raw_stream(t):
    return torch._C._cuda_getCurrentRawStream(t.device.index)


def _matrix(t, name, dtype, device, rows=None, cols=None):
    """Checks a 2-D tensor with contiguous rows; returns its row stride."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    shape = t.shape
    if len(shape) != 2 or (rows is not None and shape[0] != rows) or (cols is not None and shape[1] != cols):
        raise ValueError(f"{name} has shape {tuple(shape)}, expected "
                         f"[{'rows' if rows is None else rows}, {'columns' if cols is None else cols}]")
    ld, inner = t.stride()
    if inner != 1 and shape[1] != 1:
        raise ValueError(f"the elements of a row of {name} must be contiguous")
    return ld


def _float_type(t, name):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    code = DTYPES.get(t.dtype)
    if code is None:
        raise TypeError(f"{name} must be bfloat16, float16 or float32, got {t.dtype}")
    return code


class RouteOrder:
    """The routes r = t*K + k of T tokens sorted by expert (see sort_routes), int32:
    row_to_route [T*K], route_to_row [T*K], offsets [E+1]."""
    __slots__ = ("row_to_route", "route_to_row", "offsets", "T", "K", "E")

    def __init__(self, row_to_route: torch.Tensor, route_to_row: torch.Tensor, offsets: torch.Tensor,
                 T: int, K: int, E: int):
        _need(offsets, "offsets", torch.int32, (E + 1,))
        _need(row_to_route, "row_to_route", torch.int32, (T * K,), offsets.device)
        _need(route_to_row, "route_to_row", torch.int32, (T * K,), offsets.device)
        self._set(row_to_route, route_to_row, offsets, T, K, E)

    def _set(self, row_to_route, route_to_row, offsets, T, K, E):
        self.row_to_route, self.route_to_row, self.offsets = row_to_route, route_to_row, offsets
        self.T, self.K, self.E = T, K, E
        return self

    def tensors(self):
        return self.row_to_route, self.route_to_row, self.offsets


def _order(order, device, T=None):
    if not isinstance(order, RouteOrder):
        raise TypeError("order must be a RouteOrder (see sort_routes)")
    if order.offsets.device != device:
        raise ValueError(f"order is on {order.offsets.device}, expected {device}")
    if T is not None and order.T != T:
        raise ValueError(f"order is of {order.T} tokens, expected {T}")


def _weights(w, order, device):
    if w is not None:
        _need(w, "weights", torch.float32, (order.T, order.K), device)
        return w.data_ptr()
    return None


@_on_stream
def sort_routes(ids: torch.Tensor, E: int) -> RouteOrder:
    """Stable sort of the routes r = t*K + k by expert. ids: [T, K] int32 or int64
    expert ids; an id outside [0, E) drops its route. Rows offsets[e] ..
    offsets[e+1]-1 hold the routes of expert e in ascending order; row_to_route is
    -1 behind the last row, route_to_row -1 for a dropped route."""
    if ids.dtype not in (torch.int32, torch.int64):
        raise TypeError(f"ids must be int32 or int64, got {ids.dtype}")
    if ids.dim() != 2:
        raise ValueError(f"ids must be [T, K], got {tuple(ids.shape)}")
    _need(ids, "ids", ids.dtype)
    T, K = ids.shape
    n = _lib.moe_sort_workspace_bytes(T, K, E)
    if n == 0:
        raise MoeError(1, _lib.moe_last_error().decode())
    R = T * K
    # one allocation: the workspace (whole int32 words), then the maps and the offsets
    ws = n // 4
    whole = torch.empty(ws + 2 * R + E + 1, dtype=torch.int32, device=ids.device)
    p = whole.data_ptr()
    _check(_lib.moe_sort_routes(ids.data_ptr(), int(ids.dtype == torch.int64), T, K, E, p, n, p + n,
                                p + n + 4 * R, p + n + 8 * R, _raw_stream(ids)))
    _, row_to_route, route_to_row, offsets = whole.split_with_sizes((ws, R, R, E + 1))
    return RouteOrder.__new__(RouteOrder)._set(row_to_route, route_to_row, offsets, T, K, E)


@_on_stream
def dispatch(x: torch.Tensor, order: RouteOrder, weights=None, out=None) -> torch.Tensor:
    """Rows of the experts from token rows x [T, H]: out[row(t,k)] = weights[t,k] * x[t]
    (weights [T, K] fp32, or None for copies). out is [T*K, H]; its rows from
    offsets[E] on are left as they were (uninitialised if out is allocated here)."""
    dt = _float_type(x, "x")
    ld = _matrix(x, "x", x.dtype, x.device)
    T, H = x.shape
    _order(order, x.device, T)
    w = _weights(weights, order, x.device)
    if out is None:
        out = torch.empty((T * order.K, H), dtype=x.dtype, device=x.device)
    ld_out = _matrix(out, "out", x.dtype, x.device, T * order.K, H)
    _check(_lib.moe_dispatch(x.data_ptr(), ld, dt, order.route_to_row.data_ptr(), w, T, order.K, H,
                             out.data_ptr(), ld_out, _raw_stream(x)))
    return out


@_on_stream
def dispatch_grad(drows: torch.Tensor, order: RouteOrder, x=None, weights=None, out=None):
    """Gradients of dispatch: (dx [T, H], dweights [T, K] fp32 or None). dweights needs
    weights and x (the dispatched tokens); with weights alone only dx is computed."""
    dt = _float_type(drows, "drows")
    ld = _matrix(drows, "drows", drows.dtype, drows.device)
    dev, H = drows.device, drows.shape[1]
    _order(order, dev)
    T, K = order.T, order.K
    if drows.shape[0] != T * K:
        raise ValueError(f"drows has {drows.shape[0]} rows, expected T*K = {T * K}")
    w = _weights(weights, order, dev)
    if x is not None and weights is None:
        raise ValueError("x is only used for the gradient of weights, which are missing")
    ldx = _matrix(x, "x", drows.dtype, dev, T, H) if x is not None else 0
    dw = torch.empty((T, K), dtype=torch.float32, device=dev) if x is not None else None
    if out is None:
        out = torch.empty((T, H), dtype=drows.dtype, device=dev)
    ld_out = _matrix(out, "out", drows.dtype, dev, T, H)
    _check(_lib.moe_dispatch_grad(drows.data_ptr(), ld, dt, order.route_to_row.data_ptr(), w,
                                  x.data_ptr() if x is not None else None, ldx, T, K, H, out.data_ptr(),
                                  ld_out, dw.data_ptr() if dw is not None else None, _raw_stream(drows)))
    return out, dw


@_on_stream
def combine(rows: torch.Tensor, order: RouteOrder, weights=None, out=None) -> torch.Tensor:
    """Token rows from the experts' rows [T*K, H]: y[t] = sum_k weights[t,k] * rows[row(t,k)]
    over the routes that are kept (weights [T, K] fp32, or None for 1). fp32 sums in
    k order, one rounding to the type of rows. See also finalize."""
    dt = _float_type(rows, "rows")
    ld = _matrix(rows, "rows", rows.dtype, rows.device)
    dev, H = rows.device, rows.shape[1]
    _order(order, dev)
    T, K = order.T, order.K
    if rows.shape[0] != T * K:
        raise ValueError(f"rows has {rows.shape[0]} rows, expected T*K = {T * K}")
    w = _weights(weights, order, dev)
    if out is None:
        out = torch.empty((T, H), dtype=rows.dtype, device=dev)
    ld_out = _matrix(out, "out", rows.dtype, dev, T, H)
    _check(_lib.moe_combine(rows.data_ptr(), ld, dt, order.route_to_row.data_ptr(), w, T, K, H,
                            out.data_ptr(), ld_out, _raw_stream(rows)))
    return out


@_on_stream
def combine_grad(dy: torch.Tensor, order: RouteOrder, rows=None, weights=None, out=None):
    """Gradients of combine: (drows [T*K, H], dweights [T, K] fp32 or None). drows'
    rows from offsets[E] on are left as they were. dweights needs weights and rows
    (the combined rows)."""
    dt = _float_type(dy, "dy")
    ld = _matrix(dy, "dy", dy.dtype, dy.device)
    dev = dy.device
    T, H = dy.shape
    _order(order, dev, T)
    K = order.K
    w = _weights(weights, order, dev)
    if rows is not None and weights is None:
        raise ValueError("rows is only used for the gradient of weights, which are missing")
    ldr = _matrix(rows, "rows", dy.dtype, dev, T * K, H) if rows is not None else 0
    dw = torch.empty((T, K), dtype=torch.float32, device=dev) if rows is not None else None
    if out is None:
        out = torch.empty((T * K, H), dtype=dy.dtype, device=dev)
    ld_out = _matrix(out, "out", dy.dtype, dev, T * K, H)
    _check(_lib.moe_combine_grad(dy.data_ptr(), ld, dt, order.route_to_row.data_ptr(), w,
                                 rows.data_ptr() if rows is not None else None, ldr, T, K, H, out.data_ptr(),
                                 ld_out, dw.data_ptr() if dw is not None else None, _raw_stream(dy)))
    return out, dw


@_on_stream
def quantize_int8(x: torch.Tensor, out=None):
    """Symmetric 8-bit quantization of each row of x [M, N]: (codes int8 [M, N], scales
    fp32 [M]) with scales = max|x| / 127 and codes = x / scale rounded to nearest, ties
    to even. A row with an infinity or a NaN has that as its scale and codes 0."""
    dt = _float_type(x, "x")
    ld = _matrix(x, "x", x.dtype, x.device)
    M, N = x.shape
    if out is None:
        out = torch.empty((M, N), dtype=torch.int8, device=x.device)
    ld_out = _matrix(out, "out", torch.int8, x.device, M, N)
    scales = torch.empty(M, dtype=torch.float32, device=x.device)
    _check(_lib.moe_int_quantize(x.data_ptr(), ld, dt, M, N, out.data_ptr(), ld_out, scales.data_ptr(),
                                 _raw_stream(x)))
    return out, scales


def _int8_out(out, out_dtype, M, N, dev):
    if out is None:
        out = torch.empty((M, N), dtype=out_dtype or torch.bfloat16, device=dev)
    elif out_dtype is not None and isinstance(out, torch.Tensor) and out.dtype != out_dtype:
        raise TypeError(f"out is {out.dtype}, out_dtype {out_dtype}")
    dt = _float_type(out, "out")
    return out, dt, _matrix(out, "out", out.dtype, dev, M, N)


@_on_stream
def int8_matmul(a: torch.Tensor, a_scale: torch.Tensor, b: torch.Tensor, b_scale: torch.Tensor, bias=None,
                out_dtype=None, out=None) -> torch.Tensor:
    """y = a_scale[:, None] * b_scale * (a @ b.T) + bias for int8 a [M, K] (see
    quantize_int8) and b [N, K], fp32 a_scale [M], b_scale [N] and bias [N] (or None):
    exact integer sums, fp32 scaling, one rounding to out_dtype (bfloat16 unless
    given). K and the row strides are multiples of 16."""
    lda = _matrix(a, "a", torch.int8, a.device)
    dev = a.device
    M, K = a.shape
    ldb = _matrix(b, "b", torch.int8, dev, None, K)
    N = b.shape[0]
    _need(a_scale, "a_scale", torch.float32, (M,), dev)
    _need(b_scale, "b_scale", torch.float32, (N,), dev)
    if bias is not None:
        _need(bias, "bias", torch.float32, (N,), dev)
    out, dt, ldy = _int8_out(out, out_dtype, M, N, dev)
    _check(_lib.moe_int_matmul(a.data_ptr(), lda, a_scale.data_ptr(), b.data_ptr(), ldb, b_scale.data_ptr(),
                               bias.data_ptr() if bias is not None else None, M, N, K, dt, out.data_ptr(),
                               ldy, _raw_stream(a)))
    return out


@_on_stream
def int8_grouped_matmul(a: torch.Tensor, a_scale: torch.Tensor, b: torch.Tensor, b_scale: torch.Tensor,
                        order: RouteOrder, gather: bool = False, bias=None, out_dtype=None,
                        out=None) -> torch.Tensor:
    """int8_matmul expert by expert over sorted routes: row r of the result [T*K, N], of
    expert e, is row r of a [T*K, K] times b[e] ([E, N, K] int8, b_scale and bias [E, N]).
    gather: a holds the tokens' rows [T, K] (a_scale [T]) and row r reads the one of its
    route. Rows from offsets[E] on are left as they were (uninitialised if out is
    allocated here)."""
    lda = _matrix(a, "a", torch.int8, a.device)
    dev = a.device
    _order(order, dev)
    M, E = order.T * order.K, order.E
    a_rows, K = a.shape
    if a_rows != (order.T if gather else M):
        raise ValueError(f"a has {a_rows} rows, expected {order.T if gather else M}")
    if not isinstance(b, torch.Tensor) or b.dim() != 3 or b.shape[0] != E or b.shape[2] != K:
        raise ValueError(f"b must be a tensor [{E}, N, {K}]")
    N = b.shape[1]
    if b.dtype != torch.int8:
        raise TypeError(f"b must be torch.int8, got {b.dtype}")
    if b.device != dev:
        raise ValueError(f"b is on {b.device}, expected {dev}")
    be, ldb, inner = b.stride()
    if inner != 1 and K != 1:
        raise ValueError("the elements of a row of b must be contiguous")
    _need(a_scale, "a_scale", torch.float32, (a_rows,), dev)
    _need(b_scale, "b_scale", torch.float32, (E, N), dev)
    if bias is not None:
        _need(bias, "bias", torch.float32, (E, N), dev)
    out, dt, ldy = _int8_out(out, out_dtype, M, N, dev)
    _check(_lib.moe_int_grouped_matmul(a.data_ptr(), lda, a_scale.data_ptr(), a_rows, b.data_ptr(), ldb, be,
                                       b_scale.data_ptr(), bias.data_ptr() if bias is not None else None,
                                       order.offsets.data_ptr(),
                                       order.row_to_route.data_ptr() if gather else None, order.K, M, N, K, E,
                                       dt, out.data_ptr(), ldy, _raw_stream(a)))
    return out
