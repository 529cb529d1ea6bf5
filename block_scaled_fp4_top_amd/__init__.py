"""Block-scaled (NVFP4 / MXFP8) MoE layer forward for MI355X: Python binding.

Argument marshalling only: tensors are checked (dtype, contiguity, shape,
device) and their device pointers handed to the C ABI in include/moe_fp4.h;
every step of the layer runs in the HIP library libmoe_fp4.so. There is no
fallback: if the library is missing, importing the binding fails.
"""
from __future__ import annotations

import ctypes
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


_MOST = (1 << 31) - 1  # the library takes sizes as int32, which ctypes would cut off silently


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
    if R > _MOST or H > _MOST:
        raise ValueError(f"permuted_out has shape {tuple(permuted_out.shape)}, sizes must fit 32 bits")
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
    if rows > _MOST or cols > _MOST:
        raise ValueError(f"v has shape {tuple(v.shape)}, sizes must fit 32 bits")
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
# contiguous. Gradients are functions of their own: autograd records nothing, and a
# result requires no gradient whatever its inputs require.
# (Small calls are bound by the host, so what a call has made itself is not
# checked again.)
# ---------------------------------------------------------------------------
DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
_current_device = torch._C._cuda_getDevice
_raw_stream = torch._C._cuda_getCurrentRawStream


def _elsewhere(f, args, stream):
    """f(*args) with the device of its first argument and `stream` current: for a call
    on another device or stream than the current ones."""
    first = args[0]
    if not isinstance(first, torch.Tensor):
        raise TypeError("the first argument must be a torch.Tensor")
    dev = first.device
    if not first.is_cuda:
        raise ValueError("the tensors must be on a GPU")
    if stream is None:
        with torch.cuda.device(dev):
            return f(*args)
    if stream.device != dev:
        raise ValueError(f"the stream is on {stream.device}, the tensors on {dev}")
    with torch.cuda.stream(stream):
        got = f(*args)
        if not torch.cuda.is_current_stream_capturing():
            for t in args:  # may be freed while the stream still reads them
                for u in t.tensors() if isinstance(t, RouteOrder) else (t,):
                    if isinstance(u, torch.Tensor):
                        u.record_stream(stream)
    return got


def _device_index(t):
    """The index of a tensor's GPU; -1 for anything else (which _elsewhere refuses)."""
    return t.get_device() if isinstance(t, torch.Tensor) else -1


def _matrix(t, name, dtype, index, rows=None, cols=None):
    """Checks a 2-D tensor with contiguous rows on GPU `index`; returns its row stride."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.get_device() != index:
        raise ValueError(f"{name} is on {t.device}, expected cuda:{index}")
    shape = t.shape
    if len(shape) != 2 or (rows is not None and shape[0] != rows) or (cols is not None and shape[1] != cols):
        raise ValueError(f"{name} has shape {tuple(shape)}, expected "
                         f"[{'rows' if rows is None else rows}, {'columns' if cols is None else cols}]")
    if shape[0] > _MOST or shape[1] > _MOST:
        raise ValueError(f"{name} has shape {tuple(shape)}, sizes must fit 32 bits")
    ld, inner = t.stride()
    if inner != 1 and shape[1] != 1:
        raise ValueError(f"the elements of a row of {name} must be contiguous")
    return ld


def _vector(t, name, index, shape):
    """Checks a contiguous fp32 tensor of this shape; returns its address."""
    if t.__class__ is torch.Tensor and t.dtype is torch.float32 and t.get_device() == index and t.shape == shape \
            and t.is_contiguous():
        return t.data_ptr()
    _need(t, name, torch.float32, shape, torch.device("cuda", index))
    return t.data_ptr()


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
    __slots__ = ("row_to_route", "route_to_row", "offsets", "T", "K", "E", "index")

    def __init__(self, row_to_route: torch.Tensor, route_to_row: torch.Tensor, offsets: torch.Tensor,
                 T: int, K: int, E: int):
        if max(T, K, E, T * K) > _MOST:
            raise ValueError(f"T={T}, K={K}, E={E}: sizes must fit 32 bits")
        _need(offsets, "offsets", torch.int32, (E + 1,))
        _need(row_to_route, "row_to_route", torch.int32, (T * K,), offsets.device)
        _need(route_to_row, "route_to_row", torch.int32, (T * K,), offsets.device)
        self._set(row_to_route, route_to_row, offsets, T, K, E)

    def _set(self, row_to_route, route_to_row, offsets, T, K, E):
        self.row_to_route, self.route_to_row, self.offsets = row_to_route, route_to_row, offsets
        self.T, self.K, self.E = T, K, E
        self.index = offsets.get_device()
        return self

    def tensors(self):
        return self.row_to_route, self.route_to_row, self.offsets


def _order(order, index, T=None):
    if not isinstance(order, RouteOrder):
        raise TypeError("order must be a RouteOrder (see sort_routes)")
    if order.index != index:
        raise ValueError(f"order is on cuda:{order.index}, expected cuda:{index}")
    if T is not None and order.T != T:
        raise ValueError(f"order is of {order.T} tokens, expected {T}")


def sort_routes(ids: torch.Tensor, E: int, stream=None) -> RouteOrder:
    """Stable sort of the routes r = t*K + k by expert. ids: [T, K] int32 or int64
    expert ids; an id outside [0, E) drops its route. Rows offsets[e] ..
    offsets[e+1]-1 hold the routes of expert e in ascending order; row_to_route is
    -1 behind the last row, route_to_row -1 for a dropped route."""
    dev = _device_index(ids)
    if stream is not None or dev < 0 or dev != _current_device():
        return _elsewhere(sort_routes, (ids, E), stream)
    wide = ids.dtype == torch.int64
    if not wide and ids.dtype != torch.int32:
        raise TypeError(f"ids must be int32 or int64, got {ids.dtype}")
    if ids.dim() != 2:
        raise ValueError(f"ids must be [T, K], got {tuple(ids.shape)}")
    if not ids.is_contiguous():
        raise ValueError("ids must be contiguous")
    T, K = ids.shape
    if T > _MOST or K > _MOST or abs(E) > _MOST:
        raise ValueError(f"T={T}, K={K}, E={E}: sizes must fit 32 bits")
    n = _lib.moe_sort_workspace_bytes(T, K, E)
    if n == 0:
        raise MoeError(1, _lib.moe_last_error().decode())
    R = T * K
    # one allocation: the workspace (whole int32 words), then the maps and the offsets
    ws = n // 4
    whole = torch.empty(ws + 2 * R + E + 1, dtype=torch.int32, device=ids.device)
    p = whole.data_ptr()
    _check(_lib.moe_sort_routes(ids.data_ptr(), wide, T, K, E, p, n, p + n, p + n + 4 * R, p + n + 8 * R,
                                _raw_stream(dev)))
    _, row_to_route, route_to_row, offsets = whole.split_with_sizes((ws, R, R, E + 1))
    return RouteOrder.__new__(RouteOrder)._set(row_to_route, route_to_row, offsets, T, K, E)


def dispatch(x: torch.Tensor, order: RouteOrder, weights=None, out=None, stream=None) -> torch.Tensor:
    """Rows of the experts from token rows x [T, H]: out[row(t,k)] = weights[t,k] * x[t]
    (weights [T, K] fp32, or None for copies). out is [T*K, H]; its rows from
    offsets[E] on are left as they were (uninitialised if out is allocated here)."""
    dev = _device_index(x)
    if stream is not None or dev < 0 or dev != _current_device():
        return _elsewhere(dispatch, (x, order, weights, out), stream)
    dt = _float_type(x, "x")
    ld = _matrix(x, "x", x.dtype, dev)
    T, H = x.shape
    _order(order, dev, T)
    K = order.K
    w = None if weights is None else _vector(weights, "weights", dev, (T, K))
    if out is None:
        out, ld_out = torch.empty((T * K, H), dtype=x.dtype, device=x.device), H
    else:
        ld_out = _matrix(out, "out", x.dtype, dev, T * K, H)
    _check(_lib.moe_dispatch(x.data_ptr(), ld, dt, order.route_to_row.data_ptr(), w, T, K, H,
                             out.data_ptr(), ld_out, _raw_stream(dev)))
    return out


def dispatch_grad(drows: torch.Tensor, order: RouteOrder, x=None, weights=None, out=None, stream=None):
    """Gradients of dispatch: (dx [T, H], dweights [T, K] fp32 or None). dweights needs
    weights and x (the dispatched tokens); with weights alone only dx is computed."""
    dev = _device_index(drows)
    if stream is not None or dev < 0 or dev != _current_device():
        return _elsewhere(dispatch_grad, (drows, order, x, weights, out), stream)
    dt = _float_type(drows, "drows")
    _order(order, dev)
    T, K = order.T, order.K
    ld = _matrix(drows, "drows", drows.dtype, dev, T * K)
    H = drows.shape[1]
    w = None if weights is None else _vector(weights, "weights", dev, (T, K))
    xp, ldx, dw, dwp = None, 0, None, None
    if x is not None:
        if weights is None:
            raise ValueError("x is only used for the gradient of weights, which are missing")
        ldx, xp = _matrix(x, "x", drows.dtype, dev, T, H), x.data_ptr()
        dw = torch.empty((T, K), dtype=torch.float32, device=drows.device)
        dwp = dw.data_ptr()
    if out is None:
        out, ld_out = torch.empty((T, H), dtype=drows.dtype, device=drows.device), H
    else:
        ld_out = _matrix(out, "out", drows.dtype, dev, T, H)
    _check(_lib.moe_dispatch_grad(drows.data_ptr(), ld, dt, order.route_to_row.data_ptr(), w, xp, ldx, T, K, H,
                                  out.data_ptr(), ld_out, dwp, _raw_stream(dev)))
    return out, dw


def combine(rows: torch.Tensor, order: RouteOrder, weights=None, out=None, stream=None) -> torch.Tensor:
    """Token rows from the experts' rows [T*K, H]: y[t] = sum_k weights[t,k] * rows[row(t,k)]
    over the routes that are kept (weights [T, K] fp32, or None for 1). fp32 sums in
    k order, one rounding to the type of rows. See also finalize."""
    dev = _device_index(rows)
    if stream is not None or dev < 0 or dev != _current_device():
        return _elsewhere(combine, (rows, order, weights, out), stream)
    dt = _float_type(rows, "rows")
    _order(order, dev)
    T, K = order.T, order.K
    ld = _matrix(rows, "rows", rows.dtype, dev, T * K)
    H = rows.shape[1]
    w = None if weights is None else _vector(weights, "weights", dev, (T, K))
    if out is None:
        out, ld_out = torch.empty((T, H), dtype=rows.dtype, device=rows.device), H
    else:
        ld_out = _matrix(out, "out", rows.dtype, dev, T, H)
    _check(_lib.moe_combine(rows.data_ptr(), ld, dt, order.route_to_row.data_ptr(), w, T, K, H,
                            out.data_ptr(), ld_out, _raw_stream(dev)))
    return out


def combine_grad(dy: torch.Tensor, order: RouteOrder, rows=None, weights=None, out=None, stream=None):
    """Gradients of combine: (drows [T*K, H], dweights [T, K] fp32 or None). drows'
    rows from offsets[E] on are left as they were. dweights needs weights and rows
    (the combined rows)."""
    dev = _device_index(dy)
    if stream is not None or dev < 0 or dev != _current_device():
        return _elsewhere(combine_grad, (dy, order, rows, weights, out), stream)
    dt = _float_type(dy, "dy")
    ld = _matrix(dy, "dy", dy.dtype, dev)
    T, H = dy.shape
    _order(order, dev, T)
    K = order.K
    w = None if weights is None else _vector(weights, "weights", dev, (T, K))
    rp, ldr, dw, dwp = None, 0, None, None
    if rows is not None:
        if weights is None:
            raise ValueError("rows is only used for the gradient of weights, which are missing")
        ldr, rp = _matrix(rows, "rows", dy.dtype, dev, T * K, H), rows.data_ptr()
        dw = torch.empty((T, K), dtype=torch.float32, device=dy.device)
        dwp = dw.data_ptr()
    if out is None:
        out, ld_out = torch.empty((T * K, H), dtype=dy.dtype, device=dy.device), H
    else:
        ld_out = _matrix(out, "out", dy.dtype, dev, T * K, H)
    _check(_lib.moe_combine_grad(dy.data_ptr(), ld, dt, order.route_to_row.data_ptr(), w, rp, ldr, T, K, H,
                                 out.data_ptr(), ld_out, dwp, _raw_stream(dev)))
    return out, dw


def quantize_int8(x: torch.Tensor, out=None, stream=None):
    """Symmetric 8-bit quantization of each row of x [M, N]: (codes int8 [M, N], scales
    fp32 [M]) with scales = max|x| / 127 and codes = x / scale rounded to nearest, ties
    to even. A row with an infinity or a NaN has that as its scale and codes 0."""
    dev = _device_index(x)
    if stream is not None or dev < 0 or dev != _current_device():
        return _elsewhere(quantize_int8, (x, out), stream)
    dt = _float_type(x, "x")
    ld = _matrix(x, "x", x.dtype, dev)
    M, N = x.shape
    if out is None:
        out, ld_out = torch.empty((M, N), dtype=torch.int8, device=x.device), N
    else:
        ld_out = _matrix(out, "out", torch.int8, dev, M, N)
    scales = torch.empty(M, dtype=torch.float32, device=x.device)
    _check(_lib.moe_int_quantize(x.data_ptr(), ld, dt, M, N, out.data_ptr(), ld_out, scales.data_ptr(),
                                 _raw_stream(dev)))
    return out, scales


def _int8_out(out, out_dtype, M, N, t, dev):
    if out is None:
        dt = DTYPES.get(torch.bfloat16 if out_dtype is None else out_dtype)
        if dt is None:
            raise TypeError(f"out_dtype must be bfloat16, float16 or float32, got {out_dtype}")
        return torch.empty((M, N), dtype=out_dtype or torch.bfloat16, device=t.device), dt, N
    dt = _float_type(out, "out")
    if out_dtype is not None and out.dtype != out_dtype:
        raise TypeError(f"out is {out.dtype}, out_dtype {out_dtype}")
    return out, dt, _matrix(out, "out", out.dtype, dev, M, N)


def int8_matmul(a: torch.Tensor, a_scale: torch.Tensor, b: torch.Tensor, b_scale: torch.Tensor, bias=None,
                out_dtype=None, out=None, stream=None) -> torch.Tensor:
    """y = a_scale[:, None] * b_scale * (a @ b.T) + bias for int8 a [M, K] (see
    quantize_int8) and b [N, K], fp32 a_scale [M], b_scale [N] and bias [N] (or None):
    exact integer sums, fp32 scaling, one rounding to out_dtype (bfloat16 unless
    given). K and the row strides are multiples of 16."""
    dev = _device_index(a)
    if stream is not None or dev < 0 or dev != _current_device():
        return _elsewhere(int8_matmul, (a, a_scale, b, b_scale, bias, out_dtype, out), stream)
    lda = _matrix(a, "a", torch.int8, dev)
    M, K = a.shape
    ldb = _matrix(b, "b", torch.int8, dev, None, K)
    N = b.shape[0]
    sa, sb = _vector(a_scale, "a_scale", dev, (M,)), _vector(b_scale, "b_scale", dev, (N,))
    bp = None if bias is None else _vector(bias, "bias", dev, (N,))
    out, dt, ldy = _int8_out(out, out_dtype, M, N, a, dev)
    _check(_lib.moe_int_matmul(a.data_ptr(), lda, sa, b.data_ptr(), ldb, sb, bp, M, N, K, dt, out.data_ptr(),
                               ldy, _raw_stream(dev)))
    return out


def int8_grouped_matmul(a: torch.Tensor, a_scale: torch.Tensor, b: torch.Tensor, b_scale: torch.Tensor,
                        order: RouteOrder, gather: bool = False, bias=None, out_dtype=None,
                        out=None, stream=None) -> torch.Tensor:
    """int8_matmul expert by expert over sorted routes: row r of the result [T*K, N], of
    expert e, is row r of a [T*K, K] times b[e] ([E, N, K] int8, b_scale and bias [E, N]).
    gather: a holds the tokens' rows [T, K] (a_scale [T]) and row r reads the one of its
    route. Rows from offsets[E] on are left as they were (uninitialised if out is
    allocated here)."""
    dev = _device_index(a)
    if stream is not None or dev < 0 or dev != _current_device():
        return _elsewhere(int8_grouped_matmul, (a, a_scale, b, b_scale, order, gather, bias, out_dtype, out), stream)
    _order(order, dev)
    M, E = order.T * order.K, order.E
    rows = order.T if gather else M
    lda = _matrix(a, "a", torch.int8, dev, rows)
    K = a.shape[1]
    if not isinstance(b, torch.Tensor) or b.dim() != 3 or b.shape[0] != E or b.shape[2] != K:
        raise ValueError(f"b must be a tensor [{E}, N, {K}]")
    if b.dtype != torch.int8:
        raise TypeError(f"b must be torch.int8, got {b.dtype}")
    if b.get_device() != dev:
        raise ValueError(f"b is on {b.device}, expected cuda:{dev}")
    N = b.shape[1]
    if N > _MOST:
        raise ValueError(f"b has shape {tuple(b.shape)}, sizes must fit 32 bits")
    be, ldb, inner = b.stride()
    if inner != 1 and K != 1:
        raise ValueError("the elements of a row of b must be contiguous")
    sa, sb = _vector(a_scale, "a_scale", dev, (rows,)), _vector(b_scale, "b_scale", dev, (E, N))
    bp = None if bias is None else _vector(bias, "bias", dev, (E, N))
    out, dt, ldy = _int8_out(out, out_dtype, M, N, a, dev)
    _check(_lib.moe_int_grouped_matmul(a.data_ptr(), lda, sa, rows, b.data_ptr(), ldb, be, sb, bp,
                                       order.offsets.data_ptr(),
                                       order.row_to_route.data_ptr() if gather else None, order.K, M, N, K, E,
                                       dt, out.data_ptr(), ldy, _raw_stream(dev)))
    return out
