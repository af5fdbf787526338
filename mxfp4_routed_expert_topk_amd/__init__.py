"""Python binding of libmoe_mxfp4.so: the routed-expert MXFP4 MoE layer on
AMD MI355X (gfx950).

Argument marshalling only: every step of the layer runs in the HIP library.
torch provides device memory and the current stream.  If the library has not
been built, importing the low-level entry points raises at once; there is no
other execution path.

Names follow the C ABI in include/moe_mxfp4.h:
  query_sizes(cfg)                      -> (repacked_bytes, workspace_bytes)
  Plan(cfg, w13_codes, w13_scales, w2_codes, w2_scales)     (moe_mxfp4_plan)
  Plan.forward(hidden, topk_ids, topk_weights, out=None, acc=None)
  Plan.forward_noalloc(...)             the same, scratch in the library (moe_mxfp4_forward_noalloc)
  Plan.route(topk_ids)                  -> (counts, offsets, perm, rowpos)
  Plan.workspace_region(region)         -> the workspace bytes of an intermediate (MXFP8 h)
  mxfp8_quantize(x_bf16)                -> (codes, scales)
  router_topk(logits, k)                -> (topk_ids, topk_weights)  (moe_router_topk)
  mxfp4_quantize(x)                     -> (codes, scales)           (moe_mxfp4_quantize)
  mxfp4_dequantize(codes, scales)       -> the values they stand for (moe_mxfp4_dequantize)
  mxfp4_matmul(a_codes, a_scales, b_codes, b_scales)  -> A B^T       (moe_mxfp4_matmul)
  grouped_matmul(x, w, offsets)         rows sorted by group times the group's matrix (moe_grouped_matmul)
  grouped_matmul_backward(dy, x, w, offsets)          -> (dx, dw)    (moe_grouped_matmul_backward)
  router_select(logits, k, ...)         -> (topk_ids, topk_weights)  (moe_router_select)
  router_select_backward(dweights, logits, ids, ...)  -> dlogits     (moe_router_select_backward)
  mxfp4_linear(x, codes, scales)        bf16 rows times an MXFP4 matrix, plain or gated (moe_mxfp4_linear)
  expert_combine(y, rowpos, weights)    weighted sum of each token's rows (moe_expert_combine)
  expert_combine_backward(dout, y, rowpos, perm, weights)  -> (dy, dweights)  (moe_expert_combine_backward)
  probe_memory(kind, src, dst, sink)    peak micro-benchmarks (moe_probe_memory / moe_probe_mfma)
  probe_mfma(kind, iters, sink)         -> flops of the launch
"""
from __future__ import annotations

import ctypes
import dataclasses
import os
import warnings
from typing import Optional

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libmoe_mxfp4.so")

MOE_ACT_BF16 = 0
MOE_ACT_MXFP8 = 1
STATUS_NAMES = {0: "MOE_OK", 1: "MOE_ERR_ARG", 2: "MOE_ERR_SHAPE", 3: "MOE_ERR_ALIGN", 4: "MOE_ERR_CAPACITY",
                5: "MOE_ERR_SCALE_BYTE", 6: "MOE_ERR_WORKSPACE", 7: "MOE_ERR_UNSUPPORTED", 8: "MOE_ERR_HIP",
                9: "MOE_ERR_TIMEOUT"}
MOE_WS_H_CODES = 0
MOE_WS_H_SCALES = 1
EXPORTS = ("moe_mxfp4_query_sizes", "moe_mxfp4_plan", "moe_mxfp4_forward", "moe_mxfp4_forward_noalloc",
           "moe_mxfp4_forward_fused",
           "moe_mxfp4_fused_status", "moe_mxfp4_route", "moe_mxfp4_workspace_region", "moe_mxfp8_quantize",
           "moe_router_topk", "moe_mxfp4_quantize", "moe_mxfp4_dequantize", "moe_mxfp4_matmul",
           "moe_grouped_matmul", "moe_grouped_matmul_backward", "moe_grouped_matmul_workspace",
           "moe_grouped_matmul_backward_workspace", "moe_router_select", "moe_router_select_backward",
           "moe_mxfp4_linear", "moe_expert_combine", "moe_expert_combine_backward",
           "moe_probe_memory", "moe_probe_mfma", "moe_probe_mfma_f8f4_blocks",
           "moe_mxfp4_set_stage_events",
           "moe_mxfp4_destroy", "moe_mxfp4_last_error")
_STATUS_FNS = tuple(n for n in EXPORTS if n not in ("moe_mxfp4_destroy", "moe_mxfp4_last_error") and not n.endswith("_workspace"))


class MoeError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{STATUS_NAMES.get(status, status)}: {message}")
        self.status = status
        self.message = message


class _Config(ctypes.Structure):
    _fields_ = [("hidden", ctypes.c_int32), ("intermediate", ctypes.c_int32), ("num_experts", ctypes.c_int32),
                ("top_k", ctypes.c_int32), ("max_tokens", ctypes.c_int32), ("act", ctypes.c_int32)]


@dataclasses.dataclass(frozen=True)
class Config:
    hidden: int
    intermediate: int
    num_experts: int
    top_k: int
    max_tokens: int
    act: int = MOE_ACT_BF16

    def c(self) -> _Config:
        return _Config(self.hidden, self.intermediate, self.num_experts, self.top_k, self.max_tokens, self.act)


_lib = None


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load the HIP library (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise ImportError(f"libmoe_mxfp4.so not found at {path}; build it with "
                          f"`python -m mxfp4_routed_expert_topk_amd.build`")
    lib = ctypes.CDLL(path)
    vp, i32, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
    cfgp = ctypes.POINTER(_Config)
    lib.moe_mxfp4_query_sizes.argtypes = [cfgp, ctypes.POINTER(sz), ctypes.POINTER(sz)]
    lib.moe_mxfp4_plan.argtypes = [cfgp, vp, vp, vp, vp, vp, sz, vp, ctypes.POINTER(vp)]
    lib.moe_mxfp4_forward.argtypes = [vp, vp, vp, vp, i32, vp, vp, vp, sz, vp]
    lib.moe_mxfp4_forward_fused.argtypes = [vp, vp, vp, vp, i32, vp, vp, vp, sz, vp]
    lib.moe_mxfp4_forward_noalloc.argtypes = [vp, vp, vp, vp, i32, vp, vp, vp]
    lib.moe_mxfp4_fused_status.argtypes = [vp, vp, sz, vp]
    lib.moe_mxfp4_route.argtypes = [vp, vp, i32, vp, vp, vp, vp, vp, sz, vp]
    lib.moe_mxfp4_workspace_region.argtypes = [vp, i32, ctypes.POINTER(sz), ctypes.POINTER(sz)]
    lib.moe_mxfp8_quantize.argtypes = [vp, i32, i32, vp, vp, vp]
    lib.moe_router_topk.argtypes = [vp, i32, i32, i32, vp, vp, vp]
    i64 = ctypes.c_int64
    lib.moe_mxfp4_quantize.argtypes = [vp, i32, i32, i32, i64, vp, vp, vp]
    lib.moe_mxfp4_dequantize.argtypes = [vp, vp, i32, i32, i32, vp, vp]
    lib.moe_mxfp4_matmul.argtypes = [vp, vp, vp, vp, i32, i32, i32, i32, vp, vp]
    lib.moe_grouped_matmul.argtypes = [vp, i64, vp, vp, i32, i32, i32, i32, vp, vp, sz, vp]
    lib.moe_grouped_matmul_backward.argtypes = [vp, i64, vp, i64, vp, vp, i32, i32, i32, i32, vp, vp, i32, vp, sz, vp]
    lib.moe_grouped_matmul_workspace.argtypes = [i32] * 4
    lib.moe_grouped_matmul_backward_workspace.argtypes = [i32] * 6
    lib.moe_grouped_matmul_workspace.restype = lib.moe_grouped_matmul_backward_workspace.restype = sz
    f32 = ctypes.c_float
    lib.moe_router_select.argtypes = [vp, i32, i64, i32, i32, i32, i32, vp, i32, i32, i32, i32, f32, vp, vp, vp]
    lib.moe_router_select_backward.argtypes = [vp, vp, i32, i64, vp, i32, i32, i32, i32, i32, f32, vp, vp]
    lib.moe_mxfp4_linear.argtypes = [vp, i64, vp, vp, i32, i32, i32, i32, i32, vp, vp]
    lib.moe_expert_combine.argtypes = [vp, i64, i32, vp, vp, i32, i32, i32, i32, vp, vp]
    lib.moe_expert_combine_backward.argtypes = [vp, i32, i64, vp, i64, i32, vp, vp, vp, i32, i32, i32, vp, vp, vp]
    lib.moe_probe_memory.argtypes = [i32, vp, vp, sz, vp, i32, vp]
    lib.moe_probe_mfma.argtypes = [i32, i32, vp, i32, ctypes.POINTER(ctypes.c_double), vp]
    lib.moe_probe_mfma_f8f4_blocks.argtypes = [vp, vp, vp, vp, vp, vp, i32, vp]
    lib.moe_mxfp4_set_stage_events.argtypes = [vp, ctypes.POINTER(vp), i32]
    lib.moe_mxfp4_destroy.argtypes = [vp]
    lib.moe_mxfp4_destroy.restype = None
    lib.moe_mxfp4_last_error.argtypes = []
    lib.moe_mxfp4_last_error.restype = ctypes.c_char_p
    for name in _STATUS_FNS:
        getattr(lib, name).restype = ctypes.c_int
    _lib = lib
    return lib


def _check(status: int) -> None:
    if status != 0:
        raise MoeError(status, load_library().moe_mxfp4_last_error().decode())


def _ptr(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


MOE_ERR_ARG, MOE_ERR_SHAPE = 1, 2


def _arg_error(msg: str):
    return MoeError(MOE_ERR_ARG, msg)


def _need(t, name: str, dtype, rows_min: int, cols: Optional[int], device, ndim: int = 2):
    """Raise MoeError(MOE_ERR_ARG) unless `t` is a contiguous tensor of `dtype`
    on `device`, shaped [>= rows_min, cols] (cols None: any)."""
    import torch
    if not isinstance(t, torch.Tensor):
        raise _arg_error(f"{name} must be a torch.Tensor, got {type(t).__name__}")
    if t.dtype != dtype:
        raise _arg_error(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != ndim:
        raise _arg_error(f"{name} must have {ndim} dimensions, got shape {tuple(t.shape)}")
    if device is not None and t.device != device:
        raise _arg_error(f"{name} must be on {device}, got {t.device}")
    if not t.is_contiguous():
        raise _arg_error(f"{name} must be contiguous")
    if ndim == 2:
        if t.shape[0] < rows_min:
            raise _arg_error(f"{name} must have at least {rows_min} rows, got shape {tuple(t.shape)}")
        if cols is not None and t.shape[1] != cols:
            raise _arg_error(f"{name} must have {cols} columns, got shape {tuple(t.shape)}")
    elif t.numel() < rows_min:
        raise _arg_error(f"{name} must hold at least {rows_min} elements, got {t.numel()}")


def _too_large(**sizes):
    """The refusal of sizes of which one is 2^31 or more: ctypes would pass its
    low 32 bits on."""
    return MoeError(MOE_ERR_SHAPE, "sizes must be below 2^31, got " + ", ".join(f"{n}={v}" for n, v in sizes.items()))


def _need_int32(**values):
    """Raise MoeError(MOE_ERR_SHAPE) for a value that no int32 holds, negative
    ones too: ctypes would pass its low 32 bits on."""
    if any(not -1 << 31 <= v < 1 << 31 for v in values.values()):
        raise MoeError(MOE_ERR_SHAPE, "values must be below 2^31 and at least -2^31, got "
                       + ", ".join(f"{n}={v}" for n, v in values.items()))


def _stream(stream=None) -> int:
    import torch
    s = torch.cuda.current_stream() if stream is None else stream
    return s.cuda_stream


def query_sizes(cfg: Config):
    lib = load_library()
    rb, wb = ctypes.c_size_t(), ctypes.c_size_t()
    _check(lib.moe_mxfp4_query_sizes(ctypes.byref(cfg.c()), ctypes.byref(rb), ctypes.byref(wb)))
    return rb.value, wb.value


class Plan:
    """A plan over repacked weights.  Holds the repacked buffer and the
    forward workspace as torch uint8 tensors on the current device."""

    def __init__(self, cfg: Config, w13_codes, w13_scales, w2_codes, w2_scales, stream=None):
        import torch
        lib = load_library()
        self.cfg = cfg
        self.repacked_bytes, self.workspace_bytes = query_sizes(cfg)
        dev = w13_codes.device
        self.repacked = torch.empty(self.repacked_bytes, dtype=torch.uint8, device=dev)
        # zero-filled: the fused forward keeps its counters here and starts from zeros
        self.workspace = torch.zeros(self.workspace_bytes, dtype=torch.uint8, device=dev)
        h = ctypes.c_void_p()
        _check(lib.moe_mxfp4_plan(ctypes.byref(cfg.c()), _ptr(w13_codes), _ptr(w13_scales), _ptr(w2_codes),
                                  _ptr(w2_scales), _ptr(self.repacked), self.repacked_bytes, _stream(stream),
                                  ctypes.byref(h)))
        self._h = h
        self._events = None

    def close(self):
        if getattr(self, "_h", None) and self._h.value:
            load_library().moe_mxfp4_destroy(self._h)
            self._h = ctypes.c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def _forward_args(self, hidden, topk_ids, topk_weights, out, acc, num_tokens, workspace):
        """Check the tensors of a forward against the plan (dtype, shape, device,
        contiguity; MoeError(MOE_ERR_ARG) otherwise) and allocate `out` if None."""
        import torch
        c = self.cfg
        dev = self.workspace.device
        if not isinstance(hidden, torch.Tensor) or hidden.dim() != 2:
            raise _arg_error("hidden must be a 2-D torch.Tensor [T, hidden]")
        T = hidden.shape[0] if num_tokens is None else int(num_tokens)
        if T < 0 or T > hidden.shape[0]:
            raise _arg_error(f"num_tokens must be in [0, {hidden.shape[0]}] (rows of hidden), got {T}")
        _need(hidden, "hidden", torch.bfloat16, T, c.hidden, dev)
        _need(topk_ids, "topk_ids", torch.int32, T, c.top_k, dev)
        _need(topk_weights, "topk_weights", torch.float32, T, c.top_k, dev)
        if out is None:
            out = torch.empty((hidden.shape[0], c.hidden), dtype=torch.bfloat16, device=dev)
        _need(out, "out", torch.bfloat16, T, c.hidden, dev)
        if acc is not None:
            _need(acc, "acc", torch.float32, T, c.hidden, dev)
        ws = self.workspace if workspace is None else workspace
        _need(ws, "workspace", torch.uint8, 0, None, dev, ndim=1)
        return T, out, ws

    def forward(self, hidden, topk_ids, topk_weights, out=None, acc=None, num_tokens=None, stream=None,
                workspace=None):
        T, out, ws = self._forward_args(hidden, topk_ids, topk_weights, out, acc, num_tokens, workspace)
        _check(load_library().moe_mxfp4_forward(self._h, _ptr(hidden), _ptr(topk_ids), _ptr(topk_weights), T,
                                                _ptr(acc), _ptr(out), _ptr(ws), ws.numel(), _stream(stream)))
        return out

    def forward_noalloc(self, hidden, topk_ids, topk_weights, out=None, acc=None, num_tokens=None, stream=None):
        """The same forward with the library's fixed scratch instead of a
        workspace (moe_mxfp4_forward_noalloc); pass `out` to allocate nothing."""
        T, out, _ = self._forward_args(hidden, topk_ids, topk_weights, out, acc, num_tokens, None)
        _check(load_library().moe_mxfp4_forward_noalloc(self._h, _ptr(hidden), _ptr(topk_ids), _ptr(topk_weights), T,
                                                        _ptr(acc), _ptr(out), _stream(stream)))
        return out

    def forward_fused(self, hidden, topk_ids, topk_weights, out=None, acc=None, num_tokens=None, stream=None,
                      workspace=None):
        """The same forward in one kernel launch (bf16 plans, at most 256 routes)."""
        T, out, ws = self._forward_args(hidden, topk_ids, topk_weights, out, acc, num_tokens, workspace)
        _check(load_library().moe_mxfp4_forward_fused(self._h, _ptr(hidden), _ptr(topk_ids), _ptr(topk_weights),
                                                      T, _ptr(acc), _ptr(out), _ptr(ws), ws.numel(),
                                                      _stream(stream)))
        return out

    def fused_status(self, stream=None, workspace=None):
        """Raise MoeError(MOE_ERR_TIMEOUT) if the last fused forward's waits timed out (synchronises)."""
        ws = self.workspace if workspace is None else workspace
        _check(load_library().moe_mxfp4_fused_status(self._h, _ptr(ws), ws.numel(), _stream(stream)))

    def route(self, topk_ids, num_tokens=None, stream=None):
        import torch
        dev = self.workspace.device
        if not isinstance(topk_ids, torch.Tensor) or topk_ids.dim() != 2:
            raise _arg_error("topk_ids must be a 2-D torch.Tensor [T, top_k]")
        T = topk_ids.shape[0] if num_tokens is None else int(num_tokens)
        if T < 0 or T > topk_ids.shape[0]:
            raise _arg_error(f"num_tokens must be in [0, {topk_ids.shape[0]}] (rows of topk_ids), got {T}")
        _need(topk_ids, "topk_ids", torch.int32, T, self.cfg.top_k, dev)
        E, n = self.cfg.num_experts, max(1, T * self.cfg.top_k)
        counts = torch.empty(E, dtype=torch.int32, device=dev)
        offsets = torch.empty(E + 1, dtype=torch.int32, device=dev)
        perm = torch.full((n,), -7, dtype=torch.int32, device=dev)
        rowpos = torch.empty(n, dtype=torch.int32, device=dev)
        _check(load_library().moe_mxfp4_route(self._h, _ptr(topk_ids), T, _ptr(counts), _ptr(offsets), _ptr(perm),
                                              _ptr(rowpos), _ptr(self.workspace), self.workspace.numel(),
                                              _stream(stream)))
        return counts, offsets, perm, rowpos

    def workspace_region(self, region, workspace=None):
        """The uint8 view of `workspace` (default: the plan's) holding an
        intermediate of the last forward on it (MOE_WS_H_CODES: MXFP8 h codes
        [T_max*k, I]; MOE_WS_H_SCALES: their E8M0 bytes [T_max*k, I/32])."""
        off, nb = ctypes.c_size_t(), ctypes.c_size_t()
        _check(load_library().moe_mxfp4_workspace_region(self._h, int(region), ctypes.byref(off), ctypes.byref(nb)))
        ws = self.workspace if workspace is None else workspace
        return ws[off.value: off.value + nb.value]

    def set_stage_events(self, events):
        """events: list of 5 torch.cuda.Event(enable_timing=True) or None to stop."""
        lib = load_library()
        if not events:
            _check(lib.moe_mxfp4_set_stage_events(self._h, None, 0))
            self._events = None
            return
        for ev in events:
            if not ev.cuda_event:      # torch creates the HIP event on its first record
                ev.record()
        arr = (ctypes.c_void_p * len(events))(*[ev.cuda_event for ev in events])
        self._events = (events, arr)   # keep alive while set
        _check(lib.moe_mxfp4_set_stage_events(self._h, arr, len(events)))


def router_topk(logits, top_k, ids=None, weights=None, stream=None):
    """topk_ids int32 [T, k] and topk_weights fp32 [T, k] from fp32 logits [T, E]
    (moe_router_topk)."""
    import torch
    if not isinstance(logits, torch.Tensor) or logits.dim() != 2:
        raise _arg_error("logits must be a 2-D torch.Tensor [T, num_experts]")
    T, E = logits.shape
    if (T | E) >> 31:
        raise _too_large(num_tokens=T, num_experts=E)
    _need(logits, "logits", torch.float32, T, E, logits.device)
    ids = torch.empty((T, top_k), dtype=torch.int32, device=logits.device) if ids is None else ids
    weights = torch.empty((T, top_k), dtype=torch.float32, device=logits.device) if weights is None else weights
    _need(ids, "topk_ids", torch.int32, T, top_k, logits.device)
    _need(weights, "topk_weights", torch.float32, T, top_k, logits.device)
    _check(load_library().moe_router_topk(_ptr(logits), T, E, top_k, _ptr(ids), _ptr(weights), _stream(stream)))
    return ids, weights


def mxfp8_quantize(x_bf16, stream=None):
    import torch
    if not isinstance(x_bf16, torch.Tensor) or x_bf16.dim() != 2:
        raise _arg_error("x must be a 2-D torch.Tensor [rows, cols]")
    rows, cols = x_bf16.shape
    if (rows | cols) >> 31:
        raise _too_large(rows=rows, cols=cols)
    _need(x_bf16, "x", torch.bfloat16, rows, cols, x_bf16.device)
    codes = torch.empty((rows, cols), dtype=torch.uint8, device=x_bf16.device)
    scales = torch.empty((rows, max(cols // 32, 0)), dtype=torch.uint8, device=x_bf16.device)
    _check(load_library().moe_mxfp8_quantize(_ptr(x_bf16), rows, cols, _ptr(codes), _ptr(scales), _stream(stream)))
    return codes, scales


MOE_BF16, MOE_F32 = 0, 1

# The entry points below serve single tokens too, where a call's own time on
# the host counts (an empty launch takes 3.5 us of it): checks compare what is
# cheap to read first and word the error only once one has failed.


def _dtype_code(dtype, name: str) -> int:
    import torch
    if dtype is torch.bfloat16:
        return MOE_BF16
    if dtype is torch.float32:
        return MOE_F32
    raise _arg_error(f"{name} must be torch.bfloat16 or torch.float32, got {dtype}")


def _need_shape(t, name: str, dtype, shape, like):
    """Raise MoeError(MOE_ERR_ARG) unless `t` is a contiguous tensor of `dtype`
    and exactly `shape` on the device of the tensor `like`."""
    try:
        if t.dtype is dtype and t.shape == shape and t.get_device() == like.get_device() and t.is_contiguous():
            return
    except AttributeError:   # not a tensor
        pass
    import torch
    if not isinstance(t, torch.Tensor):
        raise _arg_error(f"{name} must be a torch.Tensor, got {type(t).__name__}")
    if t.dtype != dtype:
        raise _arg_error(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise _arg_error(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.device != like.device:
        raise _arg_error(f"{name} must be on {like.device}, got {t.device}")
    raise _arg_error(f"{name} must be contiguous")


def _rows(t, name: str, dtypes, cols: Optional[int], like):
    """The row stride (elements) of a matrix whose rows are contiguous;
    MoeError(MOE_ERR_ARG) otherwise."""
    try:
        if t.is_contiguous() and t.dtype in dtypes and t.dim() == 2 and (cols is None or t.shape[1] == cols) \
                and (like is None or t.get_device() == like.get_device()):
            return t.shape[1]
    except AttributeError:   # not a tensor
        pass
    import torch
    if not isinstance(t, torch.Tensor):
        raise _arg_error(f"{name} must be a torch.Tensor, got {type(t).__name__}")
    if t.dtype not in dtypes:
        raise _arg_error(f"{name} must be {' or '.join(map(str, dtypes))}, got {t.dtype}")
    if t.dim() != 2 or (cols is not None and t.shape[1] != cols):
        raise _arg_error(f"{name} must be [rows, {'cols' if cols is None else cols}], got shape {tuple(t.shape)}")
    if like is not None and t.get_device() != like.get_device():
        raise _arg_error(f"{name} must be on {like.device}, got {t.device}")
    row_stride, step = t.stride()
    if step != 1 and t.shape[1] > 1:
        raise _arg_error(f"the rows of {name} must be contiguous, got strides {t.stride()}")
    return row_stride if t.shape[0] > 1 else t.shape[1]


def _apart(out, name: str, *inputs):
    """Raise MoeError(MOE_ERR_ARG) if the memory of the contiguous `out` and of
    an input overlap; inputs are given as (name, tensor), each contiguous or a
    matrix of contiguous rows."""
    lo = out.data_ptr()
    hi = lo + out.nbytes
    for other, t in inputs:
        at = t.data_ptr()
        if at < hi and at + t.nbytes > lo or at < lo and not t.is_contiguous() and t.numel() and \
                at + ((t.shape[0] - 1) * t.stride(0) + t.shape[1]) * t.element_size() > lo:
            if lo != hi and t.numel():
                raise _arg_error(f"{name} must not overlap {other}")


def _new(shape, dtype, like, stream):
    """An uninitialised tensor on the device of `like`, from the memory of
    `stream` if one is given."""
    import torch
    if stream is None:
        return like.new_empty(*shape, dtype=dtype)   # torch reads a tuple of sizes 0.4 us slower
    with torch.cuda.stream(stream):
        return like.new_empty(*shape, dtype=dtype)


def _launch(fn, args, like, stream, tensors):
    """fn(*args, stream) on `stream`, or on the current stream of the tensors'
    device, with that device current.  On a given stream the tensors' memory is
    kept from other use until the stream has passed this point."""
    import torch
    index = like.get_device()
    if index < 0:
        raise _arg_error(f"tensors must be on a GPU, got {like.device}")
    if stream is None:
        # the address behind torch.cuda.current_stream(index), without the
        # 2.7 us of building the Stream object
        at = torch._C._cuda_getCurrentRawStream(index)
    elif stream.device != like.device:
        raise _arg_error(f"stream is of {stream.device}, the tensors are on {like.device}")
    else:
        at = stream.cuda_stream
    if index == torch._C._cuda_getDevice():
        status = fn(*args, at)
    else:
        with torch.cuda.device(index):
            status = fn(*args, at)
    if status:
        _check(status)
    if stream is not None:
        for t in tensors:
            t.record_stream(stream)


def mxfp4_quantize(x, codes=None, scales=None, stream=None):
    """codes uint8 [rows, cols/2] and scales uint8 [rows, cols/32] of a bf16 or
    fp32 matrix [rows, cols], cols a multiple of 32 (moe_mxfp4_quantize).  The
    rows of x must be contiguous; they may be a slice of wider ones."""
    import torch
    ld = _rows(x, "x", (torch.bfloat16, torch.float32), None, None)
    rows, cols = x.shape
    if cols <= 0 or cols % 32:
        raise MoeError(MOE_ERR_SHAPE, f"cols must be a positive multiple of 32, got {cols}")
    if (rows | cols) >> 31:
        raise _too_large(rows=rows, cols=cols)
    if codes is None:
        codes = _new((rows, cols // 2), torch.uint8, x, stream)
    else:
        _need_shape(codes, "codes", torch.uint8, (rows, cols // 2), x)
        _apart(codes, "codes", ("x", x))
    if scales is None:
        scales = _new((rows, cols // 32), torch.uint8, x, stream)
    else:
        _need_shape(scales, "scales", torch.uint8, (rows, cols // 32), x)
        _apart(scales, "scales", ("x", x), ("codes", codes))
    code = MOE_BF16 if x.dtype is torch.bfloat16 else MOE_F32
    _launch(load_library().moe_mxfp4_quantize,
            (x.data_ptr(), code, rows, cols, ld, codes.data_ptr(), scales.data_ptr()), x, stream, (x, codes, scales))
    return codes, scales


def _mxfp4_operand(codes, scales, codes_name: str, scales_name: str, like):
    """(rows, K) of an MXFP4 operand, its tensors checked."""
    import torch
    try:
        rows, half = shape = codes.shape
        if half and not half % 16 and not (rows | 2 * half) >> 31 and codes.dtype is scales.dtype is torch.uint8 \
                and scales.shape == (rows, half // 16) \
                and codes.get_device() == scales.get_device() == like.get_device() \
                and codes.is_contiguous() and scales.is_contiguous():
            return rows, 2 * half
    except (AttributeError, ValueError):   # not tensors, or not 2-D
        pass
    if not isinstance(codes, torch.Tensor) or codes.dim() != 2:
        raise _arg_error(f"{codes_name} must be a 2-D torch.Tensor [rows, cols/2]")
    _need_shape(codes, codes_name, torch.uint8, shape, like)
    if half == 0 or half % 16:
        raise MoeError(MOE_ERR_SHAPE, f"{codes_name} must have a positive multiple of 16 columns, got {half}")
    _need_shape(scales, scales_name, torch.uint8, (rows, half // 16), like)
    if (rows | 2 * half) >> 31:
        raise _too_large(rows=rows, cols=2 * half)
    return rows, 2 * half


def _float_out(out, name: str, shape, dtype, like, stream, *inputs):
    """(out, its type code): a new tensor of `dtype` (default bf16), or the given
    one checked against shape, dtype and the inputs' memory."""
    import torch
    if out is None:
        if dtype is None:
            dtype, code = torch.bfloat16, MOE_BF16
        else:
            code = _dtype_code(dtype, "dtype" if name == "out" else name + "_dtype")
        return _new(shape, dtype, like, stream), code
    code = _dtype_code(getattr(out, "dtype", None) if dtype is None else dtype, name)
    _need_shape(out, name, out.dtype if dtype is None else dtype, shape, like)
    _apart(out, name, *inputs)
    return out, code


def mxfp4_dequantize(codes, scales, dtype=None, out=None, stream=None):
    """The values [rows, cols] that codes [rows, cols/2] and scales [rows, cols/32]
    stand for, in bf16 (default) or fp32, exact (moe_mxfp4_dequantize)."""
    rows, cols = _mxfp4_operand(codes, scales, "codes", "scales", codes)
    out, code = _float_out(out, "out", (rows, cols), dtype, codes, stream, ("codes", codes), ("scales", scales))
    _launch(load_library().moe_mxfp4_dequantize,
            (codes.data_ptr(), scales.data_ptr(), rows, cols, code, out.data_ptr()), codes, stream,
            (codes, scales, out))
    return out


def mxfp4_matmul(a_codes, a_scales, b_codes, b_scales, dtype=None, out=None, stream=None):
    """A B^T [m, n] of two MXFP4 matrices A [m, k] and B [n, k], summed in fp32 and
    rounded once to bf16 (default) or left in fp32 (moe_mxfp4_matmul)."""
    m, k = _mxfp4_operand(a_codes, a_scales, "a_codes", "a_scales", a_codes)
    n, kb = _mxfp4_operand(b_codes, b_scales, "b_codes", "b_scales", a_codes)
    if kb != k:
        raise MoeError(MOE_ERR_SHAPE, f"A has {k} columns and B {kb}")
    out, code = _float_out(out, "out", (m, n), dtype, a_codes, stream, ("a_codes", a_codes), ("a_scales", a_scales),
                           ("b_codes", b_codes), ("b_scales", b_scales))
    _launch(load_library().moe_mxfp4_matmul,
            (a_codes.data_ptr(), a_scales.data_ptr(), b_codes.data_ptr(), b_scales.data_ptr(), m, n, k, code,
             out.data_ptr()), a_codes, stream, (a_codes, a_scales, b_codes, b_scales, out))
    return out


# No reduction of at most this many terms (a group's, of rows) is split by the
# grouped entries, whatever the other sizes: their workspace sizes, a question
# that costs a small call 0.5 us, are asked for above it only.
_LONGEST_WHOLE_SUM = 3000


def _grouped(w, offsets):
    import torch
    try:
        groups, n, k = shape = w.shape
        if w.dtype is torch.bfloat16 and offsets.dtype is torch.int32 and offsets.shape == (groups + 1,) \
                and w.get_device() == offsets.get_device() and w.is_contiguous() and offsets.is_contiguous():
            return shape
    except (AttributeError, ValueError):   # not tensors, or w not 3-D
        pass
    if not isinstance(w, torch.Tensor) or w.dim() != 3:
        raise _arg_error("w must be a 3-D torch.Tensor [num_groups, n, k]")
    _need_shape(w, "w", torch.bfloat16, w.shape, w)
    _need_shape(offsets, "offsets", torch.int32, (w.shape[0] + 1,), w)
    return w.shape


def grouped_matmul(x, w, offsets, out=None, stream=None):
    """out [rows, n] bf16 with out[r] = w[e] @ x[r] for offsets[e] <= r < offsets[e+1]
    (moe_grouped_matmul): x [rows, k] bf16 (its rows contiguous), w [num_groups, n, k]
    bf16, offsets [num_groups + 1] int32 on the device, as Plan.route gives them.
    Rows outside every group are left as they were (undefined in a new `out`).
    No autograd graph is recorded: grouped_matmul_backward gives the gradients.  A
    call that autograd would have recorded warns; under torch.no_grad(), or inside
    a torch.autograd.Function, it does not."""
    import torch
    groups, n, k = _grouped(w, offsets)
    ld = _rows(x, "x", (torch.bfloat16,), k, w)
    rows = x.shape[0]
    if (rows | groups | n | k) >> 31:
        raise _too_large(rows=rows, num_groups=groups, n=n, k=k)
    if out is None:
        out = _new((rows, n), torch.bfloat16, x, stream)
    else:
        _need_shape(out, "out", torch.bfloat16, (rows, n), w)
        _apart(out, "out", ("x", x), ("w", w), ("offsets", offsets))
    if (x.requires_grad or w.requires_grad) and torch.is_grad_enabled():
        warnings.warn("grouped_matmul records no autograd graph: the gradients are grouped_matmul_backward's", stacklevel=2)
    lib, used, space, size = load_library(), (x, w, offsets, out), None, 0
    if k > _LONGEST_WHOLE_SUM:
        size = lib.moe_grouped_matmul_workspace(rows, groups, n, k)
        if size:
            space = _new((size,), torch.uint8, x, stream)
            used += (space,)
            space = space.data_ptr()
    _launch(lib.moe_grouped_matmul,
            (x.data_ptr(), ld, w.data_ptr(), offsets.data_ptr(), rows, groups, n, k, out.data_ptr(), space, size), w,
            stream, used)
    return out


def grouped_matmul_backward(dy, x, w, offsets, dx=None, dw=None, dw_dtype=None, need_dx=True, need_dw=True,
                            stream=None):
    """(dx, dw) of grouped_matmul for dy [rows, n] bf16: dx [rows, k] bf16 (rows
    outside every group are left as they were), dw [num_groups, n, k] in fp32
    (default) or bf16, zero for an empty group (moe_grouped_matmul_backward).
    need_dx / need_dw False: that gradient is not computed and returned as None
    (x is not read without need_dw and may then be None)."""
    import torch
    groups, n, k = _grouped(w, offsets)
    lddy = _rows(dy, "dy", (torch.bfloat16,), n, w)
    rows = dy.shape[0]
    if (rows | groups | n | k) >> 31:
        raise _too_large(rows=rows, num_groups=groups, n=n, k=k)
    used = [dy, w, offsets]
    ldx, code, x_at, dw_at, dx_at = k, MOE_F32, None, None, None
    if need_dw:
        ldx = _rows(x, "x", (torch.bfloat16,), k, w)
        if x.shape[0] != rows:
            raise _arg_error(f"x must have dy's {rows} rows, got shape {tuple(x.shape)}")
        if dw is None and dw_dtype is None:
            dw_dtype = torch.float32
        dw, code = _float_out(dw, "dw", (groups, n, k), dw_dtype, w, stream, ("dy", dy), ("x", x), ("w", w),
                              ("offsets", offsets))
        x_at, dw_at = x.data_ptr(), dw.data_ptr()
        used += [x, dw]
    elif dw is not None:
        raise _arg_error("dw is given, but need_dw is False")
    if need_dx:
        if dx is None:
            dx = _new((rows, k), torch.bfloat16, w, stream)
        else:
            _need_shape(dx, "dx", torch.bfloat16, (rows, k), w)
            _apart(dx, "dx", ("dy", dy), ("w", w), ("offsets", offsets))
            if need_dw:
                _apart(dx, "dx", ("x", x), ("dw", dw))
        dx_at = dx.data_ptr()
        used.append(dx)
    elif dx is not None:
        raise _arg_error("dx is given, but need_dx is False")
    lib, space = load_library(), None
    size = 0
    if n > _LONGEST_WHOLE_SUM or rows > _LONGEST_WHOLE_SUM * groups:
        size = lib.moe_grouped_matmul_backward_workspace(rows, groups, n, k, need_dx, need_dw)
    if size:
        used.append(_new((size,), torch.uint8, w, stream))
        space = used[-1].data_ptr()
    _launch(lib.moe_grouped_matmul_backward,
            (dy.data_ptr(), lddy, x_at, ldx, w.data_ptr(), offsets.data_ptr(), rows, groups, n, k, dx_at, dw_at, code,
             space, size), w, stream, used)
    return dx, dw


def _warn_no_graph(name: str, gradient: str, *tensors):
    """Warn where autograd would have recorded the call."""
    import torch
    if torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in tensors):
        warnings.warn(f"{name} records no autograd graph{gradient}", stacklevel=3)


MOE_SCORE_SOFTMAX, MOE_SCORE_SIGMOID = 0, 1


def _bad_score(score):
    return _arg_error(f"score must be MOE_SCORE_SOFTMAX (0) or MOE_SCORE_SIGMOID (1), got {score!r}")


def _logits(logits):
    """(rows, experts, row stride, type code) of a router's logits."""
    import torch
    ld = _rows(logits, "logits", (torch.float32, torch.bfloat16), None, None)
    rows, experts = logits.shape
    if (rows | experts) >> 31:
        raise _too_large(num_tokens=rows, num_experts=experts)
    return rows, experts, ld, MOE_F32 if logits.dtype is torch.float32 else MOE_BF16


def router_select(logits, top_k, score=MOE_SCORE_SOFTMAX, bias=None, num_groups=1, group_limit=1, group_top=1,
                  renormalize=True, scale=1.0, ids=None, weights=None, stream=None):
    """topk_ids int32 [T, k] and topk_weights fp32 [T, k] from logits [T, E] in fp32
    or bf16 (moe_router_select).  Experts are ranked by score (softmax over the
    row, or sigmoid) plus bias fp32 [E]; of num_groups equal runs of experts the
    group_limit with the largest sums of their group_top best are kept; weights
    are scale times the selected scores, which do not contain the bias,
    renormalised to a sum of 1 by default.  An expert with a logit of -inf or NaN
    is never selected; slots for which no expert is left get id -1 and weight 0.
    No autograd graph is recorded: router_select_backward gives the gradient (a
    call that autograd would have recorded warns)."""
    import torch
    rows, experts, ld, code = _logits(logits)
    if (top_k | num_groups | group_limit | group_top) >> 31:   # too large, or negative, which the library refuses
        _need_int32(top_k=top_k, num_groups=num_groups, group_limit=group_limit, group_top=group_top)
    if score != MOE_SCORE_SOFTMAX and score != MOE_SCORE_SIGMOID:
        raise _bad_score(score)
    if not 0 < top_k <= experts:
        raise MoeError(MOE_ERR_SHAPE, f"top_k must be in [1, {experts}], got {top_k}")
    shape = (rows, top_k)
    used = [logits]
    if bias is not None:
        _need_shape(bias, "bias", torch.float32, (experts,), logits)
        used.append(bias)
    if ids is None:
        ids = _new(shape, torch.int32, logits, stream)
    else:
        _need_shape(ids, "ids", torch.int32, shape, logits)
        _apart(ids, "ids", *zip(("logits", "bias"), used))
    if weights is None:
        weights = _new(shape, torch.float32, logits, stream)
    else:
        _need_shape(weights, "weights", torch.float32, shape, logits)
        _apart(weights, "weights", ("ids", ids), *zip(("logits", "bias"), used))
    if logits.requires_grad:
        _warn_no_graph("router_select", ": the gradient is router_select_backward's", logits)
    _launch(load_library().moe_router_select,
            (logits.data_ptr(), code, ld, rows, experts, top_k, score, _ptr(bias), num_groups, group_limit, group_top,
             bool(renormalize), scale, ids.data_ptr(), weights.data_ptr()), logits, stream, (*used, ids, weights))
    return ids, weights


def router_select_backward(dweights, logits, ids, score=MOE_SCORE_SOFTMAX, renormalize=True, scale=1.0, dlogits=None,
                           stream=None):
    """The gradient [T, E] of router_select's logits, in their type, for dweights
    fp32 [T, k] and the ids int32 [T, k] that it gave; score, renormalize and
    scale as there (moe_router_select_backward)."""
    import torch
    rows, experts, ld, code = _logits(logits)
    if score != MOE_SCORE_SOFTMAX and score != MOE_SCORE_SIGMOID:
        raise _bad_score(score)
    if not isinstance(ids, torch.Tensor) or ids.dim() != 2:
        raise _arg_error("ids must be a 2-D torch.Tensor [T, top_k]")
    shape = (rows, ids.shape[1])
    if shape[1] >> 31:
        raise _too_large(top_k=shape[1])
    _need_shape(ids, "ids", torch.int32, shape, logits)
    _need_shape(dweights, "dweights", torch.float32, shape, logits)
    if dlogits is None:
        dlogits = _new((rows, experts), logits.dtype, logits, stream)
    else:
        _need_shape(dlogits, "dlogits", logits.dtype, (rows, experts), logits)
        _apart(dlogits, "dlogits", ("dweights", dweights), ("logits", logits), ("ids", ids))
    _launch(load_library().moe_router_select_backward,
            (dweights.data_ptr(), logits.data_ptr(), code, ld, ids.data_ptr(), rows, experts, shape[1], score,
             bool(renormalize), scale, dlogits.data_ptr()), logits, stream, (dweights, logits, ids, dlogits))
    return dlogits


def mxfp4_linear(x, codes, scales, gate=False, dtype=None, out=None, stream=None):
    """x W^T [m, n] of bf16 rows x [m, k] (contiguous, or a slice of wider ones) and
    an MXFP4 matrix W [n, k] (codes uint8 [n, k/2], scales uint8 [n, k/32]), summed
    in fp32 and rounded once to bf16 (default) or left in fp32 (moe_mxfp4_linear).
    gate: W is a fused w1||w3 and the result silu(x w1^T) * (x w3^T) [m, n/2].
    No autograd graph is recorded (a call that autograd would have recorded
    warns): the weights are four-bit constants."""
    import torch
    n, k = _mxfp4_operand(codes, scales, "codes", "scales", codes)
    ld = _rows(x, "x", (torch.bfloat16,), k, codes)
    m = x.shape[0]
    if m >> 31:
        raise _too_large(m=m)
    if gate and n % 2:
        raise MoeError(MOE_ERR_SHAPE, f"a gated product needs an even n, got {n}")
    out, code = _float_out(out, "out", (m, n // 2 if gate else n), dtype, codes, stream, ("x", x), ("codes", codes),
                           ("scales", scales))
    if x.requires_grad:
        _warn_no_graph("mxfp4_linear", "", x)
    _launch(load_library().moe_mxfp4_linear,
            (x.data_ptr(), ld, codes.data_ptr(), scales.data_ptr(), m, n, k, bool(gate), code, out.data_ptr()), codes,
            stream, (x, codes, scales, out))
    return out


def _routes(rowpos, weights, like):
    """(tokens, top_k) of rowpos and the weights, if there are any."""
    import torch
    if not isinstance(rowpos, torch.Tensor) or rowpos.dim() != 2:
        raise _arg_error("rowpos must be a 2-D torch.Tensor [T, top_k]")
    shape = rowpos.shape
    _need_shape(rowpos, "rowpos", torch.int32, shape, like)
    if weights is not None:
        _need_shape(weights, "weights", torch.float32, shape, like)
    return shape


def expert_combine(y, rowpos, weights=None, dtype=None, out=None, stream=None):
    """out [T, hidden]: each token's sum over its slots of weights[t, s] times the row
    rowpos[t, s] of y [rows, hidden] bf16, in fp32 and rounded once to bf16
    (default) or left in fp32 (moe_expert_combine).  rowpos int32 [T, k] as
    Plan.route gives it (reshaped); a value outside [0, rows) is no route.
    weights fp32 [T, k], None: all 1.  No autograd graph is recorded:
    expert_combine_backward gives the gradients (a call that autograd would have
    recorded warns)."""
    import torch
    ld = _rows(y, "y", (torch.bfloat16,), None, None)
    rows, hidden = y.shape
    tokens, top_k = _routes(rowpos, weights, y)
    if (rows | hidden | tokens | top_k) >> 31:
        raise _too_large(rows=rows, hidden=hidden, num_tokens=tokens, top_k=top_k)
    used = [("y", y), ("rowpos", rowpos)]
    if weights is not None:
        used.append(("weights", weights))
    out, code = _float_out(out, "out", (tokens, hidden), dtype, y, stream, *used)
    if y.requires_grad or weights is not None and weights.requires_grad:
        _warn_no_graph("expert_combine", ": the gradients are expert_combine_backward's", y, weights)
    _launch(load_library().moe_expert_combine,
            (y.data_ptr(), ld, rows, rowpos.data_ptr(), _ptr(weights), tokens, top_k, hidden, code, out.data_ptr()), y,
            stream, (*(t for _, t in used), out))
    return out


def expert_combine_backward(dout, y, rowpos, perm=None, weights=None, dy=None, dweights=None, need_dy=True,
                            need_dw=True, stream=None):
    """(dy, dweights) of expert_combine for dout [T, hidden] in bf16 or fp32: dy
    [rows, hidden] bf16, dy[r] = weights[t, s] * dout[t] for the route t * k + s =
    perm[r] (rows without one are left as they were, undefined in a new dy);
    dweights fp32 [T, k], 0 for no route (moe_expert_combine_backward).  rowpos
    int32 [T, k] and perm int32 [rows] as Plan.route gives them.  need_dy /
    need_dw False: that gradient is not computed and returned as None (perm is
    read for dy only and y for dweights only; either may then be None).  With
    weights None and need_dw False, dy is the rows of dout in the experts' order."""
    import torch
    if not (need_dy or need_dw):
        raise _arg_error("need_dy or need_dw must be True")
    ld = _rows(dout, "dout", (torch.bfloat16, torch.float32), None, None)
    tokens, top_k = _routes(rowpos, weights, dout)
    hidden = dout.shape[1]
    if dout.shape[0] != tokens:
        raise _arg_error(f"dout must have rowpos's {tokens} rows, got shape {tuple(dout.shape)}")
    used = [("dout", dout), ("rowpos", rowpos)]
    if weights is not None:
        used.append(("weights", weights))
    rows, ldy, y_at, dy_at, perm_at, dw_at = None, hidden, None, None, None, None
    if need_dw:
        ldy = _rows(y, "y", (torch.bfloat16,), hidden, dout)
        rows, y_at = y.shape[0], y.data_ptr()
        used.append(("y", y))
    elif dweights is not None:
        raise _arg_error("dweights is given, but need_dw is False")
    if need_dy:
        if rows is None:
            if not isinstance(perm, torch.Tensor) or perm.dim() != 1:
                raise _arg_error("perm must be a 1-D torch.Tensor [rows]")
            rows = perm.shape[0]
        _need_shape(perm, "perm", torch.int32, (rows,), dout)
        perm_at = perm.data_ptr()
        used.append(("perm", perm))
        if dy is None:
            dy = _new((rows, hidden), torch.bfloat16, dout, stream)
        else:
            _need_shape(dy, "dy", torch.bfloat16, (rows, hidden), dout)
            _apart(dy, "dy", *used)
        dy_at = dy.data_ptr()
    elif dy is not None:
        raise _arg_error("dy is given, but need_dy is False")
    if need_dw:
        if dweights is None:
            dweights = _new((tokens, top_k), torch.float32, dout, stream)
        else:
            _need_shape(dweights, "dweights", torch.float32, (tokens, top_k), dout)
            _apart(dweights, "dweights", *used, *((("dy", dy),) if need_dy else ()))
        dw_at = dweights.data_ptr()
    if (rows | hidden | tokens | top_k) >> 31:
        raise _too_large(rows=rows, hidden=hidden, num_tokens=tokens, top_k=top_k)
    _launch(load_library().moe_expert_combine_backward,
            (dout.data_ptr(), MOE_F32 if dout.dtype is torch.float32 else MOE_BF16, ld, y_at, ldy, rows,
             rowpos.data_ptr(), perm_at, _ptr(weights), tokens, top_k, hidden, dy_at, dw_at), dout, stream,
            [t for _, t in used] + [t for t in (dy, dweights) if t is not None])
    return dy, dweights


MOE_PROBE_READ, MOE_PROBE_READ_NT, MOE_PROBE_COPY = 0, 1, 2
MOE_PROBE_MFMA_BF16, MOE_PROBE_MFMA_F8F4 = 0, 1


def probe_memory(kind, src, dst, sink, grid, stream=None):
    """One launch of a memory probe over src (and dst): moe_probe_memory."""
    nbytes = src.numel() * src.element_size()
    _check(load_library().moe_probe_memory(int(kind), _ptr(src), _ptr(dst), nbytes, _ptr(sink), int(grid),
                                           _stream(stream)))


def probe_mfma(kind, iters, sink, grid, stream=None):
    """One launch of an MFMA probe: moe_probe_mfma; returns its flops."""
    fl = ctypes.c_double()
    _check(load_library().moe_probe_mfma(int(kind), int(iters), _ptr(sink), int(grid), ctypes.byref(fl),
                                         _stream(stream)))
    return fl.value


def probe_mfma_f8f4_blocks(a_lanes, b_lanes, a_scales, b_scales, c, stream=None):
    """d = one scaled MFMA per problem (moe_probe_mfma_f8f4_blocks); tensors in lane order."""
    import torch
    n = a_lanes.shape[0]
    dev = a_lanes.device
    _need(a_lanes, "a_lanes", torch.uint8, n, None, dev, ndim=3)
    _need(b_lanes, "b_lanes", torch.uint8, n, None, dev, ndim=3)
    _need(a_scales, "a_scales", torch.uint8, n, 64, dev)
    _need(b_scales, "b_scales", torch.uint8, n, 64, dev)
    _need(c, "c", torch.float32, n, None, dev, ndim=3)
    if a_lanes.shape[1:] != (64, 32) or b_lanes.shape[1:] != (64, 16) or c.shape[1:] != (64, 4):
        raise _arg_error("operands must be a [n,64,32], b [n,64,16], c [n,64,4]")
    d = torch.empty_like(c)
    _check(load_library().moe_probe_mfma_f8f4_blocks(_ptr(a_lanes), _ptr(b_lanes), _ptr(a_scales), _ptr(b_scales),
                                                     _ptr(c), _ptr(d), n, _stream(stream)))
    return d
