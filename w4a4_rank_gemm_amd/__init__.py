"""w4a4_rank_gemm_amd -- the fused W4A4 + low-rank linear of TwinQuant on MI355X.

A thin ctypes binding of libtwq (include/twq.h): it checks tensor dtypes and
devices, allocates outputs with torch on the input's device, and passes raw
pointers and the current HIP stream. Every step of the layer runs in the HIP
kernels of libtwq; there is no fallback. If libtwq.so has not been built, or no
GPU is present, the calls raise.

    Y = s_X s_W (Q_X Q_W) + (X L1) L2

(TwinQuant, page 1, section 2, eqs. (1)-(3); fused as in page 1, section 4.3.)
"""
from __future__ import annotations

import ctypes
import functools
import os
import threading

import torch

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "lib", "libtwq.so")

TWQ_OK = 0
STATUS_NAMES = {0: "TWQ_OK", 1: "TWQ_ERR_NULL", 2: "TWQ_ERR_SHAPE", 3: "TWQ_ERR_ALIGN",
                4: "TWQ_ERR_UNSUPPORTED", 5: "TWQ_ERR_HIP", 6: "TWQ_ERR_WORKSPACE"}

# every symbol include/twq.h declares
EXPORTS = ("twq_status_string", "twq_last_error_string", "twq_last_hip_error", "twq_version",
           "twq_quantize_act_workspace_bytes", "twq_quantize_act", "twq_pack_weight",
           "twq_dual_linear", "twq_debug_residual_acc", "twq_linear_workspace_bytes",
           "twq_linear", "twq_quantize_act_grouped", "twq_pack_weight_grouped", "twq_dual_linear_grouped",
           "twq_linear_grouped_workspace_bytes", "twq_linear_grouped", "twq_quantize_act_a8",
           "twq_dual_linear_a8", "twq_linear_a8_workspace_bytes", "twq_linear_a8", "twq_debug_residual_acc_a8",
           "twq_pack_lowrank_int4",
           "twq_quantize_act_lr4", "twq_debug_lr4_h", "twq_dual_linear_lr4", "twq_linear_lr4_workspace_bytes",
           "twq_linear_lr4", "twq_debug_linear_lr4_main", "twq_debug_linear_main",
           "twq_debug_linear_grouped_main", "twq_debug_linear_a8_main", "twq_linear_noalloc_max_bytes",
           "twq_linear_noalloc", "twq_fold_workspace_bytes", "twq_fold_lowrank", "twq_adapter_plan_bytes",
           "twq_adapter_plan", "twq_adapters_workspace_bytes", "twq_adapters", "twq_adapters_grad_workspace_bytes",
           "twq_adapters_grad", "twq_checkpoint_act", "twq_restore_act", "twq_linear_dx_workspace_bytes",
           "twq_linear_dx", "twq_linear_a16_workspace_bytes", "twq_linear_a16", "twq_moe_route_workspace_bytes",
           "twq_moe_route", "twq_moe_experts_workspace_bytes", "twq_moe_experts", "twq_moe_workspace_bytes", "twq_moe")

GROUP = 128  # group size of the group-wise entry points


class TwqError(RuntimeError):
    def __init__(self, status: int, where: str, detail: str = ""):
        self.status = status
        msg = f"{where}: {STATUS_NAMES.get(status, status)}"
        if detail:
            msg += f" ({detail})"
        super().__init__(msg)


_lib = None
_lock = threading.Lock()
_P, _I, _S, _T, _F = ctypes.c_void_p, ctypes.c_int64, ctypes.c_size_t, ctypes.c_int, ctypes.c_float


def lib() -> ctypes.CDLL:
    """The loaded libtwq.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        with _lock:
            if _lib is None:
                if not os.path.exists(LIB_PATH):
                    raise ImportError(f"libtwq.so is not built ({LIB_PATH}); run "
                                      "`python -m w4a4_rank_gemm_amd.build`")
                L = ctypes.CDLL(LIB_PATH)
                L.twq_status_string.restype = ctypes.c_char_p
                L.twq_status_string.argtypes = [ctypes.c_int]
                L.twq_last_error_string.restype = ctypes.c_char_p
                L.twq_last_error_string.argtypes = []
                L.twq_last_hip_error.restype = ctypes.c_char_p
                L.twq_last_hip_error.argtypes = []
                L.twq_version.restype = ctypes.c_int
                L.twq_quantize_act_workspace_bytes.restype = _S
                L.twq_quantize_act_workspace_bytes.argtypes = [_I, _I, _I]
                L.twq_quantize_act.restype = ctypes.c_int
                L.twq_quantize_act.argtypes = [_P, _I, _I, _P, _P, _P, _I, _P, _P, _S, _P]
                L.twq_pack_weight.restype = ctypes.c_int
                L.twq_pack_weight.argtypes = [_P, _I, _I, _P, _P, _P]
                L.twq_dual_linear.restype = ctypes.c_int
                L.twq_dual_linear.argtypes = [_P, _P, _P, _P, _P, _P, _I, _P, _I, _I, _I, _P]
                L.twq_debug_residual_acc.restype = ctypes.c_int
                L.twq_debug_residual_acc.argtypes = [_P, _P, _P, _I, _I, _I, _P]
                L.twq_linear_workspace_bytes.restype = _S
                L.twq_linear_workspace_bytes.argtypes = [_I, _I, _I, _I]
                L.twq_linear.restype = ctypes.c_int
                L.twq_linear.argtypes = [_P, _P, _P, _P, _P, _I, _P, _I, _I, _I, _P, _S, _P]
                L.twq_quantize_act_grouped.restype = ctypes.c_int
                L.twq_quantize_act_grouped.argtypes = [_P, _I, _I, _I, _P, _P, _P, _I, _P, _P, _S, _P]
                L.twq_pack_weight_grouped.restype = ctypes.c_int
                L.twq_pack_weight_grouped.argtypes = [_P, _I, _I, _I, _P, _P, _P]
                L.twq_dual_linear_grouped.restype = ctypes.c_int
                L.twq_dual_linear_grouped.argtypes = [_P, _P, _P, _P, _P, _P, _I, _P, _I, _I, _I, _I, _P]
                L.twq_linear_grouped_workspace_bytes.restype = _S
                L.twq_linear_grouped_workspace_bytes.argtypes = [_I, _I, _I, _I, _I]
                L.twq_linear_grouped.restype = ctypes.c_int
                L.twq_linear_grouped.argtypes = [_P, _P, _P, _P, _P, _I, _P, _I, _I, _I, _I, _P, _S, _P]
                L.twq_quantize_act_a8.restype = ctypes.c_int
                L.twq_quantize_act_a8.argtypes = [_P, _I, _I, _P, _P, _P, _I, _P, _P, _S, _P]
                L.twq_dual_linear_a8.restype = ctypes.c_int
                L.twq_dual_linear_a8.argtypes = [_P, _P, _P, _P, _P, _P, _I, _P, _I, _I, _I, _P]
                L.twq_linear_a8_workspace_bytes.restype = _S
                L.twq_linear_a8_workspace_bytes.argtypes = [_I, _I, _I, _I]
                L.twq_linear_a8.restype = ctypes.c_int
                L.twq_linear_a8.argtypes = [_P, _P, _P, _P, _P, _I, _P, _I, _I, _I, _P, _S, _P]
                L.twq_debug_residual_acc_a8.restype = ctypes.c_int
                L.twq_debug_residual_acc_a8.argtypes = [_P, _P, _P, _I, _I, _I, _P]
                L.twq_pack_lowrank_int4.restype = ctypes.c_int
                L.twq_pack_lowrank_int4.argtypes = [_P, _P, _I, _I, _I, _P, _P, _P, _P, _P, _P]
                L.twq_quantize_act_lr4.restype = ctypes.c_int
                L.twq_quantize_act_lr4.argtypes = [_P, _I, _I, _P, _P, _I, _P, _P, _P, _P, _P]
                L.twq_debug_lr4_h.restype = ctypes.c_int
                L.twq_debug_lr4_h.argtypes = [_P, _I, _I, _P, _P, _I, _P, _P, _P, _P, _P, _P]
                L.twq_linear_lr4_workspace_bytes.restype = _S
                L.twq_linear_lr4_workspace_bytes.argtypes = [_I, _I, _I, _I]
                for nm in ("twq_linear_lr4", "twq_debug_linear_lr4_main"):
                    getattr(L, nm).restype = ctypes.c_int
                    getattr(L, nm).argtypes = [_P, _P, _P, _P, _P, _P, _I, _P, _I, _I, _I, _P, _S, _P]
                L.twq_dual_linear_lr4.restype = ctypes.c_int
                L.twq_dual_linear_lr4.argtypes = [_P, _P, _P, _P, _P, _P, _P, _I, _P, _I, _I, _I, _P]
                for nm in ("twq_debug_linear_main", "twq_debug_linear_a8_main"):
                    getattr(L, nm).restype = ctypes.c_int
                    getattr(L, nm).argtypes = [_P, _P, _P, _P, _P, _I, _P, _I, _I, _I, _P, _S, _P]
                L.twq_fold_workspace_bytes.restype = _S
                L.twq_fold_workspace_bytes.argtypes = [_I, _I, _I]
                L.twq_fold_lowrank.restype = ctypes.c_int
                L.twq_fold_lowrank.argtypes = [_P, _P, _P, _P, _P, _P, _I, _I, _I, _P, _P, _P, _P, _S, _P]
                L.twq_linear_noalloc_max_bytes.restype = _S
                L.twq_linear_noalloc_max_bytes.argtypes = []
                L.twq_linear_noalloc.restype = ctypes.c_int
                L.twq_linear_noalloc.argtypes = [_P, _P, _P, _P, _P, _I, _P, _I, _I, _I, _P]
                L.twq_debug_linear_grouped_main.restype = ctypes.c_int
                L.twq_debug_linear_grouped_main.argtypes = [_P, _P, _P, _P, _P, _I, _P, _I, _I, _I, _I, _P, _S, _P]
                for nm, args in (("twq_adapter_plan_bytes", [_I] * 2), ("twq_adapters_workspace_bytes", [_I] * 5),
                                 ("twq_adapters_grad_workspace_bytes", [_I] * 5),
                                 ("twq_linear_dx_workspace_bytes", [_I] * 4), ("twq_linear_a16_workspace_bytes", [_I] * 5),
                                 ("twq_moe_route_workspace_bytes", [_I] * 4),
                                 ("twq_moe_experts_workspace_bytes", [_I] * 5), ("twq_moe_workspace_bytes", [_I] * 5)):
                    getattr(L, nm).restype = _S
                    getattr(L, nm).argtypes = args
                for nm, args in (("twq_adapter_plan", [_P, _I, _I, _P, _S, _P]),
                                 ("twq_adapters", [_P] * 5 + [_S] + [_P] * 3 + [_I] * 5 + [_T, _P, _S, _P]),
                                 ("twq_adapters_grad", [_P] * 9 + [_S] + [_P] * 4 + [_I] * 5 + [_T, _P, _S, _P]),
                                 ("twq_checkpoint_act", [_P, _I, _I, _T, _P, _P, _P]),
                                 ("twq_restore_act", [_P, _P, _I, _I, _T, _P, _P]),
                                 ("twq_linear_dx", [_P] * 5 + [_I, _P, _I, _I, _I, _T, _P, _S, _P]),
                                 ("twq_linear_a16", [_P] * 5 + [_I, _P, _I, _I, _I, _I, _T, _P, _S, _P]),
                                 ("twq_moe_route", [_P] * 3 + [_I] * 4 + [_T, _T, _F, _T] + [_P] * 3 + [_S, _P]),
                                 ("twq_moe_experts", [_P] * 8 + [_I] * 6 + [_T, _P, _S, _P]),
                                 ("twq_moe", [_P] * 8 + [_I] * 6 + [_T, _T, _F, _T, _P, _S, _P])):
                    getattr(L, nm).restype = ctypes.c_int
                    getattr(L, nm).argtypes = args
                _lib = L
    return _lib


def _check(status: int, where: str):
    if status != TWQ_OK:
        detail = lib().twq_last_error_string().decode() if status == 5 else ""
        raise TwqError(status, where, detail)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(dev: torch.device):
    return ctypes.c_void_p(torch.cuda.current_stream(dev).cuda_stream)


def _need(t: torch.Tensor, name: str, dtype: torch.dtype, ndim: int):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be on a GPU (got {t.device})")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype} (got {t.dtype})")
    if t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims (got {tuple(t.shape)})")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


# One workspace per (device, stream): calls sharing a workspace must not overlap,
# and eager calls enqueued on one stream never do. New workspaces start zeroed.
# Captured calls take theirs from their graph's memory: a graph may be replayed on any
# stream, and after the workspace of its capture stream was replaced by a larger one.
_workspaces: dict = {}


def _workspace(dev: torch.device, nbytes: int):
    if nbytes == 0:
        return None, 0
    if torch.cuda.is_current_stream_capturing():
        return torch.empty(nbytes, dtype=torch.uint8, device=dev), nbytes
    key = (dev.index, torch.cuda.current_stream(dev).cuda_stream)
    ws = _workspaces.get(key)
    if ws is None or ws.numel() < nbytes:
        ws = torch.zeros(max(nbytes, 1 << 20), dtype=torch.uint8, device=dev)
        _workspaces[key] = ws
    return ws, ws.numel()


def quantize_act(x: torch.Tensor, l1t: torch.Tensor | None = None):
    """X fp16 [b][m] -> (Q_X u8 [b][m/2], s_X f32 [b], T f32 [b][r] or None)."""
    _need(x, "x", torch.float16, 2)
    b, m = x.shape
    r = 0
    if l1t is not None:
        _need(l1t, "l1t", torch.float16, 2)
        r = l1t.shape[0]
        if l1t.shape[1] != m or l1t.device != x.device:
            raise ValueError("l1t must be [r][m] on x's device")
    dev = x.device
    qx = torch.empty((b, m // 2), dtype=torch.uint8, device=dev)
    sx = torch.empty((b,), dtype=torch.float32, device=dev)
    t = torch.empty((b, r), dtype=torch.float32, device=dev) if r else None
    L = lib()
    ws, wsb = _workspace(dev, L.twq_quantize_act_workspace_bytes(b, m, r))
    _check(L.twq_quantize_act(_ptr(x), b, m, _ptr(qx), _ptr(sx), _ptr(l1t), r, _ptr(t),
                              _ptr(ws), wsb, _stream(dev)), "twq_quantize_act")
    return qx, sx, t


def pack_weight(w_res: torch.Tensor):
    """W_res f32 [n][m] -> (Q_W u8 [n][m/2], s_W f32 [n]).

    Q_W's n*m/2 bytes are in the library's 16-channel panel layout (twq.h), not one
    channel per row: the tensor's shape only records n and m."""
    _need(w_res, "w_res", torch.float32, 2)
    n, m = w_res.shape
    dev = w_res.device
    qw = torch.empty((n, m // 2), dtype=torch.uint8, device=dev)
    sw = torch.empty((n,), dtype=torch.float32, device=dev)
    _check(lib().twq_pack_weight(_ptr(w_res), n, m, _ptr(qw), _ptr(sw), _stream(dev)),
           "twq_pack_weight")
    return qw, sw


def dual_linear(qx, sx, qw, sw, t=None, l2t=None, out: torch.Tensor | None = None):
    """The fused layer: Y fp16 [b][n] from the packed operands and the low-rank pair."""
    _need(qx, "qx", torch.uint8, 2)
    _need(qw, "qw", torch.uint8, 2)
    _need(sx, "sx", torch.float32, 1)
    _need(sw, "sw", torch.float32, 1)
    b, kb = qx.shape
    n = qw.shape[0]
    m = 2 * kb
    if qw.shape[1] != kb or sx.shape[0] != b or sw.shape[0] != n:
        raise ValueError("inconsistent shapes of qx/sx/qw/sw")
    r = 0
    if l2t is not None or t is not None:
        _need(t, "t", torch.float32, 2)
        _need(l2t, "l2t", torch.float16, 2)
        r = l2t.shape[1]
        if t.shape != (b, r) or l2t.shape[0] != n:
            raise ValueError("t must be [b][r] and l2t [n][r]")
    dev = qx.device
    for name, ten in (("sx", sx), ("qw", qw), ("sw", sw), ("t", t), ("l2t", l2t)):
        if ten is not None and ten.device != dev:
            raise ValueError(f"{name} is on {ten.device}, qx on {dev}")
    y = out if out is not None else torch.empty((b, n), dtype=torch.float16, device=dev)
    _need(y, "out", torch.float16, 2)
    if y.shape != (b, n):
        raise ValueError("out must be [b][n]")
    _check(lib().twq_dual_linear(_ptr(qx), _ptr(sx), _ptr(qw), _ptr(sw), _ptr(t), _ptr(l2t), r,
                                 _ptr(y), b, m, n, _stream(dev)), "twq_dual_linear")
    return y


def linear(x: torch.Tensor, qw, sw, l1t=None, l2t=None, out: torch.Tensor | None = None):
    """The whole layer in one call (twq_linear): Y fp16 [b][n] from fp16 X, the packed
    residual weight and the fp16 low-rank pair; Q_X, s_X and T live in the workspace."""
    _need(x, "x", torch.float16, 2)
    _need(qw, "qw", torch.uint8, 2)
    _need(sw, "sw", torch.float32, 1)
    b, m = x.shape
    n = qw.shape[0]
    if qw.shape[1] != m // 2 or sw.shape[0] != n:
        raise ValueError("inconsistent shapes of x/qw/sw")
    r = 0
    if l1t is not None or l2t is not None:
        _need(l1t, "l1t", torch.float16, 2)
        _need(l2t, "l2t", torch.float16, 2)
        r = l1t.shape[0]
        if l1t.shape[1] != m or l2t.shape != (n, r):
            raise ValueError("l1t must be [r][m] and l2t [n][r]")
    dev = x.device
    for name, ten in (("qw", qw), ("sw", sw), ("l1t", l1t), ("l2t", l2t)):
        if ten is not None and ten.device != dev:
            raise ValueError(f"{name} is on {ten.device}, x on {dev}")
    y = out if out is not None else torch.empty((b, n), dtype=torch.float16, device=dev)
    _need(y, "out", torch.float16, 2)
    if y.shape != (b, n):
        raise ValueError("out must be [b][n]")
    L = lib()
    ws, wsb = _workspace(dev, L.twq_linear_workspace_bytes(b, m, n, r))
    _check(L.twq_linear(_ptr(x), _ptr(qw), _ptr(sw), _ptr(l1t), _ptr(l2t), r, _ptr(y), b, m, n,
                        _ptr(ws), wsb, _stream(dev)), "twq_linear")
    return y


def linear_noalloc(x: torch.Tensor, qw, sw, l1t=None, l2t=None, out: torch.Tensor | None = None):
    """twq_linear_noalloc: the one-call layer on the library's own per-GPU scratch array
    (no workspace, no allocation inside the call). Only `out`, if not given, is allocated
    here, before the call; pass `out` to allocate nothing. Calls that may overlap on one
    GPU share the scratch and must be serialized by the caller."""
    _need(x, "x", torch.float16, 2)
    _need(qw, "qw", torch.uint8, 2)
    _need(sw, "sw", torch.float32, 1)
    b, m = x.shape
    n = qw.shape[0]
    if qw.shape[1] != m // 2 or sw.shape[0] != n:
        raise ValueError("inconsistent shapes of x/qw/sw")
    r = 0
    if l1t is not None or l2t is not None:
        _need(l1t, "l1t", torch.float16, 2)
        _need(l2t, "l2t", torch.float16, 2)
        r = l1t.shape[0]
        if l1t.shape[1] != m or l2t.shape != (n, r):
            raise ValueError("l1t must be [r][m] and l2t [n][r]")
    dev = x.device
    for name, ten in (("qw", qw), ("sw", sw), ("l1t", l1t), ("l2t", l2t)):
        if ten is not None and ten.device != dev:
            raise ValueError(f"{name} is on {ten.device}, x on {dev}")
    y = out if out is not None else torch.empty((b, n), dtype=torch.float16, device=dev)
    _need(y, "out", torch.float16, 2)
    if y.shape != (b, n):
        raise ValueError("out must be [b][n]")
    with torch.cuda.device(dev):
        _check(lib().twq_linear_noalloc(_ptr(x), _ptr(qw), _ptr(sw), _ptr(l1t), _ptr(l2t), r, _ptr(y), b, m, n,
                                        _stream(dev)), "twq_linear_noalloc")
    return y


# ---- group-wise scales (groups of GROUP along K; scales group-major) ----

def quantize_act_grouped(x: torch.Tensor, l1t: torch.Tensor | None = None, g: int = GROUP):
    """X fp16 [b][m] -> (Q_X u8 [b][m/2], s_X f32 [m/g][b], T f32 [b][r] or None)."""
    _need(x, "x", torch.float16, 2)
    b, m = x.shape
    r = 0
    if l1t is not None:
        _need(l1t, "l1t", torch.float16, 2)
        r = l1t.shape[0]
        if l1t.shape[1] != m or l1t.device != x.device:
            raise ValueError("l1t must be [r][m] on x's device")
    dev = x.device
    qx = torch.empty((b, m // 2), dtype=torch.uint8, device=dev)
    sx = torch.empty((m // g, b), dtype=torch.float32, device=dev)
    t = torch.empty((b, r), dtype=torch.float32, device=dev) if r else None
    L = lib()
    ws, wsb = _workspace(dev, L.twq_quantize_act_workspace_bytes(b, m, r))
    _check(L.twq_quantize_act_grouped(_ptr(x), b, m, g, _ptr(qx), _ptr(sx), _ptr(l1t), r, _ptr(t),
                                      _ptr(ws), wsb, _stream(dev)), "twq_quantize_act_grouped")
    return qx, sx, t


def pack_weight_grouped(w_res: torch.Tensor, g: int = GROUP):
    """W_res f32 [n][m] -> (Q_W u8 [n][m/2] in the panel layout, s_W f32 [m/g][n])."""
    _need(w_res, "w_res", torch.float32, 2)
    n, m = w_res.shape
    dev = w_res.device
    qw = torch.empty((n, m // 2), dtype=torch.uint8, device=dev)
    sw = torch.empty((m // g, n), dtype=torch.float32, device=dev)
    _check(lib().twq_pack_weight_grouped(_ptr(w_res), n, m, g, _ptr(qw), _ptr(sw), _stream(dev)),
           "twq_pack_weight_grouped")
    return qw, sw


def dual_linear_grouped(qx, sx, qw, sw, t=None, l2t=None, out: torch.Tensor | None = None, g: int = GROUP):
    """The fused layer with group-wise scales: Y fp16 [b][n]."""
    _need(qx, "qx", torch.uint8, 2)
    _need(qw, "qw", torch.uint8, 2)
    _need(sx, "sx", torch.float32, 2)
    _need(sw, "sw", torch.float32, 2)
    b, kb = qx.shape
    n = qw.shape[0]
    m = 2 * kb
    if qw.shape[1] != kb or sx.shape != (m // g, b) or sw.shape != (m // g, n):
        raise ValueError("inconsistent shapes of qx/sx/qw/sw")
    r = 0
    if l2t is not None or t is not None:
        _need(t, "t", torch.float32, 2)
        _need(l2t, "l2t", torch.float16, 2)
        r = l2t.shape[1]
        if t.shape != (b, r) or l2t.shape[0] != n:
            raise ValueError("t must be [b][r] and l2t [n][r]")
    dev = qx.device
    y = out if out is not None else torch.empty((b, n), dtype=torch.float16, device=dev)
    _need(y, "out", torch.float16, 2)
    if y.shape != (b, n):
        raise ValueError("out must be [b][n]")
    _check(lib().twq_dual_linear_grouped(_ptr(qx), _ptr(sx), _ptr(qw), _ptr(sw), _ptr(t), _ptr(l2t), r,
                                         _ptr(y), b, m, n, g, _stream(dev)), "twq_dual_linear_grouped")
    return y


def linear_grouped(x: torch.Tensor, qw, sw, l1t=None, l2t=None, out: torch.Tensor | None = None, g: int = GROUP):
    """The whole group-wise layer in one call (twq_linear_grouped): Y fp16 [b][n]."""
    _need(x, "x", torch.float16, 2)
    _need(qw, "qw", torch.uint8, 2)
    _need(sw, "sw", torch.float32, 2)
    b, m = x.shape
    n = qw.shape[0]
    if qw.shape[1] != m // 2 or sw.shape != (m // g, n):
        raise ValueError("inconsistent shapes of x/qw/sw")
    r = 0
    if l1t is not None or l2t is not None:
        _need(l1t, "l1t", torch.float16, 2)
        _need(l2t, "l2t", torch.float16, 2)
        r = l1t.shape[0]
        if l1t.shape[1] != m or l2t.shape != (n, r):
            raise ValueError("l1t must be [r][m] and l2t [n][r]")
    dev = x.device
    y = out if out is not None else torch.empty((b, n), dtype=torch.float16, device=dev)
    _need(y, "out", torch.float16, 2)
    if y.shape != (b, n):
        raise ValueError("out must be [b][n]")
    L = lib()
    ws, wsb = _workspace(dev, L.twq_linear_grouped_workspace_bytes(b, m, n, r, g))
    _check(L.twq_linear_grouped(_ptr(x), _ptr(qw), _ptr(sw), _ptr(l1t), _ptr(l2t), r, _ptr(y), b, m, n, g,
                                _ptr(ws), wsb, _stream(dev)), "twq_linear_grouped")
    return y


# ---- W4A8: 8-bit activation codes (int8 [b][m]), 4-bit residual weight ----

def quantize_act_a8(x: torch.Tensor, l1t: torch.Tensor | None = None):
    """X fp16 [b][m] -> (Q_X int8 [b][m], s_X f32 [b], T f32 [b][r] or None)."""
    _need(x, "x", torch.float16, 2)
    b, m = x.shape
    r = 0
    if l1t is not None:
        _need(l1t, "l1t", torch.float16, 2)
        r = l1t.shape[0]
        if l1t.shape[1] != m or l1t.device != x.device:
            raise ValueError("l1t must be [r][m] on x's device")
    dev = x.device
    qx = torch.empty((b, m), dtype=torch.int8, device=dev)
    sx = torch.empty((b,), dtype=torch.float32, device=dev)
    t = torch.empty((b, r), dtype=torch.float32, device=dev) if r else None
    L = lib()
    ws, wsb = _workspace(dev, L.twq_quantize_act_workspace_bytes(b, m, r))
    _check(L.twq_quantize_act_a8(_ptr(x), b, m, _ptr(qx), _ptr(sx), _ptr(l1t), r, _ptr(t),
                                 _ptr(ws), wsb, _stream(dev)), "twq_quantize_act_a8")
    return qx, sx, t


def dual_linear_a8(qx, sx, qw, sw, t=None, l2t=None, out: torch.Tensor | None = None):
    """The fused W4A8 layer: Y fp16 [b][n]."""
    _need(qx, "qx", torch.int8, 2)
    _need(qw, "qw", torch.uint8, 2)
    _need(sx, "sx", torch.float32, 1)
    _need(sw, "sw", torch.float32, 1)
    b, m = qx.shape
    n = qw.shape[0]
    if qw.shape[1] != m // 2 or sx.shape[0] != b or sw.shape[0] != n:
        raise ValueError("inconsistent shapes of qx/sx/qw/sw")
    r = 0
    if l2t is not None or t is not None:
        _need(t, "t", torch.float32, 2)
        _need(l2t, "l2t", torch.float16, 2)
        r = l2t.shape[1]
        if t.shape != (b, r) or l2t.shape[0] != n:
            raise ValueError("t must be [b][r] and l2t [n][r]")
    dev = qx.device
    y = out if out is not None else torch.empty((b, n), dtype=torch.float16, device=dev)
    _need(y, "out", torch.float16, 2)
    if y.shape != (b, n):
        raise ValueError("out must be [b][n]")
    _check(lib().twq_dual_linear_a8(_ptr(qx), _ptr(sx), _ptr(qw), _ptr(sw), _ptr(t), _ptr(l2t), r,
                                    _ptr(y), b, m, n, _stream(dev)), "twq_dual_linear_a8")
    return y


def linear_a8(x: torch.Tensor, qw, sw, l1t=None, l2t=None, out: torch.Tensor | None = None):
    """The whole W4A8 layer in one call (twq_linear_a8): Y fp16 [b][n]."""
    _need(x, "x", torch.float16, 2)
    _need(qw, "qw", torch.uint8, 2)
    _need(sw, "sw", torch.float32, 1)
    b, m = x.shape
    n = qw.shape[0]
    if qw.shape[1] != m // 2 or sw.shape[0] != n:
        raise ValueError("inconsistent shapes of x/qw/sw")
    r = 0
    if l1t is not None or l2t is not None:
        _need(l1t, "l1t", torch.float16, 2)
        _need(l2t, "l2t", torch.float16, 2)
        r = l1t.shape[0]
        if l1t.shape[1] != m or l2t.shape != (n, r):
            raise ValueError("l1t must be [r][m] and l2t [n][r]")
    dev = x.device
    y = out if out is not None else torch.empty((b, n), dtype=torch.float16, device=dev)
    _need(y, "out", torch.float16, 2)
    if y.shape != (b, n):
        raise ValueError("out must be [b][n]")
    L = lib()
    ws, wsb = _workspace(dev, L.twq_linear_a8_workspace_bytes(b, m, n, r))
    _check(L.twq_linear_a8(_ptr(x), _ptr(qw), _ptr(sw), _ptr(l1t), _ptr(l2t), r, _ptr(y), b, m, n,
                           _ptr(ws), wsb, _stream(dev)), "twq_linear_a8")
    return y


def debug_residual_acc_a8(qx, qw):
    """int32 [b][n] = Q_X (8-bit) . Q_W^T (4-bit) computed by the W4A8 main loop."""
    _need(qx, "qx", torch.int8, 2)
    _need(qw, "qw", torch.uint8, 2)
    b, m = qx.shape
    n = qw.shape[0]
    acc = torch.empty((b, n), dtype=torch.int32, device=qx.device)
    _check(lib().twq_debug_residual_acc_a8(_ptr(qx), _ptr(qw), _ptr(acc), b, m, n, _stream(qx.device)),
           "twq_debug_residual_acc_a8")
    return acc


def debug_residual_acc(qx, qw):
    """int32 [b][n] = Q_X . Q_W^T computed by the fused kernel's main loop."""
    _need(qx, "qx", torch.uint8, 2)
    _need(qw, "qw", torch.uint8, 2)
    b, kb = qx.shape
    n = qw.shape[0]
    acc = torch.empty((b, n), dtype=torch.int32, device=qx.device)
    _check(lib().twq_debug_residual_acc(_ptr(qx), _ptr(qw), _ptr(acc), b, 2 * kb, n,
                                        _stream(qx.device)), "twq_debug_residual_acc")
    return acc


def pack_lowrank_int4(l1t: torch.Tensor, l2t: torch.Tensor):
    """fp16 L1^T [r][m], L2^T [n][r] -> dict ql1 [r][m/2], sl1 [r], ql2 [n][r/2], sl2 [r], c [r].

    ql1 is in the panel layout of pack_weight (it is the weight operand of H = Q_X Q_L1^T)."""
    _need(l1t, "l1t", torch.float16, 2)
    _need(l2t, "l2t", torch.float16, 2)
    r, m = l1t.shape
    n = l2t.shape[0]
    if l2t.shape[1] != r:
        raise ValueError("l2t must be [n][r]")
    dev = l1t.device
    out = {"ql1": torch.empty((r, m // 2), dtype=torch.uint8, device=dev),
           "sl1": torch.empty((r,), dtype=torch.float32, device=dev),
           "ql2": torch.empty((n, r // 2), dtype=torch.uint8, device=dev),
           "sl2": torch.empty((r,), dtype=torch.float32, device=dev),
           "c": torch.empty((r,), dtype=torch.float32, device=dev)}
    _check(lib().twq_pack_lowrank_int4(_ptr(l1t), _ptr(l2t), r, m, n, _ptr(out["ql1"]), _ptr(out["sl1"]),
                                       _ptr(out["ql2"]), _ptr(out["sl2"]), _ptr(out["c"]), _stream(dev)),
           "twq_pack_lowrank_int4")
    return out


def quantize_act_lr4(x: torch.Tensor, lp: dict, debug_h: bool = False):
    """X fp16 [b][m] and the packed int4 factors (pack_lowrank_int4) -> (Q_X u8 [b][m/2],
    s_X f32 [b], Q_H u8 [b][r/2], s_H f32 [b]); H = Q_X Q_L1^T is requantized on chip.
    debug_h: through the test export twq_debug_lr4_h, which also returns the int32 H."""
    _need(x, "x", torch.float16, 2)
    ql1, c = lp["ql1"], lp["c"]
    _need(ql1, "ql1", torch.uint8, 2)
    _need(c, "c", torch.float32, 1)
    b, m = x.shape
    r = ql1.shape[0]
    if ql1.shape[1] != m // 2 or c.shape[0] != r:
        raise ValueError("ql1 must be [r][m/2] and c [r]")
    dev = x.device
    qx = torch.empty((b, m // 2), dtype=torch.uint8, device=dev)
    sx = torch.empty((b,), dtype=torch.float32, device=dev)
    qh = torch.empty((b, r // 2), dtype=torch.uint8, device=dev)
    sh = torch.empty((b,), dtype=torch.float32, device=dev)
    if debug_h:
        h = torch.empty((b, r), dtype=torch.int32, device=dev)
        _check(lib().twq_debug_lr4_h(_ptr(x), b, m, _ptr(ql1), _ptr(c), r, _ptr(h), _ptr(qx), _ptr(sx), _ptr(qh),
                                     _ptr(sh), _stream(dev)), "twq_debug_lr4_h")
        return qx, sx, qh, sh, h
    _check(lib().twq_quantize_act_lr4(_ptr(x), b, m, _ptr(ql1), _ptr(c), r, _ptr(qx), _ptr(sx), _ptr(qh), _ptr(sh),
                                      _stream(dev)), "twq_quantize_act_lr4")
    return qx, sx, qh, sh


def linear_lr4(x: torch.Tensor, qw, sw, lp: dict, out: torch.Tensor | None = None):
    """The whole layer with the int4 low-rank branch in one call (twq_linear_lr4)."""
    _need(x, "x", torch.float16, 2)
    _need(qw, "qw", torch.uint8, 2)
    _need(sw, "sw", torch.float32, 1)
    b, m = x.shape
    n = qw.shape[0]
    ql1, c, ql2 = lp["ql1"], lp["c"], lp["ql2"]
    r = ql1.shape[0]
    if qw.shape[1] != m // 2 or sw.shape[0] != n or ql1.shape[1] != m // 2 or ql2.shape != (n, r // 2):
        raise ValueError("inconsistent shapes of x/qw/sw/ql1/ql2")
    dev = x.device
    y = out if out is not None else torch.empty((b, n), dtype=torch.float16, device=dev)
    _need(y, "out", torch.float16, 2)
    L = lib()
    ws, wsb = _workspace(dev, L.twq_linear_lr4_workspace_bytes(b, m, n, r))
    _check(L.twq_linear_lr4(_ptr(x), _ptr(qw), _ptr(sw), _ptr(ql1), _ptr(c), _ptr(ql2), r, _ptr(y), b, m, n,
                            _ptr(ws), wsb, _stream(dev)), "twq_linear_lr4")
    return y


def dual_linear_lr4(qx, sx, qw, sw, qh, sh, ql2, out: torch.Tensor | None = None):
    """The fused layer with the int4 low-rank branch: Y fp16 [b][n]."""
    for name, t, dt in (("qx", qx, torch.uint8), ("qw", qw, torch.uint8), ("qh", qh, torch.uint8),
                        ("ql2", ql2, torch.uint8)):
        _need(t, name, dt, 2)
    _need(sx, "sx", torch.float32, 1)
    _need(sw, "sw", torch.float32, 1)
    _need(sh, "sh", torch.float32, 1)
    b, kb = qx.shape
    n = qw.shape[0]
    r = 2 * qh.shape[1]
    if ql2.shape != (n, r // 2) or sh.shape[0] != b:
        raise ValueError("qh must be [b][r/2], ql2 [n][r/2], sh [b]")
    y = out if out is not None else torch.empty((b, n), dtype=torch.float16, device=qx.device)
    _check(lib().twq_dual_linear_lr4(_ptr(qx), _ptr(sx), _ptr(qw), _ptr(sw), _ptr(qh), _ptr(sh), _ptr(ql2), r,
                                     _ptr(y), b, 2 * kb, n, _stream(qx.device)), "twq_dual_linear_lr4")
    return y


# ---- low-rank adapters beside the shared layer, and training them over it ----

TYPES = {torch.float16: 0, torch.bfloat16: 1}  # TWQ_F16, TWQ_BF16


def _type(t, name: str) -> int:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype not in TYPES:
        raise TypeError(f"{name} must be torch.float16 or torch.bfloat16 (got {t.dtype})")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a GPU (got {t.device})")
    if t.dim() != 2:
        raise ValueError(f"{name} must have 2 dims (got {tuple(t.shape)})")
    return TYPES[t.dtype]


def _want(t: torch.Tensor, name: str, dtype: torch.dtype, shape: tuple, index: int):
    """t is a contiguous GPU tensor of this type and shape on GPU `index`. One comparison in the
    usual case: these calls are short enough for their checks to be seen."""
    if (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.get_device() == index
            and t.is_contiguous()):
        return
    _need(t, name, dtype, len(shape))
    if tuple(t.shape) != shape:
        raise ValueError(f"{name} must be {list(shape)} (got {list(t.shape)})")
    raise ValueError(f"{name} is on {t.device}, not on GPU {index}")


def _addr(t):
    return None if t is None else t.data_ptr()


def _launch(index: int, where: str, fn, *args):
    """fn(*args, stream) on GPU `index`'s current stream, with that GPU current."""
    stream = torch._C._cuda_getCurrentRawStream(index)
    if torch._C._cuda_getDevice() == index:
        status = fn(*args, stream)
    else:
        with torch.cuda.device(index):
            status = fn(*args, stream)
    if status != TWQ_OK:
        _check(status, where)


@functools.lru_cache(maxsize=4096)
def _sizes(name: str, *sizes) -> int:
    return getattr(lib(), name)(*sizes)


def _scratch(like: torch.Tensor, nbytes: int):
    """Workspace of one call, from torch's allocator: its memory belongs to the call's place in
    the stream (or to the graph that captures it), so neither other calls nor other captured
    graphs share it."""
    return like.new_empty(nbytes, dtype=torch.uint8) if nbytes else None


def _apart(out: torch.Tensor, name: str, *others):
    """out shares no memory with any of the others."""
    lo, hi = out.data_ptr(), out.data_ptr() + out.numel() * out.element_size()
    for t in others:
        if t is not None and t.data_ptr() < hi and lo < t.data_ptr() + t.numel() * t.element_size():
            raise ValueError(f"{name} overlaps an input it must not share memory with")


class AdapterPlan:
    """A batch's token rows grouped by adapter (adapter_plan)."""

    def __init__(self, data: torch.Tensor, b: int, count: int):
        self.data, self.b, self.count = data, b, count


def adapter_plan(index: torch.Tensor, count: int) -> AdapterPlan:
    """index int32 [b], each token row's adapter (outside [0, count): none) -> the plan that
    adapters and adapters_grad take; made once for all layers that see the same rows."""
    _need(index, "index", torch.int32, 1)
    b, gpu = index.shape[0], index.get_device()
    L = lib()
    if not 0 <= count <= 4096:
        raise ValueError(f"count must lie in [0, 4096] (got {count})")
    data = torch.empty(L.twq_adapter_plan_bytes(b, count), dtype=torch.uint8, device=index.device)
    _launch(gpu, "twq_adapter_plan", L.twq_adapter_plan, _addr(index), b, count, _addr(data), data.numel())
    return AdapterPlan(data, b, count)


def _adapter_shapes(at, bt, plan: AdapterPlan, scale, b: int, dtype: torch.dtype, gpu: int):
    if not isinstance(plan, AdapterPlan):
        raise TypeError("plan must come from adapter_plan")
    if plan.b != b or plan.data.get_device() != gpu:
        raise ValueError(f"plan is for {plan.b} rows on {plan.data.device}, not {b} on GPU {gpu}")
    for t, name in ((at, "at"), (bt, "bt")):
        if not isinstance(t, torch.Tensor) or t.dim() != 3:
            _need(t, name, dtype, 3)
    _, r, m = at.shape
    n = bt.shape[1]
    _want(at, "at", dtype, (plan.count, r, m), gpu)
    _want(bt, "bt", dtype, (plan.count, n, r), gpu)
    if scale is not None:
        _want(scale, "scale", torch.float32, (plan.count,), gpu)
    return m, n, r


def adapters(x: torch.Tensor, at: torch.Tensor, bt: torch.Tensor, plan: AdapterPlan, y: torch.Tensor | None,
             scale: torch.Tensor | None = None, out: torch.Tensor | None = None, keep_h: bool = False):
    """out[i] = y[i] + scale[a] (x[i] at[a]^T) bt[a]^T for each token row i with adapter a of
    the plan; out[i] = y[i] without one.

    x [b][m], y [b][n] (None: zeros), at [count][r][m], bt [count][n][r]: all fp16 or all bf16.
    out may be y. keep_h: also returns x at^T, f32 [b][r], which adapters_grad needs. As with every
    call here no autograd graph is recorded: the gradients are adapters_grad's and linear_dx's."""
    ty = _type(x, "x")
    dt, gpu, b = x.dtype, x.get_device(), x.shape[0]
    m, n, r = _adapter_shapes(at, bt, plan, scale, b, dt, gpu)
    _want(x, "x", dt, (b, m), gpu)
    if y is not None:
        _want(y, "y", dt, (b, n), gpu)
    if out is None:
        out = x.new_empty((b, n))
    else:
        _want(out, "out", dt, (b, n), gpu)
        _apart(out, "out", x, at, bt, scale, None if y is None or y.data_ptr() == out.data_ptr() else y)
    h = x.new_empty((b, r), dtype=torch.float32) if keep_h else None
    L = lib()
    wsb = _sizes("twq_adapters_workspace_bytes", b, m, n, r, plan.count)
    ws = _scratch(x, wsb)
    _launch(gpu, "twq_adapters", L.twq_adapters, x.data_ptr(), at.data_ptr(), bt.data_ptr(), _addr(scale),
            plan.data.data_ptr(), plan.data.numel(), _addr(y), out.data_ptr(), _addr(h), b, m, n, r, plan.count, ty,
            _addr(ws), wsb)
    return (out, h) if keep_h else out


def adapters_grad(dy: torch.Tensor, x, h: torch.Tensor, at: torch.Tensor, bt: torch.Tensor, plan: AdapterPlan,
                  scale: torch.Tensor | None = None, dx: torch.Tensor | None = None, out: torch.Tensor | None = None):
    """The gradients of adapters(): (dat [count][r][m], dbt [count][n][r], dX [b][m]).

    x: the activations [b][m], or their checkpoint (qc, sc) from checkpoint_act; h from
    adapters(keep_h=True). dX = dx + the adapters' share (dx None: zeros), written to out if
    given (out may be dx). Adapters without rows get zero gradients."""
    ty = _type(dy, "dy")
    dt, gpu, b = dy.dtype, dy.get_device(), dy.shape[0]
    m, n, r = _adapter_shapes(at, bt, plan, scale, b, dt, gpu)
    _want(dy, "dy", dt, (b, n), gpu)
    _want(h, "h", torch.float32, (b, r), gpu)
    qc = sc = None
    if isinstance(x, (tuple, list)):
        qc, sc = x
        x = None
        _want(qc, "qc", torch.int8, (b, m), gpu)
        _want(sc, "sc", torch.float32, (m // GROUP, b), gpu)
    else:
        _want(x, "x", dt, (b, m), gpu)
    if dx is not None:
        _want(dx, "dx", dt, (b, m), gpu)
    if out is None:
        out = dy.new_empty((b, m))
    else:
        _want(out, "out", dt, (b, m), gpu)
        _apart(out, "out", dy, x, qc, sc, h, at, bt, scale, None if dx is None or dx.data_ptr() == out.data_ptr() else dx)
    dat, dbt = torch.empty_like(at), torch.empty_like(bt)
    L = lib()
    wsb = _sizes("twq_adapters_grad_workspace_bytes", b, m, n, r, plan.count)
    ws = _scratch(dy, wsb)
    _launch(gpu, "twq_adapters_grad", L.twq_adapters_grad, dy.data_ptr(), _addr(x), _addr(qc), _addr(sc), h.data_ptr(),
            at.data_ptr(), bt.data_ptr(), _addr(scale), plan.data.data_ptr(), plan.data.numel(), _addr(dx), out.data_ptr(),
            dat.data_ptr(), dbt.data_ptr(), b, m, n, r, plan.count, ty, _addr(ws), wsb)
    return dat, dbt, out


def checkpoint_act(x: torch.Tensor):
    """x fp16 or bf16 [b][m] -> (codes int8 [b][m], scales f32 [m/128][b]): the activations in
    8 bits, one scale per token and 128 elements."""
    ty = _type(x, "x")
    _need(x, "x", x.dtype, 2)
    b, m = x.shape
    qc = x.new_empty((b, m), dtype=torch.int8)
    sc = x.new_empty((m // GROUP, b), dtype=torch.float32)
    _launch(x.get_device(), "twq_checkpoint_act", lib().twq_checkpoint_act, x.data_ptr(), b, m, ty, qc.data_ptr(),
            sc.data_ptr())
    return qc, sc


def restore_act(qc: torch.Tensor, sc: torch.Tensor, dtype: torch.dtype = torch.float16,
                out: torch.Tensor | None = None) -> torch.Tensor:
    """The activations of checkpoint_act again, codes times scales, in fp16 or bf16."""
    _need(qc, "qc", torch.int8, 2)
    (b, m), gpu = qc.shape, qc.get_device()
    _want(sc, "sc", torch.float32, (m // GROUP, b), gpu)
    if out is None:
        out = qc.new_empty((b, m), dtype=dtype)
    else:
        _want(out, "out", dtype, (b, m), gpu)
        _apart(out, "out", qc, sc)
    _launch(gpu, "twq_restore_act", lib().twq_restore_act, qc.data_ptr(), sc.data_ptr(), b, m, _type(out, "out"),
            out.data_ptr())
    return out


def linear_dx(dy: torch.Tensor, qw: torch.Tensor, sw: torch.Tensor, l1t=None, l2t=None,
              out: torch.Tensor | None = None) -> torch.Tensor:
    """The layer's input gradient: dX [b][m] = dY (s_W Q_W)^T + (dY L2^T) L1^T, with the packed
    weight of pack_weight and the low-rank pair of linear; dY and dX fp16 or bf16."""
    ty = _type(dy, "dy")
    _need(qw, "qw", torch.uint8, 2)
    b, gpu, dt = dy.shape[0], dy.get_device(), dy.dtype
    n, m = qw.shape[0], 2 * qw.shape[1]
    _want(dy, "dy", dt, (b, n), gpu)
    _want(qw, "qw", torch.uint8, (n, m // 2), gpu)
    _want(sw, "sw", torch.float32, (n,), gpu)
    r = 0
    if l1t is not None or l2t is not None:
        _need(l1t, "l1t", torch.float16, 2)
        r = l1t.shape[0]
        _want(l1t, "l1t", torch.float16, (r, m), gpu)
        _want(l2t, "l2t", torch.float16, (n, r), gpu)
    if out is None:
        out = dy.new_empty((b, m))
    else:
        _want(out, "out", dt, (b, m), gpu)
        _apart(out, "out", dy, qw, sw, l1t, l2t)
    L = lib()
    wsb = _sizes("twq_linear_dx_workspace_bytes", b, m, n, r)
    ws = _scratch(dy, wsb)
    _launch(gpu, "twq_linear_dx", L.twq_linear_dx, dy.data_ptr(), qw.data_ptr(), sw.data_ptr(), _addr(l1t), _addr(l2t), r,
            out.data_ptr(), b, m, n, ty, _addr(ws), wsb)
    return out


# ---- the packed weight with 16-bit activations, and routed layers of packed experts ----

SCORES = {"softmax": 0, "sigmoid": 1}  # TWQ_SOFTMAX, TWQ_SIGMOID
MOE_TOKENS = 256                       # tokens of one routed call


def linear_a16(x: torch.Tensor, qw: torch.Tensor, sw: torch.Tensor, l1t=None, l2t=None,
               out: torch.Tensor | None = None, g: int = GROUP) -> torch.Tensor:
    """The group-wise layer with unquantized activations (W4A16): Y [b][n] = X (s_W Q_W)^T +
    (X L1) L2, with the packed weight of pack_weight_grouped and the fp16 pair of linear; X and Y
    fp16 or bf16. As elsewhere here no autograd graph is recorded."""
    ty = _type(x, "x")
    _need(qw, "qw", torch.uint8, 2)
    dt, gpu = x.dtype, x.get_device()
    (b, m), n = x.shape, qw.shape[0]
    _want(x, "x", dt, (b, m), gpu)
    _want(qw, "qw", torch.uint8, (n, m // 2), gpu)
    _want(sw, "sw", torch.float32, (m // g, n), gpu)
    r = 0
    if l1t is not None or l2t is not None:
        _need(l1t, "l1t", torch.float16, 2)
        r = l1t.shape[0]
        _want(l1t, "l1t", torch.float16, (r, m), gpu)
        _want(l2t, "l2t", torch.float16, (n, r), gpu)
    if out is None:
        out = x.new_empty((b, n))
    else:
        _want(out, "out", dt, (b, n), gpu)
        _apart(out, "out", x, qw, sw, l1t, l2t)
    L = lib()
    wsb = _sizes("twq_linear_a16_workspace_bytes", b, m, n, r, g)
    ws = _scratch(x, wsb)
    _launch(gpu, "twq_linear_a16", L.twq_linear_a16, x.data_ptr(), qw.data_ptr(), sw.data_ptr(), _addr(l1t), _addr(l2t), r,
            out.data_ptr(), b, m, n, g, ty, _addr(ws), wsb)
    return out


def pack_experts(w: torch.Tensor):
    """W f32 [experts][n][m] -> (codes u8 [experts][n][m/2], scales f32 [m/128][experts * n]): each
    expert's matrix as pack_weight_grouped packs it, the scales of all experts side by side."""
    _need(w, "w", torch.float32, 3)
    e, n, m = w.shape
    if n % 16 or m % GROUP:
        raise ValueError(f"n must be a multiple of 16 and m of {GROUP} (got {n}, {m})")
    with torch.cuda.device(w.device):
        qw, sw = pack_weight_grouped(w.view(e * n, m))
    return qw.view(e, n, m // 2), sw


def _router(x, wr, k: int, bias, score: str, gpu: int):
    if score not in SCORES:
        raise ValueError(f"score must be one of {sorted(SCORES)} (got {score!r})")
    if not isinstance(wr, torch.Tensor) or wr.dim() != 2:
        _need(wr, "wr", x.dtype, 2)
    b, m = x.shape
    experts = wr.shape[0]
    _want(x, "x", x.dtype, (b, m), gpu)
    _want(wr, "wr", x.dtype, (experts, m), gpu)
    if bias is not None:
        _want(bias, "bias", torch.float32, (experts,), gpu)
    return b, m, experts


def _experts(x, gate_up, down, gpu: int):
    (q1, s1), (q2, s2) = gate_up, down
    for t, name in ((q1, "gate_up codes"), (q2, "down codes")):
        if not isinstance(t, torch.Tensor) or t.dim() != 3:
            _need(t, name, torch.uint8, 3)
    m, (experts, n1, _) = x.shape[1], q1.shape
    f = n1 // 2
    _want(q1, "gate_up codes", torch.uint8, (experts, 2 * f, m // 2), gpu)
    _want(s1, "gate_up scales", torch.float32, (m // GROUP, experts * 2 * f), gpu)
    _want(q2, "down codes", torch.uint8, (experts, m, f // 2), gpu)
    _want(s2, "down scales", torch.float32, (f // GROUP, experts * m), gpu)
    return q1, s1, q2, s2, experts, f


def _routed_out(x, out, *inputs):
    if out is None:
        return torch.empty_like(x)
    _want(out, "out", x.dtype, tuple(x.shape), x.get_device())
    _apart(out, "out", x, *inputs)
    return out


def moe_route(x: torch.Tensor, wr: torch.Tensor, k: int, bias: torch.Tensor | None = None, score: str = "softmax",
              norm: bool = True, scale: float = 1.0):
    """The router of a routed layer, for up to MOE_TOKENS tokens: (ids int32 [b][k], weights f32 [b][k]).

    Logits x wr^T (binary64; wr [experts][m] of x's type), scores p = softmax or sigmoid of
    them. A token's experts are the k with the largest logits, or with a bias (f32 [experts]) the
    largest p + bias, best first, the lowest index first among equals; weights are p, divided by
    their sum if norm, times scale."""
    ty, gpu = _type(x, "x"), x.get_device()
    b, m, experts = _router(x, wr, k, bias, score, gpu)
    ids, weights = x.new_empty((b, k), dtype=torch.int32), x.new_empty((b, k), dtype=torch.float32)
    L = lib()
    wsb = _sizes("twq_moe_route_workspace_bytes", b, m, experts, k)
    ws = _scratch(x, wsb)
    _launch(gpu, "twq_moe_route", L.twq_moe_route, x.data_ptr(), wr.data_ptr(), _addr(bias), b, m, experts, k, SCORES[score],
            int(norm), scale, ty, ids.data_ptr(), weights.data_ptr(), _addr(ws), wsb)
    return ids, weights


def moe_experts(x: torch.Tensor, ids: torch.Tensor, weights: torch.Tensor, gate_up, down,
                out: torch.Tensor | None = None) -> torch.Tensor:
    """The experts' part of a routed layer for a given choice (moe_route's, or any other router's):
    Y [b][m], y_i = sum_j weights_ij D_e (silu(G_e x_i) * (U_e x_i)) with e = ids_ij.

    x [b][m] fp16 or bf16, at most MOE_TOKENS rows; ids int32 [b][k] (outside [0, experts): none),
    weights f32 [b][k]; gate_up = pack_experts([experts][2 f][m], f rows of G and then f of U an
    expert), down = pack_experts([experts][m][f])."""
    ty, gpu = _type(x, "x"), x.get_device()
    b, m = x.shape
    _want(x, "x", x.dtype, (b, m), gpu)
    q1, s1, q2, s2, experts, f = _experts(x, gate_up, down, gpu)
    _need(ids, "ids", torch.int32, 2)
    k = ids.shape[1]
    _want(ids, "ids", torch.int32, (b, k), gpu)
    _want(weights, "weights", torch.float32, (b, k), gpu)
    out = _routed_out(x, out, ids, weights, q1, s1, q2, s2)
    L = lib()
    wsb = _sizes("twq_moe_experts_workspace_bytes", b, m, f, experts, k)
    ws = _scratch(x, wsb)
    _launch(gpu, "twq_moe_experts", L.twq_moe_experts, x.data_ptr(), ids.data_ptr(), weights.data_ptr(), q1.data_ptr(),
            s1.data_ptr(), q2.data_ptr(), s2.data_ptr(), out.data_ptr(), b, m, f, experts, k, GROUP, ty, _addr(ws), wsb)
    return out


def moe(x: torch.Tensor, wr: torch.Tensor, k: int, gate_up, down, bias: torch.Tensor | None = None, score: str = "softmax",
        norm: bool = True, scale: float = 1.0, out: torch.Tensor | None = None) -> torch.Tensor:
    """The whole routed layer in one call (twq_moe): moe_route, then moe_experts on its choice."""
    ty, gpu = _type(x, "x"), x.get_device()
    b, m, experts = _router(x, wr, k, bias, score, gpu)
    q1, s1, q2, s2, held, f = _experts(x, gate_up, down, gpu)
    if held != experts:
        raise ValueError(f"wr routes to {experts} experts, gate_up holds {held}")
    out = _routed_out(x, out, wr, bias, q1, s1, q2, s2)
    L = lib()
    wsb = _sizes("twq_moe_workspace_bytes", b, m, f, experts, k)
    ws = _scratch(x, wsb)
    _launch(gpu, "twq_moe", L.twq_moe, x.data_ptr(), wr.data_ptr(), _addr(bias), q1.data_ptr(), s1.data_ptr(), q2.data_ptr(),
            s2.data_ptr(), out.data_ptr(), b, m, f, experts, k, GROUP, SCORES[score], int(norm), scale, ty, _addr(ws), wsb)
    return out


class RoutedLayer:
    """A routed layer (mixture of experts) with packed experts, resident on one GPU: the router's
    weight wr [experts][m], the experts' gate and up rows [experts][2 f][m] and down rows
    [experts][m][f] in binary32."""

    def __init__(self, wr: torch.Tensor, gate_up: torch.Tensor, down: torch.Tensor, k: int, bias: torch.Tensor | None = None,
                 score: str = "softmax", norm: bool = True, scale: float = 1.0):
        self.wr, self.bias = wr, bias
        self.gate_up, self.down = pack_experts(gate_up), pack_experts(down)
        self.k, self.score, self.norm, self.scale = k, score, norm, scale

    def __call__(self, x: torch.Tensor, out: torch.Tensor | None = None) -> torch.Tensor:
        return moe(x, self.wr, self.k, self.gate_up, self.down, self.bias, self.score, self.norm, self.scale, out=out)

    def route(self, x: torch.Tensor):
        """The experts of each token and their weights (moe_route)."""
        return moe_route(x, self.wr, self.k, self.bias, self.score, self.norm, self.scale)


class DualLinear:
    """A packed layer: Q_W, s_W and the fp16 low-rank pair, resident on one GPU."""

    def __init__(self, w_res: torch.Tensor, l1t: torch.Tensor | None, l2t: torch.Tensor | None):
        self.qw, self.sw = pack_weight(w_res)
        self.l1t = l1t
        self.l2t = l2t
        self.n, self.m = w_res.shape
        self.r = 0 if l1t is None else l1t.shape[0]

    def __call__(self, x: torch.Tensor, out: torch.Tensor | None = None) -> torch.Tensor:
        return linear(x, self.qw, self.sw, self.l1t if self.r else None, self.l2t if self.r else None, out=out)

    def adapted(self, x: torch.Tensor, at: torch.Tensor, bt: torch.Tensor, plan: AdapterPlan,
                scale: torch.Tensor | None = None, out: torch.Tensor | None = None, keep_h: bool = False):
        """The layer with each token row's adapter on top (adapters, in place on the layer's output)."""
        y = self(x, out=out)
        return adapters(x, at, bt, plan, y, scale, out=y, keep_h=keep_h)

    def grad_input(self, dy: torch.Tensor, out: torch.Tensor | None = None) -> torch.Tensor:
        """The frozen layer's input gradient (linear_dx)."""
        return linear_dx(dy, self.qw, self.sw, self.l1t if self.r else None, self.l2t if self.r else None, out=out)
