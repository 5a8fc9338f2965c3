"""Thin Python binding of libbeam_moe.so (argument marshalling only).

Every step of the layer runs in the library's CUDA kernels; this module only
checks tensor dtypes/devices, hands raw device pointers and the current torch
stream to the C ABI, and raises ``BeamError`` on a non-OK status.  There is no
fallback: without the compiled library every entry point raises.
"""
from __future__ import annotations

import ctypes
import os
import threading

import torch

from .config import BeamMoEConfig, CConfig

_HERE = os.path.dirname(os.path.abspath(__file__))
# BEAM_MOE_DEVICE_CHECKS=1 loads the debug build with device-side bounds
# checks (group_limited_routed_gb300.build.build(checked=True)) instead
_LIB_PATH = os.path.join(_HERE, "_build_checked" if os.environ.get("BEAM_MOE_DEVICE_CHECKS") == "1"
                         else "_build", "libbeam_moe.so")
_lock = threading.Lock()
_lib = None

_P = ctypes.c_void_p
_I64 = ctypes.c_int64
_SZ = ctypes.c_size_t
_ST = ctypes.c_int

STATUS = {0: "ok", 1: "invalid argument", 2: "unsupported", 3: "workspace too small",
          4: "CUDA error", 5: "device-side wait timed out", 6: "device-side check failed"}

EXPORTS = ("beam_moe_workspace_size", "beam_moe_workspace_layout", "beam_moe_route",
           "beam_moe_select", "beam_moe_forward", "beam_moe_forward_routed",
           "beam_moe_forward_noalloc", "beam_moe_forward_nvfp4", "beam_moe_nvfp4_pack_scales",
           "beam_moe_check_status", "beam_moe_set_stage_events", "beam_moe_set_debug",
           "beam_moe_kernels_per_forward", "beam_status_string", "beam_moe_ep_dispatch",
           "beam_moe_ep_workspace_size", "beam_moe_ep_experts", "beam_moe_ep_combine",
           "beam_moe_forward_boundary", "beam_moe_forward_nvfp4_a16",
           "beam_moe_ep_experts_nvfp4", "beam_moe_forward_fp8", "beam_moe_fp8_quantize_rows",
           "beam_moe_ep_experts_fp8", "beam_moe_forward_nvfp4_boundary",
           "beam_moe_forward_nvfp4_a16_boundary", "beam_moe_forward_fp8_boundary",
           "beam_moe_forward_mxfp8", "beam_moe_forward_mxfp8_boundary",
           "beam_moe_grouped_matmul_workspace_size", "beam_moe_grouped_matmul",
           "beam_moe_grouped_matmul_dx", "beam_moe_grouped_matmul_dw", "beam_moe_swiglu",
           "beam_moe_swiglu_grad", "beam_moe_orthogonalize_workspace_size",
           "beam_moe_orthogonalize")


class BeamError(RuntimeError):
    def __init__(self, code: int, where: str):
        super().__init__(f"{where}: {STATUS.get(code, 'unknown')} (status {code})")
        self.code = code


class _Layout(ctypes.Structure):
    _fields_ = [(n, ctypes.c_size_t) for n in (
        "status", "logits", "topk_idx", "topk_w", "counts", "offsets", "perm_src", "pair_row",
        "perm_w", "x_perm", "h", "x_fp4", "x_sf", "h_fp4", "h_sf", "y", "x_fp8", "x_scale",
        "h_fp8", "h_scale", "total")]


class _Boundary(ctypes.Structure):
    _fields_ = [("residual", ctypes.c_void_p), ("post_norm_w", ctypes.c_void_p),
                ("next_norm_w", ctypes.c_void_p), ("next_input", ctypes.c_void_p),
                ("eps", ctypes.c_float), ("residual_index", ctypes.c_int32)]


class _Fp4Weight(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("sf", ctypes.c_void_p), ("global_scale", ctypes.c_void_p)]


class _Fp8Weight(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("scale", ctypes.c_void_p)]


class _Mxfp8Weight(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("sf", ctypes.c_void_p)]


class _Grouped(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("n_groups", ctypes.c_int32), ("N", ctypes.c_int32),
                ("K", ctypes.c_int32), ("dtype", ctypes.c_int32), ("out_dtype", ctypes.c_int32),
                ("x_ld", ctypes.c_int64), ("y_ld", ctypes.c_int64),
                ("w_stride_e", ctypes.c_int64), ("w_stride_n", ctypes.c_int64),
                ("w_stride_k", ctypes.c_int64)]


class _Gate(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("F", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("gate_ld", ctypes.c_int64), ("up_ld", ctypes.c_int64)]


class _Ortho(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("rows", ctypes.c_int32), ("cols", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("out_dtype", ctypes.c_int32),
                ("steps", ctypes.c_int32), ("a", ctypes.c_float), ("b", ctypes.c_float),
                ("c", ctypes.c_float), ("eps", ctypes.c_float), ("stride_batch", ctypes.c_int64),
                ("stride_row", ctypes.c_int64), ("stride_col", ctypes.c_int64)]


def library_path() -> str:
    return _LIB_PATH


def lib():
    """Load libbeam_moe.so; raises if it has not been built."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(_LIB_PATH):
            raise RuntimeError(
                f"{_LIB_PATH} is missing: build it with group_limited_routed_gb300.build.build() "
                "(there is no non-CUDA fallback)")
        L = ctypes.CDLL(_LIB_PATH)
        cfgp = ctypes.POINTER(CConfig)
        L.beam_moe_workspace_size.argtypes = [cfgp, _I64, ctypes.c_int32]
        L.beam_moe_workspace_size.restype = _SZ
        L.beam_moe_workspace_layout.argtypes = [cfgp, _I64, ctypes.c_int32, ctypes.POINTER(_Layout)]
        L.beam_moe_workspace_layout.restype = _ST
        L.beam_moe_route.argtypes = [cfgp, _P, _P, _P, _I64, _P, _P, _P, _P, _SZ, _P]
        L.beam_moe_route.restype = _ST
        L.beam_moe_select.argtypes = [cfgp, _P, _P, _I64, _P, _P, _P, _SZ, _P]
        L.beam_moe_select.restype = _ST
        L.beam_moe_forward.argtypes = [cfgp, _P, _P, _P, _P, _P, _P, _P, _I64, _P, _SZ, _P]
        L.beam_moe_forward.restype = _ST
        L.beam_moe_forward_routed.argtypes = [cfgp, _P, _P, _P, _P, _P, _P, _P, _I64, _P, _SZ, _P]
        L.beam_moe_forward_routed.restype = _ST
        L.beam_moe_forward_noalloc.argtypes = [cfgp, _P, _P, _P, _P, _P, _P, _P, _I64, _P]
        L.beam_moe_forward_noalloc.restype = _ST
        fp4p = ctypes.POINTER(_Fp4Weight)
        L.beam_moe_forward_nvfp4.argtypes = [cfgp, _P, _P, _P, fp4p, fp4p, fp4p, _P, _I64, _P,
                                             _SZ, _P]
        L.beam_moe_forward_nvfp4.restype = _ST
        L.beam_moe_forward_nvfp4_a16.argtypes = [cfgp, _P, _P, _P, fp4p, fp4p, fp4p, _P, _I64,
                                                 _P, _SZ, _P]
        L.beam_moe_forward_nvfp4_a16.restype = _ST
        fp8p = ctypes.POINTER(_Fp8Weight)
        L.beam_moe_forward_fp8.argtypes = [cfgp, _P, _P, _P, fp8p, fp8p, fp8p, _P, _I64, _P,
                                           _SZ, _P]
        L.beam_moe_forward_fp8.restype = _ST
        mxp = ctypes.POINTER(_Mxfp8Weight)
        L.beam_moe_forward_mxfp8.argtypes = [cfgp, _P, _P, _P, mxp, mxp, mxp, _P, _I64, _P,
                                             _SZ, _P]
        L.beam_moe_forward_mxfp8.restype = _ST
        L.beam_moe_fp8_quantize_rows.argtypes = [_P, _I64, ctypes.c_int32, _P, _P, _P]
        L.beam_moe_ep_experts_fp8.argtypes = [cfgp, ctypes.c_int32, ctypes.c_int32, _P, _P, _P,
                                              fp8p, fp8p, fp8p, _P, _I64, _P, _SZ, _P]
        L.beam_moe_ep_experts_fp8.restype = _ST
        L.beam_moe_fp8_quantize_rows.restype = _ST
        L.beam_moe_nvfp4_pack_scales.argtypes = [_P, _I64, _I64, _P, _P]
        L.beam_moe_nvfp4_pack_scales.restype = _ST
        L.beam_moe_check_status.argtypes = [_P, _P]
        L.beam_moe_check_status.restype = _ST
        L.beam_moe_set_stage_events.argtypes = [ctypes.POINTER(_P), ctypes.c_int32]
        L.beam_moe_set_stage_events.restype = _ST
        L.beam_moe_set_debug.argtypes = [ctypes.c_uint32, ctypes.c_int32]
        L.beam_moe_set_debug.restype = _ST
        L.beam_moe_kernels_per_forward.argtypes = [cfgp, _I64, ctypes.c_int32, ctypes.c_int32]
        L.beam_moe_kernels_per_forward.restype = ctypes.c_int32
        L.beam_moe_forward_boundary.argtypes = [cfgp, _P, _P, _P, _P, _P, _P, _P, _I64,
                                                ctypes.POINTER(_Boundary), _P, _SZ, _P]
        L.beam_moe_forward_boundary.restype = _ST
        for name, wp in (("beam_moe_forward_nvfp4_boundary", fp4p),
                         ("beam_moe_forward_nvfp4_a16_boundary", fp4p),
                         ("beam_moe_forward_fp8_boundary", fp8p),
                         ("beam_moe_forward_mxfp8_boundary", mxp)):
            f = getattr(L, name)
            f.argtypes = [cfgp, _P, _P, _P, wp, wp, wp, _P, _I64, ctypes.POINTER(_Boundary), _P,
                          _SZ, _P]
            f.restype = _ST
        L.beam_moe_ep_dispatch.argtypes = [cfgp, _P, _P, _P, _I64, ctypes.c_int32, _P, _P, _P, _P,
                                           _P, _SZ, _P]
        L.beam_moe_ep_dispatch.restype = _ST
        L.beam_moe_ep_workspace_size.argtypes = [cfgp, ctypes.c_int32, _I64, ctypes.c_int32]
        L.beam_moe_ep_workspace_size.restype = _SZ
        L.beam_moe_ep_experts.argtypes = [cfgp, ctypes.c_int32, ctypes.c_int32, _P, _P, _P, _P, _P,
                                          _P, _P, _I64, _P, _SZ, _P]
        L.beam_moe_ep_experts.restype = _ST
        L.beam_moe_ep_experts_nvfp4.argtypes = [cfgp, ctypes.c_int32, ctypes.c_int32, _P, _P, _P,
                                                fp4p, fp4p, fp4p, _P, _I64, _P, _SZ, _P]
        L.beam_moe_ep_experts_nvfp4.restype = _ST
        L.beam_moe_ep_combine.argtypes = [cfgp, _P, _I64, _P, _P, _SZ, _P]
        L.beam_moe_ep_combine.restype = _ST
        gp = ctypes.POINTER(_Grouped)
        L.beam_moe_grouped_matmul_workspace_size.argtypes = [gp, ctypes.c_int32]
        L.beam_moe_grouped_matmul_workspace_size.restype = _SZ
        for name in ("beam_moe_grouped_matmul", "beam_moe_grouped_matmul_dx"):
            f = getattr(L, name)
            f.argtypes = [gp, _P, _P, _P, _P, _P, _SZ, _P]
            f.restype = _ST
        L.beam_moe_grouped_matmul_dw.argtypes = [gp, _P, _P, _P, ctypes.c_int32, _P, _P, _SZ, _P]
        L.beam_moe_grouped_matmul_dw.restype = _ST
        ap = ctypes.POINTER(_Gate)
        L.beam_moe_swiglu.argtypes = [ap, _P, _P, _P, _P, _I64, _P]
        L.beam_moe_swiglu.restype = _ST
        L.beam_moe_swiglu_grad.argtypes = [ap, _P, _I64, _P, _P, _P, _P, _I64, _P, _I64, _P, _P]
        L.beam_moe_swiglu_grad.restype = _ST
        L.beam_moe_orthogonalize_workspace_size.argtypes = [ctypes.c_int32] * 4
        L.beam_moe_orthogonalize_workspace_size.restype = _SZ
        L.beam_moe_orthogonalize.argtypes = [ctypes.POINTER(_Ortho), _P, _P, _P, _SZ, _P]
        L.beam_moe_orthogonalize.restype = _ST
        L.beam_status_string.argtypes = [_ST]
        L.beam_status_string.restype = ctypes.c_char_p
        _lib = L
        return L


def _cfg(cfg) -> CConfig:
    return CConfig.of(cfg)


def _check(code: int, where: str):
    if code != 0:
        raise BeamError(code, where)


def _stream(stream) -> int:
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _dev(t: torch.Tensor, dtype, name: str) -> int:
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def workspace_size(cfg, T_max: int, weight_fmt: int = 0) -> int:
    c = _cfg(cfg)
    n = lib().beam_moe_workspace_size(ctypes.byref(c), int(T_max), int(weight_fmt))
    if n == 0:
        raise BeamError(1, "beam_moe_workspace_size")
    return int(n)


def layout(cfg, T_max: int, weight_fmt: int = 0) -> dict:
    c = _cfg(cfg)
    out = _Layout()
    _check(lib().beam_moe_workspace_layout(ctypes.byref(c), int(T_max), int(weight_fmt),
                                           ctypes.byref(out)), "beam_moe_workspace_layout")
    return {n: int(getattr(out, n)) for n, _ in _Layout._fields_}


class Workspace:
    """Caller-owned device workspace sized for up to T_max tokens."""

    def __init__(self, cfg, T_max: int, device=None, weight_fmt: int = 0):
        self.cfg = cfg
        self.T_max = int(T_max)
        self.nbytes = workspace_size(cfg, T_max, weight_fmt)
        self.buf = torch.zeros(self.nbytes, dtype=torch.uint8,
                               device=device if device is not None else torch.device("cuda"))
        self.layout = layout(cfg, T_max, weight_fmt)

    @property
    def ptr(self) -> int:
        return self.buf.data_ptr()

    def view(self, name: str, dtype, shape) -> torch.Tensor:
        """A tensor view of one intermediate buffer (see beam_moe_ws_layout_t)."""
        off = self.layout[name]
        n = 1
        for s in shape:
            n *= int(s)
        nbytes = n * torch.tensor([], dtype=dtype).element_size()
        return self.buf[off:off + nbytes].view(dtype).view(*shape)


def _ws(cfg, T, ws, device):
    if ws is None:
        ws = Workspace(cfg, max(int(T), 1), device)
    return ws


def route(cfg, hidden, router_w, corr_bias, ws: Workspace | None = None, want_logits=False,
          stream=None):
    """Router + group-limited selection -> (idx [T,k] int32, w [T,k] f32[, logits])."""
    T = hidden.shape[0]
    ws = _ws(cfg, T, ws, hidden.device)
    idx = torch.empty(T, cfg.topk, dtype=torch.int32, device=hidden.device)
    w = torch.empty(T, cfg.topk, dtype=torch.float32, device=hidden.device)
    logits = torch.empty(T, cfg.n_experts, dtype=torch.float32, device=hidden.device) \
        if want_logits else None
    c = _cfg(cfg)
    _check(lib().beam_moe_route(ctypes.byref(c), _dev(hidden, torch.bfloat16, "hidden"),
                                _dev(router_w, torch.float32, "router_w"),
                                _dev(corr_bias, torch.float32, "corr_bias"), T, idx.data_ptr(),
                                w.data_ptr(), None if logits is None else logits.data_ptr(),
                                ws.ptr, ws.nbytes, _stream(stream)), "beam_moe_route")
    return (idx, w, logits) if want_logits else (idx, w)


def select(cfg, logits, corr_bias, ws: Workspace | None = None, stream=None):
    """Selection alone on given FP32 logits -> (idx, w)."""
    T = logits.shape[0]
    ws = _ws(cfg, T, ws, logits.device)
    idx = torch.empty(T, cfg.topk, dtype=torch.int32, device=logits.device)
    w = torch.empty(T, cfg.topk, dtype=torch.float32, device=logits.device)
    c = _cfg(cfg)
    _check(lib().beam_moe_select(ctypes.byref(c), _dev(logits, torch.float32, "logits"),
                                 _dev(corr_bias, torch.float32, "corr_bias"), T, idx.data_ptr(),
                                 w.data_ptr(), ws.ptr, ws.nbytes, _stream(stream)),
           "beam_moe_select")
    return idx, w


def forward(cfg, hidden, router_w, corr_bias, w_gate, w_up, w_down, out=None,
            ws: Workspace | None = None, stream=None):
    """The whole layer.  ``hidden`` may be a (pinned) host tensor: it is then
    copied to the weights' device and the output copied back to the host."""
    host_in = not hidden.is_cuda
    dev = w_gate.device
    x = hidden.to(dev, non_blocking=True) if host_in else hidden
    T = x.shape[0]
    ws = _ws(cfg, T, ws, dev)
    o = torch.empty(T, cfg.d, dtype=torch.bfloat16, device=dev) if (out is None or host_in) else out
    c = _cfg(cfg)
    _check(lib().beam_moe_forward(ctypes.byref(c), _dev(x, torch.bfloat16, "hidden"),
                                  _dev(router_w, torch.float32, "router_w"),
                                  _dev(corr_bias, torch.float32, "corr_bias"),
                                  _dev(w_gate, torch.bfloat16, "w_gate"),
                                  _dev(w_up, torch.bfloat16, "w_up"),
                                  _dev(w_down, torch.bfloat16, "w_down"), o.data_ptr(), T,
                                  ws.ptr, ws.nbytes, _stream(stream)), "beam_moe_forward")
    if host_in:
        if out is None:
            out = torch.empty(o.shape, dtype=o.dtype, pin_memory=True)
        out.copy_(o, non_blocking=True)
        return out
    return o


def forward_boundary(cfg, hidden, router_w, corr_bias, w_gate, w_up, w_down, residual,
                     post_norm_w, next_norm_w, eps: float, n: int, out=None, next_input=None,
                     ws: Workspace | None = None, stream=None, a16: bool = False):
    """The layer followed by the decoder's sublayer boundary (post-norm, n-th
    depth-scaled residual add, next pre-norm) in its combine kernel.  Returns
    (out, next_input); ``residual`` is overwritten with the new stream.

    The expert format follows the weights: BF16 tensors, ``Fp4Weight`` (NVFP4
    activations, or F16 ones with ``a16=True``), ``Fp8Weight`` or
    ``Mxfp8Weight``."""
    T = hidden.shape[0]
    dev = hidden.device
    if isinstance(w_gate, Fp4Weight):
        fmt, name = (NVFP4_A16, "beam_moe_forward_nvfp4_a16_boundary") if a16 else \
            (NVFP4, "beam_moe_forward_nvfp4_boundary")
        wts = tuple(ctypes.byref(x._c) for x in (w_gate, w_up, w_down))
    elif isinstance(w_gate, Fp8Weight):
        fmt, name = FP8, "beam_moe_forward_fp8_boundary"
        wts = tuple(ctypes.byref(x._c) for x in (w_gate, w_up, w_down))
    elif isinstance(w_gate, Mxfp8Weight):
        fmt, name = MXFP8, "beam_moe_forward_mxfp8_boundary"
        wts = tuple(ctypes.byref(x._c) for x in (w_gate, w_up, w_down))
    else:
        fmt, name = BF16, "beam_moe_forward_boundary"
        wts = (_dev(w_gate, torch.bfloat16, "w_gate"), _dev(w_up, torch.bfloat16, "w_up"),
               _dev(w_down, torch.bfloat16, "w_down"))
    if ws is None:
        ws = Workspace(cfg, max(int(T), 1), dev, weight_fmt=fmt)
    o = torch.empty(T, cfg.d, dtype=torch.bfloat16, device=dev) if out is None else out
    nx = torch.empty(T, cfg.d, dtype=torch.bfloat16, device=dev) if next_input is None \
        else next_input
    b = _Boundary(_dev(residual, torch.bfloat16, "residual"),
                  _dev(post_norm_w, torch.bfloat16, "post_norm_w"),
                  _dev(next_norm_w, torch.bfloat16, "next_norm_w"),
                  _dev(nx, torch.bfloat16, "next_input"), float(eps), int(n))
    c = _cfg(cfg)
    _check(getattr(lib(), name)(ctypes.byref(c), _dev(hidden, torch.bfloat16, "hidden"),
                                _dev(router_w, torch.float32, "router_w"),
                                _dev(corr_bias, torch.float32, "corr_bias"), *wts, o.data_ptr(),
                                T, ctypes.byref(b), ws.ptr, ws.nbytes, _stream(stream)), name)
    return o, nx


def forward_routed(cfg, hidden, topk_idx, topk_w, w_gate, w_up, w_down, out=None,
                   ws: Workspace | None = None, stream=None):
    """Experts + combine with a given routing (routing replay)."""
    T = hidden.shape[0]
    ws = _ws(cfg, T, ws, hidden.device)
    o = torch.empty(T, cfg.d, dtype=torch.bfloat16, device=hidden.device) if out is None else out
    c = _cfg(cfg)
    _check(lib().beam_moe_forward_routed(ctypes.byref(c), _dev(hidden, torch.bfloat16, "hidden"),
                                         _dev(topk_idx, torch.int32, "topk_idx"),
                                         _dev(topk_w, torch.float32, "topk_w"),
                                         _dev(w_gate, torch.bfloat16, "w_gate"),
                                         _dev(w_up, torch.bfloat16, "w_up"),
                                         _dev(w_down, torch.bfloat16, "w_down"), o.data_ptr(), T,
                                         ws.ptr, ws.nbytes, _stream(stream)),
           "beam_moe_forward_routed")
    return o


def forward_noalloc(cfg, hidden, router_w, corr_bias, w_gate, w_up, w_down, out=None,
                    stream=None):
    """The whole layer without a workspace: for callers that cannot allocate
    device memory (the library's fixed 32 MiB device array holds the
    intermediates; small batches only, see beam_moe.h).  Calls overlapping on
    the GPU race on that array."""
    T = hidden.shape[0]
    o = torch.empty(T, cfg.d, dtype=torch.bfloat16, device=hidden.device) if out is None else out
    c = _cfg(cfg)
    _check(lib().beam_moe_forward_noalloc(ctypes.byref(c), _dev(hidden, torch.bfloat16, "hidden"),
                                          _dev(router_w, torch.float32, "router_w"),
                                          _dev(corr_bias, torch.float32, "corr_bias"),
                                          _dev(w_gate, torch.bfloat16, "w_gate"),
                                          _dev(w_up, torch.bfloat16, "w_up"),
                                          _dev(w_down, torch.bfloat16, "w_down"), o.data_ptr(),
                                          T, _stream(stream)), "beam_moe_forward_noalloc")
    return o


BF16 = 0
NVFP4 = 1
NVFP4_A16 = 2


def pack_scales(sf: torch.Tensor, stream=None) -> torch.Tensor:
    """Block scales [..., rows, S] (uint8, row-major: E4M3 for NVFP4, E8M0 for
    MXFP8) -> the blocked order the tensor cores take
    (beam_moe_nvfp4_pack_scales); same shape and dtype."""
    src = sf.contiguous()
    S = src.shape[-1]
    rows = src.numel() // S
    dst = torch.empty_like(src)
    _check(lib().beam_moe_nvfp4_pack_scales(_dev(src, torch.uint8, "sf"), rows, S,
                                            dst.data_ptr(), _stream(stream)),
           "beam_moe_nvfp4_pack_scales")
    return dst


class Fp4Weight:
    """One NVFP4 projection: codes q [E, N, K/2], blocked scales, global scales [E]."""

    def __init__(self, q: torch.Tensor, sf_rowmajor: torch.Tensor, gs: torch.Tensor,
                 stream=None):
        self.q = q.contiguous()
        self.sf = pack_scales(sf_rowmajor, stream)
        self.gs = gs.contiguous().float()
        self._c = _Fp4Weight(_dev(self.q, torch.uint8, "q"), self.sf.data_ptr(),
                             _dev(self.gs, torch.float32, "global_scale"))

    @classmethod
    def of(cls, d: dict, stream=None) -> "Fp4Weight":
        return cls(d["q"], d["sf"], d["gs"], stream)


def forward_nvfp4(cfg, hidden, router_w, corr_bias, gate: Fp4Weight, up: Fp4Weight,
                  down: Fp4Weight, out=None, ws: Workspace | None = None, stream=None):
    """The whole layer with NVFP4 experts (activations quantised to NVFP4)."""
    T = hidden.shape[0]
    if ws is None:
        ws = Workspace(cfg, max(int(T), 1), hidden.device, weight_fmt=NVFP4)
    o = torch.empty(T, cfg.d, dtype=torch.bfloat16, device=hidden.device) if out is None else out
    c = _cfg(cfg)
    _check(lib().beam_moe_forward_nvfp4(ctypes.byref(c), _dev(hidden, torch.bfloat16, "hidden"),
                                        _dev(router_w, torch.float32, "router_w"),
                                        _dev(corr_bias, torch.float32, "corr_bias"),
                                        ctypes.byref(gate._c), ctypes.byref(up._c),
                                        ctypes.byref(down._c), o.data_ptr(), T, ws.ptr, ws.nbytes,
                                        _stream(stream)), "beam_moe_forward_nvfp4")
    return o


def forward_nvfp4_a16(cfg, hidden, router_w, corr_bias, gate: Fp4Weight, up: Fp4Weight,
                      down: Fp4Weight, out=None, ws: Workspace | None = None, stream=None):
    """The whole layer with NVFP4 expert weights and 16-bit (F16) activations."""
    T = hidden.shape[0]
    if ws is None:
        ws = Workspace(cfg, max(int(T), 1), hidden.device, weight_fmt=NVFP4_A16)
    o = torch.empty(T, cfg.d, dtype=torch.bfloat16, device=hidden.device) if out is None else out
    c = _cfg(cfg)
    _check(lib().beam_moe_forward_nvfp4_a16(ctypes.byref(c), _dev(hidden, torch.bfloat16, "hidden"),
                                            _dev(router_w, torch.float32, "router_w"),
                                            _dev(corr_bias, torch.float32, "corr_bias"),
                                            ctypes.byref(gate._c), ctypes.byref(up._c),
                                            ctypes.byref(down._c), o.data_ptr(), T, ws.ptr,
                                            ws.nbytes, _stream(stream)),
           "beam_moe_forward_nvfp4_a16")
    return o


FP8 = 3


class Fp8Weight:
    """One dynamic-FP8 projection: E4M3 codes q [E, N, K] (uint8) and one
    FP32 scale per output row [E, N]."""

    def __init__(self, q: torch.Tensor, scale: torch.Tensor):
        self.q = q.contiguous()
        self.scale = scale.contiguous()
        self._c = _Fp8Weight(_dev(self.q, torch.uint8, "q"),
                             _dev(self.scale, torch.float32, "scale"))

    @classmethod
    def of(cls, d: dict) -> "Fp8Weight":
        return cls(d["q"], d["s"])


def forward_fp8(cfg, hidden, router_w, corr_bias, gate: Fp8Weight, up: Fp8Weight,
                down: Fp8Weight, out=None, ws: Workspace | None = None, stream=None):
    """The whole layer with dynamic FP8 experts (E4M3 weights with per-row
    scales; token rows and h quantised per row at run time)."""
    T = hidden.shape[0]
    if ws is None:
        ws = Workspace(cfg, max(int(T), 1), hidden.device, weight_fmt=FP8)
    o = torch.empty(T, cfg.d, dtype=torch.bfloat16, device=hidden.device) if out is None else out
    c = _cfg(cfg)
    _check(lib().beam_moe_forward_fp8(ctypes.byref(c), _dev(hidden, torch.bfloat16, "hidden"),
                                      _dev(router_w, torch.float32, "router_w"),
                                      _dev(corr_bias, torch.float32, "corr_bias"),
                                      ctypes.byref(gate._c), ctypes.byref(up._c),
                                      ctypes.byref(down._c), o.data_ptr(), T, ws.ptr, ws.nbytes,
                                      _stream(stream)), "beam_moe_forward_fp8")
    return o


MXFP8 = 4


class Mxfp8Weight:
    """One MXFP8 projection: E4M3 codes q [E, N, K] (uint8) and E8M0 scales,
    one per 32 along K, given row-major [E, N, K/32] and kept in the blocked
    order the tensor cores take (beam_moe_nvfp4_pack_scales)."""

    def __init__(self, q: torch.Tensor, sf_rowmajor: torch.Tensor, stream=None):
        self.q = q.contiguous()
        self.sf = pack_scales(sf_rowmajor, stream)
        self._c = _Mxfp8Weight(_dev(self.q, torch.uint8, "q"), self.sf.data_ptr())

    @classmethod
    def of(cls, d: dict, stream=None) -> "Mxfp8Weight":
        return cls(d["q"], d["s"], stream)


def forward_mxfp8(cfg, hidden, router_w, corr_bias, gate: Mxfp8Weight, up: Mxfp8Weight,
                  down: Mxfp8Weight, out=None, ws: Workspace | None = None, stream=None):
    """The whole layer with MXFP8 experts (activations quantised to MX blocks)."""
    T = hidden.shape[0]
    if ws is None:
        ws = Workspace(cfg, max(int(T), 1), hidden.device, weight_fmt=MXFP8)
    o = torch.empty(T, cfg.d, dtype=torch.bfloat16, device=hidden.device) if out is None else out
    c = _cfg(cfg)
    _check(lib().beam_moe_forward_mxfp8(ctypes.byref(c), _dev(hidden, torch.bfloat16, "hidden"),
                                        _dev(router_w, torch.float32, "router_w"),
                                        _dev(corr_bias, torch.float32, "corr_bias"),
                                        ctypes.byref(gate._c), ctypes.byref(up._c),
                                        ctypes.byref(down._c), o.data_ptr(), T, ws.ptr, ws.nbytes,
                                        _stream(stream)), "beam_moe_forward_mxfp8")
    return o


def fp8_quantize_rows(x: torch.Tensor, stream=None):
    """BF16 rows [n, cols] -> (E4M3 codes uint8 [n, cols], FP32 scales [n]),
    the FP8 path's activation rule (beam_moe_fp8_quantize_rows)."""
    n, cols = x.shape
    q = torch.empty(n, cols, dtype=torch.uint8, device=x.device)
    sc = torch.empty(n, dtype=torch.float32, device=x.device)
    _check(lib().beam_moe_fp8_quantize_rows(_dev(x, torch.bfloat16, "x"), n, cols, q.data_ptr(),
                                            sc.data_ptr(), _stream(stream)),
           "beam_moe_fp8_quantize_rows")
    return q, sc


def check_status(ws: Workspace, stream=None) -> int:
    """Synchronise and return (and clear) the latched device status code."""
    return int(lib().beam_moe_check_status(ws.ptr, _stream(stream)))


def set_stage_events(events) -> None:
    """Record 8 torch.cuda.Event objects at the step boundaries of later calls
    (None switches it off)."""
    if events is None:
        _check(lib().beam_moe_set_stage_events(None, 0), "beam_moe_set_stage_events")
        return
    arr = (_P * len(events))(*[e.cuda_event for e in events])
    _check(lib().beam_moe_set_stage_events(arr, len(events)), "beam_moe_set_stage_events")


def set_debug(wait_limit_us: int = 0, withhold_first_load: bool = False) -> None:
    _check(lib().beam_moe_set_debug(int(wait_limit_us), int(bool(withhold_first_load))),
           "beam_moe_set_debug")


def kernels_per_forward(cfg, T: int, weight_fmt: int = 0, routed: bool = False) -> int:
    c = _cfg(cfg)
    return int(lib().beam_moe_kernels_per_forward(ctypes.byref(c), int(T), int(weight_fmt),
                                                  int(bool(routed))))


# ------------------------------------------------------------ expert parallelism
def ep_dispatch(cfg, hidden, router_w, corr_bias, n_ranks: int, ws: Workspace | None = None,
                stream=None):
    """Route this rank's tokens and pack one row per (token, slot) pair in
    owner order -> (send_x [T*k, d] bf16, send_expert [T*k] int32,
    send_w [T*k] f32, send_counts [n_ranks] int32, ws).  Keep ``ws`` for
    :func:`ep_combine`."""
    T = hidden.shape[0]
    dev = hidden.device
    ws = _ws(cfg, T, ws, dev)
    TK = T * cfg.topk
    send_x = torch.empty(TK, cfg.d, dtype=torch.bfloat16, device=dev)
    send_e = torch.empty(TK, dtype=torch.int32, device=dev)
    send_w = torch.empty(TK, dtype=torch.float32, device=dev)
    counts = torch.empty(n_ranks, dtype=torch.int32, device=dev)
    c = _cfg(cfg)
    _check(lib().beam_moe_ep_dispatch(ctypes.byref(c), _dev(hidden, torch.bfloat16, "hidden"),
                                      _dev(router_w, torch.float32, "router_w"),
                                      _dev(corr_bias, torch.float32, "corr_bias"), T,
                                      int(n_ranks), send_x.data_ptr(), send_e.data_ptr(),
                                      send_w.data_ptr(), counts.data_ptr(), ws.ptr, ws.nbytes,
                                      _stream(stream)), "beam_moe_ep_dispatch")
    return send_x, send_e, send_w, counts, ws


class EpWorkspace:
    """Device workspace of :func:`ep_experts` for up to M_max received rows."""

    def __init__(self, cfg, n_ranks: int, M_max: int, device=None, weight_fmt: int = 0):
        c = _cfg(cfg)
        self.nbytes = int(lib().beam_moe_ep_workspace_size(ctypes.byref(c), int(n_ranks),
                                                           int(M_max), int(weight_fmt)))
        self.weight_fmt = int(weight_fmt)
        if self.nbytes == 0:
            raise BeamError(1, "beam_moe_ep_workspace_size")
        self.M_max = int(M_max)
        self.buf = torch.zeros(self.nbytes, dtype=torch.uint8,
                               device=device if device is not None else torch.device("cuda"))

    @property
    def ptr(self) -> int:
        return self.buf.data_ptr()


def ep_experts(cfg, n_ranks: int, rank: int, x_recv, expert_recv, w_recv, w_gate, w_up, w_down,
               ws: EpWorkspace | None = None, out=None, stream=None):
    """This rank's experts on its received rows -> y_recv [M, d] f32 (weighted)."""
    M = x_recv.shape[0]
    dev = x_recv.device
    if ws is None or ws.M_max < M:
        ws = EpWorkspace(cfg, n_ranks, max(M, 1), dev)
    y = torch.empty(M, cfg.d, dtype=torch.float32, device=dev) if out is None else out
    if M == 0:
        return y
    c = _cfg(cfg)
    _check(lib().beam_moe_ep_experts(ctypes.byref(c), int(n_ranks), int(rank),
                                     _dev(x_recv, torch.bfloat16, "x_recv"),
                                     _dev(expert_recv, torch.int32, "expert_recv"),
                                     _dev(w_recv, torch.float32, "w_recv"),
                                     _dev(w_gate, torch.bfloat16, "w_gate"),
                                     _dev(w_up, torch.bfloat16, "w_up"),
                                     _dev(w_down, torch.bfloat16, "w_down"),
                                     _dev(y, torch.float32, "y_recv"), M, ws.ptr, ws.nbytes,
                                     _stream(stream)), "beam_moe_ep_experts")
    return y


def ep_experts_nvfp4(cfg, n_ranks: int, rank: int, x_recv, expert_recv, w_recv, gate: Fp4Weight,
                     up: Fp4Weight, down: Fp4Weight, ws: EpWorkspace | None = None, out=None,
                     stream=None):
    """This rank's NVFP4 experts on its received rows -> y_recv [M, d] f32."""
    M = x_recv.shape[0]
    dev = x_recv.device
    if ws is None or ws.M_max < M or ws.weight_fmt != NVFP4:
        ws = EpWorkspace(cfg, n_ranks, max(M, 1), dev, weight_fmt=NVFP4)
    y = torch.empty(M, cfg.d, dtype=torch.float32, device=dev) if out is None else out
    if M == 0:
        return y
    c = _cfg(cfg)
    _check(lib().beam_moe_ep_experts_nvfp4(ctypes.byref(c), int(n_ranks), int(rank),
                                           _dev(x_recv, torch.bfloat16, "x_recv"),
                                           _dev(expert_recv, torch.int32, "expert_recv"),
                                           _dev(w_recv, torch.float32, "w_recv"),
                                           ctypes.byref(gate._c), ctypes.byref(up._c),
                                           ctypes.byref(down._c),
                                           _dev(y, torch.float32, "y_recv"), M, ws.ptr,
                                           ws.nbytes, _stream(stream)),
           "beam_moe_ep_experts_nvfp4")
    return y


def ep_experts_fp8(cfg, n_ranks: int, rank: int, x_recv, expert_recv, w_recv, gate: Fp8Weight,
                   up: Fp8Weight, down: Fp8Weight, ws: EpWorkspace | None = None, out=None,
                   stream=None):
    """This rank's dynamic-FP8 experts on its received rows -> y_recv [M, d] f32."""
    M = x_recv.shape[0]
    dev = x_recv.device
    if ws is None or ws.M_max < M or ws.weight_fmt != FP8:
        ws = EpWorkspace(cfg, n_ranks, max(M, 1), dev, weight_fmt=FP8)
    y = torch.empty(M, cfg.d, dtype=torch.float32, device=dev) if out is None else out
    if M == 0:
        return y
    c = _cfg(cfg)
    _check(lib().beam_moe_ep_experts_fp8(ctypes.byref(c), int(n_ranks), int(rank),
                                         _dev(x_recv, torch.bfloat16, "x_recv"),
                                         _dev(expert_recv, torch.int32, "expert_recv"),
                                         _dev(w_recv, torch.float32, "w_recv"),
                                         ctypes.byref(gate._c), ctypes.byref(up._c),
                                         ctypes.byref(down._c),
                                         _dev(y, torch.float32, "y_recv"), M, ws.ptr,
                                         ws.nbytes, _stream(stream)),
           "beam_moe_ep_experts_fp8")
    return y


def ep_combine(cfg, y_back, T: int, ws: Workspace, out=None, stream=None):
    """The owner's combine of the returned rows -> out [T, d] bf16."""
    dev = ws.buf.device
    o = torch.empty(T, cfg.d, dtype=torch.bfloat16, device=dev) if out is None else out
    if T == 0:
        return o
    c = _cfg(cfg)
    _check(lib().beam_moe_ep_combine(ctypes.byref(c), _dev(y_back, torch.float32, "y_back"), T,
                                     o.data_ptr(), ws.ptr, ws.nbytes, _stream(stream)),
           "beam_moe_ep_combine")
    return o


# ---------------------------------------------------------------- training
_DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}


class OpWorkspace:
    """Caller-owned device workspace of one training operator (a status word,
    then scratch); calls that share it must be on one stream."""

    def __init__(self, nbytes: int, device=None):
        self.nbytes = int(nbytes)
        self.buf = torch.empty(self.nbytes, dtype=torch.uint8,
                               device=device if device is not None else torch.device("cuda"))
        self.buf[:256].zero_()

    @property
    def ptr(self) -> int:
        return self.buf.data_ptr()


def _type(dtype, name: str, allowed) -> int:
    if dtype not in allowed:
        raise TypeError(f"{name} must be one of {', '.join(map(str, allowed))}, got {dtype}")
    return _DTYPES[dtype]


_HALVES = (torch.bfloat16, torch.float16)


def _rows2d(t: torch.Tensor, name: str, dtype=None, width=None) -> int:
    """Check a CUDA matrix with contiguous rows; returns its row stride."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != 2 or (width is not None and t.shape[1] != width):
        raise ValueError(f"{name} must be a matrix"
                         + (f" with {width} columns" if width is not None else "")
                         + f", got shape {tuple(t.shape)}")
    if t.shape[1] > 1 and t.stride(1) != 1:
        raise ValueError(f"{name} must have contiguous rows, got strides {t.stride()}")
    ld = t.stride(0) if t.shape[0] > 1 else t.shape[1]
    if ld < t.shape[1]:
        raise ValueError(f"{name} must not have overlapping rows, got strides {t.stride()}")
    return ld


def _same_device(first: torch.Tensor, **others) -> None:
    for name, t in others.items():
        if isinstance(t, torch.Tensor) and t.device != first.device:
            raise ValueError(f"{name} must be on {first.device}, got {t.device}")


def _offsets(offsets, n_groups=None) -> int:
    ptr = _dev(offsets, torch.int32, "offsets")
    if offsets.dim() != 1 or offsets.numel() < 2:
        raise ValueError("offsets must be a vector of at least 2 boundaries, "
                         f"got shape {tuple(offsets.shape)}")
    if n_groups is not None and offsets.numel() != n_groups + 1:
        raise ValueError(f"offsets must hold {n_groups + 1} boundaries, got {offsets.numel()}")
    return ptr


def _grouped_desc(rows, E, N, K, dtype, out_dtype, x_ld, y_ld, w_strides) -> _Grouped:
    if not 1 <= E <= 1024:
        raise ValueError(f"1 to 1024 groups, got {E}")
    return _Grouped(rows, E, N, K, _type(dtype, "operands", _HALVES),
                    _type(out_dtype, "out_dtype", (dtype, torch.float32)), x_ld, y_ld, *w_strides)


def _w_strides(w, dtype) -> tuple:
    if not isinstance(w, torch.Tensor) or not w.is_cuda:
        raise TypeError("w must be a CUDA tensor")
    if w.dtype != dtype:
        raise TypeError(f"w must be {dtype}, got {w.dtype}")
    if w.dim() != 3 or w.numel() == 0:
        raise ValueError(f"w must be [groups, N, K], got shape {tuple(w.shape)}")
    E, N, K = w.shape
    e, n, k = w.stride()
    if K == 1 and n != 1:
        k = 1
    if N == 1 and k != 1:
        n = 1
    if k == 1 and (N == 1 or n >= K):
        n = K if N == 1 else n
    elif n == 1 and (K == 1 or k >= N):
        k = N if K == 1 else k
    else:
        raise ValueError(f"w must be contiguous along N or K, got strides {w.stride()}")
    return (e if E > 1 else N * K), n, k


def grouped_matmul_workspace_size(rows: int, n_groups: int, N: int, K: int,
                                  dtype=torch.bfloat16, unaligned: bool = False) -> int:
    """Workspace bytes of the grouped products on contiguous operands (with
    ``unaligned``, of views whose base or strides are not 16-byte multiples)."""
    d = _grouped_desc(rows, n_groups, N, K, dtype, dtype, K, N, (N * K, K, 1))
    n = lib().beam_moe_grouped_matmul_workspace_size(ctypes.byref(d), int(unaligned))
    if n == 0:
        raise BeamError(1, "beam_moe_grouped_matmul_workspace_size")
    return int(n)


def _op_ws(ws, device, size) -> "OpWorkspace":
    return OpWorkspace(size(), device) if ws is None else ws


def _grouped_ws(ws, d, device, *operands):
    def size():
        odd = any(t.data_ptr() % 16 for t in operands)
        n = lib().beam_moe_grouped_matmul_workspace_size(ctypes.byref(d), int(odd))
        if n == 0:
            raise BeamError(1, "beam_moe_grouped_matmul_workspace_size")
        return n
    return _op_ws(ws, device, size)


def _grouped_rows(a, a_name, w, offsets, out, out_dtype, ws, transpose):
    """y = x W^T or, with ``transpose``, dx = dy W, group by group."""
    strides = _w_strides(w, a.dtype if isinstance(a, torch.Tensor) else None)
    E, N, K = w.shape
    width_in, width_out = (N, K) if transpose else (K, N)
    ld = _rows2d(a, a_name, width=width_in)
    _same_device(a, w=w, offsets=offsets, out=out)
    dt = out_dtype if out_dtype is not None else out.dtype if out is not None else a.dtype
    off = _offsets(offsets, E)
    if out is None:
        out = torch.empty(a.shape[0], width_out, dtype=dt, device=a.device)
    out_ld = _rows2d(out, "out", dt, width_out)
    if out.shape[0] != a.shape[0]:
        raise ValueError(f"out must have {a.shape[0]} rows, got {out.shape[0]}")
    x_ld, y_ld = (out_ld, ld) if transpose else (ld, out_ld)
    d = _grouped_desc(a.shape[0], E, N, K, a.dtype, dt, x_ld, y_ld, strides)
    ws = _grouped_ws(ws, d, a.device, a, w)
    return d, off, out, ws


def grouped_matmul(x, w, offsets, out=None, out_dtype=None, ws: OpWorkspace | None = None,
                   stream=None):
    """y[r] = W[e] x[r] for the rows offsets[e] <= r < offsets[e + 1] of every
    group e; rows outside all groups are zero.

    x [rows, K] and w [E, N, K] are BF16 or F16 (w contiguous along N or K, so
    ``w.transpose(1, 2)`` of a [E, K, N] tensor is read in place), offsets
    int32 [E + 1].  y [rows, N] has x's type or FP32."""
    d, off, y, ws = _grouped_rows(x, "x", w, offsets, out, out_dtype, ws, False)
    with torch.cuda.device(x.device):
        _check(lib().beam_moe_grouped_matmul(ctypes.byref(d), x.data_ptr(), w.data_ptr(), off,
                                             y.data_ptr(), ws.ptr, ws.nbytes, _stream(stream)),
               "beam_moe_grouped_matmul")
    return y


def grouped_matmul_dx(dy, w, offsets, out=None, out_dtype=None, ws: OpWorkspace | None = None,
                      stream=None):
    """The input gradient of ``grouped_matmul``: dx[r] = W[e]^T dy[r]."""
    d, off, dx, ws = _grouped_rows(dy, "dy", w, offsets, out, out_dtype, ws, True)
    with torch.cuda.device(dy.device):
        _check(lib().beam_moe_grouped_matmul_dx(ctypes.byref(d), dy.data_ptr(), w.data_ptr(), off,
                                                dx.data_ptr(), ws.ptr, ws.nbytes,
                                                _stream(stream)), "beam_moe_grouped_matmul_dx")
    return dx


def grouped_matmul_dw(dy, x, offsets, out=None, accumulate: bool = False, out_dtype=None,
                      ws: OpWorkspace | None = None, stream=None):
    """The weight gradient of ``grouped_matmul``: dW[e] = sum over the rows of
    group e of dy[r] x[r]^T, [E, N, K] in the operands' type or FP32; zero for
    a group without rows.  ``accumulate`` adds to ``out`` (FP32)."""
    y_ld = _rows2d(dy, "dy")
    x_ld = _rows2d(x, "x", dy.dtype)
    if x.shape[0] != dy.shape[0]:
        raise ValueError(f"x and dy must have the same rows, got {x.shape[0]} and {dy.shape[0]}")
    _same_device(dy, x=x, offsets=offsets, out=out)
    off = _offsets(offsets)
    E, N, K = offsets.numel() - 1, dy.shape[1], x.shape[1]
    dt = out_dtype if out_dtype is not None else out.dtype if out is not None else dy.dtype
    if accumulate and (out is None or dt != torch.float32):
        raise ValueError("accumulate needs an FP32 out to add to")
    d = _grouped_desc(x.shape[0], E, N, K, dy.dtype, dt, x_ld, y_ld, (N * K, K, 1))
    if out is None:
        out = torch.empty(E, N, K, dtype=dt, device=dy.device)
    if tuple(out.shape) != (E, N, K):
        raise ValueError(f"out must be {(E, N, K)}, got {tuple(out.shape)}")
    dst = _dev(out, dt, "out")
    if ws is None:
        # W takes no part: describe one that needs no copy
        d.w_stride_n, d.w_stride_e = (K + 7) // 8 * 8, (K + 7) // 8 * 8 * N
    ws = _grouped_ws(ws, d, dy.device, dy, x)
    with torch.cuda.device(dy.device):
        _check(lib().beam_moe_grouped_matmul_dw(ctypes.byref(d), dy.data_ptr(), x.data_ptr(), off,
                                                int(accumulate), dst, ws.ptr, ws.nbytes,
                                                _stream(stream)), "beam_moe_grouped_matmul_dw")
    return out


def _row_weight(row_weight, rows: int):
    if row_weight is None:
        return None
    ptr = _dev(row_weight, torch.float32, "row_weight")
    if tuple(row_weight.shape) != (rows,):
        raise ValueError(f"row_weight must be [{rows}], got {tuple(row_weight.shape)}")
    return ptr


def _gate_desc(gate, up):
    g_ld = _rows2d(gate, "gate")
    u_ld = _rows2d(up, "up", gate.dtype, gate.shape[1])
    if up.shape[0] != gate.shape[0]:
        raise ValueError(f"gate and up must have the same rows, got {gate.shape[0]} "
                         f"and {up.shape[0]}")
    return _Gate(gate.shape[0], gate.shape[1], _type(gate.dtype, "gate", _HALVES), g_ld, u_ld)


def _like(out, like, name):
    if out is None:
        out = torch.empty(like.shape, dtype=like.dtype, device=like.device)
    ld = _rows2d(out, name, like.dtype, like.shape[1])
    if out.shape[0] != like.shape[0]:
        raise ValueError(f"{name} must have {like.shape[0]} rows, got {out.shape[0]}")
    _same_device(like, **{name: out})
    return out, ld


def swiglu(gate, up, row_weight=None, out=None, stream=None):
    """h = row_weight[r] * silu(gate) * up (BF16 or F16 [rows, F], row strides
    free; FP32 inside, rounded once).  Without row_weight the factor is 1."""
    d = _gate_desc(gate, up)
    _same_device(gate, up=up, row_weight=row_weight)
    h, h_ld = _like(out, gate, "out")
    w = _row_weight(row_weight, gate.shape[0])
    with torch.cuda.device(gate.device):
        _check(lib().beam_moe_swiglu(ctypes.byref(d), gate.data_ptr(), up.data_ptr(), w,
                                     h.data_ptr(), h_ld, _stream(stream)), "beam_moe_swiglu")
    return h


def swiglu_grad(dh, gate, up, row_weight=None, out=None, stream=None):
    """The gradient of ``swiglu``: (dgate, dup) and, with row_weight, its own
    gradient (FP32 [rows]).  ``out``: (dgate, dup) to write to; they may be
    gate and up themselves."""
    d = _gate_desc(gate, up)
    dh_ld = _rows2d(dh, "dh", gate.dtype, gate.shape[1])
    if dh.shape[0] != gate.shape[0]:
        raise ValueError(f"dh must have {gate.shape[0]} rows, got {dh.shape[0]}")
    _same_device(gate, up=up, dh=dh, row_weight=row_weight)
    dg, dg_ld = _like(None if out is None else out[0], gate, "dgate")
    du, du_ld = _like(None if out is None else out[1], gate, "dup")
    w = _row_weight(row_weight, gate.shape[0])
    dw = None if w is None else torch.empty(gate.shape[0], dtype=torch.float32, device=gate.device)
    with torch.cuda.device(gate.device):
        _check(lib().beam_moe_swiglu_grad(ctypes.byref(d), dh.data_ptr(), dh_ld, gate.data_ptr(),
                                          up.data_ptr(), w, dg.data_ptr(), dg_ld, du.data_ptr(),
                                          du_ld, None if dw is None else dw.data_ptr(),
                                          _stream(stream)), "beam_moe_swiglu_grad")
    return (dg, du) if dw is None else (dg, du, dw)


def orthogonalize_workspace_size(batch: int, rows: int, cols: int, dtype=torch.float32) -> int:
    """Workspace bytes of ``orthogonalize`` (FP32 input needs the most)."""
    n = lib().beam_moe_orthogonalize_workspace_size(
        batch, rows, cols, _type(dtype, "m", _HALVES + (torch.float32,)))
    if n == 0:
        raise BeamError(1, "beam_moe_orthogonalize_workspace_size")
    return int(n)


def orthogonalize(m, steps: int = 5, coeffs=(3.4445, -4.7750, 2.0315), eps: float = 1e-7,
                  out=None, out_dtype=None, ws: OpWorkspace | None = None, stream=None):
    """The update m [..., R, C] orthogonalised matrix by matrix: X = M / (|M|_F
    + eps), then ``steps`` times X <- a X + (b A + c A^2) X with A = X X^T (the
    Muon optimiser's Newton-Schulz products).

    m is BF16, F16 or FP32 with any strides; the result is BF16 or F16
    (``out_dtype``; m's own 16-bit type, BF16 for FP32) and accurate to about
    2e-3 of its norm."""
    if not isinstance(m, torch.Tensor) or not m.is_cuda:
        raise TypeError("m must be a CUDA tensor")
    if m.dim() < 2:
        raise ValueError(f"m must be a matrix or a stack of them, got shape {tuple(m.shape)}")
    kind = _type(m.dtype, "m", _HALVES + (torch.float32,))
    dt = out_dtype if out_dtype is not None else out.dtype if out is not None else \
        m.dtype if m.dtype in _HALVES else torch.bfloat16
    out_kind = _type(dt, "out_dtype", _HALVES)
    R, C = m.shape[-2:]
    stack = m if m.dim() == 3 else m.reshape(-1, R, C) if m.numel() else m.new_empty(0, R, C)
    batch = stack.shape[0]
    if out is None:
        out = torch.empty(m.shape, dtype=dt, device=m.device)
    if out.shape != m.shape:
        raise ValueError(f"out must be {tuple(m.shape)}, got {tuple(out.shape)}")
    _same_device(m, out=out)
    dst = _dev(out, dt, "out")
    if m.numel() == 0:
        return out
    d = _Ortho(batch, R, C, kind, out_kind, int(steps), *(float(v) for v in coeffs), float(eps),
               *stack.stride())
    ws = _op_ws(ws, m.device, lambda: orthogonalize_workspace_size(batch, R, C, m.dtype))
    with torch.cuda.device(m.device):
        _check(lib().beam_moe_orthogonalize(ctypes.byref(d), stack.data_ptr(), dst, ws.ptr,
                                            ws.nbytes, _stream(stream)), "beam_moe_orthogonalize")
    return out
