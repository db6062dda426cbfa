"""Thin Python binding of libmoe_gb300 (the C ABI declared in include/moe.h).

Argument marshalling only: every step of the MoE layer runs in the library's CUDA
kernels.  PyTorch supplies device memory (tensors), streams and the current device.
Functions take torch CUDA tensors (or raw device addresses as ints, or None for NULL)
and raise ``MoEError`` when the library returns a status other than MOE_OK.

There is no fallback: if the shared library has not been built, or cannot be
loaded, every call raises.
"""

from __future__ import annotations

import ctypes
import os
from typing import Optional

__all__ = [
    "MoEConfig", "MoEError", "F32", "BF16", "FLAG_FUSED_COMBINE", "FLAG_CAPACITY", "FLAG_FP8", "library_path", "load", "workspace_size",
    "route", "permute", "permute_noalloc", "grouped_ffn", "expert_gate_up", "expert_gate_up_gather", "quantize_fp8", "expert_gate_up_fp8", "expert_down_fp8", "layer_forward_fp8", "expert_down", "combine", "layer_forward", "workspace_views",
    "RouteConfig", "SCORE_SOFTMAX", "SCORE_SIGMOID", "route_scored", "route_scored_backward",
    "combine_backward", "LinearConfig", "ACT_NONE", "ACT_RELU", "ACT_GELU", "ACT_GELU_TANH",
    "ACT_SILU", "linear_workspace_size", "linear", "linear_backward",
    "GroupedConfig", "ACT_SWIGLU", "grouped_linear_workspace_size", "grouped_linear",
    "grouped_linear_backward", "BlockNormConfig", "GATE_NONE", "GATE_VALUE", "GATE_LOGISTIC",
    "block_norm_workspace_size", "block_norm", "block_norm_backward",
    "GradList", "clip_grad_norm_workspace_size", "clip_grad_norm",
    "sync_check", "debug_wait_timeout", "status_string", "version",
]

F32 = 0
BF16 = 1
# moe_config_t.flags: fuse the combine into the down projection (bf16 layers; y is then
# correct to fp32 rounding but not bitwise reproducible run to run)
FLAG_FUSED_COMBINE = 1
FLAG_CAPACITY = 2
FLAG_FP8 = 4
# moe_route_config_t.score
SCORE_SOFTMAX = 0
SCORE_SIGMOID = 1
# moe_linear_config_t.activation
ACT_NONE = 0
ACT_RELU = 1
ACT_GELU = 2
ACT_GELU_TANH = 3
ACT_SILU = 4
ACT_SWIGLU = 5  # grouped_linear only
# moe_block_norm_config_t.gate
GATE_NONE = 0
GATE_VALUE = 1
GATE_LOGISTIC = 2

_STATUS = {
    0: "MOE_OK", 1: "MOE_ERR_INVALID_ARG", 2: "MOE_ERR_UNSUPPORTED", 3: "MOE_ERR_WORKSPACE",
    4: "MOE_ERR_CUDA", 5: "MOE_ERR_TIMEOUT", 6: "MOE_ERR_INTERNAL", 7: "MOE_ERR_MISALIGNED",
}


class MoEError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {_STATUS.get(status, status)}")


class MoEConfig(ctypes.Structure):
    """moe_config_t: T, H, E, K, I, I_shared, gate_threshold, dtype, flags."""

    _fields_ = [
        ("T", ctypes.c_int32), ("H", ctypes.c_int32), ("E", ctypes.c_int32),
        ("K", ctypes.c_int32), ("I", ctypes.c_int32), ("I_shared", ctypes.c_int32),
        ("gate_threshold", ctypes.c_float), ("dtype", ctypes.c_int32), ("flags", ctypes.c_uint32),
    ]

    @classmethod
    def make(cls, T, H, E, K, I, I_shared=0, gate_threshold=0.0, dtype=BF16, flags=0):
        return cls(T, H, E, K, I, I_shared, gate_threshold, dtype, flags)

    def __repr__(self):
        return (f"MoEConfig(T={self.T}, H={self.H}, E={self.E}, K={self.K}, I={self.I}, "
                f"I_shared={self.I_shared}, theta={self.gate_threshold}, dtype={self.dtype})")


class RouteConfig(ctypes.Structure):
    """moe_route_config_t: T, E, K, groups, top_groups, group_rank, score, renormalise, scale,
    dtype, logits_stride (0 = E)."""

    _fields_ = [
        ("T", ctypes.c_int32), ("E", ctypes.c_int32), ("K", ctypes.c_int32),
        ("groups", ctypes.c_int32), ("top_groups", ctypes.c_int32),
        ("group_rank", ctypes.c_int32), ("score", ctypes.c_int32),
        ("renormalise", ctypes.c_int32), ("scale", ctypes.c_float), ("dtype", ctypes.c_int32),
        ("logits_stride", ctypes.c_int64),
    ]

    @classmethod
    def make(cls, T, E, K, groups=1, top_groups=1, group_rank=1, score=SCORE_SOFTMAX,
             renormalise=True, scale=1.0, dtype=F32, logits_stride=0):
        return cls(T, E, K, groups, top_groups, group_rank, score, int(renormalise), scale, dtype,
                   logits_stride)

    def __repr__(self):
        return (f"RouteConfig(T={self.T}, E={self.E}, K={self.K}, groups={self.groups}, "
                f"top_groups={self.top_groups}, group_rank={self.group_rank}, "
                f"score={self.score}, renormalise={self.renormalise}, scale={self.scale}, "
                f"dtype={self.dtype})")


class LinearConfig(ctypes.Structure):
    """moe_linear_config_t: rows, in_features, out_features, dtype, out_dtype, activation and
    the row strides in elements (0 = contiguous)."""

    _fields_ = [
        ("rows", ctypes.c_int32), ("in_features", ctypes.c_int32),
        ("out_features", ctypes.c_int32), ("dtype", ctypes.c_int32),
        ("out_dtype", ctypes.c_int32), ("activation", ctypes.c_int32),
        ("x_stride", ctypes.c_int64), ("w_stride", ctypes.c_int64),
        ("residual_stride", ctypes.c_int64), ("y_stride", ctypes.c_int64),
        ("z_stride", ctypes.c_int64), ("dx_stride", ctypes.c_int64),
        ("dw_stride", ctypes.c_int64),
    ]

    @classmethod
    def make(cls, rows, in_features, out_features, dtype=BF16, out_dtype=None,
             activation=ACT_NONE, x_stride=0, w_stride=0, residual_stride=0, y_stride=0,
             z_stride=0, dx_stride=0, dw_stride=0):
        return cls(rows, in_features, out_features, dtype,
                   dtype if out_dtype is None else out_dtype, activation, x_stride, w_stride,
                   residual_stride, y_stride, z_stride, dx_stride, dw_stride)

    def __repr__(self):
        return (f"LinearConfig(rows={self.rows}, in_features={self.in_features}, "
                f"out_features={self.out_features}, dtype={self.dtype}, "
                f"out_dtype={self.out_dtype}, activation={self.activation})")


class GroupedConfig(ctypes.Structure):
    """moe_grouped_config_t: rows, groups, in_features, out_features, dtype, out_dtype, dx_dtype,
    activation and the row strides in elements (0 = contiguous)."""

    _fields_ = [
        ("rows", ctypes.c_int32), ("groups", ctypes.c_int32), ("in_features", ctypes.c_int32),
        ("out_features", ctypes.c_int32), ("dtype", ctypes.c_int32),
        ("out_dtype", ctypes.c_int32), ("dx_dtype", ctypes.c_int32),
        ("activation", ctypes.c_int32), ("x_stride", ctypes.c_int64),
        ("w_stride", ctypes.c_int64), ("y_stride", ctypes.c_int64), ("z_stride", ctypes.c_int64),
        ("dx_stride", ctypes.c_int64), ("dw_stride", ctypes.c_int64),
    ]

    @classmethod
    def make(cls, rows, groups, in_features, out_features, dtype=BF16, out_dtype=None,
             dx_dtype=None, activation=ACT_NONE, x_stride=0, w_stride=0, y_stride=0, z_stride=0,
             dx_stride=0, dw_stride=0):
        return cls(rows, groups, in_features, out_features, dtype,
                   dtype if out_dtype is None else out_dtype,
                   dtype if dx_dtype is None else dx_dtype, activation, x_stride, w_stride,
                   y_stride, z_stride, dx_stride, dw_stride)

    def __repr__(self):
        return (f"GroupedConfig(rows={self.rows}, groups={self.groups}, "
                f"in_features={self.in_features}, out_features={self.out_features}, "
                f"dtype={self.dtype}, out_dtype={self.out_dtype}, dx_dtype={self.dx_dtype}, "
                f"activation={self.activation})")


class BlockNormConfig(ctypes.Structure):
    """moe_block_norm_config_t: rows, width, dtype, gate, eps, residual_scale, branch_scale and the
    row strides in elements (0 = contiguous)."""

    _fields_ = [
        ("rows", ctypes.c_int32), ("width", ctypes.c_int32), ("dtype", ctypes.c_int32),
        ("gate", ctypes.c_int32), ("eps", ctypes.c_float), ("residual_scale", ctypes.c_float),
        ("branch_scale", ctypes.c_float), ("x_stride", ctypes.c_int64),
        ("residual_stride", ctypes.c_int64), ("sum_stride", ctypes.c_int64),
        ("y_stride", ctypes.c_int64), ("dx_stride", ctypes.c_int64),
        ("dresidual_stride", ctypes.c_int64),
    ]

    @classmethod
    def make(cls, rows, width, dtype=BF16, eps=1e-6, residual_scale=1.0, branch_scale=1.0,
             gate=GATE_NONE, x_stride=0, residual_stride=0, sum_stride=0, y_stride=0, dx_stride=0,
             dresidual_stride=0):
        return cls(rows, width, dtype, gate, eps, residual_scale, branch_scale, x_stride,
                   residual_stride, sum_stride, y_stride, dx_stride, dresidual_stride)

    def __repr__(self):
        return (f"BlockNormConfig(rows={self.rows}, width={self.width}, dtype={self.dtype}, "
                f"gate={self.gate}, eps={self.eps}, residual_scale={self.residual_scale}, "
                f"branch_scale={self.branch_scale})")


class _Grad(ctypes.Structure):
    """moe_grad_t."""

    _fields_ = [("grad", ctypes.c_void_p), ("out", ctypes.c_void_p), ("size", ctypes.c_int64),
                ("dtype", ctypes.c_int32), ("out_dtype", ctypes.c_int32)]


class GradList:
    """The tensors of clip_grad_norm, contiguous bf16 or float32 on one GPU; outs: as many tensors of
    the same sizes (the gradients themselves to clip in place), or None for the norm alone.  Holds
    the tensors, whose storage it names.  Results that overlap one another, or another tensor's
    gradient, are refused: they would be scaled in no fixed order.

    Making a list asks every tensor a dozen questions: some 8 us each on the host, 1.2 ms for 150,
    where clipping them takes 0.6 ms of the GPU.  So make it once, over gradients that stay where
    they are (kept and zeroed, not set to None, between the steps), and pass it every step."""

    def __init__(self, grads, outs=None):
        self.grads = list(grads)
        self.outs = None if outs is None else list(outs)
        if self.outs is not None and len(self.outs) != len(self.grads):
            raise ValueError("as many results as gradients")
        self.array = (_Grad * max(1, len(self.grads)))()
        for i, g in enumerate(self.grads):
            o = None if self.outs is None else self.outs[i]
            for t in (g, o):
                if t is not None and not t.is_contiguous():
                    raise ValueError("gradients and results must be contiguous")
            if o is not None and o.numel() != g.numel():
                raise ValueError("a result of another size than its gradient")
            # (tensors without elements have no place: their addresses are all 0)
            if (o is not None and g.numel() > 0 and o.data_ptr() == g.data_ptr()
                    and o.dtype != g.dtype):
                raise ValueError("a result in its gradient's place but of another type")
            self.array[i] = _Grad(g.data_ptr(), None if o is None else o.data_ptr(), g.numel(),
                                  _dtype_of(g), _dtype_of(g if o is None else o))
            for t in (g, o):
                if t is not None and not t.is_cuda:
                    raise ValueError("gradients and results must be on the GPU")
                if t is not None and t.device != self.grads[0].device:
                    raise ValueError("gradients and results must be on one GPU")
        self._refuse_overlaps()

    def _refuse_overlaps(self):
        spans = []  # (first byte, end, written)
        for g, o in zip(self.grads, self.outs or []):
            in_place = o is not None and o.data_ptr() == g.data_ptr()
            for t, written in ((None if in_place else g, False), (o, True)):
                if t is not None and t.numel() > 0:
                    at = t.data_ptr()
                    spans.append((at, at + t.numel() * t.element_size(), written))
        any_end = written_end = 0  # of the spans that start before
        for at, end, written in sorted(spans):
            if at < (any_end if written else written_end):
                raise ValueError("a result overlaps another tensor of the list")
            any_end = max(any_end, end)
            if written:
                written_end = max(written_end, end)

    def __len__(self):
        return len(self.grads)


def _dtype_of(t) -> int:
    name = str(t.dtype)
    if name == "torch.bfloat16":
        return BF16
    if name == "torch.float32":
        return F32
    raise ValueError(f"bfloat16 or float32, not {name}")


def library_path(debug: bool = False) -> str:
    """The release library, or with ``debug`` the bounds-checking build (-DMOE_DEBUG)."""
    return os.path.join(os.path.dirname(os.path.abspath(__file__)),
                        "_build_debug" if debug else "_build", "libmoe_gb300.so")


_LIB: Optional[ctypes.CDLL] = None

_P = ctypes.c_void_p
_CFG = ctypes.POINTER(MoEConfig)
_RCFG = ctypes.POINTER(RouteConfig)
_LCFG = ctypes.POINTER(LinearConfig)
_GCFG = ctypes.POINTER(GroupedConfig)
_NCFG = ctypes.POINTER(BlockNormConfig)
_SIGS = {
    "moe_workspace_size": [_CFG, ctypes.POINTER(ctypes.c_size_t)],
    "moe_route": [_CFG, _P, _P, _P, _P, _P, _P, _P],
    "moe_permute": [_CFG, _P, _P, _P, _P, _P, _P, _P, _P, ctypes.c_size_t, _P],
    "moe_permute_noalloc": [_CFG, _P, _P, _P, _P, _P, _P, _P, _P],
    "moe_grouped_ffn": [_CFG, _P, _P, _P, _P, _P, _P, ctypes.c_size_t, _P],
    "moe_expert_gate_up": [_CFG, _P, _P, _P, _P, _P, ctypes.c_size_t, _P],
    "moe_expert_gate_up_gather": [_CFG, _P, _P, _P, _P, _P, _P, ctypes.c_size_t, _P],
    "moe_quantize_fp8": [_P, ctypes.c_int64, ctypes.c_int32, _P, _P, _P],
    "moe_expert_gate_up_fp8": [_CFG, _P, _P, _P, _P, _P, _P, _P, ctypes.c_size_t, _P],
    "moe_expert_down_fp8": [_CFG, _P, _P, _P, _P, _P, _P, _P, ctypes.c_size_t, _P],
    "moe_layer_forward_fp8": [_CFG, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P,
                              ctypes.c_size_t, _P],
    "moe_expert_down": [_CFG, _P, _P, _P, _P, _P, ctypes.c_size_t, _P],
    "moe_combine": [_CFG, _P, _P, _P, _P, _P, _P, _P],
    "moe_layer_forward": [_CFG, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, ctypes.c_size_t, _P],
    "moe_workspace_views": [_CFG, _P] + [ctypes.POINTER(_P)] * 10,
    "moe_route_scored": [_RCFG, _P, _P, _P, _P, _P],
    "moe_route_scored_backward": [_RCFG, _P, _P, _P, _P, _P],
    "moe_combine_backward": [_CFG, _P, _P, _P, _P, _P, _P, _P],
    "moe_linear_workspace_size": [_LCFG, ctypes.POINTER(ctypes.c_size_t)],
    "moe_linear": [_LCFG, _P, _P, _P, _P, _P, _P, _P, ctypes.c_size_t, _P],
    "moe_linear_backward": [_LCFG, _P, _P, _P, _P, _P, _P, _P, _P, ctypes.c_size_t, _P],
    "moe_grouped_linear_workspace_size": [_GCFG, ctypes.POINTER(ctypes.c_size_t)],
    "moe_grouped_linear": [_GCFG, _P, _P, _P, _P, _P, _P, ctypes.c_size_t, _P],
    "moe_grouped_linear_backward": [_GCFG, _P, _P, _P, _P, _P, _P, _P, _P, ctypes.c_size_t, _P],
    "moe_block_norm_workspace_size": [_NCFG, ctypes.POINTER(ctypes.c_size_t)],
    "moe_block_norm": [_NCFG] + [_P] * 9,
    "moe_block_norm_backward": [_NCFG] + [_P] * 15 + [ctypes.c_size_t, _P],
    "moe_clip_grad_norm_workspace_size": [ctypes.c_int, ctypes.POINTER(ctypes.c_size_t)],
    "moe_clip_grad_norm": [_P, ctypes.c_int, ctypes.c_float, ctypes.c_float, ctypes.c_float, _P,
                           _P, ctypes.c_size_t, _P],
    "moe_sync_check": [_P],
    "moe_debug_wait_timeout": [ctypes.c_uint, _P, _P],
    "moe_status_string": [ctypes.c_int],
    "moe_version": [],
    "moe_kernel_launch_count": [],
    "moe_debug_set_fault": [ctypes.c_char_p, ctypes.c_int],
}


def load(path: Optional[str] = None) -> ctypes.CDLL:
    """Load libmoe_gb300.so (built by ``build.py``); raises if it is missing."""
    global _LIB
    if _LIB is not None:
        return _LIB
    path = path or library_path()
    if not os.path.exists(path):
        raise RuntimeError(f"libmoe_gb300.so not built ({path}); run "
                           "`python -c 'import __graft_entry__ as g; g.build()'` first")
    _LIB = _open(path)
    return _LIB


def _open(path: str) -> ctypes.CDLL:
    lib = ctypes.CDLL(path)
    for name, args in _SIGS.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = (ctypes.c_char_p if name in ("moe_status_string", "moe_version") else
                      ctypes.c_ulonglong if name == "moe_kernel_launch_count" else ctypes.c_int)
    return lib


def load_debug() -> ctypes.CDLL:
    """A handle on the bounds-checking build (``build.build(debug=True)``), separate from
    the release library that ``load()`` returns; raises if it is not built."""
    path = library_path(debug=True)
    if not os.path.exists(path):
        raise RuntimeError(f"debug build of libmoe_gb300.so missing ({path})")
    return _open(path)


def _ptr(t) -> Optional[int]:
    return t if t is None or isinstance(t, int) else t.data_ptr()


def _stream(stream) -> Optional[int]:
    if stream is None:
        import torch
        try:
            # the raw handle of torch's current stream: building a torch.cuda.Stream for it takes
            # 3 us, as long as a small call's launch
            return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
        except AttributeError:  # the names are not public: a torch that has them no longer
            return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(status: int, where: str):
    if status != 0:
        raise MoEError(status, where)


def status_string(status: int) -> str:
    return load().moe_status_string(status).decode()


def version() -> str:
    return load().moe_version().decode()


def kernel_launch_count() -> int:
    """Kernels the library has launched in this process (moe_kernel_launch_count)."""
    return int(load().moe_kernel_launch_count())


def debug_set_fault(point: Optional[str], n: int = 1) -> None:
    """Arm (or with point None, disarm) the host-side fault injector: the n-th pass through
    `point` returns MOE_ERR_CUDA (moe_debug_set_fault)."""
    _check(load().moe_debug_set_fault(point.encode() if point else None, int(n)),
           "moe_debug_set_fault")


def workspace_size(cfg: MoEConfig) -> int:
    n = ctypes.c_size_t(0)
    _check(load().moe_workspace_size(ctypes.byref(cfg), ctypes.byref(n)), "moe_workspace_size")
    return n.value


def route(cfg, x, w_router, router_bias, logits, topk_ids, topk_w, stream=None):
    _check(load().moe_route(ctypes.byref(cfg), _ptr(x), _ptr(w_router), _ptr(router_bias),
                            _ptr(logits), _ptr(topk_ids), _ptr(topk_w), _stream(stream)),
           "moe_route")


def permute(cfg, x, topk_ids, counts, offsets, perm, inv, x_perm, ws, ws_bytes=None, stream=None):
    nb = ws.numel() * ws.element_size() if ws_bytes is None else ws_bytes
    _check(load().moe_permute(ctypes.byref(cfg), _ptr(x), _ptr(topk_ids), _ptr(counts),
                              _ptr(offsets), _ptr(perm), _ptr(inv), _ptr(x_perm), _ptr(ws), nb,
                              _stream(stream)), "moe_permute")


def permute_noalloc(cfg, x, topk_ids, counts, offsets, perm, inv, x_perm, stream=None):
    """moe_permute for callers that cannot allocate: no workspace; the library's fixed
    scratch array is used instead (shared by all calls on a device, so overlapping calls
    must be serialised by the caller)."""
    _check(load().moe_permute_noalloc(ctypes.byref(cfg), _ptr(x), _ptr(topk_ids), _ptr(counts),
                                      _ptr(offsets), _ptr(perm), _ptr(inv), _ptr(x_perm),
                                      _stream(stream)), "moe_permute_noalloc")


def grouped_ffn(cfg, x_perm, offsets, w_gate_up, w_down, out_perm, ws, ws_bytes=None, stream=None):
    nb = ws.numel() * ws.element_size() if ws_bytes is None else ws_bytes
    _check(load().moe_grouped_ffn(ctypes.byref(cfg), _ptr(x_perm), _ptr(offsets), _ptr(w_gate_up),
                                  _ptr(w_down), _ptr(out_perm), _ptr(ws), nb, _stream(stream)),
           "moe_grouped_ffn")


def expert_gate_up(cfg, x_perm, offsets, w_gate_up, h, ws, ws_bytes=None, stream=None):
    nb = ws.numel() * ws.element_size() if ws_bytes is None else ws_bytes
    _check(load().moe_expert_gate_up(ctypes.byref(cfg), _ptr(x_perm), _ptr(offsets),
                                     _ptr(w_gate_up), _ptr(h), _ptr(ws), nb, _stream(stream)),
           "moe_expert_gate_up")


def expert_gate_up_gather(cfg, x, perm, offsets, w_gate_up, h, ws, ws_bytes=None, stream=None):
    nb = ws.numel() * ws.element_size() if ws_bytes is None else ws_bytes
    _check(load().moe_expert_gate_up_gather(ctypes.byref(cfg), _ptr(x), _ptr(perm), _ptr(offsets),
                                            _ptr(w_gate_up), _ptr(h), _ptr(ws), nb,
                                            _stream(stream)),
           "moe_expert_gate_up_gather")


def quantize_fp8(x, codes, scales, stream=None):
    """Per-row E4M3 codes and float32 scales of a bf16 [rows, cols] tensor."""
    rows, cols = x.shape[0], x.numel() // max(1, x.shape[0])
    _check(load().moe_quantize_fp8(_ptr(x), rows, cols, _ptr(codes), _ptr(scales), _stream(stream)),
           "moe_quantize_fp8")


def expert_gate_up_fp8(cfg, x_codes, x_scales, offsets, w_codes, w_scales, h, ws, ws_bytes=None,
                       stream=None):
    nb = ws.numel() * ws.element_size() if ws_bytes is None else ws_bytes
    _check(load().moe_expert_gate_up_fp8(ctypes.byref(cfg), _ptr(x_codes), _ptr(x_scales),
                                         _ptr(offsets), _ptr(w_codes), _ptr(w_scales), _ptr(h),
                                         _ptr(ws), nb, _stream(stream)),
           "moe_expert_gate_up_fp8")


def expert_down_fp8(cfg, h_codes, h_scales, offsets, w_codes, w_scales, out_perm, ws,
                    ws_bytes=None, stream=None):
    nb = ws.numel() * ws.element_size() if ws_bytes is None else ws_bytes
    _check(load().moe_expert_down_fp8(ctypes.byref(cfg), _ptr(h_codes), _ptr(h_scales),
                                      _ptr(offsets), _ptr(w_codes), _ptr(w_scales),
                                      _ptr(out_perm), _ptr(ws), nb, _stream(stream)),
           "moe_expert_down_fp8")


def layer_forward_fp8(cfg, x, w_router, router_bias, w_gate_up_codes, w_gate_up_scales,
                      w_down_codes, w_down_scales, w_shared_gate_up, w_shared_down, y, y_f32, ws,
                      ws_bytes=None, stream=None):
    nb = ws.numel() * ws.element_size() if ws_bytes is None else ws_bytes
    _check(load().moe_layer_forward_fp8(
        ctypes.byref(cfg), _ptr(x), _ptr(w_router), _ptr(router_bias), _ptr(w_gate_up_codes),
        _ptr(w_gate_up_scales), _ptr(w_down_codes), _ptr(w_down_scales), _ptr(w_shared_gate_up),
        _ptr(w_shared_down), _ptr(y), _ptr(y_f32), _ptr(ws), nb, _stream(stream)),
        "moe_layer_forward_fp8")


def expert_down(cfg, h, offsets, w_down, out_perm, ws, ws_bytes=None, stream=None):
    nb = ws.numel() * ws.element_size() if ws_bytes is None else ws_bytes
    _check(load().moe_expert_down(ctypes.byref(cfg), _ptr(h), _ptr(offsets), _ptr(w_down),
                                  _ptr(out_perm), _ptr(ws), nb, _stream(stream)),
           "moe_expert_down")


def combine(cfg, out_perm, inv, topk_w, shared_out, y, y_f32=None, stream=None):
    _check(load().moe_combine(ctypes.byref(cfg), _ptr(out_perm), _ptr(inv), _ptr(topk_w),
                              _ptr(shared_out), _ptr(y), _ptr(y_f32), _stream(stream)),
           "moe_combine")


def layer_forward(cfg, x, w_router, router_bias, w_gate_up, w_down, w_shared_gate_up,
                  w_shared_down, y, y_f32, ws, ws_bytes=None, stream=None):
    nb = ws.numel() * ws.element_size() if ws_bytes is None else ws_bytes
    _check(load().moe_layer_forward(ctypes.byref(cfg), _ptr(x), _ptr(w_router), _ptr(router_bias),
                                    _ptr(w_gate_up), _ptr(w_down), _ptr(w_shared_gate_up),
                                    _ptr(w_shared_down), _ptr(y), _ptr(y_f32), _ptr(ws), nb,
                                    _stream(stream)), "moe_layer_forward")


def route_scored(cfg, logits, expert_bias, topk_ids, topk_w, stream=None):
    """Expert ids and weights from scores (softmax or sigmoid, balance bias, groups)."""
    _check(load().moe_route_scored(ctypes.byref(cfg), _ptr(logits), _ptr(expert_bias),
                                   _ptr(topk_ids), _ptr(topk_w), _stream(stream)),
           "moe_route_scored")


def route_scored_backward(cfg, logits, topk_ids, d_topk_w, d_logits, stream=None):
    """d_logits from the gradient of route_scored's weights."""
    _check(load().moe_route_scored_backward(ctypes.byref(cfg), _ptr(logits), _ptr(topk_ids),
                                            _ptr(d_topk_w), _ptr(d_logits), _stream(stream)),
           "moe_route_scored_backward")


def combine_backward(cfg, dy, out_perm, inv, topk_w, d_out_perm, d_topk_w, stream=None):
    """Gradients of combine: the expert rows' (or None) and the route weights' (or None)."""
    _check(load().moe_combine_backward(ctypes.byref(cfg), _ptr(dy), _ptr(out_perm), _ptr(inv),
                                       _ptr(topk_w), _ptr(d_out_perm), _ptr(d_topk_w),
                                       _stream(stream)), "moe_combine_backward")


def linear_workspace_size(cfg: LinearConfig) -> int:
    n = ctypes.c_size_t(0)
    _check(load().moe_linear_workspace_size(ctypes.byref(cfg), ctypes.byref(n)),
           "moe_linear_workspace_size")
    return n.value


def _ws(ws, ws_bytes):
    if ws_bytes is not None:
        return ws_bytes
    return 0 if ws is None else ws.numel() * ws.element_size()


def linear(cfg, x, w, bias, residual, y, z=None, ws=None, ws_bytes=None, stream=None):
    """y = act(x w^T + bias) + residual; z (optional) receives the value before act."""
    _check(load().moe_linear(ctypes.byref(cfg), _ptr(x), _ptr(w), _ptr(bias), _ptr(residual),
                             _ptr(y), _ptr(z), _ptr(ws), _ws(ws, ws_bytes), _stream(stream)),
           "moe_linear")


def linear_backward(cfg, dy, x, w, z, dx, dw, dbias, ws=None, ws_bytes=None, stream=None):
    """dx, dw and dbias (each may be None) of linear; z is what linear stored."""
    _check(load().moe_linear_backward(ctypes.byref(cfg), _ptr(dy), _ptr(x), _ptr(w), _ptr(z),
                                      _ptr(dx), _ptr(dw), _ptr(dbias), _ptr(ws),
                                      _ws(ws, ws_bytes), _stream(stream)),
           "moe_linear_backward")


def grouped_linear_workspace_size(cfg: GroupedConfig) -> int:
    n = ctypes.c_size_t(0)
    _check(load().moe_grouped_linear_workspace_size(ctypes.byref(cfg), ctypes.byref(n)),
           "moe_grouped_linear_workspace_size")
    return n.value


def grouped_linear(cfg, x, offsets, w, y, z=None, ws=None, ws_bytes=None, stream=None):
    """y_r = x_r w_g^T for the rows of every group g, or silu(gate) * up of it (ACT_SWIGLU; z
    optionally receives the value before the activation)."""
    _check(load().moe_grouped_linear(ctypes.byref(cfg), _ptr(x), _ptr(offsets), _ptr(w), _ptr(y),
                                     _ptr(z), _ptr(ws), _ws(ws, ws_bytes), _stream(stream)),
           "moe_grouped_linear")


def grouped_linear_backward(cfg, dy, x, offsets, w, z, dx, dw, ws=None, ws_bytes=None,
                            stream=None):
    """dx and dw (each may be None) of grouped_linear; z is what grouped_linear stored.  With
    dx_dtype=F32 a bf16 ACT_SWIGLU layer keeps 24 bits of dz for dx and 16 for dw, in about twice
    the time of BF16, which rounds dz."""
    _check(load().moe_grouped_linear_backward(
        ctypes.byref(cfg), _ptr(dy), _ptr(x), _ptr(offsets), _ptr(w), _ptr(z), _ptr(dx),
        _ptr(dw), _ptr(ws), _ws(ws, ws_bytes), _stream(stream)), "moe_grouped_linear_backward")


def block_norm_workspace_size(cfg: BlockNormConfig) -> int:
    n = ctypes.c_size_t(0)
    _check(load().moe_block_norm_workspace_size(ctypes.byref(cfg), ctypes.byref(n)),
           "moe_block_norm_workspace_size")
    return n.value


def block_norm(cfg, x, residual, post_weight, gate, channel_scale, norm_weight, sum, y,
               stream=None):
    """sum = residual_scale * residual + branch_scale * gate * channel_scale * postnorm(x) and
    y = norm(sum) * norm_weight (either may be None)."""
    _check(load().moe_block_norm(ctypes.byref(cfg), _ptr(x), _ptr(residual), _ptr(post_weight),
                                 _ptr(gate), _ptr(channel_scale), _ptr(norm_weight), _ptr(sum),
                                 _ptr(y), _stream(stream)), "moe_block_norm")


def block_norm_backward(cfg, dy, dsum, x, sum, post_weight, gate, channel_scale, norm_weight, dx,
                        dresidual, dgate, dpost_weight, dchannel_scale, dnorm_weight, ws=None,
                        ws_bytes=None, stream=None):
    """The gradients of block_norm (each output may be None) from dy and dsum (one may be None)."""
    _check(load().moe_block_norm_backward(
        ctypes.byref(cfg), _ptr(dy), _ptr(dsum), _ptr(x), _ptr(sum), _ptr(post_weight), _ptr(gate),
        _ptr(channel_scale), _ptr(norm_weight), _ptr(dx), _ptr(dresidual), _ptr(dgate),
        _ptr(dpost_weight), _ptr(dchannel_scale), _ptr(dnorm_weight), _ptr(ws),
        _ws(ws, ws_bytes), _stream(stream)), "moe_block_norm_backward")


def clip_grad_norm_workspace_size(grads) -> int:
    """For a GradList, or a number of tensors."""
    n = ctypes.c_size_t(0)
    count = grads if isinstance(grads, int) else len(grads)
    _check(load().moe_clip_grad_norm_workspace_size(count, ctypes.byref(n)),
           "moe_clip_grad_norm_workspace_size")
    return n.value


def clip_grad_norm(grads: GradList, max_norm, norm, ws, grad_scale=1.0, eps=1e-6, ws_bytes=None,
                   stream=None):
    """norm[0] = grad_scale * 2-norm of all gradients; results = gradients * grad_scale *
    min(1, max_norm / (norm + eps))."""
    _check(load().moe_clip_grad_norm(ctypes.addressof(grads.array), len(grads), grad_scale,
                                     max_norm, eps, _ptr(norm), _ptr(ws), _ws(ws, ws_bytes),
                                     _stream(stream)), "moe_clip_grad_norm")


def workspace_views(cfg, ws) -> dict:
    """Device addresses (ints) of the intermediates a moe_layer_forward left in `ws`."""
    names = ["logits", "topk_ids", "topk_w", "counts", "offsets", "perm", "inv", "x_perm",
             "out_perm", "shared_out"]
    outs = [_P() for _ in names]
    _check(load().moe_workspace_views(ctypes.byref(cfg), _ptr(ws), *[ctypes.byref(o) for o in outs]),
           "moe_workspace_views")
    return {n: o.value for n, o in zip(names, outs)}


def debug_wait_timeout(limit_us, done, stream=None):
    """Self-test of the bounded device-side waits: a wait that nothing completes gives up
    after limit_us and records MOE_ERR_TIMEOUT for the next sync_check()."""
    _check(load().moe_debug_wait_timeout(limit_us, _ptr(done), _stream(stream)),
           "moe_debug_wait_timeout")


def sync_check(stream=None):
    _check(load().moe_sync_check(_stream(stream)), "moe_sync_check")
