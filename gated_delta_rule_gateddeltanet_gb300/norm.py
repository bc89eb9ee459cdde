"""Python binding of the root-mean-square norm of include/gdn.h, forward and backward.

    rms_norm(...)          / RMSNormCall         -> output, or (output[, residual_out][, scale])
    rms_norm_backward(...) / RMSNormBackwardCall -> (dx, dweight[, dgate])
"""
from __future__ import annotations

import ctypes

import torch

from . import GdnError, _check, _ptr, _shape, _token_stride, load_library
from .attention import _Call, _heads_out, _io

OUT_DTYPE = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2, torch.float8_e4m3fn: 3, torch.int8: 4}

_i32, _i64, _f32, _p = ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_void_p


class RMSNormArgs(ctypes.Structure):
    """Mirror of ``gdn_rms_norm_args``."""
    _fields_ = [("total_tokens", _i32), ("num_heads", _i32), ("head_dim", _i32), ("io_dtype", _i32),
                ("out_dtype", _i32), ("scale_group", _i32), ("eps", _f32), ("weight_offset", _f32),
                ("x_stride", _i64), ("residual_stride", _i64), ("gate_stride", _i64), ("x", _p), ("residual", _p),
                ("gate", _p), ("weight", _p), ("residual_out", _p), ("output", _p), ("scale", _p)]


class RMSNormBackwardArgs(ctypes.Structure):
    """Mirror of ``gdn_rms_norm_backward_args``."""
    _fields_ = [("total_tokens", _i32), ("num_heads", _i32), ("head_dim", _i32), ("io_dtype", _i32), ("eps", _f32),
                ("weight_offset", _f32), ("x_stride", _i64), ("dy_stride", _i64), ("gate_stride", _i64),
                ("d_residual_stride", _i64), ("x", _p), ("dy", _p), ("gate", _p), ("d_residual", _p), ("weight", _p),
                ("dx", _p), ("dgate", _p), ("dweight", _p), ("workspace", _p), ("workspace_bytes", ctypes.c_size_t)]


ENTRY_POINTS = {"gdn_rms_norm": RMSNormArgs, "gdn_rms_norm_backward": RMSNormBackwardArgs}


def declare(lib):
    """Argument types of this module's entry points (called when the library is loaded)."""
    for name, args in ENTRY_POINTS.items():
        f = getattr(lib, name)
        f.restype, f.argtypes = _i32, [ctypes.POINTER(args), _p]
    f = lib.gdn_rms_norm_backward_workspace_size
    f.restype, f.argtypes = _i32, [ctypes.POINTER(RMSNormBackwardArgs), ctypes.POINTER(ctypes.c_size_t)]


def _rows(t, name):
    """[T, C] as [T, 1, C]; [T, heads, d] as it is."""
    if t is None or t.dim() == 3:
        return t
    if t.dim() != 2:
        raise ValueError(f"{name} must be [T, heads, d] or [T, C]")
    return t.unsqueeze(1)


def _like(t, name, x):
    """Token stride of an input of x's shape and type."""
    _check(t, name, dtype=x.dtype, device=x.device, contiguous=False)
    _shape(t, name, x.shape)
    return _token_stride(t, name, x.shape[1] * x.shape[2])


def _geometry(args, x, weight, eps, weight_offset):
    args.total_tokens, args.num_heads, args.head_dim = x.shape
    args.io_dtype, args.eps, args.weight_offset = _io(x, "x"), float(eps), float(weight_offset)
    _check(weight, "weight", dtype=torch.float32, device=x.device)
    _shape(weight, "weight", (x.shape[2],))
    args.weight = _ptr(weight)
    args.x_stride, args.x = _like(x, "x", x), _ptr(x)


def _workspace_size(args):
    n = ctypes.c_size_t(0)
    rc = load_library().gdn_rms_norm_backward_workspace_size(ctypes.byref(args), ctypes.byref(n))
    if rc != 0:
        raise GdnError(rc, "gdn_rms_norm_backward_workspace_size")
    return int(n.value)


class RMSNormCall(_Call):
    """Root-mean-square norm of every head's row (C ABI ``gdn_rms_norm``).  x:
    [T, heads, d], or [T, C] for whole tokens, fp16 / bf16 / fp32, token stride
    free; ``weight`` [d] fp32 or None, ``weight_offset`` is added to it.  With
    ``residual`` (as x) the sum is normalised and returned too (``residual_out``
    may be x or residual).  ``gate`` (as x) multiplies the result by silu(gate).
    ``out_dtype`` torch.float8_e4m3fn or torch.int8 gives 8-bit rows with fp32
    scales, one a token ([T]) or one for every ``scale_group`` channels ([T, heads
    * d / scale_group]).  ``outputs`` is output, or the tuple (output[,
    residual_out][, scale])."""

    def __init__(self, x, weight=None, *, eps=1e-6, weight_offset=0.0, residual=None, gate=None, out_dtype=None,
                 scale_group=0, output=None, residual_out=None, scale=None):
        flat = x
        x = _rows(x, "x")
        a, dev = RMSNormArgs(), x.device
        _geometry(a, x, weight, eps, weight_offset)
        T, H, d = x.shape
        if out_dtype is None:
            out_dtype = x.dtype if output is None else output.dtype
        if out_dtype not in OUT_DTYPE:
            raise TypeError(f"unsupported output dtype {out_dtype}")
        eight = out_dtype in (torch.float8_e4m3fn, torch.int8)
        a.out_dtype, a.scale_group = OUT_DTYPE[out_dtype], int(scale_group)
        for name, t in (("residual", residual), ("gate", gate)):
            if t is not None:
                t = _rows(t, name)
                setattr(a, name + "_stride", _like(t, name, x))
                setattr(a, name, _ptr(t))
        if output is None:
            output = torch.empty(flat.shape, dtype=out_dtype, device=dev)
        _check(output, "output", dtype=out_dtype, device=dev)
        _shape(output, "output", flat.shape)
        outputs = [output]
        if residual is not None:
            residual_out = _heads_out(residual_out, "residual_out", flat, dev)
            _check(residual_out, "residual_out")
            outputs.append(residual_out)
        elif residual_out is not None:
            raise ValueError("residual_out without residual")
        if eight:
            if a.scale_group < 0 or (a.scale_group and d % a.scale_group):
                raise ValueError(f"scale_group must divide a row's {d} channels, got {scale_group}")
            shape = (T, H * d // a.scale_group) if a.scale_group else (T,)
            if scale is None:
                scale = torch.empty(shape, dtype=torch.float32, device=dev)
            _check(scale, "scale", dtype=torch.float32, device=dev)
            _shape(scale, "scale", shape)
            outputs.append(scale)
        elif scale is not None or scale_group:
            raise ValueError("scale and scale_group go with 8-bit outputs")
        a.output, a.residual_out, a.scale = _ptr(output), _ptr(residual_out), _ptr(scale)
        self._resolve("gdn_rms_norm", a, tuple(outputs) if len(outputs) > 1 else output, (x, weight, residual, gate), dev)


def rms_norm(x, weight=None, **kw):
    """``RMSNormCall(...).launch()``: returns output, or (output[, residual_out][, scale])."""
    return RMSNormCall(x, weight, **kw).launch()


class RMSNormBackwardCall(_Call):
    """Gradients of the norm (C ABI ``gdn_rms_norm_backward``).  dy: the
    output's gradient, x: what was normalised (the forward call's x, or its
    residual_out), ``d_residual``: the gradient that reaches residual_out from
    elsewhere; weight, gate, eps and weight_offset as in that call.  ``outputs`` is
    (dx, dweight) or (dx, dweight, dgate); dx is the gradient of x and of residual
    alike, dweight [d] fp32 is None without a weight."""

    def __init__(self, dy, x, weight=None, *, eps=1e-6, weight_offset=0.0, gate=None, d_residual=None, dx=None,
                 dweight=None, dgate=None, workspace=None):
        flat = x
        x = _rows(x, "x")
        a, dev = RMSNormBackwardArgs(), x.device
        _geometry(a, x, weight, eps, weight_offset)
        for name, t in (("dy", dy), ("gate", gate), ("d_residual", d_residual)):
            if t is not None:
                t = _rows(t, name)
                setattr(a, name + "_stride", _like(t, name, x))
                setattr(a, name, _ptr(t))
        dx = _heads_out(dx, "dx", flat, dev)
        _check(dx, "dx")
        if gate is not None:
            dgate = _heads_out(dgate, "dgate", flat, dev)
            _check(dgate, "dgate")
        elif dgate is not None:
            raise ValueError("dgate without gate")
        if weight is not None:
            if dweight is None:
                dweight = torch.empty_like(weight)
            _check(dweight, "dweight", dtype=torch.float32, device=dev)
            _shape(dweight, "dweight", weight.shape)
            a.dweight = _ptr(dweight)
            if workspace is None:
                workspace = torch.empty(_workspace_size(a), dtype=torch.uint8, device=dev)
            _check(workspace, "workspace", device=dev)
            a.workspace, a.workspace_bytes = _ptr(workspace), workspace.numel() * workspace.element_size()
        elif dweight is not None:
            raise ValueError("dweight without weight")
        a.dx, a.dgate = _ptr(dx), _ptr(dgate)
        self._resolve("gdn_rms_norm_backward", a, (dx, dweight) if gate is None else (dx, dweight, dgate),
                      (dy, x, weight, gate, d_residual, workspace), dev)


def rms_norm_backward(dy, x, weight=None, **kw):
    """``RMSNormBackwardCall(...).launch()``: returns (dx, dweight[, dgate])."""
    return RMSNormBackwardCall(dy, x, weight, **kw).launch()
