"""Python binding of the gated linear recurrence of include/gdn.h, forward and backward.

As in ``attention.py``: it checks types, devices and shapes, allocates outputs
that the caller did not pass, and calls the library on the current torch stream;
every operator has a function and a call object whose ``launch()`` is one C-ABI call.

    linear_recurrence(...)          / LinearRecurrenceCall         -> (output, final_state[, checkpoints])
    linear_recurrence_backward(...) / LinearRecurrenceBackwardCall -> (dx, da, db, d_initial_state[, dA_log, ddt_bias])
"""
from __future__ import annotations

import ctypes

import torch

from . import GATE_MODE, _check, _ptr, _row_stride, _shape
from .attention import _Call, _cu_seqlens, _int32, _io, _status

CHECKPOINT = 64  # GDN_RECURRENCE_CHECKPOINT

_i32, _i64, _p = ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p


class LinearRecurrenceArgs(ctypes.Structure):
    """Mirror of ``gdn_linear_recurrence_args``."""
    _fields_ = [("num_seqs", _i32), ("total_tokens", _i32), ("channels", _i32), ("num_state_slots", _i32),
                ("io_dtype", _i32), ("gate_mode", _i32), ("unit_input", _i32), ("max_seqlen", _i32),
                ("x_stride", _i64), ("a_stride", _i64), ("b_stride", _i64), ("x", _p), ("a", _p), ("b", _p),
                ("A_log", _p), ("dt_bias", _p), ("cu_seqlens", _p), ("state_slots", _p), ("initial_state", _p),
                ("final_state", _p), ("output", _p), ("checkpoints", _p), ("status", _p)]


class LinearRecurrenceBackwardArgs(ctypes.Structure):
    """Mirror of ``gdn_linear_recurrence_backward_args``."""
    _fields_ = [("num_seqs", _i32), ("total_tokens", _i32), ("channels", _i32), ("num_state_slots", _i32),
                ("io_dtype", _i32), ("gate_mode", _i32), ("unit_input", _i32),
                ("x_stride", _i64), ("a_stride", _i64), ("b_stride", _i64), ("dy_stride", _i64),
                ("x", _p), ("a", _p), ("b", _p), ("dy", _p), ("A_log", _p), ("dt_bias", _p), ("cu_seqlens", _p),
                ("state_slots", _p), ("initial_state", _p), ("checkpoints", _p), ("d_final_state", _p), ("dx", _p),
                ("da", _p), ("db", _p), ("dA_log", _p), ("ddt_bias", _p), ("d_initial_state", _p), ("status", _p)]


ENTRY_POINTS = {"gdn_linear_recurrence": LinearRecurrenceArgs,
                "gdn_linear_recurrence_backward": LinearRecurrenceBackwardArgs}


def declare(lib):
    """Argument types of this module's entry points (called when the library is loaded)."""
    for name, args in ENTRY_POINTS.items():
        f = getattr(lib, name)
        f.restype, f.argtypes = _i32, [ctypes.POINTER(args), _p]


def _tokens(t, name, shape, dtype, device):
    """Token stride of a [T, C] input whose channels are contiguous (a slice of a fused projection may be)."""
    _check(t, name, dtype=dtype, device=device, contiguous=False)
    _shape(t, name, shape)
    if t.numel() and t.shape[1] > 1 and t.stride(1) != 1:
        raise ValueError(f"{name}: channels must be contiguous")
    return _row_stride(t, name, shape[1])


def _output(t, name, shape, dtype, device):
    """A contiguous output, allocated if absent."""
    if t is None:
        t = torch.empty(shape, dtype=dtype, device=device)
    _check(t, name, dtype=dtype, device=device)
    _shape(t, name, shape, leading_at_least=True)
    return t


def _states(t, name, slots, channels, device):
    _check(t, name, dtype=torch.float32, device=device)
    _shape(t, name, (slots, channels), leading_at_least=True)


def _inputs(args, x, a, b, cu_seqlens, A_log, dt_bias, gate_mode, unit_input, initial_state, state_slots, num_seqs,
            num_state_slots, status, states):
    """Fills what both directions have in common; returns (T, C, B, slots, the gates' type).  ``states``: state tensors,
    the first of which that is given says how many slots there are."""
    dev = x.device
    if x.dim() != 2:
        raise ValueError("x must be [T, C]")
    T, C = x.shape
    args.io_dtype, args.gate_mode, args.unit_input = _io(x, "x"), GATE_MODE[gate_mode], int(bool(unit_input))
    gate_dtype = x.dtype if gate_mode == "raw" else torch.float32
    args.x_stride = _tokens(x, "x", (T, C), x.dtype, dev)
    args.a_stride = _tokens(a, "a", (T, C), gate_dtype, dev)
    if b is not None:
        args.b_stride = _tokens(b, "b", (T, C), gate_dtype, dev)
    if gate_mode == "raw" and (A_log is None or dt_bias is None):
        raise ValueError("raw gates need A_log and dt_bias")
    if gate_mode != "raw" and (A_log is not None or dt_bias is not None):
        raise ValueError("A_log and dt_bias go with raw gates")
    for name, t in (("A_log", A_log), ("dt_bias", dt_bias)):
        _check(t, name, dtype=torch.float32, device=dev)
        _shape(t, name, (C,))
    if cu_seqlens is not None:
        B = _cu_seqlens(cu_seqlens, dev)
        if num_seqs is not None and int(num_seqs) != B:
            raise ValueError(f"num_seqs is {num_seqs}, cu_seqlens has {B} sequences")
    elif num_seqs is None:
        raise ValueError("without cu_seqlens, num_seqs says how many sequences of equal length there are")
    else:
        B = _int32(num_seqs, "num_seqs")
    _check(state_slots, "state_slots", dtype=torch.int32, device=dev)
    _shape(state_slots, "state_slots", (B,))
    _status(status, dev)
    slots = next((t.shape[0] for t in states if t is not None), B) if num_state_slots is None else num_state_slots
    args.num_seqs, args.total_tokens, args.channels = B, T, C
    args.num_state_slots = _int32(slots, "num_state_slots")
    _states(initial_state, "initial_state", slots, C, dev)
    args.x, args.a, args.b, args.A_log, args.dt_bias = _ptr(x), _ptr(a), _ptr(b), _ptr(A_log), _ptr(dt_bias)
    args.cu_seqlens, args.state_slots, args.initial_state = _ptr(cu_seqlens), _ptr(state_slots), _ptr(initial_state)
    args.status = _ptr(status)
    return T, C, B, slots, gate_dtype


def _checkpoint_shape(T, C):
    return (T + CHECKPOINT - 1) // CHECKPOINT, C


class LinearRecurrenceCall(_Call):
    """The gated linear recurrence over a packed batch (C ABI
    ``gdn_linear_recurrence``).  x: [T, C] fp16 / bf16 / fp32; a, b: [T, C], raw
    gate inputs in x's type with ``A_log`` and ``dt_bias`` [C] fp32, or fp32
    decays and input weights with ``gate_mode="precomputed"``; b may be None (an
    input weight of 1).  Token strides are free.  ``unit_input`` multiplies the
    input weight by sqrt(1 - decay^2).  cu_seqlens: [B + 1] int32, or None with
    ``num_seqs`` sequences of equal length.  ``initial_state`` [slots, C] fp32 or
    None (zeros); ``final_state`` may be the same tensor (in place);
    ``write_final_state=False`` writes none.  A launch writes the batch's slots only:
    the other rows of a ``final_state`` that this object allocated are ``initial_state``'s at
    its construction.  ``return_checkpoints`` keeps what the backward pass needs.  ``outputs`` is (output, final_state), or (output,
    final_state, checkpoints)."""

    def __init__(self, x, a, b=None, cu_seqlens=None, *, A_log=None, dt_bias=None, gate_mode="raw", unit_input=False,
                 initial_state=None, final_state=None, state_slots=None, num_seqs=None, num_state_slots=None,
                 output=None, checkpoints=None, return_checkpoints=False, max_seqlen=0, write_final_state=True,
                 status=None):
        args, dev = LinearRecurrenceArgs(), x.device
        T, C, B, slots, _ = _inputs(args, x, a, b, cu_seqlens, A_log, dt_bias, gate_mode, unit_input, initial_state,
                                    state_slots, num_seqs, num_state_slots, status, (initial_state, final_state))
        args.max_seqlen = _int32(max_seqlen or 0, "max_seqlen")
        if not write_final_state:
            if final_state is not None:
                raise ValueError("final_state with write_final_state=False")
        elif final_state is None:
            final_state = (torch.zeros((slots, C), dtype=torch.float32, device=dev) if initial_state is None
                           else initial_state.clone())
        _states(final_state, "final_state", slots, C, dev)
        output = _output(output, "output", (T, C), x.dtype, dev)
        if checkpoints is not None or return_checkpoints:
            checkpoints = _output(checkpoints, "checkpoints", _checkpoint_shape(T, C), torch.float32, dev)
        args.output, args.final_state, args.checkpoints = _ptr(output), _ptr(final_state), _ptr(checkpoints)
        self._resolve("gdn_linear_recurrence", args,
                      (output, final_state) if checkpoints is None else (output, final_state, checkpoints),
                      (x, a, b, cu_seqlens, A_log, dt_bias, initial_state, state_slots, status), dev)


def linear_recurrence(x, a, b=None, cu_seqlens=None, **kw):
    """``LinearRecurrenceCall(...).launch()``: returns (output, final_state[, checkpoints])."""
    return LinearRecurrenceCall(x, a, b, cu_seqlens, **kw).launch()


class LinearRecurrenceBackwardCall(_Call):
    """Gradients of the gated linear recurrence (C ABI
    ``gdn_linear_recurrence_backward``).  dy: [T, C], the output's gradient;
    ``checkpoints`` from the forward call; ``d_final_state`` [slots, C] fp32 or None
    (zeros); everything else as that call was given it (its initial states must not
    have been overwritten in place).  ``outputs`` is (dx, da, db, d_initial_state),
    and (.., dA_log, ddt_bias) with raw gates; db is None without b.  A launch writes the
    batch's slots of d_initial_state only.  ``max_seqlen`` is taken so that the forward call's keywords can be
    passed on; nothing depends on it."""

    def __init__(self, dy, x, a, b, checkpoints, cu_seqlens=None, *, A_log=None, dt_bias=None, gate_mode="raw",
                 unit_input=False, initial_state=None, state_slots=None, num_seqs=None, num_state_slots=None,
                 d_final_state=None, dx=None, da=None, db=None, d_initial_state=None, dA_log=None, ddt_bias=None,
                 max_seqlen=0, status=None):
        args, dev = LinearRecurrenceBackwardArgs(), x.device
        T, C, B, slots, gate_dtype = _inputs(args, x, a, b, cu_seqlens, A_log, dt_bias, gate_mode, unit_input,
                                             initial_state, state_slots, num_seqs, num_state_slots, status,
                                             (initial_state, d_final_state, d_initial_state))
        args.dy_stride = _tokens(dy, "dy", (T, C), x.dtype, dev)
        _check(checkpoints, "checkpoints", dtype=torch.float32, device=dev)
        _shape(checkpoints, "checkpoints", _checkpoint_shape(T, C), leading_at_least=True)
        _states(d_final_state, "d_final_state", slots, C, dev)
        if d_initial_state is None:
            d_initial_state = torch.zeros((slots, C), dtype=torch.float32, device=dev)
        _states(d_initial_state, "d_initial_state", slots, C, dev)
        if db is not None and b is None:
            raise ValueError("db without b")
        dx = _output(dx, "dx", (T, C), x.dtype, dev)
        da = _output(da, "da", (T, C), gate_dtype, dev)
        db = None if b is None else _output(db, "db", (T, C), gate_dtype, dev)
        outputs = (dx, da, db, d_initial_state)
        if gate_mode == "raw":
            dA_log = _output(dA_log, "dA_log", (C,), torch.float32, dev)
            ddt_bias = _output(ddt_bias, "ddt_bias", (C,), torch.float32, dev)
            outputs += (dA_log, ddt_bias)
        elif dA_log is not None or ddt_bias is not None:
            raise ValueError("dA_log and ddt_bias go with raw gates")
        args.dy, args.checkpoints, args.d_final_state = _ptr(dy), _ptr(checkpoints), _ptr(d_final_state)
        args.dx, args.da, args.db, args.d_initial_state = _ptr(dx), _ptr(da), _ptr(db), _ptr(d_initial_state)
        args.dA_log, args.ddt_bias = _ptr(dA_log), _ptr(ddt_bias)
        self._resolve("gdn_linear_recurrence_backward", args, outputs,
                      (dy, x, a, b, checkpoints, cu_seqlens, A_log, dt_bias, initial_state, state_slots, d_final_state,
                       status), dev)


def linear_recurrence_backward(dy, x, a, b, checkpoints, cu_seqlens=None, **kw):
    """``LinearRecurrenceBackwardCall(...).launch()``: returns (dx, da, db, d_initial_state[, dA_log, ddt_bias])."""
    return LinearRecurrenceBackwardCall(dy, x, a, b, checkpoints, cu_seqlens, **kw).launch()
