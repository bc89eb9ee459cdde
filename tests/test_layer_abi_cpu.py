"""CPU checks of the C ABI and binding of the gated linear recurrence and the root-mean-square norm: struct
layouts match the header, argument errors return before any launch, and the binding refuses tensors whose
types, shapes or strides do not fit.  No call here reaches a kernel."""
import ctypes
import os
import subprocess

import pytest
import torch

import gated_delta_rule_gateddeltanet_gb300 as gdn
from gated_delta_rule_gateddeltanet_gb300 import norm, recurrence
from gated_delta_rule_gateddeltanet_gb300.recurrent_step import RecurrentStep

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
NULL, DTYPE, SHAPE, ALIGN, WORKSPACE, ARG = 1, 2, 3, 4, 5, 8
FAKE = 0x1000  # never dereferenced: every case fails its host check first, or has nothing to do


@pytest.fixture(scope="module", autouse=True)
def lib():
    from gated_delta_rule_gateddeltanet_gb300 import build
    build.build()
    return gdn.load_library()


STRUCTS = {"gdn_linear_recurrence_args": recurrence.LinearRecurrenceArgs,
           "gdn_linear_recurrence_backward_args": recurrence.LinearRecurrenceBackwardArgs,
           "gdn_rms_norm_args": norm.RMSNormArgs, "gdn_rms_norm_backward_args": norm.RMSNormBackwardArgs}


def test_struct_layouts_match_c(tmp_path):
    body = 'printf("CHECKPOINT %d\\n", GDN_RECURRENCE_CHECKPOINT);'
    for name, cls in STRUCTS.items():
        body += "".join(f'printf("{name}.{f} %zu\\n", offsetof({name}, {f}));' for f, _ in cls._fields_)
        body += f'printf("{name} %zu\\n", sizeof({name}));'
    src = tmp_path / "layout.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "gdn.h"\nint main(void){' + body + "return 0;}\n")
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-std=c11", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    got = dict(line.split() for line in subprocess.run([str(exe)], capture_output=True, text=True,
                                                       check=True).stdout.splitlines())
    assert int(got["CHECKPOINT"]) == recurrence.CHECKPOINT
    for name, cls in STRUCTS.items():
        assert int(got[name]) == ctypes.sizeof(cls)
        for f, _ in cls._fields_:
            assert int(got[f"{name}.{f}"]) == getattr(cls, f).offset, (name, f)


def _set(a, kw):
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def test_null_argument_structs(lib):
    for name in (*recurrence.ENTRY_POINTS, *norm.ENTRY_POINTS):
        assert getattr(lib, name)(None, None) == NULL
    n = ctypes.c_size_t(0)
    assert lib.gdn_rms_norm_backward_workspace_size(None, ctypes.byref(n)) == NULL
    assert lib.gdn_rms_norm_backward_workspace_size(ctypes.byref(norm.RMSNormBackwardArgs()), None) == NULL


RECURRENCE_REFUSALS = [
    (dict(io_dtype=3), DTYPE), (dict(io_dtype=-1), DTYPE), (dict(gate_mode=2), ARG), (dict(unit_input=2), ARG),
    (dict(unit_input=1, gate_mode=1), ARG), (dict(num_seqs=-1), SHAPE), (dict(num_seqs=65536), SHAPE),
    (dict(total_tokens=-1), SHAPE), (dict(total_tokens=(1 << 30) + 1), SHAPE), (dict(channels=0), SHAPE), (dict(channels=(1 << 24) + 1), SHAPE),
    (dict(num_state_slots=0), SHAPE), (dict(state_slots=None, num_state_slots=1), SHAPE),
    (dict(cu_seqlens=None, total_tokens=101), SHAPE), (dict(x_stride=63), SHAPE), (dict(a_stride=1), SHAPE),
    (dict(b_stride=-64), SHAPE), (dict(x=None), NULL), (dict(a=None), NULL), (dict(A_log=None), NULL),
    (dict(dt_bias=None), NULL), (dict(x=FAKE + 1), ALIGN), (dict(a=FAKE + 1), ALIGN), (dict(b=FAKE + 1), ALIGN),
    (dict(gate_mode=1, a=FAKE + 2), ALIGN), (dict(initial_state=FAKE + 2), ALIGN), (dict(A_log=FAKE + 1), ALIGN),
]


def _recurrence(cls):
    a = cls()
    a.num_seqs, a.total_tokens, a.channels, a.num_state_slots, a.io_dtype = 2, 100, 64, 2, 1
    for f in ("x", "a", "b", "A_log", "dt_bias", "cu_seqlens", "state_slots", "initial_state"):
        setattr(a, f, FAKE)
    return a


@pytest.mark.parametrize("kw,code", RECURRENCE_REFUSALS + [
    (dict(max_seqlen=-1), SHAPE), (dict(output=None), NULL), (dict(output=FAKE + 1), ALIGN), (dict(final_state=FAKE + 1), ALIGN),
    (dict(checkpoints=FAKE + 1), ALIGN), (dict(num_seqs=0), 0),
])
def test_recurrence_refusals(lib, kw, code):
    a = _recurrence(recurrence.LinearRecurrenceArgs)
    a.output = FAKE
    assert lib.gdn_linear_recurrence(ctypes.byref(_set(a, kw)), None) == code


@pytest.mark.parametrize("kw,code", RECURRENCE_REFUSALS + [
    (dict(dy_stride=1), SHAPE), (dict(dy=None), NULL), (dict(dx=None), NULL), (dict(da=None), NULL), (dict(db=None), NULL),
    (dict(checkpoints=None), NULL), (dict(b=None), ARG), (dict(gate_mode=1, dA_log=FAKE), ARG),
    (dict(gate_mode=1, ddt_bias=FAKE), ARG), (dict(dx=FAKE + 1), ALIGN), (dict(dA_log=FAKE + 1), ALIGN),
    (dict(d_initial_state=FAKE, d_final_state=FAKE), ARG), (dict(d_final_state=FAKE + 2), ALIGN),
])
def test_recurrence_backward_refusals(lib, kw, code):
    a = _recurrence(recurrence.LinearRecurrenceBackwardArgs)
    for f in ("dy", "checkpoints", "dx", "da", "db"):
        setattr(a, f, FAKE)
    assert lib.gdn_linear_recurrence_backward(ctypes.byref(_set(a, kw)), None) == code


NORM_REFUSALS = [
    (dict(io_dtype=3), DTYPE), (dict(total_tokens=-1), SHAPE), (dict(num_heads=0), SHAPE), (dict(head_dim=0), SHAPE),
    (dict(num_heads=1 << 20, head_dim=1 << 12), SHAPE), (dict(eps=0.0), ARG), (dict(eps=-1.0), ARG), (dict(eps=float("nan")), ARG),
    (dict(eps=float("inf")), ARG), (dict(weight_offset=float("inf")), ARG), (dict(x_stride=255), SHAPE), (dict(gate_stride=2), SHAPE),
    (dict(x=None), NULL), (dict(x=FAKE + 1), ALIGN), (dict(weight=FAKE + 2), ALIGN), (dict(gate=FAKE + 1), ALIGN),
]


@pytest.mark.parametrize("kw,code", NORM_REFUSALS + [
    (dict(out_dtype=0), DTYPE), (dict(out_dtype=2), DTYPE), (dict(out_dtype=7), DTYPE), (dict(scale_group=64), ARG),
    (dict(out_dtype=3, scale=FAKE, scale_group=16), ARG), (dict(out_dtype=3, scale=FAKE, scale_group=-32), ARG),
    (dict(out_dtype=4, scale=FAKE, scale_group=64, head_dim=96, gate_stride=0), SHAPE), (dict(out_dtype=3), NULL), (dict(scale=FAKE), ARG),
    (dict(output=None), NULL), (dict(residual=3 * FAKE), NULL), (dict(residual_out=3 * FAKE), ARG), (dict(residual_stride=3), SHAPE),
    (dict(output=FAKE, x_stride=300), ARG), (dict(output=5 * FAKE, gate_stride=300), ARG),
    (dict(residual=3 * FAKE, residual_out=3 * FAKE, residual_stride=300), ARG),
    (dict(residual=3 * FAKE, residual_out=FAKE, x_stride=300), ARG),
    (dict(residual=3 * FAKE, residual_out=3 * FAKE, output=3 * FAKE), ARG),
    (dict(residual=3 * FAKE, residual_out=5 * FAKE), ARG),
    (dict(out_dtype=3, scale=FAKE, output=FAKE), ARG), (dict(out_dtype=4, scale=FAKE, output=5 * FAKE), ARG),
    (dict(total_tokens=0, x=None, output=None), 0),
])
def test_norm_refusals(lib, kw, code):
    a = norm.RMSNormArgs()
    a.total_tokens, a.num_heads, a.head_dim, a.io_dtype, a.out_dtype, a.eps = 4, 2, 128, 1, 1, 1e-6
    a.x, a.output, a.weight, a.gate = FAKE, 2 * FAKE, FAKE, 5 * FAKE
    assert lib.gdn_rms_norm(ctypes.byref(_set(a, kw)), None) == code


@pytest.mark.parametrize("kw,code", NORM_REFUSALS + [
    (dict(dy=None), NULL), (dict(dx=None), NULL), (dict(dgate=None), NULL), (dict(gate=None), ARG), (dict(weight=None), ARG),
    (dict(dy_stride=3), SHAPE), (dict(d_residual_stride=3), SHAPE), (dict(dx=FAKE), ARG), (dict(dx=6 * FAKE), ARG),
    (dict(dgate=5 * FAKE), ARG), (dict(dgate=2 * FAKE), ARG), (dict(workspace=None), WORKSPACE), (dict(workspace_bytes=16), WORKSPACE),
    (dict(workspace=FAKE + 8), ALIGN), (dict(dx=2 * FAKE + 1), ALIGN),
])
def test_norm_backward_refusals(lib, kw, code):
    a = norm.RMSNormBackwardArgs()
    a.total_tokens, a.num_heads, a.head_dim, a.io_dtype, a.eps = 4, 2, 128, 1, 1e-6
    a.x, a.dy, a.weight, a.gate, a.dx, a.dgate, a.dweight = FAKE, 6 * FAKE, FAKE, 5 * FAKE, 2 * FAKE, 3 * FAKE, 4 * FAKE
    a.workspace, a.workspace_bytes = FAKE, 1 << 30
    assert lib.gdn_rms_norm_backward(ctypes.byref(_set(a, kw)), None) == code


def z(*s, dtype=torch.float16):
    return torch.zeros(*s, dtype=dtype)


def f(*s):
    return z(*s, dtype=torch.float32)


CU = torch.tensor([0, 2, 6], dtype=torch.int32)


def _call(**kw):
    args = dict(x=z(6, 8), a=z(6, 8), b=z(6, 8), cu_seqlens=CU, A_log=f(8), dt_bias=f(8))
    return gdn.LinearRecurrenceCall(**{**args, **kw})


def test_recurrence_binding_accepts():
    wide = z(6, 24)
    x, a, b = wide.split(8, 1)
    call = _call(x=x, a=a, b=b)
    assert (call.args.x_stride, call.args.num_seqs, call.args.num_state_slots) == (24, 2, 2)
    assert call.outputs[0].shape == (6, 8) and call.outputs[1].shape == (2, 8) and len(call.outputs) == 2
    assert _call(return_checkpoints=True).outputs[2].shape == (1, 8)
    assert _call(cu_seqlens=None, num_seqs=3).args.num_seqs == 3
    pool = f(5, 8)
    assert _call(initial_state=pool, final_state=pool, state_slots=torch.tensor([4, 1], dtype=torch.int32)).outputs[1] is pool
    assert _call(write_final_state=False).outputs[1] is None
    pre = dict(a=f(6, 8), b=None, A_log=None, dt_bias=None, gate_mode="precomputed")
    assert _call(**pre).args.gate_mode == 1


@pytest.mark.parametrize("kw,error", [
    (dict(x=z(6, 8, dtype=torch.int32)), TypeError), (dict(x=z(6, 2, 4)), ValueError), (dict(a=f(6, 8)), TypeError),
    (dict(b=z(5, 8)), ValueError), (dict(x=z(1, 8).expand(6, 8)), ValueError), (dict(a=z(8, 6).t()), ValueError),
    (dict(A_log=None), ValueError), (dict(A_log=z(8)), TypeError), (dict(dt_bias=f(7)), ValueError),
    (dict(gate_mode="precomputed", a=f(6, 8), b=f(6, 8)), ValueError), (dict(gate_mode="precomputed", A_log=None, dt_bias=None), TypeError),
    (dict(cu_seqlens=CU.long()), TypeError), (dict(cu_seqlens=CU[None]), ValueError), (dict(cu_seqlens=None), ValueError),
    (dict(num_seqs=3), ValueError), (dict(state_slots=CU), ValueError), (dict(initial_state=f(2, 7)), ValueError),
    (dict(initial_state=z(2, 8)), TypeError), (dict(initial_state=f(8, 2).t()), ValueError), (dict(output=z(5, 8)), ValueError),
    (dict(output=z(6, 16)[:, :8]), ValueError), (dict(final_state=f(2, 8), write_final_state=False), ValueError),
    (dict(checkpoints=f(1, 7)), ValueError), (dict(max_seqlen=1 << 31), ValueError), (dict(status=f(1)), TypeError),
    (dict(initial_state=f(3, 8), final_state=f(2, 8)), ValueError),
])
def test_recurrence_binding_refuses(kw, error):
    with pytest.raises(error):
        _call(**kw)


def _back(**kw):
    args = dict(dy=z(6, 8), x=z(6, 8), a=z(6, 8), b=z(6, 8), checkpoints=f(1, 8), cu_seqlens=CU, A_log=f(8), dt_bias=f(8))
    return gdn.LinearRecurrenceBackwardCall(**{**args, **kw})


@pytest.mark.parametrize("kw,error", [
    (dict(dy=f(6, 8)), TypeError), (dict(dy=z(1, 8).expand(6, 8)), ValueError), (dict(checkpoints=f(0, 8)), ValueError),
    (dict(checkpoints=z(1, 8)), TypeError), (dict(initial_state=f(2, 8), d_final_state=f(1, 8)), ValueError), (dict(b=None, db=z(6, 8)), ValueError),
    (dict(dx=f(6, 8)), TypeError), (dict(dA_log=f(7)), ValueError),
    (dict(gate_mode="precomputed", a=f(6, 8), b=f(6, 8), A_log=None, dt_bias=None, dA_log=f(8)), ValueError),
])
def test_recurrence_backward_binding_refuses(kw, error):
    assert len(_back().outputs) == 6 and _back(b=None).outputs[2] is None
    with pytest.raises(error):
        _back(**kw)


@pytest.mark.parametrize("kw,error", [
    (dict(x=z(6, 8, dtype=torch.float64)), TypeError), (dict(x=z(8)), ValueError), (dict(weight=z(8)), TypeError),
    (dict(weight=f(7)), ValueError), (dict(residual=z(6, 7)), ValueError), (dict(residual=f(6, 8)), TypeError),
    (dict(gate=z(1, 8).expand(6, 8)), ValueError), (dict(x=z(8, 6).t()), ValueError), (dict(out_dtype=torch.float32), gdn.GdnError),
    (dict(out_dtype=torch.int16), TypeError), (dict(residual_out=z(6, 8)), ValueError), (dict(scale=f(6)), ValueError),
    (dict(scale_group=32), ValueError), (dict(out_dtype=torch.int8, scale_group=3), ValueError),
    (dict(out_dtype=torch.int8, scale=f(5)), ValueError), (dict(out_dtype=torch.int8, output=z(6, 8)), TypeError),
    (dict(output=z(5, 8)), ValueError), (dict(residual=z(6, 8), residual_out=z(6, 16)[:, :8]), ValueError),
])
def test_norm_binding_refuses(lib, kw, error):
    args = dict(x=z(6, 8), weight=f(8))
    assert gdn.RMSNormCall(**args).outputs.shape == (6, 8)
    assert gdn.RMSNormCall(z(6, 2, 64), out_dtype=torch.int8, scale_group=32).outputs[1].shape == (6, 4)
    with pytest.raises(error):
        call = gdn.RMSNormCall(**{**args, **kw})
        rc = lib.gdn_rms_norm(ctypes.byref(call.args), None)  # (refused by its types)
        assert rc != 0
        raise gdn.GdnError(rc, "gdn_rms_norm")


@pytest.mark.parametrize("kw,error", [
    (dict(dy=f(6, 8)), TypeError), (dict(dgate=z(6, 8)), ValueError), (dict(weight=None, dweight=f(8)), ValueError),
    (dict(dweight=f(7)), ValueError), (dict(dx=z(6, 16)[:, :8]), ValueError), (dict(d_residual=z(6, 7)), ValueError),
])
def test_norm_backward_binding_refuses(kw, error):
    args = dict(dy=z(6, 8), x=z(6, 8), weight=f(8))
    assert [t.shape for t in gdn.RMSNormBackwardCall(**args).outputs] == [(6, 8), (8,)]
    assert gdn.RMSNormBackwardCall(**{**args, "weight": None}).outputs[1] is None
    with pytest.raises(error):
        gdn.RMSNormBackwardCall(**{**args, **kw})


def test_host_tensors_are_refused_at_launch():
    step = RecurrentStep(f(8, 4), None, z(3, 8, 3), f(8), f(8), f(3, 8), f(8), seqs=2, head_dim=8)
    for call in (_call(), _back(), gdn.RMSNormCall(z(6, 8)), gdn.RMSNormBackwardCall(z(6, 8), z(6, 8)), step):
        with pytest.raises(ValueError, match="GPU"):
            call.launch()


@pytest.mark.parametrize("kw", [dict(head_dim=3), dict(seqs=4)])
def test_recurrent_step_refuses(kw):
    with pytest.raises(ValueError):
        RecurrentStep(f(8, 4), None, z(3, 8, 3), f(8), f(8), f(3, 8), f(8), **{**dict(seqs=2, head_dim=8), **kw})
