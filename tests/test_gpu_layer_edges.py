"""Uses of the gated linear recurrence and the root-mean-square norm beside the ordinary ones: infinite gates, state
slots given twice (debug build), a process's first call inside a capture, calls on two streams at once, and more heads
than one grid dimension holds."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import gated_delta_rule_gateddeltanet_gb300 as gdn
from gpu_common import dev
from layer_common import DTYPES, Recurrence

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("unit", [False, True])
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("dtype", DTYPES)
def test_infinite_gates(dtype, sign, unit):
    """a at infinity is a decay of 0 or 1, b an input weight of 1 or 0; in 64 bits a gate of 10,000 is the same."""
    case = Recurrence([150, 3], 68, dtype, unit=unit)
    for t in (case.a, case.b):
        t[3::5] = sign * float("inf")
    y, final, chk = case.forward(return_checkpoints=True)
    grads = case.backward(chk)
    for t in (case.a, case.b):
        t[torch.isinf(t)] = sign * 1e4
    case.check_forward(y, final)
    case.check_backward(grads)


def test_duplicate_slots_are_flagged_by_the_debug_build(monkeypatch):
    from gated_delta_rule_gateddeltanet_gb300 import build
    library = gdn.load_library(build.build(debug=True))
    gdn.load_library()
    case = Recurrence([20, 3, 40], 32)
    _, _, chk = case.forward(return_checkpoints=True)
    monkeypatch.setattr(gdn, "_lib", library)
    for same in (False, True):
        if same:
            case.slots[2] = case.slots[0]
        for call in (lambda s: case.forward(status=s), lambda s: case.backward(chk, status=s)):
            status = torch.zeros(1, dtype=torch.int32, device=dev())
            call(status)
            assert bool(status.item() & gdn.DEVERR["dup_slot"]) == same


FIRST = """
import torch
import gated_delta_rule_gateddeltanet_gb300 as gdn
x, a, b = (torch.randn(400, 1024, device="cuda").bfloat16() for _ in range(3))
cu = torch.tensor([0, 390, 400], dtype=torch.int32, device="cuda")
kw = dict(A_log=torch.zeros(1024, device="cuda"), dt_bias=torch.zeros(1024, device="cuda"))
w = torch.ones(1024, device="cuda")
def run():
    y, final, chk = gdn.linear_recurrence(x, a, b, cu, **kw, return_checkpoints=True)
    grads = gdn.linear_recurrence_backward(y, x, a, b, chk, cu, **kw)
    return [y, final, *grads, gdn.rms_norm(y, w), *gdn.rms_norm_backward(y, x, w)]
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    captured = run()
graph.replay()
for got, want in zip(captured, run(), strict=True):
    assert (got is None and want is None) or torch.equal(got, want)
"""


def test_a_process_may_capture_its_first_calls():
    out = subprocess.run([sys.executable, "-c", FIRST], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert out.returncode == 0, out.stderr[-2000:]


def test_two_streams_at_once():
    cases = [Recurrence([700, 90], 260, torch.bfloat16, seed=s) for s in (1, 2)]
    weight = torch.ones(260, device=dev())

    def run(case):
        y, final, chk = case.forward(return_checkpoints=True)
        return [y, final, *case.backward(chk), gdn.rms_norm(y, weight), *gdn.rms_norm_backward(case.dy, y, weight)]

    want = [run(c) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    for _ in range(3):
        got = []
        for case, stream in zip(cases, streams):
            with torch.cuda.stream(stream):
                got.append(run(case))
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            assert all(torch.equal(a, b) for a, b in zip(g, w, strict=True) if a is not None)


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float8_e4m3fn])
def test_more_heads_than_a_grid_dimension_holds(out):
    T, H, d = 4 * 65535 + 9, 8, 128
    x = torch.randn(T, H, d, device=dev(), dtype=torch.bfloat16)
    w = torch.rand(d, device=dev())
    kw = {} if out == torch.bfloat16 else dict(out_dtype=out, scale_group=d)
    every = gdn.rms_norm(x, w, **kw)
    every = every if isinstance(every, tuple) else (every,)
    for lo, hi in ((0, 33), (T // 2 - 17, T // 2 + 16), (T - 33, T)):
        part = gdn.rms_norm(x[lo:hi], w, **kw)
        for e, p in zip(every, part if isinstance(part, tuple) else (part,)):
            assert torch.equal(e[lo:hi].view(torch.uint8), p.view(torch.uint8))


@pytest.mark.parametrize("lo", [-9, -7, -5])
def test_decays_next_to_one_are_not_off_to_one_side(lo):
    """A long memory multiplies a decay's mean error by its length while the random part grows with the root of it, so the
    mean is held to 0.2 units of 2^-24, well inside a rounding's half (65,536 decays have a mean good to 0.01 units)."""
    C = 1 << 16
    g = torch.Generator("cpu").manual_seed(5)
    a, A_log = lo + 2 * torch.rand(1, C, generator=g), torch.log(1 + 15 * torch.rand(C, generator=g))
    want = np.exp(-np.exp(A_log.double().numpy()) * np.log1p(np.exp(a.double().numpy())))
    zero = torch.zeros(C, device=dev())
    for T in (1, 17):  # a decay alone, by a thread and by a tile: the tokens after the first keep the state
        rows = torch.full((T, C), -200.0)
        rows[0] = a[0]
        _, final = gdn.linear_recurrence(torch.zeros(T, C, device=dev()), rows.to(dev()), None, None, A_log=A_log.to(dev()),
                                         dt_bias=zero, initial_state=torch.ones(1, C, device=dev()), num_seqs=1)
        assert abs(((final.double().cpu().numpy() - want) / 2.0 ** -24).mean()) < 0.2
