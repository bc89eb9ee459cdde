"""Helpers of the tests of the gated linear recurrence and the root-mean-square norm: inputs, and
results held to the oracle's bounds (oracle/layers.py) plus the rounding of what is stored."""
import numpy as np
import torch

import gated_delta_rule_gateddeltanet_gb300 as gdn
from attention_common import f64, rounding
from gpu_common import dev
from oracle import layers as ol

DTYPES = [torch.bfloat16, torch.float16, torch.float32]


def held(got, want, err, what, dtype=None):
    """got within the oracle's error bound of want, and what rounding want to its type changes."""
    got_dtype = dtype or got.dtype
    g = f64(got).reshape(want.shape)
    assert np.all(np.isfinite(g)), what
    bound = err + rounding(np.abs(want) + err, got_dtype) + 2.0 ** -126
    over = np.abs(g - want) - bound
    assert over.max(initial=-1.0) <= 0, f"{what}: {over.max()} over its bound at {np.unravel_index(over.argmax(), over.shape)}"


class Recurrence:
    """Inputs of one packed batch.  extra: tokens behind the last sequence; fused: x, a, b as slices of one projection."""

    def __init__(self, lens, C, dtype=torch.float32, raw=True, unit=False, has_b=True, seed=0, initial=True, slots="shuffled",
                 extra=0, fused=False, decay=None):
        g = torch.Generator("cpu").manual_seed(seed)
        r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
        self.lens, self.C, self.raw, self.unit, self.dtype = lens, C, raw, unit, dtype
        B, T = len(lens), sum(lens) + extra
        self.B, self.T = B, T
        x, a, b = r(T, C).to(dtype), r(T, C), r(T, C)
        if raw:
            a, b = a.to(dtype), b.to(dtype)
            self.A_log = torch.log(1 + 15 * torch.rand(C, generator=g))
            self.dt_bias = torch.log(torch.expm1(1e-3 + 0.099 * torch.rand(C, generator=g)))
        else:
            a, b = torch.sigmoid(a + 3), torch.sigmoid(b)
            self.A_log = self.dt_bias = None
        if decay is not None:
            a = decay(a)
        if not has_b:
            b = None
        if fused:
            parts = [x, a] + ([b] if has_b else [])
            whole = torch.cat(parts, 1).to(dev())
            assert raw
            x, a, *rest = whole.split(C, 1)
            b = rest[0] if has_b else None
        cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
        self.spans = list(zip(cu[:-1].tolist(), cu[1:].tolist()))
        self.cu = torch.from_numpy(cu).to(dev())
        to = lambda t: None if t is None else t.to(dev())  # noqa: E731
        self.x, self.a, self.b, self.A_log, self.dt_bias = map(to, (x, a, b, self.A_log, self.dt_bias))
        self.num_slots = B + 2 if slots == "shuffled" else B
        self.slots = torch.randperm(self.num_slots, generator=g)[:B].to(torch.int32).to(dev()) if slots == "shuffled" else None
        self.initial = r(self.num_slots, C).to(dev()) if initial else None
        self.dy, self.d_final = r(T, C).to(dtype).to(dev()), r(self.num_slots, C).to(dev())

    def rows(self, pool):
        """Every sequence's row of a slot pool, in 64 bits."""
        if pool is None:
            return np.zeros((self.B, self.C))
        return f64(pool)[np.arange(self.B) if self.slots is None else self.slots.cpu().numpy()]

    def gates(self):
        n = lambda t: None if t is None else f64(t)  # noqa: E731
        return ol.Gates(n(self.a), n(self.b), n(self.A_log), n(self.dt_bias), self.raw, self.unit)

    def kw(self):
        return dict(A_log=self.A_log, dt_bias=self.dt_bias, gate_mode="raw" if self.raw else "precomputed",
                    unit_input=self.unit, initial_state=self.initial, state_slots=self.slots,
                    num_state_slots=self.num_slots)

    def forward(self, **kw):
        return gdn.linear_recurrence(self.x, self.a, self.b, self.cu, **{**self.kw(), **kw})

    def backward(self, checkpoints, **kw):
        return gdn.linear_recurrence_backward(self.dy, self.x, self.a, self.b, checkpoints, self.cu,
                                              **{**self.kw(), "d_final_state": self.d_final, **kw})

    def check_forward(self, y, final):
        n = sum(self.lens)
        h, want, *_, err, ferr, _ = ol.linear_recurrence(f64(self.x), self.gates(), self.spans, self.rows(self.initial))
        held(y[:n], h[:n], err[:n], "y")
        if final is not None:
            held(torch.from_numpy(self.rows(final)), want, ferr, "final_state", torch.float32)

    def check_backward(self, outs, d_final=True):
        n = sum(self.lens)
        x, gates = f64(self.x), self.gates()
        _, _, before, _, _, eb = ol.linear_recurrence(x, gates, self.spans, self.rows(self.initial))
        want = ol.linear_recurrence_backward(x, gates, self.spans, before, eb, f64(self.dy), self.rows(self.d_final if d_final else None))
        dx, da, db, dinit, *sums = outs
        for name, got in (("dx", dx), ("da", da), ("db", db)):
            if got is not None:
                held(got[:n], want[name][0][:n], want[name][1][:n], name)
        held(torch.from_numpy(self.rows(dinit)), *want["d_initial"], "d_initial_state", torch.float32)
        for name, got in zip(("dA_log", "ddt_bias"), sums):
            held(got, *want[name], name)
