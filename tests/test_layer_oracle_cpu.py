"""The FP64 oracle of the gated linear recurrence and the root-mean-square norm against forms of the same
formulas that share nothing with it: the unrolled sum over a sequence, and torch's derivatives in 64 bits."""
import numpy as np
import pytest
import torch

from oracle import layers as ol


def draw(T, C, B, seed=0):
    r = np.random.default_rng(seed)
    return [r.standard_normal(s) for s in ((T, C), (T, C), (T, C), (T, C), (B, C), (B, C))]


SPANS = [(0, 7), (7, 7), (7, 20), (20, 21)]


def params(C):
    r = np.random.default_rng(9)
    return np.log(r.uniform(1, 16, C)), np.log(np.expm1(r.uniform(1e-3, 0.1, C)))


@pytest.mark.parametrize("raw,unit", [(True, False), (True, True), (False, False)])
def test_the_unrolled_sum(raw, unit):
    x, a, b, _, h0, _ = draw(21, 3, 4)
    gates = ol.Gates(a, b, *(params(3) if raw else (None, None)), raw, unit)
    h, final, before, *_ = ol.linear_recurrence(x, gates, SPANS, h0)
    for k, (lo, hi) in enumerate(SPANS):
        for t in range(lo, hi):
            want = np.prod(gates.g[lo:t + 1], 0) * h0[k]
            for s in range(lo, t + 1):
                want = want + np.prod(gates.g[s + 1:t + 1], 0) * gates.w[s] * x[s]
            assert np.allclose(h[t], want, rtol=1e-12, atol=1e-12)
            assert np.allclose(before[t], h0[k] if t == lo else h[t - 1], rtol=0, atol=0)
        assert np.array_equal(final[k], h[hi - 1] if hi > lo else h0[k])
    if raw:
        rate = np.exp(params(3)[0]) * np.log1p(np.exp(a + params(3)[1]))
        assert np.allclose(gates.g, np.exp(-rate), rtol=1e-13)
        if unit:
            assert np.allclose(gates.w, np.sqrt(1 - np.exp(-2 * rate)) / (1 + np.exp(-b)), rtol=1e-9)


@pytest.mark.parametrize("raw,unit,has_b", [(True, False, True), (True, True, True), (True, True, False), (False, False, True)])
def test_gradients_are_torch_s(raw, unit, has_b):
    x, a, b, dy, h0, df = draw(21, 3, 4, seed=1)
    A, dt = params(3)
    names = ["x", "a", "b", "h0", "A", "dt"]
    leaf = {n: torch.tensor(v, requires_grad=True) for n, v in zip(names, (x, a, b, h0, A, dt))}
    if raw:
        rate = leaf["A"].exp() * torch.nn.functional.softplus(leaf["a"] + leaf["dt"])
        g, w = (-rate).exp(), torch.sigmoid(leaf["b"]) if has_b else torch.ones(21, 3, dtype=torch.float64)
        w = w * torch.sqrt(-torch.expm1(-2 * rate)) if unit else w
    else:
        g, w = leaf["a"], leaf["b"]
    loss = 0.0
    for k, (lo, hi) in enumerate(SPANS):
        h = leaf["h0"][k]
        for t in range(lo, hi):
            h = g[t] * h + w[t] * leaf["x"][t]
            loss = loss + (h * torch.tensor(dy[t])).sum()
        loss = loss + (h * torch.tensor(df[k])).sum()
    loss.backward()
    gates = ol.Gates(a, b if has_b else None, A if raw else None, dt if raw else None, raw, unit)
    *_, before, _, _, eb = ol.linear_recurrence(x, gates, SPANS, h0)
    got = ol.linear_recurrence_backward(x, gates, SPANS, before, eb, dy, df)
    pairs = [("dx", "x"), ("da", "a"), ("d_initial", "h0")] + ([("db", "b")] if has_b else [])
    pairs += [("dA_log", "A"), ("ddt_bias", "dt")] if raw else []
    for mine, name in pairs:
        assert np.allclose(got[mine][0], leaf[name].grad.numpy(), rtol=1e-9, atol=1e-11), mine
        assert np.all(got[mine][1] >= 0)


@pytest.mark.parametrize("gate", [False, True])
def test_norm_gradients_are_torch_s(gate):
    r = np.random.default_rng(2)
    s, dy, z, dr = (r.standard_normal((5, 12)) for _ in range(4))
    w = 1 + 0.3 * r.standard_normal(12)
    ts, tw, tz = (torch.tensor(v, requires_grad=True) for v in (s, w, z))
    y = torch.nn.functional.rms_norm(ts, (12,), tw, 1e-5)
    if gate:
        y = y * torch.nn.functional.silu(tz)
    got, err = ol.rms_norm(s, 1e-5, w, z if gate else None)
    assert np.allclose(got, y.detach().numpy(), rtol=1e-12) and np.all(err >= 0)
    y.backward(torch.tensor(dy))
    out = ol.rms_norm_backward(dy, s, 1e-5, w, z if gate else None, dr)
    assert np.allclose(out["dx"][0] - dr, ts.grad.numpy(), rtol=1e-9, atol=1e-12)
    assert np.allclose(out["dweight"][0], tw.grad.numpy(), rtol=1e-9, atol=1e-12)
    if gate:
        assert np.allclose(out["dgate"][0], tz.grad.numpy(), rtol=1e-9, atol=1e-12)
