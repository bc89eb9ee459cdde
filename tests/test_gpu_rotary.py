"""GPU parity of the rotary table and the rotation against the FP64 oracle: both
layouts, partial rotation, odd sizes and strides, both directions, in place, and
a token whose position is out of range."""
import numpy as np
import pytest
import torch

import gated_delta_rule_gateddeltanet_gb300 as gdn
from attention_common import f64, rounding
from gpu_common import dev
from oracle import attention as oa

pytestmark = pytest.mark.gpu

TYPES = [torch.float16, torch.bfloat16, torch.float32]


@pytest.mark.parametrize("kw", [
    {}, dict(base=1e6), dict(scaling="linear", factor=8.0), dict(scaling="ntk", factor=4.0),
    dict(scaling="by_parts", factor=8.0, original_positions=8192, beta_fast=4.0, beta_slow=1.0),
    dict(scaling="yarn", factor=16.0, original_positions=4096), dict(scaling="yarn", factor=1.0, original_positions=64),
    dict(scaling="yarn", factor=4.0, original_positions=4096, attention_factor=1.25),
])
@pytest.mark.parametrize("rotary_dim,positions", [(64, 3000), (6, 17), (128, 1)])
def test_table_is_exact_to_its_rounding(kw, rotary_dim, positions):
    """FP32 rounding of values up to the magnitude, and 64-bit angles up to `positions` (relative 2^-50)."""
    got = f64(gdn.rotary_table(positions, rotary_dim, device=dev(), **kw))
    want = oa.rotary_table(positions, rotary_dim, **kw)
    assert got.shape == want.shape
    assert np.abs(got - want).max() <= 1.5 * (2.0 ** -24 + positions * 2.0 ** -48)


def test_table_at_a_million_positions():
    got = gdn.rotary_table(1 << 20, 64, base=1e6, device=dev())[-3:]
    want = oa.rotary_table(1 << 20, 64, base=1e6)[-3:]
    assert np.abs(f64(got) - want).max() <= 2.0 ** -24 + 2.0 ** -28


def check(q, got, pos, table, interleaved, inverse):
    x = f64(q)
    want = oa.rotate(x, pos.cpu().numpy(), f64(table), interleaved, inverse)
    # |a c| + |b s| is at most |a| + |b| (cos, sin <= 1): the pair's largest magnitude twice
    r = table.shape[1]
    top = np.abs(x[..., :r]).max() * 2 if x.size else 0
    bound = rounding(want, q.dtype) * (1 + 2.0 ** -10) + 2.0 ** -23 * top
    assert np.all(np.abs(f64(got) - want) <= bound)
    assert torch.equal(got[..., r:], q[..., r:])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("hq,hk,d,r", [(8, 2, 128, 128), (4, 4, 64, 32), (3, 1, 256, 64), (5, 2, 80, 80), (2, 1, 96, 24),
                                       (1, 1, 2, 2), (3, 2, 30, 10), (7, 1, 128, 16)])
def test_rotation(dtype, interleaved, inverse, hq, hk, d, r):
    g = torch.Generator("cpu").manual_seed(d + r)
    T = 37
    q, k = (torch.randn(T, h, d, generator=g).to(dtype).to(dev()) for h in (hq, hk))
    pos = torch.randint(0, 100, (T,), generator=g, dtype=torch.int32).to(dev())
    table = gdn.rotary_table(100, r, device=dev())
    a, b = gdn.rotary(q, k, pos, table, interleaved=interleaved, inverse=inverse)
    check(q, a, pos, table, interleaved, inverse)
    check(k, b, pos, table, interleaved, inverse)
    # in place gives the same bits, and so do other strides and alignments
    q2, k2 = q.clone(), k.clone()
    gdn.rotary(q2, k2, pos, table, interleaved=interleaved, inverse=inverse, q_out=q2, k_out=k2)
    assert torch.equal(q2, a) and torch.equal(k2, b)
    fused = torch.empty(T, (hq + hk) * d + 2, dtype=dtype, device=dev())
    qf, kf = fused[:, 1:1 + hq * d].view(T, hq, d), fused[:, 1 + hq * d:1 + (hq + hk) * d].view(T, hk, d)
    qf.copy_(q), kf.copy_(k)
    gdn.rotary(qf, kf, pos, table, interleaved=interleaved, inverse=inverse, q_out=qf, k_out=kf)
    assert torch.equal(qf, a) and torch.equal(kf, b)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T", [1, 2, 1000, 20011])
def test_token_counts(dtype, T):
    q, k = torch.randn(T, 6, 64, device=dev()).to(dtype), torch.randn(T, 1, 64, device=dev()).to(dtype)
    pos = torch.randint(0, 5000, (T,), dtype=torch.int32, device=dev())
    table = gdn.rotary_table(5000, 64, device=dev())
    a, b = gdn.rotary(q, k, pos, table)
    check(q, a, pos, table, False, False)
    check(k, b, pos, table, False, False)


def test_without_keys_and_without_tokens():
    table = gdn.rotary_table(10, 32, device=dev())
    q = torch.randn(5, 2, 64, device=dev())
    pos = torch.arange(5, dtype=torch.int32, device=dev())
    a, b = gdn.rotary(q, None, pos, table)
    assert b is None
    check(q, a, pos, table, False, False)
    a, b = gdn.rotary(q[:0], q[:0], pos[:0], table)
    assert a.shape == (0, 2, 64)


@pytest.mark.parametrize("d", [64, 30])  # the vector kernel and the pair kernel
def test_positions_out_of_range_are_flagged_and_skipped(d):
    table = gdn.rotary_table(10, 10 if d == 30 else 32, device=dev())
    q = torch.randn(4, 2, d, device=dev())
    out = torch.full_like(q, 5.0)
    status = torch.zeros(1, dtype=torch.int32, device=dev())
    gdn.rotary(q, None, torch.tensor([0, 10, -1, 9], dtype=torch.int32, device=dev()), table, q_out=out, status=status)
    assert int(status) == gdn.DEVERR["position"]
    assert torch.all(out[1:3] == 5) and not torch.any(out[0] == 5) and not torch.any(out[3] == 5)


@pytest.mark.parametrize("interleaved", [False, True])
def test_gradient_against_the_formula_and_differences(interleaved):
    """The inverse rotation of g is d <rotate(x), g> / dx: against the oracle's transpose and central
    differences of the kernel itself (a linear map: the difference is exact up to FP32 rounding)."""
    g = torch.Generator("cpu").manual_seed(5)
    x, gr = torch.randn(3, 2, 16, generator=g).to(dev()), torch.randn(3, 2, 16, generator=g).to(dev())
    pos = torch.tensor([0, 7, 30], dtype=torch.int32, device=dev())
    table = gdn.rotary_table(31, 12, scaling="yarn", factor=2.0, original_positions=8, device=dev())
    grad, _ = gdn.rotary(gr, None, pos, table, interleaved=interleaved, inverse=True)
    want = oa.rotate(f64(gr), pos.cpu().numpy(), f64(table), interleaved, True)
    assert np.abs(f64(grad) - want).max() <= 2.0 ** -22 * 8
    f = lambda z: float((gdn.rotary(z, None, pos, table, interleaved=interleaved)[0].double() * gr.double()).sum())  # noqa: E731
    for idx in ((0, 0, 0), (1, 1, 3), (2, 0, 11), (2, 1, 15), (1, 0, 6)):
        e = torch.zeros_like(x)
        e[idx] = 1.0
        assert abs((f(x + e) - f(x - e)) / 2 - float(grad[idx])) <= 96 * 2.0 ** -22 * 8
