"""CPU pins of the softmax-attention oracle (oracle/attention.py): the rotation is
orthogonal and its inverse is its gradient (checked against the formula's
transpose and against differences), the scaled frequencies have their limiting
cases, the 8-bit row scales their defining bounds, and attention agrees with a
softmax written in another way."""
import math

import numpy as np
import pytest

from oracle import attention as oa


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_is_orthogonal_and_inverse_undoes_it(interleaved):
    rng = np.random.default_rng(1)
    x = rng.standard_normal((7, 3, 12))
    table = oa.rotary_table(50, 8)
    pos = rng.integers(0, 50, 7)
    y = oa.rotate(x, pos, table, interleaved)
    np.testing.assert_allclose(np.linalg.norm(y, axis=-1), np.linalg.norm(x, axis=-1), rtol=1e-13)
    np.testing.assert_array_equal(y[..., 8:], x[..., 8:])
    np.testing.assert_allclose(oa.rotate(y, pos, table, interleaved, inverse=True), x, atol=1e-13)


@pytest.mark.parametrize("interleaved", [False, True])
def test_inverse_rotation_is_the_gradient(interleaved):
    """d/dx of <rotate(x), g> by central differences (exact for a linear map up to rounding)."""
    rng = np.random.default_rng(2)
    x, g = rng.standard_normal((2, 1, 8)), rng.standard_normal((2, 1, 8))
    table, pos = oa.rotary_table(9, 6, attention_factor=1.3), np.array([3, 8])
    grad = oa.rotate(g, pos, table, interleaved, inverse=True)
    f = lambda z: (oa.rotate(z, pos, table, interleaved) * g).sum()  # noqa: E731
    for idx in np.ndindex(x.shape):
        e = np.zeros_like(x)
        e[idx] = 0.5
        assert abs(f(x + e) - f(x - e) - grad[idx]) < 1e-12


def test_positions_become_relative_in_scores():
    """<rotate(q, a), rotate(k, b)> depends on a - b alone."""
    rng = np.random.default_rng(3)
    q, k = rng.standard_normal((1, 1, 16)), rng.standard_normal((1, 1, 16))
    table = oa.rotary_table(200, 16)
    dot = lambda a, b: (oa.rotate(q, [a], table) * oa.rotate(k, [b], table)).sum()  # noqa: E731
    assert abs(dot(10, 3) - dot(150, 143)) < 1e-11


def test_scaled_frequencies_at_their_limits():
    w, _ = oa.rotary_frequencies(64)
    lin, _ = oa.rotary_frequencies(64, scaling="linear", factor=4.0)
    np.testing.assert_allclose(lin * 4, w)
    ntk, _ = oa.rotary_frequencies(64, scaling="ntk", factor=4.0)
    assert ntk[0] == w[0] and math.isclose(ntk[-1] * 4, w[-1], rel_tol=1e-12)  # slowest pair interpolated, fastest kept
    for kind in ("by_parts", "yarn"):
        v, m = oa.rotary_frequencies(64, scaling=kind, factor=4.0, original_positions=4096)
        assert v[0] == w[0] and math.isclose(v[-1] * 4, w[-1], rel_tol=1e-12)
        assert np.all(v <= w * (1 + 1e-15)) and np.all(v * 4 >= w * (1 - 1e-15))
        assert math.isclose(m, 0.1 * math.log(4) + 1 if kind == "yarn" else 1.0)


def test_row_scales_bound_their_rows():
    rng = np.random.default_rng(4)
    x = rng.standard_normal((100, 64)) * np.exp(rng.uniform(-20, 20, (100, 1)))
    top = np.abs(x).max(-1)
    s8 = oa.row_scale(x, "int8")
    np.testing.assert_allclose(top / s8, 127)
    f8 = oa.row_scale(x, "fp8")
    assert np.all(top / f8 <= 448) and np.all(top / f8 > 224)
    assert np.all(np.log2(f8) == np.round(np.log2(f8)))
    assert oa.row_scale(np.zeros((1, 64)), "fp8")[0] == 1 and np.isnan(oa.row_scale(np.full((1, 4), np.inf), "int8")[0])


@pytest.mark.parametrize("window", [0, 5])
def test_attention_against_a_masked_matrix_form(window):
    rng = np.random.default_rng(5)
    n, L, hq, hkv, d = 3, 11, 4, 2, 8
    q, k, v = rng.standard_normal((n, hq, d)), rng.standard_normal((L, hkv, d)), rng.standard_normal((L, hkv, d))
    out, lse = oa.attend(q, k, v, 0.3, window)
    kk, vv = np.repeat(k, 2, 1), np.repeat(v, 2, 1)
    s = np.einsum("nhd,lhd->hnl", q, kk) * 0.3
    pos = np.arange(L - n, L)[:, None]
    t = np.arange(L)[None]
    seen = (t <= pos) & ((t > pos - window) if window else True)
    e = np.where(seen, np.exp(s), 0.0)
    np.testing.assert_allclose(out, np.einsum("hnl,lhd->nhd", e / e.sum(-1, keepdims=True), vv), atol=1e-13)
    np.testing.assert_allclose(lse, np.log(e.sum(-1)).T, atol=1e-13)


def test_queries_before_the_cache_see_nothing():
    out, lse = oa.attend(np.ones((3, 1, 4)), np.ones((1, 1, 4)), np.ones((1, 1, 4)), 1.0)
    assert np.all(out[:2] == 0) and np.all(np.isneginf(lse[:2])) and np.all(out[2] == 1)
