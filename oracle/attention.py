"""FP64 restatement of the softmax-attention operators (numpy, from their
definitions in include/gdn.h): rotary tables and rotation, 8-bit cache rows, and
attention of each sequence's newest tokens over its cached rows."""
from __future__ import annotations

import math

import numpy as np


def rotary_frequencies(rotary_dim, base=10000.0, scaling="none", factor=1.0, original_positions=0, beta_fast=32.0,
                       beta_slow=1.0):
    """The pairs' angular frequencies and the magnitude of cos and sin."""
    i = np.arange(rotary_dim // 2, dtype=np.float64)
    if scaling == "ntk":
        base = base * factor ** (rotary_dim / (rotary_dim - 2))
    w = base ** (-2 * i / rotary_dim)
    if scaling == "linear":
        return w / factor, 1.0
    if scaling == "by_parts":
        turns = original_positions * w / (2 * math.pi)
        keep = np.clip((turns - beta_slow) / (beta_fast - beta_slow), 0, 1)
        return w * keep + w / factor * (1 - keep), 1.0
    if scaling == "yarn":
        at = lambda turns: rotary_dim * math.log(original_positions / (2 * math.pi * turns)) / (2 * math.log(base))  # noqa: E731
        lo = min(max(math.floor(at(beta_fast)), 0), rotary_dim - 1)
        hi = min(max(math.ceil(at(beta_slow)), 0), rotary_dim - 1)
        keep = 1 - np.clip((i - lo) / (hi - lo if hi > lo else 0.001), 0, 1)
        return w * keep + w / factor * (1 - keep), 0.1 * math.log(factor) + 1
    return w, 1.0


def rotary_table(positions, rotary_dim, attention_factor=0.0, **kw):
    """cos | sin, [positions, rotary_dim]."""
    w, m = rotary_frequencies(rotary_dim, **kw)
    angle = np.arange(positions, dtype=np.float64)[:, None] * w
    return np.concatenate([np.cos(angle), np.sin(angle)], 1) * (attention_factor or m)


def rotate(x, positions, table, interleaved=False, inverse=False):
    """x [T, heads, d] with its first rotary_dim channels turned."""
    x = np.asarray(x, dtype=np.float64)
    r = table.shape[1]
    row = np.asarray(table, dtype=np.float64)[positions][:, None]
    c, s = row[..., :r // 2], row[..., r // 2:] * (-1 if inverse else 1)
    y = x.copy()
    one, two = (slice(0, r, 2), slice(1, r, 2)) if interleaved else (slice(0, r // 2), slice(r // 2, r))
    y[..., one] = x[..., one] * c - x[..., two] * s
    y[..., two] = x[..., two] * c + x[..., one] * s
    return y


def row_scale(x, kind):
    """The scale of each row of x (last axis) for an "int8" or "fp8" cache (before rounding to FP32)."""
    top = np.abs(np.asarray(x, dtype=np.float64)).max(-1)
    if kind == "int8":
        scale = top / 127
    else:
        scale = np.exp2(np.maximum(np.ceil(np.log2(np.maximum(top, 1e-300) / 448)), -120))
    return np.where(np.isfinite(top), np.where(top > 0, scale, 1.0), np.nan)


def attend(q, k, v, scale, window=0):
    """q [n, Hq, d]: a sequence's newest n tokens; k, v [L, Hkv, d]: all it has
    cached.  Returns (out [n, Hq, d], lse [n, Hq])."""
    n, hq, d = q.shape
    length, hkv = k.shape[:2]
    out, lse = np.zeros((n, hq, d)), np.full((n, hq), -np.inf)
    for i in range(n):
        pos = length - n + i
        lo = max(0, pos - window + 1) if window else 0
        if pos < 0:
            continue
        for h in range(hq):
            kk, vv = k[lo:pos + 1, h // (hq // hkv)], v[lo:pos + 1, h // (hq // hkv)]
            with np.errstate(invalid="ignore"):
                s = kk @ q[i, h] * scale
                m = s.max()
                p = np.exp(s - m)
                out[i, h] = (p[:, None] * vv).sum(0) / p.sum()
                lse[i, h] = m + np.log(p.sum())
    return out, lse
