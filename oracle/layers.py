"""FP64 oracle of the gated linear recurrence and the root-mean-square norm, forward and
backward, with bounds on what FP32 arithmetic may lose (test infrastructure only).

Written token by token and row by row from the operators' formulas; shares no code
with the library.  Inputs are the values that the library was given, in 64 bits.

The bounds follow the error of each formula to first order, with u = 2^-24 (half a unit in
the last place of FP32, relative).  e^-|v| has a relative error of at most (2 |v| + 4) u: v is a
rounded sum, its product with log2(e) is rounded, each worth |v| u in the exponent, and the
base-2 exponential is good to 4 u.  The exponent of a decay, lg = -rate softplus(v), thus has one
of (2 |v| + 12) u (a polynomial of 2 u, two sums and products, rate to 4 u), g = e^lg one of |lg| times
that plus 5 u, a sigmoid of b one of (|b| + 8) u, sqrt(1 - g^2) that of lg plus 8 u.  A state's error obeys the state's own
recurrence: e_t = g e_(t-1) + (rel(g) + 4 u) g M_(t-1) + (rel(w) + 4 u) |w x|, with M the
recurrence of the magnitudes.  The 4 u cover the roundings of a step however the scan is
split: the product of decays, its use, and the sums of the parts.
"""
from __future__ import annotations

import numpy as np

U = 2.0 ** -24


def softplus(v):
    return np.maximum(v, 0.0) + np.log1p(np.exp(-np.abs(v)))


def sigmoid(v):
    e = np.exp(-np.abs(v))
    return np.where(v >= 0, 1.0, e) / (1.0 + e)


class Gates:
    """Decays g and input weights w of [T, C] gate inputs, and their relative errors."""

    def __init__(self, a, b, A_log=None, dt_bias=None, raw=True, unit=False):
        self.raw, self.unit, self.has_b = raw, unit, b is not None
        if not raw:
            self.g, self.w = a, np.ones_like(a) if b is None else b
            self.rel_g = self.rel_w = np.zeros_like(a)
            return
        self.rate, v = np.exp(A_log), a + dt_bias
        self.v = v
        self.sig_a = sigmoid(v)
        self.lg = -self.rate * softplus(v)
        self.g = np.exp(self.lg)
        self.sig_b = np.ones_like(a) if b is None else sigmoid(b)
        self.b = b
        self.factor = np.sqrt(-np.expm1(2 * self.lg)) if unit else np.ones_like(a)
        self.w = self.sig_b * self.factor
        self.rel_lg = (2 * np.abs(v) + 12) * U
        self.rel_g = np.abs(self.lg) * (self.rel_lg + 2 * U) + 5 * U
        self.rel_f = self.rel_lg + 8 * U if unit else np.zeros_like(a)
        self.rel_b = 0.0 if b is None else (np.abs(b) + 8) * U
        self.rel_w = self.rel_f + self.rel_b + U


def linear_recurrence(x, gates, spans, initial):
    """y [T, C], every sequence's last state [B, C], the states before each token, and the errors of y and
    of the last states.  spans: (begin, end) of each sequence; initial: [B, C]."""
    g, w = gates.g, gates.w
    h = np.zeros_like(x)
    before, err, err_before, mag_before = (np.zeros_like(x) for _ in range(4))
    final, final_err = initial.copy(), np.zeros_like(initial)
    for b, (lo, hi) in enumerate(spans):
        s, e, m = initial[b].copy(), np.zeros(x.shape[1]), np.abs(initial[b])
        for t in range(lo, hi):
            before[t], err_before[t], mag_before[t] = s, e, m
            u = w[t] * x[t]
            e = np.abs(g[t]) * (e + (gates.rel_g[t] + 4 * U) * m) + np.abs(u) * (gates.rel_w[t] + 4 * U)
            s = g[t] * s + u
            m = np.abs(g[t]) * m + np.abs(u)
            h[t], err[t] = s, e
        final[b], final_err[b] = s, e
    return h, final, before, err, final_err, err_before


def linear_recurrence_backward(x, gates, spans, before, err_before, dy, d_final):
    """{name: (gradient, error)} for dx, da, db, d_initial [B, C], dA_log, ddt_bias; d_final: [B, C]."""
    g, w = gates.g, gates.w
    lam, err = np.zeros_like(x), np.zeros_like(x)
    dinit, dinit_err = d_final.copy(), np.zeros_like(d_final)
    for b, (lo, hi) in enumerate(spans):
        m, e, mag = d_final[b].copy(), np.zeros(x.shape[1]), np.abs(d_final[b])
        for t in range(hi - 1, lo - 1, -1):
            lam[t] = dy[t] + m
            mag = mag + np.abs(dy[t])
            err[t] = e + 2 * U * mag
            m = g[t] * lam[t]
            e = np.abs(g[t]) * (err[t] + (gates.rel_g[t] + 4 * U) * mag)
            mag = np.abs(g[t]) * mag
        dinit[b], dinit_err[b] = m, e
    out = {"dx": (w * lam, np.abs(w) * err + np.abs(w * lam) * (gates.rel_w + 2 * U)), "d_initial": (dinit, dinit_err)}
    dg, dw = lam * before, lam * x
    dg_err = np.abs(lam) * err_before + np.abs(before) * err + np.abs(dg) * 2 * U
    dw_err = np.abs(x) * err + np.abs(dw) * 2 * U
    if not gates.raw:
        out["da"], out["db"] = (dg, dg_err), (dw, dw_err)
        return out
    dlg = dg * g
    dlg_err = np.abs(g) * dg_err + np.abs(dlg) * (gates.rel_g + 2 * U)
    if gates.unit:
        k = np.divide(gates.sig_b * g * g, gates.factor, out=np.zeros_like(g), where=gates.factor > 0)
        dlg_err = dlg_err + k * dw_err + np.abs(dw * k) * (2 * gates.rel_g + gates.rel_f + gates.rel_b + 8 * U)
        dlg = dlg - dw * k
    slope = gates.rate * gates.sig_a
    da = -dlg * slope
    da_err = dlg_err * slope + np.abs(da) * ((2 * np.abs(gates.v) + 16) * U)
    out["da"] = (da, da_err)
    if gates.has_b:
        s = gates.sig_b * sigmoid(-gates.b)
        db = dw * gates.factor * s
        # the sigmoid, and 1 less it as e^-b times it: each is relative, (|b| + 4) u the exponential's
        out["db"] = (db, gates.factor * s * dw_err + np.abs(db) * (gates.rel_f + 2 * gates.rel_b + (np.abs(gates.b) + 10) * U))
    dA = dlg * gates.lg
    dA_err = dlg_err * np.abs(gates.lg) + np.abs(dA) * (gates.rel_lg + 2 * U)
    own = np.zeros(x.shape[0], bool)
    for lo, hi in spans:
        own[lo:hi] = True
    adds = 128 + x.shape[0] / 64 + len(spans)  # roundings that a term goes through: in a tile, then over the tiles
    for name, v, e in (("dA_log", dA, dA_err), ("ddt_bias", da, da_err)):
        out[name] = (v[own].sum(0), e[own].sum(0) + adds * U * np.abs(v[own]).sum(0))
    return out


def silu(z):
    return z * sigmoid(z)


def rms_norm(s, eps, weight=None, gate=None):
    """y of rows s [.., d] and its error: the mean of the squares sums d positive terms (d / 128 + 64 of them one after
    another at most), silu's relative error is that of a sigmoid of |z|."""
    rstd = 1.0 / np.sqrt((s * s).mean(-1, keepdims=True) + eps)
    y, rel = s * rstd, (s.shape[-1] / 128 + 64) / 2 * U + 8 * U
    if weight is not None:
        y = y * weight
        rel = rel + 2 * U
    if gate is not None:
        y = y * silu(gate)
        rel = rel + (np.abs(gate) + 10) * U
    return y, np.abs(y) * rel


def rms_norm_backward(dy, s, eps, weight=None, gate=None, d_residual=None):
    """{name: (gradient, error)} for dx, dweight, dgate; rows [R, d]."""
    d = s.shape[-1]
    rstd = 1.0 / np.sqrt((s * s).mean(-1, keepdims=True) + eps)
    n, w = s * rstd, 1.0 if weight is None else weight
    rel = (d / 128 + 64) / 2 * U + 8 * U  # of rstd and n
    e, rel_e = dy, 0.0
    out = {}
    if gate is not None:
        sig = sigmoid(gate)
        e, rel_e = dy * gate * sig, (np.abs(gate) + 10) * U
        slope = sig * (1 + gate * (1 - sig))
        # the slope's terms: sig, and z (1 - sig) with the error of sig in 1 - sig
        slope_err = np.abs(slope) * (np.abs(gate) + 10) * U + sig * np.abs(gate) * ((np.abs(gate) + 10) * U + 2 * U)
        k = dy * n * w
        out["dgate"] = (k * slope, np.abs(k) * slope_err + np.abs(k * slope) * (rel + 4 * U))
    dn = e * w
    rel_dn = rel_e + 2 * U
    dot = (dn * n).mean(-1, keepdims=True)
    sums = (d / 128 + 64) * U
    dot_err = (np.abs(dn * n) * (rel_dn + rel + U)).mean(-1, keepdims=True) + sums * np.abs(dn * n).mean(-1, keepdims=True)
    dx = rstd * (dn - n * dot)
    err = rstd * (np.abs(dn) * (rel_dn + rel) + np.abs(n) * dot_err + np.abs(n * dot) * (2 * rel + 4 * U) + 2 * U * np.abs(dn)) + 2 * U * np.abs(dx)
    if d_residual is not None:
        dx = dx + d_residual
        err = err + U * np.abs(dx)
    out["dx"] = (dx, err)
    terms = (e * n).reshape(-1, d)
    rel_terms = np.broadcast_to(rel_e + rel + 2 * U, e.shape).reshape(-1, d)
    # a term is added to a running sum of its CTA's rows, those to one of the CTAs'
    adds = 32 + len(terms) / 16 + 64
    out["dweight"] = (terms.sum(0), (np.abs(terms) * rel_terms).sum(0) + adds * U * np.abs(terms).sum(0))
    return out
