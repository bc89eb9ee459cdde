"""Helpers of the softmax-attention GPU tests: paged caches with known contents
and the bounds their results are held to.

Bounds (u = half a unit in the last place, relative: FP32 2^-24, FP16 2^-11,
BF16 2^-8 of the value's binade, taken as |y| 2^-11 and |y| 2^-8; FP16 has an
absolute floor of 2^-25 below its normal range):
  rotation   each of two products and their sum is rounded in FP32: error at
             most 2^-23 (|a c| + |b s|) before the result's own rounding.
  attention  a weight's relative error is at most ln 2 times the absolute error
             of its base-2 score, plus 2^-22 for the exponential and the
             rounding of the weight itself (2^-16 as two BF16 numbers, 2^-21 as two FP16 or
             TF32 ones, 2^-11 as one FP16 number over 8-bit values).  A score of
             magnitude at most A = scale sum |q k| (all in base 2: A / ln 2) is a sum of
             d exact products whose FP32 accumulation loses at most 2^-21 of A (the
             tensor cores align each instruction's addends before they round), FP32
             inputs 2^-20 for their split.  An output is a weighted mean of values, so its
             error is at most twice the weights' error times max |v|, plus its rounding.
"""
import numpy as np
import torch

import gated_delta_rule_gateddeltanet_gb300 as gdn
from gpu_common import dev
from oracle import attention as oa

HALF_ULP = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
WEIGHT = {torch.float32: 2.0 ** -21, torch.float16: 2.0 ** -21, torch.bfloat16: 2.0 ** -16, torch.int8: 2.0 ** -11,
          torch.float8_e4m3fn: 2.0 ** -11}


def rounding(y, dtype):
    """The most that rounding y to dtype changes it."""
    return np.abs(y) * HALF_ULP[dtype] + 2.0 ** (-25 if dtype == torch.float16 else -126)


def f64(t):
    return t.detach().to(torch.float32).double().cpu().numpy()


def values(cache):
    """The numbers a cache holds, [pages, page, heads, d], for k and v."""
    out = []
    for x, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)):
        y = x.to(torch.float32)
        out.append((y if s is None else y * s[..., None]).double().cpu().numpy())
    return out


class Paged:
    """Sequences of the given lengths in a shuffled pool whose free slots hold NaN (0x7f bytes where
    the type has none), with the values every sequence reads back."""

    def __init__(self, lens, heads, d, page, dtype, *, seed=0, heads_first=False, spare=3, std=1.0, extra_cols=0):
        g = torch.Generator("cpu").manual_seed(seed)
        self.lens, self.page, self.heads, self.d = list(lens), page, heads, d
        need = [(n + page - 1) // page for n in lens]
        pages = sum(need) + spare
        order = torch.randperm(pages, generator=g).tolist()
        width = max(1, max(need)) + extra_cols
        table = torch.full((len(lens), width), -7, dtype=torch.int32)
        self.cache = gdn.PagedKVCache.allocate(pages, page, heads, d, dtype=dtype, device=dev(), heads_first=heads_first)
        used = torch.zeros(pages, page, dtype=torch.bool)
        for b, n in enumerate(lens):
            for i in range(need[b]):
                p = order.pop()
                table[b, i] = p
                used[p, :min(page, n - i * page)] = True
        for x, s in ((self.cache.k, self.cache.k_scale), (self.cache.v, self.cache.v_scale)):
            r = torch.randn(pages, page, heads, d, generator=g) * std
            if s is not None:
                r = r * torch.exp2(torch.randint(-6, 7, (pages, page, heads, 1), generator=g).float())
                top = r.abs().amax(-1)
                scale = top / 127 if dtype == torch.int8 else torch.exp2(torch.ceil(torch.log2(top / 448)))
                q = r / scale[..., None]
                r = q.round().clamp(-127, 127).to(torch.int8) if dtype == torch.int8 else q.to(dtype)
                scale[~used] = float("nan")
                s.copy_(scale)
                r.view(torch.uint8)[~used] = 0x7f
            else:
                r[~used] = float("nan")
            x.view(torch.uint8).copy_(r.view(torch.uint8)) if s is not None else x.copy_(r)
        self.table = table.to(dev())
        self.kv_lens = torch.tensor(lens, dtype=torch.int32, device=dev())

    def rows(self, b):
        """Sequence b's keys and values in 64 bits, [len, heads, d]."""
        k, v = values(self.cache)
        t = np.arange(self.lens[b])
        at = (self.table[b].cpu().numpy()[t // self.page], t % self.page)
        return k[at], v[at]


def check_attention(out, lse, q, paged, spans, scale, window=0, dtype=None):
    """Every sequence's outputs against the oracle, within the module's bound."""
    dtype = dtype or out.dtype
    k_all, v_all = values(paged.cache)
    out, q = f64(out), f64(q)
    lse = None if lse is None else f64(lse)
    at = 0
    kind = paged.cache.k.dtype
    for b, n in enumerate(spans):
        t = np.arange(paged.lens[b])
        where = (paged.table[b].cpu().numpy()[t // paged.page], t % paged.page)
        k, v = k_all[where], v_all[where]
        want, want_lse = oa.attend(q[at:at + n], k, v, scale, window)
        if n and len(t):
            kk = np.repeat(np.abs(k), q.shape[1] // k.shape[1], 1)
            most = scale * np.einsum("nhd,lhd->nhl", np.abs(q[at:at + n]), kk).max()
            score = most * 2.0 ** (-20 if kind == torch.float32 else -21)
            weight = score + 2.0 ** -22 + WEIGHT[kind]
            bound = 2 * weight * np.abs(v).max() + rounding(want, dtype)
            got = out[at:at + n]
            assert np.all(np.isfinite(got)), f"sequence {b}"
            worst = np.max(np.abs(got - want) - bound)
            assert worst <= 0, f"sequence {b}: {worst} over the bound ({np.abs(got - want).max()} of {np.abs(want).max()})"
            if lse is not None:
                seen = np.isfinite(want_lse)
                assert np.array_equal(seen, np.isfinite(lse[at:at + n]))
                tol = score + 2.0 ** -20 + np.abs(want_lse[seen]) * 2.0 ** -22
                assert np.all(np.abs(lse[at:at + n][seen] - want_lse[seen]) <= tol)
        elif n:
            assert np.all(out[at:at + n] == 0)
            if lse is not None:
                assert np.all(np.isneginf(lse[at:at + n]))
        at += n
