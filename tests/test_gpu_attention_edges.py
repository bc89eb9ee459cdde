"""Paged attention at the edges of its inputs' ranges: NaN of every bit pattern,
infinities and values next to FP32's largest, windows past every length, scores
far below zero, pages outside the pool, rows of zeros among small 8-bit values,
tokens in no sequence, weights far below the largest."""
import numpy as np
import pytest
import torch

import gated_delta_rule_gateddeltanet_gb300 as gdn
from attention_common import Paged, check_attention, f64, rounding
from gpu_common import dev
from test_gpu_paged_attention import queries, run

pytestmark = pytest.mark.gpu

F16, BF16, F32, FP8, I8 = torch.float16, torch.bfloat16, torch.float32, torch.float8_e4m3fn, torch.int8


def bits(pattern):
    """The FP32 number with this bit pattern."""
    return torch.tensor([pattern - (1 << 32 if pattern >> 31 else 0)], dtype=torch.int32, device=dev()).view(F32)[0]


def slot(p, b, t):
    return int(p.table[b, t // p.page]), t % p.page


def cu_of(spans):
    return torch.tensor(np.concatenate([[0], np.cumsum(spans)]), dtype=torch.int32, device=dev())


NANS = [0x7fffffff, 0xffffffff, 0x7fc00000, 0xffc00000, 0x7f800001, 0xff801fff, 0x7ffff000]
INFS = [0x7f800000, 0xff800000]


@pytest.mark.parametrize("n", [1, 4])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("pattern", NANS + INFS)
def test_fp32_not_finite_where_it_is_seen(pattern, d, n):
    """In a query, a seen key and a seen value, alone in its head's rows or channel; one token and a span."""
    p = Paged([40, 21], 2, d, 16, F32, seed=d)
    q = queries(2 * n, 4, d, F32)
    cu = cu_of([n, n])
    call = lambda q: gdn.paged_attention(q, p.cache, p.table, p.kv_lens, cu_seqlens=cu)  # noqa: E731
    good = call(q)
    assert torch.isfinite(good).all()
    bad_q = q.clone()
    bad_q[n - 1, 2, 5] = bits(pattern)
    out = call(bad_q)  # one row of sequence 0
    # (an infinite query has scores of both signs, and the largest is infinite)
    assert torch.isnan(out[n - 1, 2]).all()
    out[n - 1, 2] = good[n - 1, 2]
    assert torch.equal(out, good)

    page, off = slot(p, 1, 9)
    keep = p.cache.k[page, off].clone()
    p.cache.k[page, off, 1, 7] = bits(pattern)
    out = call(q)  # key head 1, so query heads 2 and 3 of sequence 1
    for i in range(n, 2 * n):
        for h in (2, 3):
            if pattern in NANS or (float(q[i, h, 7]) > 0) == (pattern == 0x7f800000):
                assert torch.isnan(out[i, h]).all()
    out[n:, 2:] = good[n:, 2:]
    assert torch.equal(out, good)
    p.cache.k[page, off] = keep

    p.cache.v[page, off, 0, 3] = bits(pattern)
    out = call(q)
    seen = out[n:, :2, 3]
    assert torch.isnan(seen).all() if pattern in NANS else not torch.isfinite(seen).any()
    out[n:, :2, 3] = good[n:, :2, 3]
    assert torch.equal(out, good)


@pytest.mark.parametrize("d,page", [(64, 16), (128, 16), (256, 16), (64, 7)])
@pytest.mark.parametrize("pattern", NANS + INFS)
def test_fp32_not_finite_where_it_is_masked(pattern, d, page):
    """In the last drafted token's key and value: the queries before it do not see it, the last does."""
    p = Paged([40, 21], 2, d, page, F32, seed=d)
    q = queries(8, 4, d, F32)
    call = lambda: gdn.paged_attention(q, p.cache, p.table, p.kv_lens, cu_seqlens=cu_of([4, 4]))  # noqa: E731
    good = call()
    for b, length in enumerate(p.lens):
        at = slot(p, b, length - 1)
        p.cache.k[at][:, 2] = bits(pattern)
        p.cache.v[at][:, ::3] = bits(pattern)
    out = call()
    for b in (0, 4):
        # (a tile with such a value is added row by row, each row's values that it does not see as zeros)
        assert (out[b:b + 3] - good[b:b + 3]).abs().max() <= 2.0 ** -20 * good.abs().max()
        assert not torch.isfinite(out[b + 3, :, ::3]).any()


def test_fp32_a_nan_key_that_the_write_rotated():
    """What arithmetic on the GPU makes of a NaN is another pattern than the host's."""
    table = gdn.rotary_table(64, 64, device=dev())
    cache = gdn.PagedKVCache.allocate(4, 16, 1, 64, dtype=F32, device=dev())
    k, v = (torch.randn(20, 1, 64, device=dev()) for _ in range(2))
    k[3, 0, 5] = float("nan")
    pos = torch.arange(20, dtype=torch.int32, device=dev())
    gdn.kv_cache_write(k, v, cache, pos, positions=pos, table=table)
    out, lse = gdn.paged_attention(queries(1, 4, 64, F32), cache, torch.arange(4, dtype=torch.int32, device=dev())[None],
                                   torch.tensor([20], dtype=torch.int32, device=dev()), return_lse=True)
    assert torch.isnan(out).all() and torch.isnan(lse).all()


@pytest.mark.parametrize("pattern", [0x7f7fefff, 0x7f7ff000, 0x7f7ff800, 0xff7ff000, 0xff7ff800])
def test_fp32_values_next_to_the_largest(pattern):
    """Finite numbers that rounding to fewer bits would take to infinity.  A lone value comes back with the error of two
    TF32 parts (2^-21) and of the weight's and the quotient's roundings; the patterns stay clear of the largest by more."""
    p = Paged([1, 1], 1, 64, 16, F32)
    x = bits(pattern)
    p.cache.v[slot(p, 0, 0)][:, 5] = x
    out = gdn.paged_attention(queries(2, 4, 64, F32), p.cache, p.table, p.kv_lens)
    assert torch.isfinite(out).all()
    assert np.all(np.abs(f64(out[0, :, 5]) / f64(x) - 1) <= 2.0 ** -19)


@pytest.mark.parametrize("which", ["key", "query"])
@pytest.mark.parametrize("pattern", [0x7f7ff000, 0x7f7fffff, 0xff7ff800])
def test_fp32_products_with_numbers_next_to_the_largest(pattern, which):
    """One channel of a key (or query) next to 2^128 against small whole multiples of 2^-126: scores of a few units."""
    p = Paged([30], 1, 64, 16, F32, seed=2)
    rows = torch.arange(30, device=dev())
    at = (p.table[0].long()[rows // 16], rows % 16)
    p.cache.k[at] = 0
    big, small = bits(pattern), torch.tensor(2.0 ** -126, device=dev())
    q = torch.zeros(1, 4, 64, device=dev())
    steps = torch.arange(30, device=dev()) % 7 - 3
    if which == "key":
        p.cache.k[at[0][4], at[1][4], 0, 9] = big
        q[0, :, 9] = small * torch.tensor([1.0, -2.0, 3.0, 0.0], device=dev())
    else:
        q[0, 1, 9] = big
        p.cache.k[at[0], at[1], 0, 9] = small * steps
    out, lse = gdn.paged_attention(q, p.cache, p.table, p.kv_lens, scale=0.25, return_lse=True)
    check_attention(out, lse, q, p, [1], 0.25)


@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 2, 2 ** 31 - 40, 1 << 20])
@pytest.mark.parametrize("kind,io", [(F16, F16), (I8, BF16), (F32, F32)])
def test_windows_past_every_length(window, kind, io):
    """Spans longer than what is cached, so that queries stand at positions far below zero less the window."""
    run(Paged([3, 1, 40, 0], 2, 64, 16, kind, seed=5), 4, io, spans=[8, 45, 60, 7], window=window)


@pytest.mark.parametrize("kind,io", [(F32, F32), (BF16, BF16), (I8, BF16), (FP8, BF16)])
@pytest.mark.parametrize("length", [1, 20, 6000])
def test_scores_far_below_zero(kind, io, length):
    """Every score the same large negative number: the mean of the values, and that number as log-sum-exp."""
    p = Paged([length], 1, 128, 16, kind, seed=3)
    p.cache.k.view(torch.uint8)[:] = 0
    if kind in (I8, FP8):  # one channel of -64 times 2^100
        p.cache.k[..., 7] = torch.full(p.cache.k.shape[:3], -64.0, device=dev()).to(kind)
        p.cache.k_scale[p.cache.k_scale == p.cache.k_scale] = 2.0 ** 100
    else:
        p.cache.k[..., 7] = -2.0 ** 60
    q = torch.zeros(1, 4, 128, dtype=io, device=dev())
    q[..., 7] = 2.0 ** 47 if kind not in (I8, FP8) else 2.0
    scale = 1.0
    out, lse = gdn.paged_attention(q, p.cache, p.table, p.kv_lens, scale=scale, return_lse=True)
    v = p.rows(0)[1]
    want = v.mean(0)[0]
    # the weights are equal: 2^-22 and their own rounding each (2^-11 for the 8-bit types, 2^-16 for BF16), and the output's
    bound = 2 * (2.0 ** -22 + (2.0 ** -11 if kind in (I8, FP8) else 2.0 ** -16)) * np.abs(v).max() + rounding(want, io)
    assert np.all(np.abs(f64(out)[0] - want) <= bound)
    assert np.all(np.abs(f64(lse) / -2.0 ** 107 - 1) <= 2.0 ** -20)


@pytest.mark.parametrize("kind,page", [(F16, 16), (F16, 7), (BF16, 32), (F32, 16), (F32, 5), (FP8, 16), (FP8, 5), (I8, 16),
                                       (I8, 7), (I8, 64)])
@pytest.mark.parametrize("entry", [-1, 10 ** 6, -2 ** 31])
@pytest.mark.parametrize("spans", [[1, 1], [3, 2]])
def test_pages_outside_the_pool_are_rows_of_zeros(kind, page, entry, spans):
    """By value: the same as over a page of the pool that holds zeros."""
    p = Paged([40, 3 * page + 3], 2, 64, page, kind, seed=14)
    io = F16 if kind in (FP8, I8) else kind
    q = queries(sum(spans), 8, 64, io)
    table = p.table.clone()
    table[1, 1] = entry
    status = torch.zeros(1, dtype=torch.int32, device=dev())
    out, lse = gdn.paged_attention(q, p.cache, table, p.kv_lens, cu_seqlens=cu_of(spans), status=status, return_lse=True)
    assert int(status) == gdn.DEVERR["page"]
    zeros = next(i for i in range(p.cache.k.shape[0]) if i not in p.table.cpu().flatten().tolist())
    for x, s in ((p.cache.k, p.cache.k_scale), (p.cache.v, p.cache.v_scale)):
        x.view(torch.uint8)[zeros] = 0
        if s is not None:
            s[zeros] = 1
    p.table[1, 1] = zeros
    check_attention(out, lse, q, p, spans, 64 ** -0.5)


@pytest.mark.parametrize("kind", [FP8, I8])
@pytest.mark.parametrize("d,length,spans", [(64, 64, [1]), (128, 300, [4]), (256, 64, [1]), (128, 6000, [1]), (64, 40, [12])])
@pytest.mark.parametrize("rows", ["first", "last", "odd", "block", "all"])
def test_zero_rows_among_small_8_bit_values(kind, d, length, spans, rows):
    """A value row of zeros has scale 1, however small the scales of the others are: it must not cost them bits."""
    p = Paged([length], 2, d, 16, kind, seed=d, std=2.0 ** -28)
    p.cache.k_scale *= 2.0 ** 28
    t = torch.arange(length, device=dev())
    pick = {"first": t < 1, "last": t >= length - 1, "odd": t % 2 == 1, "block": (t >= 16) & (t < 40), "all": t >= 0}[rows]
    t = t[pick]
    at = (p.table[0].long()[t // 16], t % 16)
    p.cache.v.view(torch.uint8)[at] = 0
    p.cache.v_scale[at] = 1
    if kind == FP8:
        p.cache.v.view(torch.uint8)[at[0][::2], at[1][::2], :, 5] = 0x80  # minus zero
    run(p, 4, BF16, spans=spans)


def test_tokens_past_the_last_sequence_are_flagged():
    """As by the library's other packed operators; the sequences are computed."""
    p = Paged([40, 50], 2, 64, 16, F16, seed=13)
    q = queries(5, 8, 64, F16)
    good = gdn.paged_attention(q, p.cache, p.table, p.kv_lens, cu_seqlens=cu_of([2, 3]))
    status = torch.zeros(1, dtype=torch.int32, device=dev())
    out = torch.full((7, 8, 64), 7.0, dtype=F16, device=dev())
    more = torch.cat([q, q[:2]])
    gdn.paged_attention(more, p.cache, p.table, p.kv_lens, cu_seqlens=cu_of([2, 3]), output=out, status=status)
    assert int(status) == gdn.DEVERR["cu_seqlens"]
    assert torch.equal(out[:5], good) and torch.all(out[5:] == 7)


@pytest.mark.parametrize("kind,io", [(F16, F16), (BF16, BF16), (F32, F32), (I8, F16), (FP8, BF16)])
@pytest.mark.parametrize("above", [10.0, 15.0, 17.0, 20.0, 24.0])
def test_one_score_far_above_many_equal_ones(kind, io, above):
    """A first token whose value is zero takes nearly all of the weight of 100,000 others, whose values are one: what
    is left for them is their weights' sum, with the error that each may have (relative, and 2^-31 of the largest
    weight as an FP16 number)."""
    n = 100000
    p = Paged([n], 1, 64, 64, kind, seed=1)
    p.cache.k.view(torch.uint8)[:] = 0
    p.cache.v.copy_(torch.ones(p.cache.v.shape, device=dev()).to(kind))
    if p.cache.k_scale is not None:
        p.cache.k_scale.fill_(0.5), p.cache.v_scale.fill_(1.0)
    at = slot(p, 0, 0)
    p.cache.v.view(torch.uint8)[at] = 0
    p.cache.k[at[0], at[1], 0, 3] = torch.tensor(16.0, device=dev()).to(kind)
    q = torch.zeros(1, 4, 64, dtype=io, device=dev())
    q[..., 3] = above / 8 if p.cache.k_scale is not None else above / 16
    out, lse = gdn.paged_attention(q, p.cache, p.table, p.kv_lens, scale=1.0, return_lse=True)
    share = (n - 1) * np.exp(-above)
    want = share / (1 + share)
    relative = {F16: 2.0 ** -21, BF16: 2.0 ** -16, F32: 2.0 ** -20, I8: 2.0 ** -11, FP8: 2.0 ** -11}[kind]
    floor = 0.0 if kind in (BF16, F32) else (n - 1) * 2.0 ** -31
    # 2^-20: 2^-22 of each numerator and of their FP32 sum's parts, in the numerator and the denominator
    bound = want * (relative + 2.0 ** -20) + floor + rounding(want, io)
    assert np.all(np.abs(f64(out) - want) <= bound)
    assert np.all(np.abs(f64(lse) - (above + np.log1p(share))) <= 2.0 ** -18)
