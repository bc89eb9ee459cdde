"""GPU parity of paged attention against the FP64 oracle, within the bounds of
attention_common: every cache type, head size and grouping, lengths around the
tiles' ends, pages that end inside a tile, spans of several query tokens, windows,
free slots that hold NaN, data errors, streams, graphs and long pools."""
import numpy as np
import pytest
import torch

import gated_delta_rule_gateddeltanet_gb300 as gdn
from attention_common import Paged, check_attention, f64
from gpu_common import dev

pytestmark = pytest.mark.gpu

F16, BF16, F32, FP8, I8 = torch.float16, torch.bfloat16, torch.float32, torch.float8_e4m3fn, torch.int8
TYPES = [(F16, F16), (BF16, BF16), (F32, F32), (F16, FP8), (BF16, FP8), (F16, I8), (BF16, I8)]
EDGES = [1, 2, 15, 16, 17, 31, 33, 63, 64, 65, 127, 128, 129, 255, 257, 300]


def queries(tokens, heads, d, dtype, seed=1):
    g = torch.Generator("cpu").manual_seed(seed)
    return torch.randn(tokens, heads, d, generator=g).to(dtype).to(dev())


def run(p, group, io, *, spans=None, window=0, scale=0.0, seed=1, std=1.0, **kw):
    spans = [1] * len(p.lens) if spans is None else spans
    q = queries(sum(spans), p.heads * group, p.d, io, seed) * std
    cu = None
    if any(n != 1 for n in spans):
        cu = torch.tensor(np.concatenate([[0], np.cumsum(spans)]), dtype=torch.int32, device=dev())
    status = torch.zeros(1, dtype=torch.int32, device=dev())
    out, lse = gdn.paged_attention(q, p.cache, p.table, p.kv_lens, cu_seqlens=cu, window=window, scale=scale,
                                   return_lse=True, status=status, **kw)
    torch.cuda.synchronize()
    assert int(status) == 0
    check_attention(out, lse, q, p, spans, scale or p.d ** -0.5, window)
    return q, out, lse


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("io,kind", TYPES)
def test_types_and_head_sizes(io, kind, d):
    run(Paged(EDGES, 2, d, 16, kind, seed=d), 4, io)


@pytest.mark.parametrize("group", [1, 3, 7, 8, 9, 16, 20, 40])
@pytest.mark.parametrize("kind", [F16, I8, F32])
def test_groups(group, kind):
    io = kind if kind in (F16, F32) else BF16
    run(Paged([1, 16, 77, 200], 3, 64, 16, kind, seed=group), group, io)


@pytest.mark.parametrize("page", [1, 3, 5, 7, 8, 12, 16, 24, 32, 48, 64, 100, 128, 1000])
@pytest.mark.parametrize("kind,d", [(F16, 128), (FP8, 64), (I8, 128), (F32, 64)])
def test_page_sizes(page, kind, d):
    io = kind if kind in (F16, F32) else F16
    run(Paged([0, 1, page, page + 1, 2 * page - 1, 150], 2, d, page, kind, seed=page, extra_cols=2), 4, io)


@pytest.mark.parametrize("kind,d", [(BF16, 128), (FP8, 256), (I8, 64), (F32, 128)])
def test_heads_first_and_token_first_layouts_agree_bit_for_bit(kind, d):
    io = BF16 if kind in (FP8, I8) else kind
    outs = []
    for heads_first in (False, True):
        p = Paged([100, 37, 300], 2, d, 32, kind, seed=3, heads_first=heads_first)
        outs.append(run(p, 4, io)[1])
    assert torch.equal(outs[0], outs[1])


@pytest.mark.parametrize("kind", [F16, BF16, F32, FP8, I8])
@pytest.mark.parametrize("spans,lens", [
    ([4, 4, 4], [4, 100, 257]), ([2, 0, 5, 1], [40, 9, 5, 130]), ([8], [8]), ([3, 3], [1, 2]),  # (longer than the cache)
    ([17, 1], [300, 64]), ([40], [120]),
])
def test_spans(kind, spans, lens):
    io = F16 if kind in (FP8, I8) else kind
    run(Paged(lens, 2, 128, 16, kind, seed=len(spans)), 5, io, spans=spans)


@pytest.mark.parametrize("window", [1, 2, 16, 33, 100, 1000])
@pytest.mark.parametrize("spans", [[1, 1, 1, 1], [4, 1, 3, 2]])
def test_windows(window, spans):
    for kind, io in ((F16, F16), (I8, BF16)):
        run(Paged([10, 64, 130, 333], 2, 64, 16, kind, seed=window), 4, io, spans=spans, window=window)


def test_empty_sequences_give_zeros():
    p = Paged([0, 5, 0, 0], 2, 128, 16, F16)
    _, out, lse = run(p, 4, F16)
    assert torch.all(out[0] == 0) and torch.all(torch.isneginf(lse[2:]))


@pytest.mark.parametrize("scale", [0.02, 0.7])
def test_scales_and_peaked_scores(scale):
    """Scores whose running maximum keeps rising, and nearly flat ones."""
    p = Paged([2000], 1, 128, 16, F16, seed=9)
    p.cache.k *= torch.linspace(0.1, 3.0, p.cache.k.shape[0], device=dev())[:, None, None, None].half()
    run(p, 8, F16, scale=scale)


@pytest.mark.parametrize("kind,io", [(F16, F16), (BF16, BF16), (F32, F32), (I8, F16), (FP8, BF16)])
def test_long_sequences_split_over_the_gpu(kind, io):
    run(Paged([9000, 33], 2, 64, 64, kind, seed=4), 8, io)
    run(Paged([5000, 1, 4001], 1, 256, 16, kind, seed=5), 2, io, spans=[2, 1, 4])


def test_many_sequences():
    rng = np.random.default_rng(0)
    run(Paged(rng.integers(0, 60, 500).tolist(), 2, 64, 16, F16, seed=6), 4, F16)


@pytest.mark.parametrize("kind,d", [(F16, 64), (BF16, 128), (F16, 256), (FP8, 64), (FP8, 256), (I8, 128), (F32, 64), (F32, 256)])
@pytest.mark.parametrize("group,page", [(4, 16), (16, 5)])
def test_ragged_batches_through_the_rings(kind, d, group, page):
    """Segments of no, one and several tiles a warp in a row, in rings of every depth (8 and 16 query rows,
    8 to 32 bits), launched again before the first launch has ended: the same bits."""
    rng = np.random.default_rng(d + group)
    lens = np.where(rng.random(180) < 0.3, rng.integers(0, 3, 180), rng.integers(0, 700, 180)).tolist()
    p = Paged(lens, 1, d, page, kind, seed=d)
    io = BF16 if kind in (FP8, I8) else kind
    q = queries(180, group, d, io)
    outs = [gdn.paged_attention(q, p.cache, p.table, p.kv_lens) for _ in range(4)]
    assert all(torch.equal(o, outs[0]) for o in outs)
    run(p, group, io)


def test_masked_places_may_hold_anything():
    """Infinities and NaN in keys and values of drafted tokens stay out of the queries before them."""
    for kind in (F16, BF16, F32):
        p = Paged([50, 20], 2, 64, 16, kind, seed=7)
        for b, length in enumerate(p.lens):
            for t, (kx, vx) in ((length - 1, (float("nan"), float("inf"))), (length - 2, (float("inf"), float("-inf")))):
                page, off = int(p.table[b, t // 16]), t % 16
                p.cache.k[page, off] = kx
                p.cache.v[page, off, :, ::3] = vx
        q = queries(8, 8, 64, kind)
        cu = torch.tensor([0, 4, 8], dtype=torch.int32, device=dev())
        out = gdn.paged_attention(q, p.cache, p.table, p.kv_lens, cu_seqlens=cu)
        # the first two queries of each sequence see none of it: the same as without those tokens
        short = torch.tensor([x - 2 for x in p.lens], dtype=torch.int32, device=dev())
        want = gdn.paged_attention(torch.cat([q[:2], q[4:6]]), p.cache, p.table, short,
                                   cu_seqlens=torch.tensor([0, 2, 4], dtype=torch.int32, device=dev()))
        assert torch.isfinite(out[:2]).all() and torch.isfinite(out[4:6]).all()
        bound = 2.0 ** -10 if kind != BF16 else 2.0 ** -7  # (two evaluations of the same values)
        assert (torch.cat([out[:2], out[4:6]]).float() - want.float()).abs().max() <= bound * want.float().abs().max()
        assert not torch.isfinite(out[3]).any(dim=-1).all()  # the last one does see it


@pytest.mark.parametrize("kind", [FP8, I8])
def test_masked_rows_that_are_not_finite_in_8_bit_caches(kind):
    """A drafted token with an infinite key and a NaN value, written by the library: queries before it stay finite."""
    p = Paged([50, 20], 2, 64, 16, kind, seed=7)
    q = queries(8, 8, 64, F16)
    cu = torch.tensor([0, 4, 8], dtype=torch.int32, device=dev())
    want = gdn.paged_attention(q, p.cache, p.table, p.kv_lens, cu_seqlens=cu)
    k, v = torch.randn(2, 2, 64, device=dev()).half(), torch.randn(2, 2, 64, device=dev()).half()
    k[:, :, 3], v[:, :, 5] = float("inf"), float("nan")
    slots = torch.tensor([int(p.table[b, (n - 1) // 16]) * 16 + (n - 1) % 16 for b, n in enumerate(p.lens)],
                         dtype=torch.int32, device=dev())
    gdn.kv_cache_write(k, v, p.cache, slots)
    out = gdn.paged_attention(q, p.cache, p.table, p.kv_lens, cu_seqlens=cu)
    for b in (0, 4):
        assert torch.equal(out[b:b + 3], want[b:b + 3]) and torch.isnan(out[b + 3]).all()


def test_infinite_values_that_are_seen_show_in_their_channel():
    """As an infinity or NaN (weights are two-part numbers: one part may be zero), and there alone."""
    p = Paged([40], 1, 64, 16, F16, seed=8)
    page, off = int(p.table[0, 0]), 3
    p.cache.v[page, off, 0, 5] = float("inf")
    out = gdn.paged_attention(queries(1, 4, 64, F16), p.cache, p.table, p.kv_lens)
    assert not torch.isfinite(out[0, :, 5]).any()
    assert torch.isfinite(out[0, :, :5]).all() and torch.isfinite(out[0, :, 6:]).all()


def test_zero_and_tiny_scales():
    """Rows of zeros whose scale is 0, and rows with scales of very different size."""
    p = Paged([200], 2, 128, 16, I8, seed=10)
    page = int(p.table[0, 2])
    for x, s in ((p.cache.k, p.cache.k_scale), (p.cache.v, p.cache.v_scale)):
        x[page, 4:7] = 0
        s[page, 4:7] = 0
        s[int(p.table[0, 1])] *= 1e-12
    run(p, 4, F16)


def test_queries_as_a_slice_of_a_fused_projection_and_strided_tables():
    p = Paged([70, 20, 5], 2, 128, 16, F16, seed=11)
    fused = torch.randn(3, 8 * 128 + 4 * 128, device=dev()).half()
    q = fused[:, :8 * 128].view(3, 8, 128)
    wide = torch.full((3, 40), -9, dtype=torch.int32, device=dev())
    wide[:, 5:5 + p.table.shape[1]] = p.table
    got = gdn.paged_attention(q, p.cache, wide[:, 5:5 + p.table.shape[1]], p.kv_lens)
    assert torch.equal(got, gdn.paged_attention(q.contiguous(), p.cache, p.table, p.kv_lens))
    check_attention(got, None, q, p, [1, 1, 1], 128 ** -0.5)


def test_same_bits_every_time_and_any_workspace():
    p = Paged([3000, 10, 900], 2, 128, 16, BF16, seed=12)
    q = queries(3, 8, 128, BF16)
    ws = gdn.paged_attention_workspace(p.cache, 8, dtype=BF16)
    outs = []
    for fill in (0, 0xff, 0x7f):
        ws.fill_(fill)
        outs.append(gdn.paged_attention(q, p.cache, p.table, p.kv_lens, workspace=ws).clone())
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


def test_data_errors_are_flagged_and_skip_their_sequence():
    p = Paged([40, 50, 30], 2, 64, 16, F16, seed=13)
    q = queries(3, 8, 64, F16)
    good = gdn.paged_attention(q, p.cache, p.table, p.kv_lens)
    for bad in (-1, 4 * 16 + 1, 2 ** 31 - 1):
        lens = p.kv_lens.clone()
        lens[1] = bad
        status = torch.zeros(1, dtype=torch.int32, device=dev())
        out = torch.full_like(good, 7.0)
        gdn.paged_attention(q, p.cache, p.table, lens, output=out, status=status)
        assert int(status) == gdn.DEVERR["kv_len"]
        assert torch.equal(out[0], good[0]) and torch.equal(out[2], good[2]) and torch.all(out[1] == 7)
    cu = torch.tensor([0, 1, 9, 3], dtype=torch.int32, device=dev())  # the second and third spans are impossible
    status = torch.zeros(1, dtype=torch.int32, device=dev())
    out = torch.full_like(good, 7.0)
    gdn.paged_attention(q, p.cache, p.table, p.kv_lens, cu_seqlens=cu, output=out, status=status)
    assert int(status) == gdn.DEVERR["cu_seqlens"] and torch.equal(out[0], good[0]) and torch.all(out[1:] == 7)


@pytest.mark.parametrize("kind,page", [(F16, 16), (I8, 16), (F16, 7), (FP8, 5)])
@pytest.mark.parametrize("entry", [-1, 10 ** 6, 2 ** 31 - 1])
def test_bad_pages_read_as_zeros_and_are_flagged(kind, page, entry):
    p = Paged([40, 2 * page + 3], 2, 64, page, kind, seed=14)
    q = queries(2, 8, 64, F16)
    good = gdn.paged_attention(q, p.cache, p.table, p.kv_lens)
    table = p.table.clone()
    table[1, 1] = entry
    status = torch.zeros(1, dtype=torch.int32, device=dev())
    out = gdn.paged_attention(q, p.cache, table, p.kv_lens, status=status)
    assert int(status) == gdn.DEVERR["page"] and torch.equal(out[0], good[0]) and torch.isfinite(out[1]).all()


def test_other_streams():
    p = Paged([2000, 100], 2, 128, 16, F16, seed=15)
    q = queries(2, 8, 128, F16)
    want = gdn.paged_attention(q, p.cache, p.table, p.kv_lens)
    side = torch.cuda.Stream()
    call = gdn.PagedAttentionCall(q, p.cache, p.table, p.kv_lens)
    side.wait_stream(torch.cuda.current_stream())
    got = call.launch(side)
    side.synchronize()
    assert torch.equal(got, want)
    with torch.cuda.stream(side):
        got = gdn.paged_attention(q, p.cache, p.table, p.kv_lens)
    side.synchronize()
    assert torch.equal(got, want)


def test_a_captured_graph_follows_the_lengths():
    p = Paged([700, 700], 2, 128, 16, F16, seed=16)
    q = queries(2, 8, 128, F16)
    call = gdn.PagedAttentionCall(q, p.cache, p.table, p.kv_lens)
    call.launch()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call.launch()
    for lens in ([1, 700], [0, 16], [350, 351], [700, 700]):
        p.kv_lens.copy_(torch.tensor(lens, dtype=torch.int32))
        p.lens = lens
        g.replay()
        torch.cuda.synchronize()
        check_attention(call.outputs, None, q, p, [1, 1], 128 ** -0.5)


@pytest.mark.parametrize("page", [16, 10])
def test_offsets_past_32_bits(page):
    """A pool of more than 2^32 bytes a half, pages at its end."""
    heads, d = 8, 128
    pages = (1 << 32) // (page * heads * d) + 5
    cache = gdn.PagedKVCache.allocate(pages, page, heads, d, dtype=I8, device=dev())
    p = Paged([100, 17], heads, d, page, I8, seed=17)
    big = torch.full_like(p.table, pages - 1)
    at = pages - 1
    for b, n in enumerate(p.lens):
        for i in range((n + page - 1) // page):
            for x, y in ((cache.k, p.cache.k), (cache.v, p.cache.v), (cache.k_scale, p.cache.k_scale),
                         (cache.v_scale, p.cache.v_scale)):
                x[at] = y[int(p.table[b, i])]
            big[b, i] = at
            at -= 1
    q = queries(2, heads * 2, d, F16)
    assert torch.equal(gdn.paged_attention(q, cache, big, p.kv_lens), gdn.paged_attention(q, p.cache, p.table, p.kv_lens))


def test_no_sequences_and_no_tokens():
    p = Paged([4], 2, 64, 16, F16)
    e = torch.empty(0, dtype=torch.int32, device=dev())
    out = gdn.paged_attention(torch.empty(0, 8, 64, dtype=F16, device=dev()), p.cache, p.table[:0], e)
    assert out.shape == (0, 8, 64)
    cu = torch.zeros(2, dtype=torch.int32, device=dev())
    out = gdn.paged_attention(torch.empty(0, 8, 64, dtype=F16, device=dev()), p.cache, p.table, p.kv_lens, cu_seqlens=cu)
    assert out.shape == (0, 8, 64)


def test_random_sweep():
    rng = np.random.default_rng(20)
    for i in range(40):
        io, kind = TYPES[rng.integers(len(TYPES))]
        d = int(rng.choice([64, 128, 256]))
        seqs = int(rng.integers(1, 9))
        lens = rng.integers(0, int(rng.choice([20, 200, 1500])), seqs).tolist()
        spans = rng.integers(0, 6, seqs).tolist() if rng.random() < 0.5 else [1] * seqs
        if sum(spans) == 0:
            spans[0] = 1
        p = Paged(lens, int(rng.integers(1, 5)), d, int(rng.choice([4, 16, 20, 32, 64])), kind, seed=i,
                  heads_first=bool(rng.random() < 0.5))
        run(p, int(rng.integers(1, 12)), io, spans=spans, window=int(rng.choice([0, 0, 50])), seed=i,
            max_seqlen=int(rng.choice([0, max(spans)])))
