"""GPU parity of the paged cache's write (rotation, quantisation) and read back
against the FP64 oracle."""
import numpy as np
import pytest
import torch

import gated_delta_rule_gateddeltanet_gb300 as gdn
from attention_common import f64, rounding, values
from gpu_common import dev
from oracle import attention as oa

pytestmark = pytest.mark.gpu

F16, BF16, F32, FP8, I8 = torch.float16, torch.bfloat16, torch.float32, torch.float8_e4m3fn, torch.int8
TYPES = [(io, kind) for io in (F16, BF16, F32) for kind in (io, FP8, I8)]


def make(T, heads, d, io, kind, page, *, heads_first=False, seed=0, spare=5):
    g = torch.Generator("cpu").manual_seed(seed)
    pages = (T + page - 1) // page + spare
    cache = gdn.PagedKVCache.allocate(pages, page, heads, d, dtype=kind, device=dev(), heads_first=heads_first)
    for x in (cache.k, cache.v):
        x.view(torch.uint8).fill_(0x55) if kind in (FP8, I8) else x.fill_(-3)
    slots = torch.randperm(pages * page, generator=g)[:T].to(torch.int32).to(dev())
    size = torch.exp2(torch.randint(-4, 5, (T, heads, 1), generator=g).float())
    k, v = ((torch.randn(T, heads, d, generator=g) * size).to(io).to(dev()) for _ in range(2))
    return cache, slots, k, v


def check_rows(cache, half, slots, x, slack=0.0):
    """The cache's rows at `slots` hold x (64 bits; `slack`: an absolute error x may have had before it was stored)."""
    page = cache.k.shape[1]
    s = slots.cpu().numpy()
    got = values(cache)[half == "v"][s // page, s % page]
    kind = cache.k.dtype
    if kind in (FP8, I8):
        scale = f64((cache.v_scale if half == "v" else cache.k_scale)[slots.long() // page, slots.long() % page])
        top = np.abs(x).max(-1)
        if kind == I8:
            np.testing.assert_allclose(scale, oa.row_scale(x, "int8"), rtol=2.0 ** -22 + slack / max(top.min(), 1e-30))
            bound = scale[..., None] * (0.5 + 1e-4)
        else:
            want = oa.row_scale(x, "fp8")
            near = np.abs(top / want - 448) <= 1 + slack  # (a row whose top is 448 scale up to rounding may go either way)
            assert np.all((scale == want) | near)
            q = np.abs(x) / scale[..., None]
            step = np.exp2(np.floor(np.log2(np.maximum(q, 2.0 ** -6))) - 3)
            bound = scale[..., None] * step * (0.5 + 1e-4)
    else:
        bound = rounding(x, kind) * (1 + 2.0 ** -10)
    assert np.all(np.abs(got - x) <= bound + slack)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("io,kind", TYPES)
def test_write_without_rotation(io, kind, d):
    for T, page, hf in ((1, 16, False), (45, 7, True), (130, 64, False)):
        cache, slots, k, v = make(T, 3, d, io, kind, page, heads_first=hf, seed=T)
        gdn.kv_cache_write(k, v, cache, slots)
        torch.cuda.synchronize()
        check_rows(cache, "k", slots, f64(k))
        check_rows(cache, "v", slots, f64(v))
        if kind == io:  # as they are: bit for bit, and nothing else is written
            at = (slots.long() // page, slots.long() % page)
            assert torch.equal(cache.k[at], k) and torch.equal(cache.v[at], v)
            cache.k[at] = -3
            assert torch.all(cache.k == -3)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("io,kind", TYPES)
@pytest.mark.parametrize("d,r", [(128, 128), (256, 64), (64, 16)])
def test_write_with_rotation(io, kind, interleaved, d, r):
    T, page = 33, 16
    cache, slots, k, v = make(T, 2, d, io, kind, page, seed=r)
    q = torch.randn(T, 6, d, device=dev()).to(io)
    pos = torch.randint(0, 300, (T,), dtype=torch.int32, device=dev())
    table = gdn.rotary_table(300, r, device=dev())
    q_out = gdn.kv_cache_write(k, v, cache, slots, positions=pos, table=table, interleaved=interleaved, q=q)
    torch.cuda.synchronize()
    want = oa.rotate(f64(k), pos.cpu().numpy(), f64(table), interleaved)
    check_rows(cache, "k", slots, want, slack=2.0 ** -22 * np.abs(f64(k)).max())
    check_rows(cache, "v", slots, f64(v))
    a, b = gdn.rotary(q, k, pos, table, interleaved=interleaved)  # the same rotation, bit for bit
    assert torch.equal(q_out, a)
    if kind == io:
        assert torch.equal(cache.k[slots.long() // page, slots.long() % page], b)
    q2 = q.clone()
    gdn.kv_cache_write(k, v, cache, slots, positions=pos, table=table, interleaved=interleaved, q=q2, q_out=q2)
    assert torch.equal(q2, a)


def test_strided_inputs_and_interleaved_halves_of_one_tensor():
    T, hk, hq, d = 20, 2, 4, 128
    fused = torch.randn(T, (hq + 2 * hk) * d, device=dev()).half()
    q, k, v = (fused[:, a * d:b * d].view(T, -1, d) for a, b in ((0, hq), (hq, hq + hk), (hq + hk, hq + 2 * hk)))
    both = torch.zeros(4, 2, 16, hk, d, dtype=F16, device=dev())
    cache = gdn.PagedKVCache(both[:, 0], both[:, 1])
    slots = torch.randperm(64, device=dev())[:T].to(torch.int32)
    gdn.kv_cache_write(k, v, cache, slots)
    at = (slots.long() // 16, slots.long() % 16)
    assert torch.equal(cache.k[at], k) and torch.equal(cache.v[at], v)
    table = gdn.rotary_table(50, 64, device=dev())
    pos = torch.arange(T, dtype=torch.int32, device=dev())
    assert torch.equal(gdn.kv_cache_write(k, v, cache, slots, positions=pos, table=table, q=q),
                       gdn.rotary(q, None, pos, table)[0])


@pytest.mark.parametrize("kind", [FP8, I8])
def test_special_rows(kind):
    """Zeros (scale 1), rows with an infinity or NaN (scale NaN: they read back as NaN), very small and very large ones."""
    cache, slots, k, v = make(8, 1, 64, F32, kind, 16)
    k[0] = 0
    k[1, 0, 7] = float("nan")
    k[2, 0, 9] = float("inf")
    k[3] = torch.randn(1, 64, device=dev()) * 1e-30
    k[4] = torch.randn(1, 64, device=dev()) * 1e30
    k[5] = 448.0
    k[6] = 1e-45
    gdn.kv_cache_write(k, v, cache, slots)
    torch.cuda.synchronize()
    at = (slots.long() // 16, slots.long() % 16)
    scale, got = f64(cache.k_scale[at])[:, 0], values(cache)[0][at[0].cpu().numpy(), at[1].cpu().numpy()][:, 0]
    assert scale[0] == 1 and np.all(got[0] == 0)
    assert np.all(np.isnan(got[1:3])) and np.all(np.isnan(scale[1:3]))
    for i in (4, 5, 7):
        x = f64(k)[i]
        assert np.abs(got[i] - x).max() <= np.abs(x).max() * (0.5 / 127 + 1e-6 if kind == I8 else 2.0 ** -4)
    assert np.abs(got[3] - f64(k)[3]).max() <= 1.1e-30 * (1 if kind == I8 else 4)  # (e4m3's scale stops at 2^-120)
    assert np.abs(got[6]).max() <= 2e-45 or kind == FP8
    if kind == FP8:
        assert scale[5] == 1 and np.all(got[5] == 448)


def test_skipped_and_bad_slots_and_positions():
    T = 6
    cache, slots, k, v = make(T, 2, 64, F16, F16, 16)
    table = gdn.rotary_table(40, 64, device=dev())
    pos = torch.tensor([0, 1, 2, 3, 40, 5], dtype=torch.int32, device=dev())
    q = torch.randn(T, 2, 64, device=dev()).half()
    total = cache.k.shape[0] * 16
    s = slots.clone()
    s[1], s[2], s[3] = -1, total, -2
    status = torch.zeros(1, dtype=torch.int32, device=dev())
    q_out = torch.full_like(q, 9.0)
    gdn.kv_cache_write(k, v, cache, s, positions=pos, table=table, q=q, q_out=q_out, status=status)
    torch.cuda.synchronize()
    assert int(status) == gdn.DEVERR["cache_slot"] | gdn.DEVERR["position"]
    want = gdn.rotary(q, None, torch.tensor([0, 1, 2, 3, 4, 5], dtype=torch.int32, device=dev()), table)[0]
    for i, written in enumerate([True, True, False, False, False, True]):  # (slot -1: the query is still rotated)
        assert torch.equal(q_out[i], want[i]) if written else torch.all(q_out[i] == 9)
    at = [(int(x) // 16, int(x) % 16) for x in slots.tolist()]
    for i in (1, 2, 3, 4):
        assert torch.all(cache.v[at[i]] == -3)
    for i in (0, 5):
        assert torch.equal(cache.v[at[i]], v[i])
    status.zero_()
    gdn.kv_cache_write(k, v, cache, torch.full_like(slots, -1), status=status)
    assert int(status) == 0


@pytest.mark.parametrize("kind", [F16, BF16, F32, FP8, I8])
@pytest.mark.parametrize("out", [F16, BF16, F32])
def test_read_back(kind, out):
    for page, d, hf, lens in ((16, 128, False, [0, 1, 40, 16]), (7, 64, True, [13, 0, 0, 50]), (64, 256, False, [200])):
        T, heads = sum(lens), 3
        io = kind if kind in (F16, BF16, F32) else F32
        pages = sum((n + page - 1) // page for n in lens)
        cache = gdn.PagedKVCache.allocate(pages + 2, page, heads, d, dtype=kind, device=dev(), heads_first=hf)
        order, width = torch.randperm(pages + 2).tolist(), max(1, max((n + page - 1) // page for n in lens)) + 1
        table = torch.full((len(lens), width), -1, dtype=torch.int32)
        slots = []
        for b, n in enumerate(lens):
            for i in range((n + page - 1) // page):
                table[b, i] = order.pop()
            slots += [int(table[b, t // page]) * page + t % page for t in range(n)]
        k, v = (torch.randn(T, heads, d, device=dev()).to(io) for _ in range(2))
        s = torch.tensor(slots, dtype=torch.int32, device=dev())
        gdn.kv_cache_write(k, v, cache, s)
        cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device=dev())
        status = torch.zeros(1, dtype=torch.int32, device=dev())
        a, b = gdn.kv_cache_read(cache, table.to(dev()), cu, T, dtype=out, status=status)
        torch.cuda.synchronize()
        assert int(status) == 0 and a.dtype == out and a.shape == (T, heads, d)
        held = values(cache)
        at = (s.cpu().numpy() // page, s.cpu().numpy() % page)
        for got, want in ((a, held[0][at]), (b, held[1][at])):
            # a product of an 8-bit value and its scale, rounded in FP32 and then to the output's type
            assert np.all(np.abs(f64(got) - want) <= rounding(want, out) * (1 + 2.0 ** -10) + np.abs(want) * 2.0 ** -24)


def test_read_back_flags_bad_pages_and_offsets():
    cache, slots, k, v = make(40, 2, 64, F16, F16, 16, spare=0)
    table = torch.tensor([[0, 99], [1, 2]], dtype=torch.int32, device=dev())
    cu = torch.tensor([0, 20, 40], dtype=torch.int32, device=dev())
    status = torch.zeros(1, dtype=torch.int32, device=dev())
    a, _ = gdn.kv_cache_read(cache, table, cu, 40, status=status)
    assert int(status) == gdn.DEVERR["page"] and torch.all(a[16:20] == 0) and torch.equal(a[20:36], cache.k[1])
    status.zero_()
    out = torch.full((60, 2, 64), 4.0, dtype=F16, device=dev())
    gdn.kv_cache_read(cache, table, torch.tensor([0, 10, 50], dtype=torch.int32, device=dev()), 60, k_out=out,
                      v_out=out.clone(), status=status)  # 40 tokens of two pages, and ten tokens of nobody
    assert int(status) == gdn.DEVERR["cu_seqlens"] and torch.equal(out[10:26], cache.k[1]) and torch.all(out[42:] == 4)


def test_offsets_past_32_bits():
    page, heads, d = 16, 8, 128
    pages = (1 << 32) // (page * heads * d) + 3
    cache = gdn.PagedKVCache.allocate(pages, page, heads, d, dtype=I8, device=dev())
    k, v = (torch.randn(5, heads, d, device=dev()) for _ in range(2))
    slots = torch.tensor([pages * page - 1 - 17 * i for i in range(5)], dtype=torch.int32, device=dev())
    gdn.kv_cache_write(k, v, cache, slots)
    table = (slots // page).view(5, 1).contiguous()
    at = (slots.long() // page, slots.long() % page)
    assert (cache.v[at].float() * cache.v_scale[at][..., None] - v).abs().max() <= v.abs().max() / 253
    cu = torch.tensor([0, 16, 32], dtype=torch.int32, device=dev())
    a, _ = gdn.kv_cache_read(cache, table[:2].contiguous(), cu, 32, dtype=F32)
    assert torch.equal(a[int(slots[0]) % page], cache.k[at][0].float() * cache.k_scale[at][0][..., None])


def test_no_tokens():
    cache, slots, k, v = make(4, 2, 64, F16, I8, 16)
    assert gdn.kv_cache_write(k[:0], v[:0], cache, slots[:0]) is None
    cu = torch.zeros(3, dtype=torch.int32, device=dev())
    a, b = gdn.kv_cache_read(cache, torch.zeros(2, 1, dtype=torch.int32, device=dev()), cu, 0)
    assert a.shape == (0, 2, 64) and a.dtype == F16


@pytest.mark.parametrize("size", [2.0 ** -140, 2.0 ** -90, 1.0, 2.0 ** 90])
def test_int8_rows_near_the_middle_of_two_integers(size):
    """FP32 rows of one channel 127 s and the others within three units in the last place of (n + 1/2) s:
    the stored integer is the FP32 quotient x / scale rounded to even, at subnormal scales too."""
    rng = np.random.default_rng(int(abs(np.log2(size))))
    T, d, page = 96, 64, 16
    top = (rng.random((T, 1)) + 0.5).astype(np.float64) * size
    x = ((rng.integers(-126, 126, (T, d)) + 0.5) * top / 127).astype(np.float32)
    x = (x.view(np.int32) + rng.integers(-3, 4, (T, d)).astype(np.int32)).view(np.float32)
    x[:, 5] = top[:, 0]
    cache = gdn.PagedKVCache.allocate(T // page, page, 1, d, dtype=I8, device=dev())
    k = torch.from_numpy(x).to(dev()).view(T, 1, d)
    gdn.kv_cache_write(k, k, cache, torch.arange(T, dtype=torch.int32, device=dev()))
    largest = np.abs(x).max(-1, keepdims=True)
    scale = largest / np.float32(127)
    # (bit patterns stepped below the smallest subnormal are NaN: such rows have a NaN scale, their integers mean nothing)
    finite = np.isfinite(x).all(-1)
    want = np.clip(np.rint(x[finite] / scale[finite]), -127, 127).astype(np.int8)
    got_scale = cache.k_scale.cpu().numpy().reshape(T, 1)
    assert scale.dtype == np.float32 and np.array_equal(got_scale, scale, equal_nan=True)
    assert np.array_equal(cache.k.cpu().numpy().reshape(T, d)[finite], want)


def test_read_back_of_many_short_and_empty_sequences():
    """Sequences of zero to three tokens, more of them than a warp probes at once, some empty at both ends."""
    lens = [0, 0] + [(7 * i) % 4 for i in range(1500)] + [0]
    T, page, B = sum(lens), 2, len(lens)
    for heads, d in ((1, 64), (3, 256)):
        pages = B * 2
        cache = gdn.PagedKVCache.allocate(pages, page, heads, d, dtype=F16, device=dev())
        cache.k.copy_(torch.randn(cache.k.shape, device=dev()))
        cache.v.copy_(torch.randn(cache.v.shape, device=dev()))
        table = torch.randperm(pages, device=dev()).view(B, 2).to(torch.int32)
        cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32).to(dev())
        k, v = gdn.kv_cache_read(cache, table, cu, T)
        seq = torch.repeat_interleave(torch.arange(B), torch.tensor(lens)).to(dev())
        pos = torch.arange(T, device=dev()) - cu[seq].long()
        at = (table[seq, pos // page].long(), pos % page)
        assert torch.equal(k, cache.k[at]) and torch.equal(v, cache.v[at])


@pytest.mark.parametrize("kind", [F16, I8])
def test_read_back_of_long_contexts(kind):
    """Enough tokens that a warp takes several (one narrow head), with a last warp that is not full."""
    T, page, d = 40001, 16, 64
    cache = gdn.PagedKVCache.allocate(T // page + 1, page, 1, d, dtype=kind, device=dev())
    x = torch.randn(T, 1, d, device=dev()).half()
    slots = torch.arange(T, dtype=torch.int32, device=dev())
    gdn.kv_cache_write(x, x.neg(), cache, slots)
    table = torch.arange(T // page + 1, dtype=torch.int32, device=dev())[None]
    k, v = gdn.kv_cache_read(cache, table, torch.tensor([0, T], dtype=torch.int32, device=dev()), T)
    if kind == F16:
        assert torch.equal(k, x) and torch.equal(v, x.neg())
    else:
        step = x.float().abs().amax(-1, keepdim=True) / 127
        assert torch.all((k.float() - x.float()).abs() <= step * 0.5001 + x.float().abs() * 2.0 ** -10)
        assert torch.equal(v, k.neg())
