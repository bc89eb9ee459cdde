"""The binding refuses what the C ABI would take for something else: views with
a stride of 0 (expanded), its word for rows without a gap, which would read or
write past the view's memory, numbers past 32 bits,
and the host's memory.  CPU tensors: nothing is launched."""
import ctypes
import types

import pytest
import torch

import gated_delta_rule_gateddeltanet_gb300 as gdn
from gated_delta_rule_gateddeltanet_gb300 import attention as at
from test_attention_abi_cpu import _kv, z


def ints(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def test_an_expanded_block_table_is_refused():
    shared = ints(1, 2).expand(3, 2)
    kw = dict(q=z(3, 8, 64), cache=_kv(), kv_lens=ints(3), workspace=torch.zeros(16, dtype=torch.uint8))
    assert gdn.PagedAttentionCall(block_table=ints(3, 4)[:, :2], **kw).args.block_table_stride == 4
    with pytest.raises(ValueError, match="block_table"):
        gdn.PagedAttentionCall(block_table=shared, **kw)
    with pytest.raises(ValueError, match="block_table"):
        gdn.KVCacheReadCall(_kv(), shared, ints(4), 10)
    # one sequence's stride is free
    one = dict(kw, q=z(1, 8, 64), kv_lens=ints(1))
    assert gdn.PagedAttentionCall(block_table=ints(2).expand(1, 2), **one).args.block_table_stride == 2


@pytest.mark.parametrize("name", ["q", "k", "q_out", "k_out"])
def test_expanded_tokens_are_refused_in_a_rotation(name):
    kw = dict(q=z(3, 4, 64), k=z(3, 2, 64), positions=ints(3), table=torch.zeros(9, 64), q_out=z(3, 4, 64), k_out=z(3, 2, 64))
    gdn.RotaryCall(**kw)
    with pytest.raises(ValueError, match=name):
        gdn.RotaryCall(**{**kw, name: kw[name][:1].expand_as(kw[name])})


@pytest.mark.parametrize("name", ["k", "v", "q", "q_out"])
def test_expanded_tokens_are_refused_in_a_write(name):
    kw = dict(k=z(3, 2, 64), v=z(3, 2, 64), cache=_kv(), slots=ints(3), positions=ints(3), table=torch.zeros(9, 64),
              q=z(3, 4, 64), q_out=z(3, 4, 64))
    gdn.KVCacheWriteCall(**kw)
    with pytest.raises(ValueError, match=name):
        gdn.KVCacheWriteCall(**{**kw, name: kw[name][:1].expand_as(kw[name])})


def test_expanded_queries_are_refused():
    kw = dict(cache=_kv(), block_table=ints(3, 2), kv_lens=ints(3), workspace=torch.zeros(16, dtype=torch.uint8))
    with pytest.raises(ValueError, match="q"):
        gdn.PagedAttentionCall(q=z(1, 8, 64).expand(3, 8, 64), **kw)


def test_expanded_tokens_are_refused_by_the_recurrence_and_the_convolution():
    t, h, d = 6, 2, 32
    f = lambda *s: torch.zeros(s)  # noqa: E731
    cu = torch.tensor([0, 6], dtype=torch.int32)
    kw = dict(q=z(t, h, d), k=z(t, h, d), v=z(t, h, d), a=f(t, h), b=f(t, h), cu_seqlens=cu)
    gdn.build_forward_args(**kw, A_log=f(h), dt_bias=f(h))
    for name in "qkv":
        with pytest.raises(ValueError, match=name):
            gdn.build_forward_args(**{**kw, name: z(1, h, d).expand(t, h, d)}, A_log=f(h), dt_bias=f(h))
    gdn.build_conv_args(z(t, 16), f(16, 4), cu)
    with pytest.raises(ValueError, match="x"):
        gdn.build_conv_args(z(1, 16).expand(t, 16), f(16, 4), cu)


def test_a_cache_of_one_expanded_row_or_scale_is_refused():
    rows = z(1, 1, 1, 64).expand(6, 16, 2, 64)
    with pytest.raises(ValueError, match="k and v"):
        gdn.PagedKVCache(rows, rows.clone().as_strided(rows.shape, rows.stride()))
    i8 = z(6, 16, 2, 64, dtype=torch.int8)
    unit = torch.ones(1, 1, 1).expand(6, 16, 2)
    with pytest.raises(ValueError, match="k_scale and v_scale"):
        gdn.PagedKVCache(i8, i8.clone(), unit, unit)
    # a scale for each head, whatever the page and token
    heads = torch.ones(2).expand(6, 16, 2)
    c = gdn.PagedKVCache(i8, i8.clone(), heads, heads).args
    assert (c.scale_page_stride, c.scale_token_stride, c.scale_head_stride) == (0, 0, 1)


@pytest.mark.parametrize("scales", [torch.ones(2).expand(6, 16, 2), torch.ones(16, 2).expand(6, 16, 2),
                                    torch.ones(6, 16, 1).expand(6, 16, 2)])
def test_rows_that_share_a_scale_are_not_written(scales):
    """Every row's scale is written: rows that share one would overwrite each other's."""
    from gated_delta_rule_gateddeltanet_gb300 import build
    build.build()
    i8 = z(6, 16, 2, 64, dtype=torch.int8)
    call = gdn.KVCacheWriteCall(z(0, 2, 64), z(0, 2, 64), gdn.PagedKVCache(i8, i8.clone(), scales, scales), ints(0))
    fn = gdn.load_library().gdn_kv_cache_write
    assert fn(ctypes.byref(call.args), None) == 3  # GDN_ERR_SHAPE, before any launch
    own = [torch.ones(6, 2, 16).transpose(1, 2) for _ in range(2)]
    call = gdn.KVCacheWriteCall(z(0, 2, 64), z(0, 2, 64), gdn.PagedKVCache(i8, i8.clone(), *own), ints(0))
    assert fn(ctypes.byref(call.args), None) == 0


def test_numbers_past_32_bits_are_refused():
    """A C struct's int32 would take them modulo 2^32: a window of 2^32 + 1 as 1."""
    kw = dict(q=z(3, 8, 64), cache=_kv(), block_table=ints(3, 2), kv_lens=ints(3), workspace=torch.zeros(16, dtype=torch.uint8))
    assert gdn.PagedAttentionCall(window=2 ** 31 - 1, **kw).args.window == 2 ** 31 - 1
    for name in ("window", "max_seqlen"):
        for n in (2 ** 31, 2 ** 32 + 1):
            with pytest.raises(ValueError, match=name):
                gdn.PagedAttentionCall(**kw, **{name: n})
    with pytest.raises(ValueError, match="max_seqlen"):
        gdn.paged_attention_workspace(_kv(), 8, max_seqlen=2 ** 32 + 1)
    with pytest.raises(ValueError, match="total_tokens"):
        gdn.KVCacheReadCall(_kv(), ints(1, 2), ints(2), 2 ** 32 + 1, k_out=z(3, 2, 64), v_out=z(3, 2, 64))
    with pytest.raises(ValueError, match="original_positions"):
        gdn.rotary_table(4, 32, scaling="yarn", factor=2.0, original_positions=2 ** 32 + 1, device="cpu")


@pytest.mark.parametrize("stream", [None, types.SimpleNamespace(cuda_stream=0)])
def test_tensors_of_the_host_are_not_launched_on(stream):
    calls = [gdn.RotaryCall(z(3, 4, 64), z(3, 2, 64), ints(3), torch.zeros(9, 64)),
             gdn.KVCacheWriteCall(z(3, 2, 64), z(3, 2, 64), _kv(), ints(3)),
             gdn.KVCacheReadCall(_kv(), ints(2, 2), ints(3), 10),
             gdn.PagedAttentionCall(z(3, 8, 64), _kv(), ints(3, 2), ints(3), workspace=torch.zeros(16, dtype=torch.uint8))]
    for call in calls:
        with pytest.raises(ValueError, match="GPU"):
            call.launch(stream)


def test_rotations_of_more_pairs_than_a_grid_holds_are_refused():
    """CTAs of 128 pairs, at most 2^31 - 1 of them.  (No call reaches a kernel here: there is no memory of that size.)"""
    from gated_delta_rule_gateddeltanet_gb300 import build
    build.build()
    a = at.RotaryArgs()
    a.total_tokens, a.num_q_heads, a.head_dim, a.rotary_dim, a.max_positions, a.io_dtype = 2 ** 31 - 1, 2, 128, 64, 99, 1
    a.q = a.q_out = a.positions = a.table = 0x1000
    assert gdn.load_library().gdn_rotary(ctypes.byref(a), None) == 3  # GDN_ERR_SHAPE
