"""The binding refuses views whose strides the C ABI would take for something
else: a stride of 0 (an expanded view) is its word for rows without a gap, which
would read or write past the view's memory.  CPU tensors: nothing is launched."""
import pytest
import torch

import gated_delta_rule_gateddeltanet_gb300 as gdn
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
