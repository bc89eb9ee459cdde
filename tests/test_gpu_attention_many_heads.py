"""Query heads whose offsets inside a token pass 32 bits."""
import pytest
import torch

import gated_delta_rule_gateddeltanet_gb300 as gdn
from gpu_common import dev

pytestmark = pytest.mark.gpu


def test_head_offsets_past_32_bits():
    """2^23 + 16 heads of 256 over one key head: a set of 16 heads repeated, whose results repeat."""
    g = torch.Generator("cpu").manual_seed(0)
    cache = gdn.PagedKVCache.allocate(3, 16, 1, 256, device=dev())
    for x in (cache.k, cache.v):
        x.copy_(torch.randn(x.shape, generator=g))
    table = torch.tensor([[2, 0]], dtype=torch.int32, device=dev())
    lens = torch.tensor([23], dtype=torch.int32, device=dev())
    few = torch.randn(1, 16, 256, generator=g).half().to(dev())
    want = gdn.paged_attention(few, cache, table, lens)
    many = few.repeat(1, (1 << 19) + 1, 1)
    out = gdn.paged_attention(many, cache, table, lens).view(-1, 16, 256)
    assert out.shape[0] == (1 << 19) + 1 and all(torch.equal(out[i:i + 4096], want.expand_as(out[i:i + 4096]))
                                                 for i in range(0, out.shape[0], 4096))
