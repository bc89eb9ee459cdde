"""The read back's packing: entries of cu_seqlens out of order are flagged wherever
they are, at every batch size, and nothing else is."""
import pytest
import torch

import gated_delta_rule_gateddeltanet_gb300 as gdn
from gpu_common import dev

pytestmark = pytest.mark.gpu


def read(entries, total, dtype=torch.int8):
    g = torch.Generator("cpu").manual_seed(0)
    cache = gdn.PagedKVCache.allocate(4, 16, 2, 64, dtype=dtype, device=dev())
    k, v = (torch.randn(64, 2, 64, generator=g).half().to(dev()) for _ in range(2))
    gdn.kv_cache_write(k, v, cache, torch.arange(64, dtype=torch.int32, device=dev()))
    cu = torch.tensor(entries, dtype=torch.int32, device=dev())
    table = torch.arange(2, dtype=torch.int32, device=dev()).repeat(len(entries) - 1, 1)
    status = torch.zeros(1, dtype=torch.int32, device=dev())
    out = gdn.kv_cache_read(cache, table, cu, total, dtype=torch.float16, status=status)
    return int(status), out


@pytest.mark.parametrize("seqs", [3, 40, 600])
def test_entries_out_of_order_are_flagged(seqs):
    good = [min(i, 20) for i in range(seqs)] + [30]
    assert read(good, 30)[0] == 0
    for at in {1, seqs // 2, seqs - 1}:
        for value in (-1, 29 if at < seqs - 1 else 31, 2 ** 31 - 1, -2 ** 31):
            bad = list(good)
            bad[at] = value
            assert read(bad, 30)[0] == gdn.DEVERR["cu_seqlens"], (at, value)


def test_ends_that_do_not_fit_the_tokens_are_flagged():
    for entries in ([1, 5, 30], [0, 5, 29], [0, 5, 31], [0, 31, 30]):
        assert read(entries, 30)[0] == gdn.DEVERR["cu_seqlens"], entries
    assert read([0, 0, 30], 30)[0] == 0 and read([0, 30, 30], 30)[0] == 0
