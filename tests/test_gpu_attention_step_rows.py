"""Rows of an attention step that have no place in the cache: idle ones, ones past
their block table's end.  The other rows are unaffected."""
import pytest
import torch

import gated_delta_rule_gateddeltanet_gb300 as gdn
from gated_delta_rule_gateddeltanet_gb300.attention_step import AttentionStep
from gpu_common import dev

pytestmark = pytest.mark.gpu


def run(lens, tokens, kind):
    """One step over a cache of fixed contents; returns the step, and the cache before it."""
    g = torch.Generator("cpu").manual_seed(1)
    cache = gdn.PagedKVCache.allocate(9, 16, 2, 64, dtype=kind, device=dev())
    k, v = (torch.randn(9 * 16, 2, 64, generator=g).half().to(dev()) for _ in range(2))
    gdn.kv_cache_write(k, v, cache, torch.arange(9 * 16, dtype=torch.int32, device=dev()))
    step = AttentionStep(cache, gdn.rotary_table(200, 64, device=dev()), seqs=3, num_q_heads=4, pages_per_seq=3, tokens=tokens)
    step.block_table.copy_(torch.arange(9, dtype=torch.int32).view(3, 3))
    for x in (step.q, step.k, step.v):
        x.copy_(torch.randn(x.shape, generator=g))
    before = cache.k.clone().view(torch.uint8)
    step.kv_lens.copy_(torch.tensor(lens, dtype=torch.int32))
    step.place()
    step.replay()
    torch.cuda.synchronize()
    return step, before


def changed(step, before):
    """Slots whose key row differs from before the step."""
    return (step.cache.k.view(torch.uint8) != before).flatten(2).any(-1).flatten().nonzero().flatten().tolist()


@pytest.mark.parametrize("kind", [torch.float16, torch.int8])
@pytest.mark.parametrize("tokens", [1, 4])
def test_idle_rows(tokens, kind):
    all_busy, _ = run([20, 20, 30], tokens, kind)
    step, before = run([20, 0, 30], tokens, kind)
    assert int(step.status) == 0
    t = tokens
    assert torch.all(step.out[t:2 * t] == 0)
    assert torch.equal(step.out[:t], all_busy.out[:t]) and torch.equal(step.out[2 * t:], all_busy.out[2 * t:])
    assert changed(step, before) == [20 - t + i for i in range(t)] + [6 * 16 + 30 - t + i for i in range(t)]


def test_fewer_cached_tokens_than_new_ones():
    step, before = run([20, 2, 30], 4, torch.float16)
    assert int(step.status) == 0
    assert torch.all(step.out[4:6] == 0) and torch.all(step.out[6:8] != 0)
    assert changed(step, before) == [16, 17, 18, 19, 48, 49, 6 * 16 + 26, 6 * 16 + 27, 6 * 16 + 28, 6 * 16 + 29]


@pytest.mark.parametrize("tokens", [1, 4])
def test_rows_past_their_table_and_pages_outside_the_pool_are_flagged(tokens):
    good, _ = run([20, 20, 30], tokens, torch.float16)
    t = tokens
    for length in (3 * 16 + 1, 3 * 16 + t, 1000, 2 ** 31 - 1):
        step, before = run([20, length, 30], t, torch.float16)
        assert int(step.status) & gdn.DEVERR["kv_len"] and int(step.status) & gdn.DEVERR["cache_slot"]
        assert torch.equal(step.out[:t], good.out[:t]) and torch.equal(step.out[2 * t:], good.out[2 * t:])
        stored = [3 * 16 + i for i in range(length - t, 3 * 16)]
        assert changed(step, before) == [20 - t + i for i in range(t)] + stored + [6 * 16 + 30 - t + i for i in range(t)]
    for entry in (-1, 9, 2 ** 31 - 1):
        step = good
        step.status.zero_()
        step.kv_lens[1] = 32
        step.block_table[1, 1] = entry
        before = step.cache.k.clone().view(torch.uint8)
        step.k.add_(1)
        step.place()
        step.replay()
        torch.cuda.synchronize()
        assert int(step.status) == gdn.DEVERR["cache_slot"] | gdn.DEVERR["page"]
        assert changed(step, before) == [20 - t + i for i in range(t)] + [6 * 16 + 30 - t + i for i in range(t)]
