"""Where ``AttentionStep.place`` puts new tokens, on the CPU (it is torch
operations on the step's buffers): sequences past the
block table's end, idle ones, pages that the pool does not have."""
import pytest
import torch

import gated_delta_rule_gateddeltanet_gb300 as gdn
from gated_delta_rule_gateddeltanet_gb300.attention_step import AttentionStep

PAGE, PAGES = 16, 8


@pytest.fixture(scope="module", autouse=True)
def library():
    from gated_delta_rule_gateddeltanet_gb300 import build
    build.build()


def step_of(lens, table, tokens=1):
    cache = gdn.PagedKVCache.allocate(PAGES, PAGE, 2, 64, device="cpu")
    step = AttentionStep(cache, torch.zeros(99, 64), seqs=len(lens), num_q_heads=4, pages_per_seq=len(table[0]), tokens=tokens)
    step.block_table.copy_(torch.tensor(table, dtype=torch.int32))
    step.kv_lens.copy_(torch.tensor(lens, dtype=torch.int32))
    step.place()
    return step.positions.view(-1, tokens).tolist(), step.slots.view(-1, tokens).tolist()


def test_tokens_inside_the_table():
    pos, slots = step_of([1, 16, 17, 32], [[3, 5]] * 4)
    assert pos == [[0], [15], [16], [31]]
    assert slots == [[48], [63], [80], [95]]
    pos, slots = step_of([4, 18], [[3, 5], [1, 2]], tokens=4)
    assert pos == [[0, 1, 2, 3], [14, 15, 16, 17]]
    assert slots == [[48, 49, 50, 51], [30, 31, 32, 33]]


def test_tokens_past_the_table_get_a_slot_outside_the_pool():
    """Which the write flags; no index leaves the table."""
    pos, slots = step_of([33, 34, 2 ** 31 - 1, 5], [[3, 5], [1, 2], [6, 7], [0, 4]], tokens=2)
    out = PAGES * PAGE
    assert slots == [[95, out], [out, out], [out, out], [3, 4]]
    assert pos[0] == [31, 32] and pos[3] == [3, 4]


def test_idle_rows_are_not_stored():
    pos, slots = step_of([0, 1, 0], [[3, 5], [1, 2], [0, 0]])
    assert pos == [[0], [0], [0]] and slots == [[-1], [16], [-1]]
    pos, slots = step_of([0, 2, 4], [[3, 5], [1, 2], [0, 0]], tokens=4)
    assert pos == [[0, 0, 0, 0], [0, 0, 0, 1], [0, 1, 2, 3]]
    assert slots == [[-1] * 4, [-1, -1, 16, 17], [0, 1, 2, 3]]


@pytest.mark.parametrize("entry", [-1, -2, PAGES, 2 ** 27 + 1, 2 ** 31 - 1, -2 ** 31])
def test_entries_outside_the_pool_give_a_slot_outside_it(entry):
    """Whatever the offset: -1 is no token's slot (it would mean not stored), a product does not wrap into the pool."""
    for length in (1, 9, 16):
        assert step_of([length, 16], [[entry, 5], [1, 2]]) == ([[length - 1], [15]], [[PAGES * PAGE], [31]])


@pytest.mark.parametrize("entry", [-1, PAGES, 2 ** 31 - 1, -2 ** 31])
def test_idle_rows_may_have_any_entries(entry):
    assert step_of([0, 16], [[entry, entry], [1, 2]]) == ([[0], [15]], [[-1], [31]])
    assert step_of([2, 0], [[1, 2], [entry] * 2], tokens=3)[1] == [[-1, 16, 17], [-1, -1, -1]]


def test_a_step_needs_a_page_a_sequence():
    cache = gdn.PagedKVCache.allocate(PAGES, PAGE, 2, 64, device="cpu")
    with pytest.raises(ValueError, match="pages_per_seq"):
        AttentionStep(cache, torch.zeros(9, 64), seqs=2, num_q_heads=4, pages_per_seq=0)
