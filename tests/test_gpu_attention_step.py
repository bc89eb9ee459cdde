"""The attention layer's decoding step, as a graph, against the FP64 oracle over
several steps of growing sequences: rotation, cache writes and attention
together, one token and four drafted tokens a step."""
import numpy as np
import pytest
import torch

import gated_delta_rule_gateddeltanet_gb300 as gdn
from attention_common import HALF_ULP, f64
from gated_delta_rule_gateddeltanet_gb300.attention_step import AttentionStep
from gpu_common import dev
from oracle import attention as oa

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tokens", [1, 4])
@pytest.mark.parametrize("kind", [torch.float16, torch.int8, torch.float8_e4m3fn])
def test_steps_of_growing_sequences(tokens, kind):
    seqs, hq, hk, d, page, steps = 3, 8, 2, 64, 16, 9
    table = gdn.rotary_table(200, 32, scaling="yarn", factor=4.0, original_positions=64, device=dev())
    cache = gdn.PagedKVCache.allocate(seqs * 5, page, hk, d, dtype=kind, device=dev(), heads_first=True)
    step = AttentionStep(cache, table, seqs=seqs, num_q_heads=hq, pages_per_seq=5, tokens=tokens)
    step.block_table.copy_(torch.randperm(seqs * 5).to(torch.int32).view(seqs, 5))
    start = torch.tensor([0, 14, 31], dtype=torch.int32)  # contexts written before, by the same call on longer spans
    g = torch.Generator("cpu").manual_seed(tokens)
    held = [[[], []] for _ in range(seqs)]  # the rows each sequence was given, rotated, in 64 bits
    for b in range(seqs):
        n = int(start[b])
        if n:
            k, v = (torch.randn(n, hk, d, generator=g).half().to(dev()) for _ in range(2))
            pos = torch.arange(n, dtype=torch.int32, device=dev())
            slots = (step.block_table[b, (pos // page).long()] * page + pos % page).to(torch.int32)
            gdn.kv_cache_write(k, v, cache, slots, positions=pos, table=table)
            held[b][0].append(oa.rotate(f64(k), np.arange(n), f64(table)))
            held[b][1].append(f64(v))
    for i in range(steps):
        for x in (step.q, step.k, step.v):
            x.copy_(torch.randn(x.shape, generator=g))
        step.kv_lens.copy_(start + (i + 1) * tokens)
        step.place()
        out = step.replay()
        torch.cuda.synchronize()
        assert int(step.status) == 0
        pos = step.positions.cpu().numpy()
        qr, kr, v = oa.rotate(f64(step.q), pos, f64(table)), oa.rotate(f64(step.k), pos, f64(table)), f64(step.v)
        for b in range(seqs):
            at = slice(b * tokens, (b + 1) * tokens)
            held[b][0].append(kr[at])
            held[b][1].append(v[at])
            k_all, v_all = np.concatenate(held[b][0]), np.concatenate(held[b][1])
            want, _ = oa.attend(qr[at], k_all, v_all, d ** -0.5)
            # what storing a row changes, relative to its largest magnitude: half a step
            row = {torch.float16: 2.0 ** -11, torch.int8: 0.5 / 127, torch.float8_e4m3fn: 2.0 ** -4}[kind]
            # a score moves by at most scale |q|_1 (row max |k| + 2^-10 max |k|) (the query is rounded to FP16), a
            # weight by that times e^that, an output by twice the weights' error times max |v| plus row max |v|
            delta = d ** -0.5 * np.abs(qr[at]).sum(-1).max() * (row + 2.0 ** -10) * np.abs(k_all).max()
            bound = (2 * delta * np.exp(delta) + row + 2 * HALF_ULP[torch.float16]) * np.abs(v_all).max()
            assert np.abs(f64(out)[at] - want).max() <= bound
        if kind == torch.float16:  # and far inside that worst case: FP16 rows behave like rounding noise
            assert np.linalg.norm(f64(out)[at] - want) <= 2.0 ** -9 * np.linalg.norm(want)


def test_capturing_writes_nothing():
    table = gdn.rotary_table(64, 64, device=dev())
    cache = gdn.PagedKVCache.allocate(4, 16, 2, 64, device=dev())
    cache.k.fill_(3), cache.v.fill_(4)
    step = AttentionStep(cache, table, seqs=2, num_q_heads=4, pages_per_seq=2)
    step.block_table.copy_(torch.tensor([[0, 1], [2, 3]], dtype=torch.int32))
    step.kv_lens.fill_(20)
    step.place()
    before = step.slots.clone()
    step.capture()
    torch.cuda.synchronize()
    assert torch.all(cache.k == 3) and torch.all(cache.v == 4) and torch.equal(step.slots, before)
    assert torch.all(step.kv_lens == 20) and int(step.status) == 0


def test_readme_attention_example_runs():
    """The README's second example as written: shapes, and the new token's attention against the oracle
    over what reading the cache back gives."""
    import os
    import re
    text = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")).read()
    scope = {}
    exec(compile(re.findall(r"```python\n(.*?)```", text, re.S)[1], "README.md", "exec"), scope)
    torch.cuda.synchronize()
    assert scope["k_all"].shape == (318, 2, 256) and scope["o1"].shape == (3, 16, 256)
    cu = torch.tensor([0, 301, 319, 321], dtype=torch.int32, device=dev())
    k, v = gdn.kv_cache_read(scope["cache"], scope["block_table"], cu, 321, dtype=torch.float32)
    for b, (i, j) in enumerate(((0, 301), (301, 319), (319, 321))):
        want, lse = oa.attend(f64(scope["q1"])[b:b + 1], f64(k)[i:j], f64(v)[i:j], 256 ** -0.5)
        # single FP16 weights (2^-11) and the output's rounding, over values of at most 5
        assert np.abs(f64(scope["o1"])[b] - want[0]).max() <= 4 * 2.0 ** -11 * np.abs(f64(v)[i:j]).max()
        assert np.abs(f64(scope["lse"])[b] - lse[0]).max() <= 2.0 ** -16 * (1 + np.abs(lse).max())
