"""Sequences of equal length without cu_seqlens: the library knows how long they are, so a call gives the bits of the
packed call that is told so."""
import pytest
import torch

import gated_delta_rule_gateddeltanet_gb300 as gdn
from layer_common import DTYPES, Recurrence

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n", [1, 3, 16, 17])
@pytest.mark.parametrize("dtype", DTYPES)
def test_equal_lengths_are_known_without_a_hint(dtype, n):
    r = Recurrence([n] * 33, 260, dtype, unit=True, seed=n)
    want = r.forward(max_seqlen=n, return_checkpoints=True)
    kw = {**r.kw(), "num_seqs": 33}
    got = gdn.linear_recurrence(r.x, r.a, r.b, **kw, return_checkpoints=True)
    assert all(torch.equal(p, q) for p, q in zip(got, want, strict=True))
    r.check_forward(*got[:2])
    r.check_backward(gdn.linear_recurrence_backward(r.dy, r.x, r.a, r.b, got[2], **kw, d_final_state=r.d_final))
