"""The largest sizes that the root-mean-square norm takes, what it refuses beyond, and the slots that a recurrent layer's step
needs: no call here reaches a kernel."""
import ctypes

import pytest
import torch

import gated_delta_rule_gateddeltanet_gb300 as gdn
from gated_delta_rule_gateddeltanet_gb300 import norm
from gated_delta_rule_gateddeltanet_gb300.recurrent_step import RecurrentStep

OK, SHAPE = 0, 3


@pytest.fixture(scope="module", autouse=True)
def lib():
    from gated_delta_rule_gateddeltanet_gb300 import build
    build.build()
    return gdn.load_library()


@pytest.mark.parametrize("heads,d,code", [(1, 2 ** 31 - 256, OK), (1, 2 ** 31 - 255, SHAPE), (1, 2 ** 31 - 1, SHAPE),
                                          (2 ** 23 - 1, 256, OK), (2 ** 23, 256, SHAPE), (2 ** 16, 2 ** 16, SHAPE)])
def test_channels_of_a_token(lib, heads, d, code):
    """A counter that steps over a row of d channels 128 at a time stays below 2^31."""
    for cls, entry in ((norm.RMSNormArgs, lib.gdn_rms_norm), (norm.RMSNormBackwardArgs, lib.gdn_rms_norm_backward)):
        a = cls()
        a.total_tokens, a.num_heads, a.head_dim, a.io_dtype, a.eps = 0, heads, d, 1, 1e-6
        if cls is norm.RMSNormArgs:
            a.out_dtype = 1
        # (no tokens, and no weight's gradient: nothing to launch)
        assert entry(ctypes.byref(a), None) == code
    n = ctypes.c_size_t(0)
    a.total_tokens = 4
    assert lib.gdn_rms_norm_backward_workspace_size(ctypes.byref(a), ctypes.byref(n)) == code
    if code == OK:
        assert n.value >= 4 * d and n.value % (4 * d) == 0


@pytest.mark.parametrize("conv_slots,state_slots,seqs", [(4, 2, 3), (2, 4, 3), (3, 3, 3), (5, 3, 3)])
def test_a_step_needs_a_slot_a_sequence_in_both_banks(conv_slots, state_slots, seqs):
    z = lambda *s: torch.zeros(*s)  # noqa: E731
    build = lambda: RecurrentStep(z(8, 4), None, z(conv_slots, 8, 3), z(8), z(8), z(state_slots, 8), z(8), seqs=seqs,  # noqa: E731
                                  head_dim=8)
    if seqs <= min(conv_slots, state_slots):
        build()
    else:
        with pytest.raises(ValueError, match="state slots"):
            build()
