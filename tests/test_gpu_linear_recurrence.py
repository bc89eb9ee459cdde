"""The gated linear recurrence on the GPU against the FP64 oracle, forward and backward, at the sizes and
packings where a scan that is split over time and channels can go wrong."""
import pytest
import torch

import gated_delta_rule_gateddeltanet_gb300 as gdn
from gpu_common import dev
from layer_common import DTYPES, Recurrence

pytestmark = pytest.mark.gpu

# one token to long ones; edges of 64-token tiles; sequences that end on, before and after them; empty ones
LENS = [[1], [64], [65], [1, 1, 1], [0, 5, 0, 0, 59, 1, 0], [63, 1, 64, 128, 2], [700], [130, 300, 1, 7], [17] * 30]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("lens", LENS, ids=str)
def test_raw_gates(lens, dtype):
    r = Recurrence(lens, 132, dtype, unit=True, seed=len(lens))
    y, final, chk = r.forward(return_checkpoints=True)
    r.check_forward(y, final)
    r.check_backward(r.backward(chk))


@pytest.mark.parametrize("raw,unit,has_b", [(True, False, True), (True, False, False), (True, True, False),
                                            (False, False, True), (False, False, False)])
@pytest.mark.parametrize("dtype", DTYPES)
def test_gate_modes(dtype, raw, unit, has_b):
    r = Recurrence([3, 0, 200, 64, 90], 136, dtype, raw, unit, has_b, seed=3)
    y, final, chk = r.forward(return_checkpoints=True)
    r.check_forward(y, final)
    outs = r.backward(chk)
    r.check_backward(outs)
    assert (outs[2] is None) == (not has_b) and len(outs) == (6 if raw else 4)


@pytest.mark.parametrize("C", [1, 3, 4, 31, 127, 128, 130, 257, 515])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_channels(C, dtype):
    r = Recurrence([70, 1, 150], C, dtype, raw=C % 2 == 0, unit=C % 4 == 0, seed=C)
    y, final, chk = r.forward(return_checkpoints=True)
    r.check_forward(y, final)
    r.check_backward(r.backward(chk))


@pytest.mark.parametrize("C", [64, 132, 129])
def test_slices_of_a_projection(C):
    r = Recurrence([100, 40], C, torch.float16, fused=True, unit=True, seed=4)
    assert r.x.stride(0) == 3 * C
    y, final, chk = r.forward(return_checkpoints=True)
    r.check_forward(y, final)
    r.check_backward(r.backward(chk))


def test_rows_that_are_not_aligned():
    """Views that begin one element into a row, and an odd distance between rows."""
    r = Recurrence([90, 33], 128, torch.bfloat16, seed=5)
    for name in ("x", "a", "b", "dy"):
        t = torch.zeros(r.T, 131, dtype=r.dtype, device=dev())[:, 1:129]
        t.copy_(getattr(r, name))
        setattr(r, name, t)
    pool = torch.zeros(r.num_slots * 128 + 1, device=dev())[1:].view(r.num_slots, 128)
    r.initial = pool.copy_(r.initial)
    y, final, chk = r.forward(return_checkpoints=True)
    r.check_forward(y, final)
    r.check_backward(r.backward(chk))


@pytest.mark.parametrize("hint", [0, 1, 3, 16, 17, 400])
def test_a_hint_changes_nothing_but_rounding(hint):
    """Also one that is too small."""
    r = Recurrence([1, 3, 0, 16, 2, 90], 100, torch.float32, unit=True, seed=6)
    y, final, chk = r.forward(max_seqlen=hint, return_checkpoints=True)
    r.check_forward(y, final)
    r.check_backward(r.backward(chk))


def test_equal_lengths_without_cu_seqlens():
    r = Recurrence([90] * 4, 64, torch.bfloat16, seed=7)
    y, final, chk = r.forward(return_checkpoints=True)
    kw = {**r.kw(), "num_seqs": 4}
    y2, f2, c2 = gdn.linear_recurrence(r.x, r.a, r.b, **kw, return_checkpoints=True)
    assert torch.equal(y, y2) and torch.equal(final, f2) and torch.equal(chk, c2)
    outs = r.backward(chk)
    for p, q in zip(outs, gdn.linear_recurrence_backward(r.dy, r.x, r.a, r.b, chk, **kw, d_final_state=r.d_final)):
        assert torch.equal(p, q)


def test_no_states():
    r = Recurrence([5, 0, 100], 72, torch.float32, initial=False, slots=None, seed=8)
    y, final, chk = r.forward(return_checkpoints=True)
    r.check_forward(y, final)
    y2, none = r.forward(write_final_state=False)
    assert none is None and torch.equal(y, y2)
    r.check_backward(r.backward(chk, d_final_state=None), d_final=False)


@pytest.mark.parametrize("lens,hint", [([1] * 7, 1), ([1] * 7, 0), ([300, 0, 2], 0)])
def test_states_in_place(lens, hint):
    """Only the batch's slots change, to the bits of a call with another buffer."""
    r = Recurrence(lens, 96, torch.bfloat16, seed=9)
    y, final, chk = r.forward(max_seqlen=hint, return_checkpoints=True)
    pool = r.initial.clone()
    y2, same, _ = r.forward(max_seqlen=hint, initial_state=pool, final_state=pool, return_checkpoints=True)
    assert same is pool and torch.equal(y, y2) and torch.equal(pool, final)
    idle = torch.ones(r.num_slots, dtype=torch.bool)
    idle[r.slots.cpu().long()] = False
    assert torch.equal(pool[idle.to(dev())], r.initial[idle.to(dev())])
    mark = torch.full_like(r.initial, 7.0)
    r.backward(chk, d_initial_state=mark)
    assert torch.all(mark[idle.to(dev())] == 7) and not torch.any(mark[r.slots.long()] == 7)
    with pytest.raises(gdn.GdnError):  # (its rows are read while others are written)
        r.backward(chk, d_final_state=mark, d_initial_state=mark)


@pytest.mark.parametrize("decay", [0.0, 1.0, -0.5, 2.0 ** -140])
def test_precomputed_decays_at_the_edges(decay):
    """No memory, all of it, decays of either sign and subnormal ones; C covers a ragged slab."""
    r = Recurrence([150, 30], 140, torch.float32, raw=False, seed=10, decay=lambda a: torch.full_like(a, decay))
    y, final, chk = r.forward(return_checkpoints=True)
    r.check_forward(y, final)
    r.check_backward(r.backward(chk))


@pytest.mark.parametrize("unit", [False, True])
@pytest.mark.parametrize("value", [-200.0, -30.0, 60.0, 200.0])
def test_raw_gates_at_the_edges(value, unit):
    """Decays that round to 1 (the unit factor is 0 or tiny) and to 0."""
    r = Recurrence([100], 64, torch.float32, unit=unit, seed=11, decay=lambda a: a * 0.1 + value)
    y, final, chk = r.forward(return_checkpoints=True)
    r.check_forward(y, final)
    r.check_backward(r.backward(chk))


def test_values_outside_a_sequence_do_not_reach_it():
    """Infinities and NaN in one sequence, and in tokens behind the last, stay there; those tokens are left as they were."""
    r = Recurrence([70, 20, 60], 64, torch.bfloat16, seed=12, extra=9)
    clean, cfinal, cchk = r.forward(return_checkpoints=True, status=torch.zeros(1, dtype=torch.int32, device=dev()))
    couts = r.backward(cchk)
    for t in (r.x, r.a, r.b, r.dy):
        t[70:90] = float("nan")
        t[75] = float("inf")
        t[150:] = float("nan")
    status = torch.zeros(1, dtype=torch.int32, device=dev())
    mark = lambda dt=r.dtype: torch.full((r.T, 64), 7.0, dtype=dt, device=dev())  # noqa: E731
    y, final, chk = r.forward(return_checkpoints=True, output=mark(), status=status)
    assert status.item() == gdn.DEVERR["cu_seqlens"]
    keep = torch.ones(r.T, dtype=torch.bool, device=dev())
    keep[70:90] = False
    keep[150:] = False
    assert torch.equal(y[keep], clean[keep]) and torch.all(y[150:] == 7)
    rows = r.slots.long()[[0, 2]]
    assert torch.equal(final[rows], cfinal[rows])
    outs = r.backward(chk, dx=mark(), da=mark(), db=mark())
    for p, q in zip(outs[:3], couts[:3]):
        assert torch.equal(p[keep], q[keep]) and torch.all(p[150:] == 7)
    assert torch.equal(outs[3][rows], couts[3][rows])


@pytest.mark.parametrize("hint", [0, 16])
def test_a_slot_out_of_range_skips_its_sequence(hint):
    r = Recurrence([10, 70, 30], 64, torch.float32, seed=13)
    clean, cfinal, cchk = r.forward(return_checkpoints=True, max_seqlen=hint)
    couts = r.backward(cchk)
    for bad in (-1, r.num_slots):
        slots = r.slots.clone()
        slots[1] = bad
        status = torch.zeros(1, dtype=torch.int32, device=dev())
        mark = lambda: torch.full((r.T, 64), 7.0, device=dev())  # noqa: E731
        y, final, chk = r.forward(state_slots=slots, status=status, output=mark(), return_checkpoints=True, max_seqlen=hint)
        assert status.item() == gdn.DEVERR["state_slot"]
        keep = torch.ones(r.T, dtype=torch.bool, device=dev())
        keep[10:80] = False
        assert torch.equal(y[keep], clean[keep]) and torch.all(y[10:80] == 7)
        rows, skipped = r.slots.long()[[0, 2]], r.slots.long()[1]
        assert torch.equal(final[rows], cfinal[rows]) and torch.equal(final[skipped], r.initial[skipped])
        status.zero_()
        outs = r.backward(cchk, state_slots=slots, status=status, dx=mark(), da=mark(), db=mark())
        assert status.item() == gdn.DEVERR["state_slot"]
        for p, q in zip(outs[:3], couts[:3]):
            assert torch.equal(p[keep], q[keep]) and torch.all(p[10:80] == 7)
        assert torch.equal(outs[3][rows], couts[3][rows])


@pytest.mark.parametrize("hint", [0, 16])
@pytest.mark.parametrize("cu", [[0, 50, 20, 110], [0, 10, 200, 110], [5, 10, 20, 110], [0, -3, 20, 110], [0, 10, 20, 200]])
def test_packing_out_of_order_is_flagged(cu, hint):
    """Nothing but the call's own tokens and slots is touched, whatever the packing says."""
    r = Recurrence([40, 40, 30], 64, torch.float32, seed=14)
    chk = r.forward(return_checkpoints=True)[2]
    cu = torch.tensor(cu, dtype=torch.int32, device=dev())
    status = torch.zeros(1, dtype=torch.int32, device=dev())
    idle = torch.ones(r.num_slots, dtype=torch.bool, device=dev())
    idle[r.slots.long()] = False
    mark = lambda: torch.full((r.T + 128, 64), 7.0, device=dev())  # noqa: E731
    y, final = gdn.linear_recurrence(r.x, r.a, r.b, cu, **r.kw(), output=mark(), status=status, max_seqlen=hint)
    assert status.item() & gdn.DEVERR["cu_seqlens"]
    assert torch.all(y[r.T:] == 7) and torch.equal(final[idle], r.initial[idle])
    status.zero_()
    outs = gdn.linear_recurrence_backward(r.dy, r.x, r.a, r.b, chk, cu, **r.kw(), dx=mark(), da=mark(), db=mark(), status=status)
    assert status.item() & gdn.DEVERR["cu_seqlens"]
    assert all(torch.all(t[r.T:] == 7) for t in outs[:3]) and torch.all(outs[3][idle] == 0)


def test_no_sequences_and_no_tokens():
    r = Recurrence([], 64, torch.bfloat16, seed=15)
    y, final, chk = r.forward(return_checkpoints=True)
    assert y.shape == (0, 64) and torch.equal(final, r.initial)
    outs = r.backward(chk)
    assert torch.all(outs[4] == 0) and torch.all(outs[5] == 0)
    r = Recurrence([0, 0], 64, torch.bfloat16, seed=16)
    _, final, chk = r.forward(return_checkpoints=True, final_state=torch.full_like(r.initial, 7.0))
    assert torch.equal(final[r.slots.long()], r.initial[r.slots.long()])
    outs = r.backward(chk)
    assert torch.equal(outs[3][r.slots.long()], r.d_final[r.slots.long()])
    assert torch.all(outs[4] == 0) and torch.all(outs[5] == 0)


def test_the_same_call_gives_the_same_bits():
    r = Recurrence([3000, 500, 2000], 260, torch.bfloat16, unit=True, seed=17)
    first = r.forward(return_checkpoints=True)
    grads = r.backward(first[2])
    for _ in range(5):
        again = r.forward(return_checkpoints=True)
        assert all(torch.equal(p, q) for p, q in zip(first, again))
        assert all(torch.equal(p, q) for p, q in zip(grads, r.backward(again[2])))


def test_long_sequences():
    r = Recurrence([9001, 1000], 40, torch.float32, unit=True, seed=18)
    y, final, chk = r.forward(return_checkpoints=True)
    r.check_forward(y, final)
    r.check_backward(r.backward(chk))


@pytest.mark.parametrize("raw", [True, False])
def test_gradients_against_differences(raw):
    """A weighted sum of the outputs moves as its gradient says, along a random direction of every input."""
    r = Recurrence([37, 90], 24, torch.float32, raw, raw, seed=19)
    chk = r.forward(return_checkpoints=True)[2]
    dx, da, db, dinit, *sums = r.backward(chk)
    g = torch.Generator(dev()).manual_seed(1)
    names = ["x", "a", "b", "initial"] + (["A_log", "dt_bias"] if raw else [])
    grads = [dx, da, db, dinit] + list(sums)
    base = {n: getattr(r, n).clone() for n in names}
    rows = r.slots.long()

    def loss():
        y, final = r.forward()
        return ((y.double() * r.dy.double()).sum() + (final[rows].double() * r.d_final[rows].double()).sum()).item()

    for name, grad in zip(names, grads):
        v = torch.randn(base[name].shape, generator=g, device=dev())
        # a central difference of step h: its error is h^2 / 6 times a third derivative, and what FP32 outputs lose over 2 h
        h = 2.0 ** -7
        moved = []
        for s in (h, -h):
            setattr(r, name, base[name] + s * v)
            moved.append(loss())
        setattr(r, name, base[name])
        slope, said = (moved[0] - moved[1]) / (2 * h), (grad.double() * v.double()).sum().item()
        size = (grad.double() * v.double()).abs().sum().item()
        assert abs(slope - said) <= 2e-3 * size, name
