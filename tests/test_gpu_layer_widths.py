"""The gated linear recurrence and the root-mean-square norm against the FP64 oracle in the forms that wide layers and
many tokens reach: four channels a lane, clusters of a single CTA over many rounds, rings that are filled again."""
import pytest
import torch

import gated_delta_rule_gateddeltanet_gb300 as gdn
from attention_common import f64
from gpu_common import dev
from layer_common import Recurrence, held
from oracle import layers as ol
from test_gpu_rms_norm import draw, weight_of

pytestmark = pytest.mark.gpu

HALF = [torch.bfloat16, torch.float16]


def check(r, **kw):
    y, final, chk = r.forward(return_checkpoints=True, **kw)
    r.check_forward(y, final)
    r.check_backward(r.backward(chk))


# past 1600 channels 16-bit rows take four channels a lane; copies of 16 bytes, 8, 4 and 2, ragged last slabs
@pytest.mark.parametrize("C", [1664, 2048, 2500, 2002, 1999])
@pytest.mark.parametrize("unit", [False, True])
@pytest.mark.parametrize("dtype", HALF)
def test_wide_layers(dtype, unit, C):
    check(Recurrence([300, 0, 1, 64, 131, 16], C, dtype, unit=unit, seed=C))


@pytest.mark.parametrize("has_b", [True, False])
@pytest.mark.parametrize("lens", [[700], [0, 5, 0, 0, 59, 1, 0], [17] * 30, [63, 1, 64, 128, 2], [1] * 200], ids=str)
def test_wide_layers_packings(lens, has_b):
    check(Recurrence(lens, 1672, torch.bfloat16, unit=True, has_b=has_b, seed=len(lens)))


@pytest.mark.parametrize("C", [1664, 1668, 1999])
def test_wide_layers_in_slices_of_a_projection(C):
    r = Recurrence([150, 90], C, torch.float16, fused=True, unit=True, seed=4)
    assert r.x.stride(0) == 3 * C
    check(r)


def test_wide_rows_that_are_not_aligned():
    """Views that begin one element into a row."""
    r = Recurrence([90, 133], 1664, torch.bfloat16, seed=5)
    for name in ("x", "a", "b", "dy"):
        t = torch.zeros(r.T, 1667, dtype=r.dtype, device=dev())[:, 1:1665]
        t.copy_(getattr(r, name))
        setattr(r, name, t)
    check(r)


@pytest.mark.parametrize("dtype,C", [(torch.bfloat16, 152 * 64 + 200), (torch.float32, 152 * 96 + 40)])
def test_more_slabs_than_pairs_of_ctas(dtype, C):
    """More slabs than clusters of two that are resident at once: one CTA takes all rounds of its slab."""
    check(Recurrence([400, 3, 0, 130], C, dtype, unit=True, seed=6))


@pytest.mark.parametrize("raw", [True, False])
def test_clusters_over_many_rounds(raw):
    """Few channels, where a cluster's 16 CTAs take 2048 (backwards 1024) tokens a round."""
    check(Recurrence([5000, 1, 3100], 36, torch.float32, raw, raw, seed=7))


# (tokens, heads, channels, dtype, gate, residual's gradient): a CTA of the backward pass takes more tokens than its ring has
# stages, several times over (a piece a thread, two, twice the threads; 8 stages to 2; the last round with idle CTAs)
RINGS = [(20700, 1, 64, torch.bfloat16, False, False), (20700, 1, 64, torch.float32, True, True),
         (8301, 1, 512, torch.float16, False, True), (4200, 16, 128, torch.bfloat16, True, True),
         (7777, 6, 256, torch.float16, True, False), (2801, 1, 2560, torch.bfloat16, True, True),
         (1111, 1, 8192, torch.bfloat16, False, True), (761, 1, 8192, torch.float32, False, True)]


@pytest.mark.parametrize("T,H,d,dtype,gated,residual", RINGS)
def test_rings_are_filled_again(T, H, d, dtype, gated, residual):
    x, dy, w = draw(T, H, d, dtype, 1), draw(T, H, d, dtype, 2), weight_of(d)
    z = draw(T, H, d, dtype, 3) if gated else None
    r = draw(T, H, d, dtype, 4) if residual else None
    dx, dw, *dz = gdn.rms_norm_backward(dy, x, w, gate=z, d_residual=r)
    n = lambda t: None if t is None else f64(t).reshape(T * H, d)  # noqa: E731
    want = ol.rms_norm_backward(n(dy), n(x), 1e-6, f64(w), n(z), n(r))
    held(dx, *want["dx"], "dx")
    held(dw, *want["dweight"], "dweight")
    if gated:
        held(dz[0], *want["dgate"], "dgate")
