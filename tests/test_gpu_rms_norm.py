"""The root-mean-square norm on the GPU against the FP64 oracle: forward in every type with the residual's
addition, the gate and 8-bit rows, and backward."""
import numpy as np
import pytest
import torch

import gated_delta_rule_gateddeltanet_gb300 as gdn
from attention_common import f64, rounding
from gpu_common import dev
from layer_common import DTYPES, held
from oracle import layers as ol

pytestmark = pytest.mark.gpu

# (tokens, heads, channels): one token to many, odd sizes, heads that share a warp, whole tokens over many warps
SHAPES = [(1, 1, 1), (3, 1, 7), (1, 1, 2048), (5, 1, 1000), (2, 1, 4096), (130, 1, 512), (3, 1, 8192), (2, 1, 20000), (2, 1, 40001),
          (1, 3, 64), (37, 18, 256), (9, 48, 128), (700, 2, 32), (4, 5, 24), (3, 2, 100), (2, 3, 512), (3, 2, 136), (2, 40, 1024)]


def draw(T, H, d, dtype, seed=0, scale=1.0):
    g = torch.Generator("cpu").manual_seed(seed)
    return (torch.randn(T, H, d, generator=g) * scale).to(dtype).to(dev())


def weight_of(d, seed=9):
    return (1 + 0.3 * torch.randn(d, generator=torch.Generator("cpu").manual_seed(seed))).to(dev())


def stored_sum(x, r):
    return x if r is None else (x.float() + r.float()).to(x.dtype)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,H,d", SHAPES)
def test_forward(T, H, d, dtype):
    x, w = draw(T, H, d, dtype, 1), weight_of(d)
    for residual, gate, weight, offset in ((None, None, w, 0.0), (draw(T, H, d, dtype, 2, 3.0), None, w, 1.0),
                                           (None, draw(T, H, d, dtype, 3), w, 0.0),
                                           (draw(T, H, d, dtype, 4), draw(T, H, d, dtype, 5), None, 0.0)):
        out = gdn.rms_norm(x, weight, eps=1e-5, weight_offset=offset, residual=residual, gate=gate)
        s = stored_sum(x, residual)
        if residual is not None:
            out, got = out
            assert torch.equal(got, s)
        y, err = ol.rms_norm(f64(s), 1e-5, None if weight is None else f64(weight) + offset, None if gate is None else f64(gate))
        held(out, y, err, "y")


EIGHT = [(torch.float8_e4m3fn, 448.0), (torch.int8, 127.0)]


def check_eight(q, scale, y, err, group, most):
    """Scales within the error of their largest magnitude; values within half a step of y / scale."""
    T = y.shape[0]
    rows, errs = (t.reshape(T, -1, group) if group else t.reshape(T, 1, -1) for t in (y, err))
    top, top_err = np.abs(rows).max(-1), errs.max(-1)
    want = np.where(top > 0, top / most, 1.0)
    got = f64(scale).reshape(want.shape)
    assert np.all(np.abs(got - want) <= np.where(top > 0, top_err / most, 0) + want * 4 * ol.U)
    z = rows / got[..., None]
    val = q.float().double().cpu().numpy().reshape(rows.shape)
    # the quotient is off by y's error and two roundings in FP32; e4m3 keeps 4 bits (2^-10 below 2^-6), int8 whole numbers
    off = errs / got[..., None] + np.abs(z) * 4 * ol.U
    half = 0.5 if most == 127 else np.maximum(np.abs(val) * 2.0 ** -4, 2.0 ** -10)
    assert np.all(np.abs(val - z) <= half + off)
    assert np.abs(val).max() <= most


@pytest.mark.parametrize("eight,most", EIGHT)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,H,d,group", [(1, 1, 2048, 0), (33, 1, 4096, 0), (3, 1, 1000, 0), (5, 1, 4096, 128), (7, 1, 96, 32),
                                         (4, 48, 128, 0), (61, 48, 128, 128), (9, 6, 64, 64), (9, 6, 64, 32), (2, 3, 20, 0),
                                         (2, 1, 20000, 32), (3, 2, 40000, 0), (5, 3, 256, 64), (300, 4, 32, 32), (2, 1, 8192, 64),
                                         (3, 5, 512, 128), (2, 130, 256, 0)])
def test_eight_bits(T, H, d, group, dtype, eight, most):
    x, r, z, w = draw(T, H, d, dtype, 1), draw(T, H, d, dtype, 2), draw(T, H, d, dtype, 3), weight_of(d)
    for residual, gate in ((None, None), (r, None), (None, z)):
        out = gdn.rms_norm(x, w, residual=residual, gate=gate, out_dtype=eight, scale_group=group)
        s = stored_sum(x, residual)
        if residual is not None:
            assert torch.equal(out[1], s)
        assert out[-1].shape == ((T, H * d // group) if group else (T,))
        y, err = ol.rms_norm(f64(s), 1e-6, f64(w), None if gate is None else f64(gate))
        check_eight(out[0], out[-1], y, err, group, most)


@pytest.mark.parametrize("eight,most", EIGHT)
@pytest.mark.parametrize("d,group", [(256, 0), (256, 64), (70, 0), (4096, 0), (4096, 128)])
def test_zeros_and_what_is_not_finite(d, group, eight, most):
    x = draw(5, 1, d, torch.float32, 1)
    x[0] = 0
    x[1, 0, 3] = float("inf")
    x[2, 0, 5] = float("nan")
    plain = gdn.rms_norm(x, eps=1e-6)
    assert torch.all(plain[0] == 0) and torch.all(torch.isnan(plain[2])) and torch.isnan(plain[1, 0, 3])
    assert torch.all(torch.isfinite(plain[3:]))
    q, scale = gdn.rms_norm(x, eps=1e-6, out_dtype=eight, scale_group=group)
    assert torch.all(scale[0] == 1) and torch.all(q[0].float() == 0)
    back = q.float().view(5, -1, group or d) * scale.view(5, -1, 1)
    assert torch.all(torch.isnan(back[2])) and torch.all(torch.isnan(back[1, 0]))
    clean = gdn.rms_norm(x[3:], eps=1e-6, out_dtype=eight, scale_group=group)
    assert torch.equal(q[3:].view(torch.uint8), clean[0].view(torch.uint8)) and torch.equal(scale[3:], clean[1])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,H,d", SHAPES)
def test_backward(T, H, d, dtype):
    x, dy, w = draw(T, H, d, dtype, 1, 2.0), draw(T, H, d, dtype, 2), weight_of(d)
    for gate, dres, weight, offset in ((None, None, w, 0.0), (None, draw(T, H, d, dtype, 3), w, 1.0),
                                       (draw(T, H, d, dtype, 4), None, w, 0.0), (draw(T, H, d, dtype, 5), draw(T, H, d, dtype, 6), None, 0.0)):
        outs = gdn.rms_norm_backward(dy, x, weight, eps=1e-5, weight_offset=offset, gate=gate, d_residual=dres)
        n = lambda t: None if t is None else f64(t).reshape(T * H, d)  # noqa: E731
        want = ol.rms_norm_backward(n(dy), n(x), 1e-5, None if weight is None else f64(weight) + offset, n(gate), n(dres))
        held(outs[0], *want["dx"], "dx")
        if weight is None:
            assert outs[1] is None
        else:
            held(outs[1], *want["dweight"], "dweight")
        if gate is not None:
            held(outs[2], *want["dgate"], "dgate")


@pytest.mark.parametrize("T,H,d", [(5000, 1, 64), (3000, 16, 128), (1500, 1, 1024)])
def test_weight_gradients_of_many_rows(T, H, d):
    x, dy, w = draw(T, H, d, torch.bfloat16, 1), draw(T, H, d, torch.bfloat16, 2), weight_of(d)
    first = gdn.rms_norm_backward(dy, x, w)
    want = ol.rms_norm_backward(f64(dy).reshape(-1, d), f64(x).reshape(-1, d), 1e-6, f64(w))
    held(first[1], *want["dweight"], "dweight")
    for _ in range(3):
        assert all(torch.equal(p, q) for p, q in zip(first, gdn.rms_norm_backward(dy, x, w)))


def test_whole_tokens_as_two_dimensions():
    x, w = draw(6, 1, 256, torch.float16, 1)[:, 0], weight_of(256)
    assert x.dim() == 2
    y, s = gdn.rms_norm(x, w, residual=x)
    assert y.shape == s.shape == x.shape
    assert torch.equal(y, gdn.rms_norm(s[:, None], w)[:, 0])
    dx, dw = gdn.rms_norm_backward(x, s, w)
    assert dx.shape == x.shape


@pytest.mark.parametrize("d,at,gap", [(128, 0, 128), (128, 1, 131), (256, 8, 264), (100, 0, 3), (2048, 8, 2064), (2048, 1, 2050)])
@pytest.mark.parametrize("dtype", [torch.float16, torch.float32])
def test_slices_and_alignment(d, at, gap, dtype):
    """Rows that begin inside wider ones, on 16-byte boundaries and off them: the results of whole tensors."""
    T, H, w = 9, 2, weight_of(d)
    ins = [draw(T, H, d, dtype, k) for k in range(4)]

    def view(t):
        wide = torch.full((T, at + H * d + gap), float("nan"), dtype=dtype, device=dev())
        v = wide[:, at:at + H * d].unflatten(1, (H, d))
        return v.copy_(t)

    x, r, z, dy = map(view, ins)
    # (a row's sum may be taken in another order by the kernel for rows off the boundaries, so not to the bit)
    y, s = gdn.rms_norm(x, w, residual=r, gate=z)
    want, err = ol.rms_norm(f64(stored_sum(ins[0], ins[1])), 1e-6, f64(w), f64(ins[2]))
    assert torch.equal(s, stored_sum(ins[0], ins[1]))
    held(y, want, err, "y")
    outs = gdn.rms_norm_backward(dy, x, w, gate=z, d_residual=r)
    n = lambda t: f64(t).reshape(T * H, d)  # noqa: E731
    back = ol.rms_norm_backward(n(ins[3]), n(ins[0]), 1e-6, f64(w), n(ins[2]), n(ins[1]))
    for name, got in zip(("dx", "dweight", "dgate"), outs):
        held(got, *back[name], name)


@pytest.mark.parametrize("T,H,d", [(7, 1, 2048), (5, 3, 128), (4, 1, 77), (3, 1, 40000)])
def test_in_place(T, H, d):
    x, r, z = (draw(T, H, d, torch.bfloat16, k) for k in range(3))
    w = weight_of(d)
    y, s = gdn.rms_norm(x, w, residual=r, gate=z)
    for into in ("x", "residual"):
        a, b, g = x.clone(), r.clone(), z.clone()
        y2, s2 = gdn.rms_norm(a, w, residual=b, gate=g, residual_out=a if into == "x" else b, output=g)
        assert torch.equal(y, y2) and torch.equal(s, s2) and y2 is g
    a = x.clone()
    plain = gdn.rms_norm(x, w)
    assert torch.equal(gdn.rms_norm(a, w, output=a), plain) and torch.equal(a, plain)


def test_no_tokens():
    x, w = draw(0, 2, 64, torch.float16), weight_of(64)
    assert gdn.rms_norm(x, w).shape == (0, 2, 64)
    dx, dw = gdn.rms_norm_backward(x, x, w)
    assert torch.all(dw == 0) and dx.shape == x.shape


def test_gradients_against_differences():
    T, H, d = 6, 3, 40
    x, z, dy, w = draw(T, H, d, torch.float32, 1), draw(T, H, d, torch.float32, 2), draw(T, H, d, torch.float32, 3), weight_of(d)
    dx, dw, dz = gdn.rms_norm_backward(dy, x, w, gate=z)
    loss = lambda x, w, z: (gdn.rms_norm(x, w, gate=z).double() * dy.double()).sum().item()  # noqa: E731
    for k, grad in enumerate((dx, dw, dz)):
        ins = [x, w, z]
        v = torch.randn(ins[k].shape, generator=torch.Generator(dev()).manual_seed(k), device=dev())
        h, moved = 2.0 ** -7, []
        for s in (h, -h):
            moved.append(loss(*[t + s * v if i == k else t for i, t in enumerate(ins)]))
        said, size = (grad.double() * v.double()).sum().item(), (grad.double() * v.double()).abs().sum().item()
        # (the step's own error is h^2 / 6 times a third derivative, 1e-5 of the gradient here; FP32 outputs lose 1e-5 over 2 h)
        assert abs((moved[0] - moved[1]) / (2 * h) - said) <= 2e-3 * size, k
