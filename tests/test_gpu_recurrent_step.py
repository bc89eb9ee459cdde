"""The recurrence and the norms as they are used together: add and norm, projections, convolution,
recurrence, gated norm in 8 bits; a prompt and then decoding steps as a captured graph; the gated norm
behind the gated delta rule.  Every stage is held to the oracle on what the stage before it gave."""
import numpy as np
import pytest
import torch

import gated_delta_rule_gateddeltanet_gb300 as gdn
from attention_common import f64
from gated_delta_rule_gateddeltanet_gb300.recurrent_step import RecurrentStep
from gpu_common import dev
from layer_common import held
from oracle import layers as ol
from test_gpu_rms_norm import EIGHT, check_eight

pytestmark = pytest.mark.gpu

C, D, K = 256, 64, 4


class Layer:
    def __init__(self, dtype, slots, seed=0):
        g = torch.Generator("cpu").manual_seed(seed)
        r = lambda *s: torch.randn(*s, generator=g).to(dev())  # noqa: E731
        self.dtype, self.r = dtype, r
        self.conv_weight, self.conv_bias = r(C, K) * 0.4, r(C) * 0.1
        self.A_log = torch.log(1 + 15 * torch.rand(C, generator=g)).to(dev())
        self.dt_bias = torch.log(torch.expm1(1e-3 + 0.099 * torch.rand(C, generator=g))).to(dev())
        self.norm = 1 + 0.2 * r(D)
        self.conv_bank = torch.zeros(slots, C, K - 1, dtype=dtype, device=dev())
        self.bank = torch.zeros(slots, C, device=dev())

    def step(self, seqs, **kw):
        return RecurrentStep(self.conv_weight, self.conv_bias, self.conv_bank, self.A_log, self.dt_bias, self.bank,
                             self.norm, seqs=seqs, head_dim=D, **kw)

    def chunk(self, projection, cu, slots, **kw):
        """The same three stages by their functions, states in place; returns (y of the convolution, h, output)."""
        x, a, b, z = projection.split(C, 1)
        y, _, _ = gdn.varlen_causal_conv_with_state(x, self.conv_weight, cu, bias=self.conv_bias, initial_state=self.conv_bank,
                                                    final_state=self.conv_bank, state_slots=slots)
        before = self.bank.clone()
        h, _ = gdn.linear_recurrence(y, a, b, cu, A_log=self.A_log, dt_bias=self.dt_bias, unit_input=True,
                                     initial_state=self.bank, final_state=self.bank, state_slots=slots)
        out = gdn.rms_norm(h.unflatten(1, (-1, D)), self.norm, gate=z.unflatten(1, (-1, D)), **kw)
        gates = ol.Gates(f64(a), f64(b), f64(self.A_log), f64(self.dt_bias), True, True)
        ends = cu.tolist()
        rows = slots.cpu().numpy()
        want, final, _, err, ferr, _ = ol.linear_recurrence(f64(y), gates, list(zip(ends, ends[1:])), f64(before)[rows])
        held(h, want, err, "h")
        held(self.bank[slots.long()], final, ferr, "state")
        return y, h, out

    def check_norm(self, h, z, out):
        y, err = ol.rms_norm(f64(h.unflatten(1, (-1, D))), 1e-6, f64(self.norm), f64(z.unflatten(1, (-1, D))))
        if isinstance(out, tuple):
            check_eight(out[0], out[1], y, err, D if out[1].dim() == 2 else 0, dict(EIGHT)[out[0].dtype])
        else:
            held(out, y, err, "out")


@pytest.mark.parametrize("dtype,kw", [(torch.float16, dict(out_dtype=torch.float8_e4m3fn, scale_group=D)),
                                      (torch.float16, dict(out_dtype=torch.int8)), (torch.float32, {})])
def test_a_prompt_and_then_steps(dtype, kw):
    layer = Layer(dtype, 5)
    slots = torch.tensor([4, 0, 2], dtype=torch.int32, device=dev())
    lens = [90, 1, 33]
    cu = torch.tensor([0, 90, 91, 124], dtype=torch.int32, device=dev())
    w_in = layer.r(C, 4 * C) * C ** -0.5

    # prompt: the residual stream's norm, the in-projection, the layer's three stages
    x, res = layer.r(sum(lens), C).to(dtype), layer.r(sum(lens), C).to(dtype)
    normed, stream = gdn.rms_norm(x, torch.ones(C, device=dev()), residual=res)
    want, err = ol.rms_norm(f64(stream), 1e-6)
    held(normed, want, err + np.abs(want) * 2 * ol.U, "norm")
    projection = (normed.float() @ w_in).to(dtype)
    _, h, out = layer.chunk(projection, cu, slots, **kw)
    layer.check_norm(h, projection[:, 3 * C:], out)

    # steps: the graph against the functions, from the same states
    step = layer.step(3, **kw)
    step.slots.copy_(slots)
    one = torch.arange(4, dtype=torch.int32, device=dev())
    for k in range(4):
        step.projection.copy_(layer.r(3, 4 * C).to(dtype))
        saved = layer.conv_bank.clone(), layer.bank.clone()
        _, h, out = layer.chunk(step.projection, one, slots, **kw)
        layer.check_norm(h, step.projection[:, 3 * C:], out)
        after = layer.conv_bank.clone(), layer.bank.clone()
        layer.conv_bank.copy_(saved[0])
        layer.bank.copy_(saved[1])
        got = step.replay()
        assert torch.equal(layer.conv_bank, after[0]) and torch.equal(layer.bank, after[1])
        if kw:
            assert torch.equal(got.view(torch.uint8), out[0].view(torch.uint8)) and torch.equal(step.scale, out[1])
        else:
            assert torch.equal(got, out)
    assert step.status.item() == 0


def test_steps_reach_what_one_prompt_reaches():
    """Token by token, four at a time and all at once: the same states up to rounding."""
    lens, T = [41, 41], 82
    projection = None
    finals = []
    for tokens in (41, 1, 4):
        layer = Layer(torch.float32, 2, seed=3)
        if projection is None:
            projection = layer.r(2, 41, 4 * C)
        if tokens == 41:
            cu = torch.tensor([0, 41, 82], dtype=torch.int32, device=dev())
            layer.chunk(projection.reshape(T, 4 * C), cu, torch.arange(2, dtype=torch.int32, device=dev()))
        else:
            first = layer.step(2, tokens=1)
            first.projection.copy_(projection[:, 0])
            first.replay()
            step = layer.step(2, tokens=tokens)
            for t in range(1, 41, tokens):
                step.projection.copy_(projection[:, t:t + tokens].reshape(2 * tokens, 4 * C))
                step.replay()
        finals.append((layer.conv_bank, layer.bank))
    for conv, bank in finals[1:]:
        assert torch.equal(conv, finals[0][0])
        # every decay and weight is within 2^-20 of the exact one, in each of the runs, and 41 of them act on a state
        assert torch.all((bank - finals[0][1]).abs() <= 2 * 41 * 2.0 ** -20 * 8)


def test_capturing_changes_no_state():
    layer = Layer(torch.float16, 3, seed=4)
    layer.bank.copy_(layer.r(3, C))
    saved = layer.conv_bank.clone(), layer.bank.clone()
    layer.step(3).capture()
    torch.cuda.synchronize()
    assert torch.equal(layer.conv_bank, saved[0]) and torch.equal(layer.bank, saved[1])


@pytest.mark.parametrize("eight,most", EIGHT)
def test_behind_the_gated_delta_rule(eight, most):
    """gdn_forward's output through the gated norm of its heads, rows in 8 bits."""
    T, Hk, Hv, d = 70, 2, 4, 128
    g = torch.Generator("cpu").manual_seed(5)
    r = lambda *s: torch.randn(*s, generator=g).to(dev())  # noqa: E731
    q, k, v, z = (r(T, h, d).half() for h in (Hk, Hk, Hv, Hv))
    out, _, _ = gdn.gdn_forward(q, k, v, r(T, Hv), r(T, Hv), torch.tensor([0, 50, 70], dtype=torch.int32, device=dev()),
                                A_log=r(Hv).abs(), dt_bias=r(Hv) - 4)
    w = 1 + 0.2 * r(d)
    for group in (0, 128):
        y8, scale = gdn.rms_norm(out, w, gate=z, out_dtype=eight, scale_group=group)
        y, err = ol.rms_norm(f64(out), 1e-6, f64(w), f64(z))
        check_eight(y8, scale, y, err, group, most)


def test_queries_and_keys_before_the_rotation():
    """The heads' norm of a fused projection's queries and keys, then gdn_rotary: strided views throughout."""
    T, Hq, Hk, d = 33, 6, 2, 64
    g = torch.Generator("cpu").manual_seed(6)
    qkv = torch.randn(T, (Hq + 2 * Hk) * d, generator=g).to(torch.bfloat16).to(dev())
    q, k, _ = (t.unflatten(1, (-1, d)) for t in qkv.split([Hq * d, Hk * d, Hk * d], 1))
    w = 1 + 0.2 * torch.randn(d, generator=g).to(dev())
    qn, kn = gdn.rms_norm(q, w, weight_offset=0.5), gdn.rms_norm(k, w, weight_offset=0.5)
    for x, got in ((q, qn), (k, kn)):
        y, err = ol.rms_norm(f64(x), 1e-6, f64(w) + 0.5)
        held(got, y, err, "norm")
    table = gdn.rotary_table(64, d, device=dev())
    pos = torch.arange(T, dtype=torch.int32, device=dev())
    a, b = gdn.rotary(qn, kn, pos, table)
    a2, b2 = gdn.rotary(qn.clone(), kn.clone(), pos, table)
    assert torch.equal(a, a2) and torch.equal(b, b2) and a.shape == q.shape


def test_streams_and_graphs():
    """Calls on another stream than the current one; a forward and a backward pass captured once and replayed on
    other inputs; two graphs that share a workspace, replayed one after the other."""
    T = 300
    g = torch.Generator(dev()).manual_seed(7)
    r = lambda *s: torch.randn(*s, generator=g, device=dev())  # noqa: E731
    x, a, b, dy = (r(T, 192).to(torch.bfloat16) for _ in range(4))
    cu = torch.tensor([0, 100, 300], dtype=torch.int32, device=dev())
    kw = dict(A_log=r(192).abs(), dt_bias=r(192) - 4, unit_input=True)
    fwd = gdn.LinearRecurrenceCall(x, a, b, cu, return_checkpoints=True, **kw)
    bwd = gdn.LinearRecurrenceBackwardCall(dy, x, a, b, fwd.outputs[2], cu, **kw)
    w = 1 + 0.1 * r(64)
    ws = torch.empty(1 << 24, dtype=torch.uint8, device=dev())
    heads = lambda t: t.unflatten(1, (3, 64))  # noqa: E731
    norms = [gdn.RMSNormBackwardCall(heads(dy), heads(t), w, gate=heads(b), workspace=ws) for t in (x, a)]

    def eager():
        return [t.clone() for c in (fwd, bwd, *norms) for t in c.launch()]

    side = torch.cuda.Stream(dev())
    want = eager()
    torch.cuda.synchronize()
    for c in (fwd, bwd, *norms):
        for t in c.outputs:
            t.fill_(0)
    torch.cuda.synchronize()
    for c in (fwd, bwd, *norms):
        c.launch(side)
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(want, [t for c in (fwd, bwd, *norms) for t in c.outputs]))

    graphs = []
    for calls in ((fwd, bwd), norms[:1], norms[1:]):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            for c in calls:
                c.launch()
        graphs.append(graph)
    for _ in range(2):
        for t in (x, a, b, dy):
            t.copy_(r(T, 192))
        want = eager()
        for c in (fwd, bwd, *norms):
            for t in c.outputs:
                t.fill_(0)
        for graph in graphs:
            graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(want, [t for c in (fwd, bwd, *norms) for t in c.outputs]))


def test_many_sequences():
    """More sequences than tokens in a tile, most of them empty or of one token, with and without a hint."""
    from layer_common import Recurrence
    g = np.random.default_rng(0)
    r = Recurrence(g.choice([0, 0, 1, 2, 5], 3000).tolist(), 40, torch.float32, unit=True, seed=8)
    for hint in (0, 5):
        y, final, chk = r.forward(max_seqlen=hint, return_checkpoints=True)
        r.check_forward(y, final)
        r.check_backward(r.backward(chk))


def test_offsets_past_32_bits():
    """Rows whose elements lie more than 2^31 from the first: the last sequence, and the last tokens, give what they
    give alone."""
    T, wide, seen = 36000, 65536, 200
    big = torch.zeros(T, wide, dtype=torch.bfloat16, device=dev())
    assert big.numel() > 2 ** 31
    g = torch.Generator(dev()).manual_seed(9)
    r = lambda *s: torch.randn(*s, generator=g, device=dev())  # noqa: E731
    tail = r(seen, wide).to(torch.bfloat16)
    big[-seen:] = tail
    A, dt = r(wide).abs(), r(wide) - 4
    cu = torch.tensor([0, T - seen, T], dtype=torch.int32, device=dev())
    h0 = r(2, wide)
    y, final = gdn.linear_recurrence(big, big, big, cu, A_log=A, dt_bias=dt, initial_state=h0)
    one = torch.tensor([0, seen], dtype=torch.int32, device=dev())
    y1, f1, chk = gdn.linear_recurrence(tail, tail, tail, one, A_log=A, dt_bias=dt, initial_state=h0[1:].clone(), return_checkpoints=True)
    # (the same tiles or other ones: FP32 rounding, and then at most one BF16 step between the two)
    assert torch.all((final[1] - f1[0]).abs() <= 2.0 ** -16 * (1 + f1[0].abs()))
    assert torch.all((y[-seen:].float() - y1.float()).abs() <= 2.0 ** -7 * (y1.float().abs() + 2.0 ** -8))
    del y
    chk2 = gdn.linear_recurrence(big, big, big, cu, A_log=A, dt_bias=dt, initial_state=h0, return_checkpoints=True)[2]
    outs = gdn.linear_recurrence_backward(big, big, big, big, chk2, cu, A_log=A, dt_bias=dt, initial_state=h0)
    ones = gdn.linear_recurrence_backward(tail, tail, tail, tail, chk, one, A_log=A, dt_bias=dt, initial_state=h0[1:].clone())
    for p, q in zip(outs[:3], ones[:3]):
        assert torch.all((p[-seen:].float() - q.float()).abs() <= 2.0 ** -6 * (q.float().abs() + 2.0 ** -6))
    del outs, chk2
    z = gdn.rms_norm(big[:, :wide // 2], eps=1e-6)  # a strided view, past 2^31 all the same
    assert torch.equal(z[-seen:], gdn.rms_norm(tail[:, :wide // 2].contiguous(), eps=1e-6))
    heads = big.unflatten(1, (-1, 128))
    z = gdn.rms_norm(heads, eps=1e-6)
    assert torch.equal(z[-seen:], gdn.rms_norm(tail.unflatten(1, (-1, 128)), eps=1e-6))
    dx, _ = gdn.rms_norm_backward(z, heads, eps=1e-6)
    assert torch.equal(dx[-seen:], gdn.rms_norm_backward(z[-seen:].contiguous(), tail.unflatten(1, (-1, 128)), eps=1e-6)[0])
