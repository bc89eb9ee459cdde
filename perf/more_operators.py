"""Cases of the gated linear recurrence (a diagonal state beside the gated delta rule's matrix state) and of the
root-mean-square norm around such layers (residual stream, output gate, rows in 8 bits), each forward and backward.

`run(state)` computes a case either in its plain form (elementary torch operations in 32 bits,
rounded once at the end) or, where `own` is set, with the calls a user makes of the library.
`exact(case, seed)` computes the same from the definitions in 64 bits.
"""
import math

import torch

own = False

DEVICE = "cuda"
GOLDEN = 0.6180339887498949
EPS = 1e-6


# ---------------------------------------------------------------------------- cases

def listed():
    return [
        # One decode step of a batch of 64 in a layer of 2560 channels: latency is all of it.
        dict(name="recurrence decode", kind="recurrence", seqs=64, lo=1, hi=1, channels=2560, dtype="bfloat16",
             mode="raw", unit=True, fused=True),
        # A packed batch of ragged prompts, gates straight from the layer's projections.
        dict(name="recurrence prompts", kind="recurrence", seqs=8, lo=100, hi=2048, channels=4096, dtype="bfloat16",
             mode="raw", unit=False, fused=True),
        # One long document: the scan has to be split over time.
        dict(name="recurrence one long", kind="recurrence", seqs=1, lo=65536, hi=65536, channels=2560, dtype="float16",
             mode="raw", unit=True, fused=False),
        # 32-bit values with decays from the program's own gates, an odd number of channels.
        dict(name="recurrence fp32 odd", kind="recurrence", seqs=5, lo=1, hi=2500, channels=1001, dtype="float32",
             mode="precomputed", unit=False, fused=False),
        # A training step's forward and backward pass over four sequences of equal length.
        dict(name="recurrence training", kind="recurrence training", seqs=4, lo=4096, hi=4096, channels=2048,
             dtype="bfloat16", mode="raw", unit=True, fused=False),
        # The same in 32 bits with the decays' own gradients, short ragged sequences.
        dict(name="recurrence training fp32", kind="recurrence training", seqs=3, lo=17, hi=700, channels=520,
             dtype="float32", mode="precomputed", unit=False, fused=False),
        # One user's decode step: the residual's addition and the norm of a single token.
        dict(name="norm one token", kind="norm", tokens=1, heads=1, head_dim=2048, dtype="bfloat16", residual=True,
             gate=False, out="bfloat16", group=0),
        # The norm before a layer's projections over a prompt batch, rows for an 8-bit product.
        dict(name="norm prompt e4m3", kind="norm", tokens=8192, heads=1, head_dim=4096, dtype="bfloat16", residual=True,
             gate=False, out="float8_e4m3fn", group=0),
        # The gated norm on the heads of a gated-delta-rule layer's output, a scale for each head.
        dict(name="norm gated heads e4m3", kind="norm", tokens=4099, heads=48, head_dim=128, dtype="float16",
             residual=False, gate=True, out="float8_e4m3fn", group=128),
        # A training step's norm of the residual stream, forward and backward.
        dict(name="norm training", kind="norm training", tokens=8192, heads=1, head_dim=4096, dtype="bfloat16",
             residual=True, gate=False),
        # The same for the gated norm of the heads.
        dict(name="norm training gated", kind="norm training", tokens=4096, heads=16, head_dim=128, dtype="float16",
             residual=False, gate=True),
        # What follows a recurrent layer's convolution: the recurrence, then the gated norm of its output.
        dict(name="layer chunk", kind="layer", seqs=16, lo=1, hi=512, channels=2048, head_dim=128, dtype="bfloat16",
             mode="raw", unit=True, fused=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))))


def draw(rng):
    kind = rng.choice(["recurrence", "recurrence", "recurrence training", "norm", "norm", "norm training", "layer"])
    dtype = rng.choice(["bfloat16", "bfloat16", "float16", "float32"])
    if kind in ("norm", "norm training"):
        heads = rng.choice([1, 1, 2, 16, 18, 40, 48])
        d = rng.choice([64, 128, 256]) if heads > 1 else rng.choice([512, 1000, 1536, 2048, 2560, 4096, 5120, 8192])
        most = 8192 * 4096 // (heads * d) // (2 if dtype == "float32" else 1)
        c = dict(kind=kind, tokens=_log_int(rng, 1, min(most, 32768)), heads=heads, head_dim=d, dtype=dtype,
                 residual=heads == 1 and rng.random() < 0.7, gate=heads > 1 and rng.random() < 0.5)
        if kind == "norm":
            c["out"] = dtype if d % 32 else rng.choice([dtype, "float8_e4m3fn"])
            c["group"] = rng.choice([0, 0, 32, 64, 128]) if c["out"] != dtype else 0
            if c["group"] and d % c["group"]:
                c["group"] = 32
        return c
    head_dim = rng.choice([64, 128, 256])
    channels = _log_int(rng, 64, 8192)
    if kind == "layer":
        channels = head_dim * max(1, channels // head_dim)
    elif rng.random() < 0.7:
        channels = 64 * max(1, channels // 64)
    most = 65536 * 2560 // channels
    seqs = _log_int(rng, 1, 256)
    hi = _log_int(rng, 1, max(1, min(most // seqs, 65536)))
    c = dict(kind=kind, seqs=seqs, lo=rng.choice([1, hi]), hi=hi, channels=channels, dtype=dtype,
             mode="raw" if rng.random() < 0.75 else "precomputed", unit=False, fused=rng.random() < 0.5)
    if c["mode"] == "raw":
        c["unit"] = rng.random() < 0.5
    if kind == "layer":
        c["head_dim"] = head_dim
    while work(c)["bytes"] > 1.3e9:  # the largest listed case's
        c["hi"] = c["hi"] * 2 // 3
        c["lo"] = min(c["lo"], c["hi"])
    return c


# ---------------------------------------------------------------------------- sizes

def _lens(case):
    """Each sequence's length: spread evenly over [lo, hi] in a scattered order."""
    lo, hi, n = case["lo"], case["hi"], case["seqs"]
    if n == 1:
        return [hi]
    return [lo + int((hi - lo + 1) * ((i + 1) * GOLDEN % 1.0)) for i in range(n)]


def _bytes(dtype):
    return {"float32": 4, "float16": 2, "bfloat16": 2, "float8_e4m3fn": 1}[dtype]


def work(case):
    io = _bytes(case["dtype"])
    if case["kind"].startswith("norm"):
        rows = case["tokens"] * case["heads"]
        n, d = rows * case["head_dim"], case["head_dim"]
        if case["kind"] == "norm":
            scales = n // case["group"] if case["group"] else case["tokens"]
            return {"bytes": n * (io * (1 + 2 * case["residual"] + case["gate"]) + _bytes(case["out"])) +
                    (4 * scales if case["out"] != case["dtype"] else 0) + 4 * d,
                    "flops": n * (4 + case["residual"] + 5 * case["gate"])}
        # forward: x (and r, z) -> y (and s); backward: dy, s (and ds, z) -> dx (and dz)
        forward = 2 + 2 * case["residual"] + case["gate"]
        backward = 3 + case["residual"] + 2 * case["gate"]
        return {"bytes": n * io * (forward + backward) + 3 * 4 * d, "flops": n * (16 + 14 * case["gate"])}
    t, c, b = sum(_lens(case)), case["channels"], case["seqs"]
    gate = io if case["mode"] == "raw" else 4
    per = {"recurrence": 2 * io + 2 * gate, "recurrence training": 5 * io + 6 * gate,
           "layer": 4 * io + 2 * gate}[case["kind"]]
    if case["kind"] == "recurrence training":
        return {"bytes": t * c * per + 3 * b * c * 4, "flops": t * c * 60}
    return {"bytes": t * c * per + 2 * b * c * 4, "flops": t * c * (20 if case["mode"] == "raw" else 3)}


# ---------------------------------------------------------------------------- inputs

def _normal(g, *shape, dtype):
    return torch.randn(*shape, generator=g, device=DEVICE).to(getattr(torch, dtype))


def prepare(case, seed):
    g = torch.Generator(DEVICE).manual_seed(seed)
    kind, dtype = case["kind"], case["dtype"]
    st = {"case": dict(case)}
    if kind.startswith("norm"):
        t, h, d = case["tokens"], case["heads"], case["head_dim"]
        st["x"] = _normal(g, t, h, d, dtype=dtype)
        st["weight"] = 1 + 0.2 * torch.randn(d, generator=g, device=DEVICE)
        st["residual"] = _normal(g, t, h, d, dtype=dtype) * 3 if case["residual"] else None
        st["gate"] = _normal(g, t, h, d, dtype=dtype) if case["gate"] else None
        if kind == "norm training":
            st["dy"] = _normal(g, t, h, d, dtype=dtype)
            st["dresidual"] = _normal(g, t, h, d, dtype=dtype) if case["residual"] else None
    else:
        lens, c, raw = _lens(case), case["channels"], case["mode"] == "raw"
        t, seqs = sum(lens), len(lens)
        z = 1 if kind == "layer" else 0
        if case["fused"] and raw:  # views of one projection's output
            st["x"], st["a"], st["b"], *rest = _normal(g, t, (3 + z) * c, dtype=dtype).split(c, 1)
            st["gate"] = rest[0] if z else None
        else:
            st["x"], st["a"], st["b"] = (_normal(g, t, c, dtype=dtype) for _ in range(3))
            st["gate"] = _normal(g, t, c, dtype=dtype) if z else None
        st["A_log"] = st["dt_bias"] = None
        if raw:
            st["A_log"] = torch.log(1 + 15 * torch.rand(c, generator=g, device=DEVICE))
            st["dt_bias"] = torch.log(torch.expm1(1e-3 + 0.099 * torch.rand(c, generator=g, device=DEVICE)))
        else:
            st["a"] = torch.sigmoid(st["a"].float() + 4)
            st["b"] = torch.sigmoid(st["b"].float())
        st["cu_seqlens"] = torch.tensor([0] + lens, device=DEVICE).cumsum(0).to(torch.int32)
        st["slots"] = torch.randperm(seqs + 3, generator=g, device=DEVICE)[:seqs].to(torch.int32)
        st["initial_state"] = torch.randn(seqs + 3, c, generator=g, device=DEVICE)
        st["longest"] = max(lens)
        if kind == "recurrence training":
            st["dy"] = _normal(g, t, c, dtype=dtype)
            st["dfinal"] = torch.randn(seqs + 3, c, generator=g, device=DEVICE)
        if kind == "layer":
            st["weight"] = 1 + 0.2 * torch.randn(case["head_dim"], generator=g, device=DEVICE)
    if own:
        _plan(st)
    return st


def _plan(st):
    """The call objects a program keeps for its fixed buffers (arguments checked and resolved once)."""
    import gated_delta_rule_gateddeltanet_gb300 as gdn

    case = st["case"]
    kind = case["kind"]
    out = dict(out_dtype=getattr(torch, case["out"]), scale_group=case["group"]) if "out" in case else {}
    if kind.startswith("norm"):
        forward = gdn.RMSNormCall(st["x"], st["weight"], eps=EPS, residual=st["residual"], gate=st["gate"], **out)
        st["calls"] = [forward]
        if kind == "norm training":
            s = forward.outputs[1] if case["residual"] else st["x"]
            st["calls"].append(gdn.RMSNormBackwardCall(st["dy"], s, st["weight"], eps=EPS, gate=st["gate"],
                                                       d_residual=st["dresidual"]))
        return
    training = kind == "recurrence training"
    args = dict(A_log=st["A_log"], dt_bias=st["dt_bias"], gate_mode=case["mode"], unit_input=case["unit"],
                initial_state=st["initial_state"], state_slots=st["slots"], max_seqlen=st["longest"])
    forward = gdn.LinearRecurrenceCall(st["x"], st["a"], st["b"], st["cu_seqlens"], return_checkpoints=training, **args)
    st["calls"] = [forward]
    if training:
        st["calls"].append(gdn.LinearRecurrenceBackwardCall(st["dy"], st["x"], st["a"], st["b"], forward.outputs[2],
                                                            st["cu_seqlens"], d_final_state=st["dfinal"], **args))
    if kind == "layer":
        d = case["head_dim"]
        heads = (forward.outputs[0].unflatten(1, (-1, d)), st["gate"].unflatten(1, (-1, d)))
        st["calls"].append(gdn.RMSNormCall(heads[0], st["weight"], eps=EPS, gate=heads[1], **out))


# ---------------------------------------------------------------------------- plain form

def _scan(g, u, longest):
    """h_t = g_t h_{t-1} + u_t along the first axis, by doubling; g is 0 where a sequence (of at most `longest`) begins."""
    step = 1
    while step < longest:
        u = torch.cat([u[:step], u[step:] + g[step:] * u[:-step]])
        g = torch.cat([g[:step], g[step:] * g[:-step]])
        step *= 2
    return u


def _gates(st):
    """(log decay or None, decay, sigmoid of the input gate, unit factor or None) in 32 bits."""
    if st["case"]["mode"] == "precomputed":
        return None, st["a"], st["b"], None
    v = st["a"].float() + st["dt_bias"]
    lg = -st["A_log"].exp() * (v.clamp(min=0) + torch.log1p(torch.exp(-v.abs())))
    unit = torch.sqrt(-torch.expm1(2 * lg)) if st["case"]["unit"] else None
    return lg, lg.exp(), 1 / (1 + torch.exp(-st["b"].float())), unit


def _ends(st):
    cu = st["cu_seqlens"].long()
    return cu[:-1], cu[1:] - 1, st["slots"].long()


def _states(st, g, w):
    """Every token's state in 32 bits."""
    first, _, slots = _ends(st)
    u = w * st["x"].float()
    u[first] += g[first] * st["initial_state"][slots]
    g = g.clone()
    g[first] = 0
    return _scan(g, u, st["longest"])


def _final(st, h):
    _, last, slots = _ends(st)
    final = st["initial_state"].clone()
    final[slots] = h[last]
    return final


def _plain_recurrence(st):
    _, g, i, unit = _gates(st)
    h = _states(st, g, i if unit is None else i * unit)
    return {"y": h.to(st["x"].dtype), "final_state": _final(st, h)}


def _plain_recurrence_training(st):
    lg, g, i, unit = _gates(st)
    w = i if unit is None else i * unit
    h = _states(st, g, w)
    out = {"y": h.to(st["x"].dtype), "final_state": _final(st, h)}
    first, last, slots = _ends(st)
    before = torch.cat([h[:1], h[:-1]])
    before[first] = st["initial_state"][slots]
    carry = torch.cat([g[1:], g[:1]])
    carry[last] = 0
    arrives = st["dy"].float().index_add(0, last, st["dfinal"][slots])
    l = _scan(carry.flip(0), arrives.flip(0), st["longest"]).flip(0)  # noqa: E741
    x = st["x"].float()
    dw = l * x
    out["dx"] = (l * w).to(st["x"].dtype)
    out["d_initial_state"] = torch.zeros_like(st["initial_state"])
    out["d_initial_state"][slots] = g[first] * l[first]
    if lg is None:
        out["da"], out["db"] = l * before, dw
        return out
    dlg = l * before * g
    di = dw
    if unit is not None:
        di = dw * unit
        dlg = dlg - torch.where(unit > 0, dw * i * g * g / unit, 0.0)
    out["db"] = (di * i * (1 - i)).to(st["b"].dtype)
    v = st["a"].float() + st["dt_bias"]
    da = -dlg * st["A_log"].exp() / (1 + torch.exp(-v))
    out["da"] = da.to(st["a"].dtype)
    out["dA_log"] = (dlg * lg).sum(0, dtype=torch.float64).float()
    out["ddt_bias"] = da.sum(0, dtype=torch.float64).float()
    return out


def _eight_bits(y, group):
    """Rows [tokens, heads, d] in 32 bits as e4m3 values and the scales of each token, or of each group of channels."""
    rows = y.flatten(1) if group == 0 else y.flatten(1).unflatten(1, (-1, group))
    top = rows.abs().amax(-1)
    scale = torch.where(top > 0, top / torch.full_like(top, 448.0), 1.0)
    q = (rows / scale[..., None]).to(torch.float8_e4m3fn)
    return {"y": q.view(y.shape), "scale": scale}


def _silu(z):
    return z / (1 + torch.exp(-z))


def _plain_norm(x, st):
    case = st["case"]
    out = {}
    s = x.float()
    if st.get("residual") is not None:  # what is normalised is the sum as it is stored
        out["residual"] = (s + st["residual"].float()).to(x.dtype)
        s = out["residual"].float()
    y = s * torch.rsqrt((s * s).mean(-1, keepdim=True) + EPS) * st["weight"]
    if st["gate"] is not None:
        y = y * _silu(st["gate"].float().view(y.shape))
    if case.get("out", case["dtype"]) == case["dtype"]:
        out["y"] = y.to(x.dtype)
    else:
        out.update(_eight_bits(y, case["group"]))
    return out


def _plain_norm_training(st):
    out = _plain_norm(st["x"], st)
    s = out.get("residual", st["x"]).float()
    r = torch.rsqrt((s * s).mean(-1, keepdim=True) + EPS)
    n, dy = s * r, st["dy"].float()
    if st["gate"] is not None:
        z = st["gate"].float()
        sig = 1 / (1 + torch.exp(-z))
        out["dgate"] = (dy * n * st["weight"] * sig * (1 + z * (1 - sig))).to(st["gate"].dtype)
        dy = dy * z * sig
    out["dweight"] = (dy * n).sum((0, 1), dtype=torch.float64).float()
    dn = dy * st["weight"]
    dx = r * (dn - n * (dn * n).mean(-1, keepdim=True))
    if st["dresidual"] is not None:
        dx = dx + st["dresidual"].float()
    out["dx"] = dx.to(st["x"].dtype)
    return out


def _plain(st):
    kind = st["case"]["kind"]
    if kind == "recurrence":
        return _plain_recurrence(st)
    if kind == "recurrence training":
        return _plain_recurrence_training(st)
    if kind == "norm":
        return _plain_norm(st["x"], st)
    if kind == "norm training":
        return _plain_norm_training(st)
    out = _plain_recurrence(st)
    out.update(_plain_norm(out["y"].unflatten(1, (-1, st["case"]["head_dim"])), st))
    return out


def run(state):
    if not own:
        return _plain(state)
    outputs = [call.launch() for call in state["calls"]]
    case = state["case"]
    kind = case["kind"]
    if kind.startswith("norm"):
        names = ["y"] + ["residual"] * case["residual"] + ["scale"] * (case.get("out", case["dtype"]) != case["dtype"])
        out = dict(zip(names, outputs[0])) if len(names) > 1 else {"y": outputs[0]}
        if kind == "norm training":
            out.update(zip(["dx", "dweight"] + ["dgate"] * case["gate"], outputs[1]))
        return out
    out = {"y": outputs[0][0], "final_state": outputs[0][1]}
    if kind == "recurrence training":
        names = ["dx", "da", "db", "d_initial_state"] + ["dA_log", "ddt_bias"] * (case["mode"] == "raw")
        out.update(zip(names, outputs[1]))
    if kind == "layer":
        out["y"] = outputs[1]
    return out


# ---------------------------------------------------------------------------- in 64 bits

def _exact_gates(st, leaves):
    """Decay and input weight in 64 bits as functions of the leaves a, b (and A_log, dt_bias)."""
    if st["case"]["mode"] == "precomputed":
        return leaves["a"], leaves["b"]
    rate = torch.exp(leaves["A_log"]) * torch.logaddexp(leaves["a"] + leaves["dt_bias"], leaves["a"].new_zeros(()))
    g, w = torch.exp(-rate), torch.sigmoid(leaves["b"])
    return g, w * torch.sqrt(-torch.expm1(-2 * rate)) if st["case"]["unit"] else w


def _exact_recurrence(st):
    """Token by token, all sequences of one length index at once."""
    names = ["a", "b"] + (["A_log", "dt_bias"] if st["case"]["mode"] == "raw" else [])
    training = st["case"]["kind"] == "recurrence training"
    leaves = {n: st[n].double().requires_grad_(training) for n in names}
    with torch.set_grad_enabled(training):
        g, w = _exact_gates(st, leaves)
    gd, x = g.detach(), st["x"].double()
    u = w.detach() * x
    cu, slots = st["cu_seqlens"].tolist(), st["slots"].long()
    lens = [b - a for a, b in zip(cu, cu[1:])]
    order = sorted(range(len(lens)), key=lambda b: -lens[b])
    at = torch.tensor([cu[b] for b in order], device=DEVICE)
    h0 = st["initial_state"].double()[slots[order]]
    h, counts = u, [sum(n > t for n in lens) for t in range(max(lens))]
    prev, last = torch.empty_like(u), h0.clone()
    for t, n in enumerate(counts):
        i = at[:n] + t
        prev[i] = last[:n]
        last[:n] = gd[i] * last[:n] + h[i]
        h[i] = last[:n]
    final = st["initial_state"].double()
    final[slots[order]] = last
    out = {"y": h, "final_state": final}
    if not training:
        return out
    lam = st["dy"].double()
    back = st["dfinal"].double()[slots[order]]
    for t in range(len(counts) - 1, -1, -1):
        i = at[:counts[t]] + t
        lam[i] += back[:counts[t]]
        back[:counts[t]] = gd[i] * lam[i]
    out["d_initial_state"] = torch.zeros_like(final)
    out["d_initial_state"][slots[order]] = back
    out["dx"] = lam * w.detach()
    grads = torch.autograd.grad([g, w], list(leaves.values()), [lam * prev, lam * x])
    names = {"a": "da", "b": "db", "A_log": "dA_log", "dt_bias": "ddt_bias"}
    out.update({names[n]: d for n, d in zip(leaves, grads)})
    return out


def _exact_norm(x, st):
    case, out = st["case"], {}
    training = case["kind"] == "norm training"
    if st.get("residual") is not None:
        x = (x.double() + st["residual"].double()).to(x.dtype)
        out["residual"] = x.double()
    x, weight = x.double().requires_grad_(training), st["weight"].double().requires_grad_(training)
    gate = None if st["gate"] is None else st["gate"].double().view(x.shape).requires_grad_(training)
    with torch.set_grad_enabled(training):
        y = x / torch.sqrt(torch.linalg.vector_norm(x, dim=-1, keepdim=True) ** 2 / x.shape[-1] + EPS) * weight
        if gate is not None:
            y = y * gate * torch.sigmoid(gate)
    if training:
        leaves = [x, weight] + ([gate] if gate is not None else [])
        dx, out["dweight"], *rest = torch.autograd.grad(y, leaves, st["dy"].double())
        out["dx"] = dx if st["dresidual"] is None else dx + st["dresidual"].double()
        if rest:
            out["dgate"] = rest[0]
        y = y.detach()
    if case.get("out", case["dtype"]) == case["dtype"]:
        return {"y": y, **out}
    rows = y.reshape(y.shape[0], -1, case["group"] or y[0].numel())
    scale = torch.linalg.vector_norm(rows, ord=math.inf, dim=-1) / 448
    scale[scale == 0] = 1
    z = rows / scale[..., None]
    step = torch.exp2(torch.floor(torch.log2(z.abs().clamp(min=2.0 ** -6))) - 3)
    return {"y": ((z / step).round() * step).view(y.shape), "scale": scale if case["group"] else scale[:, 0], **out}


def exact(case, seed):
    st = prepare(case, seed)
    if case["kind"].startswith("norm"):
        return _exact_norm(st["x"], st)
    out = _exact_recurrence(st)
    if case["kind"] == "layer":
        y = out["y"].to(st["x"].dtype).unflatten(1, (-1, case["head_dim"]))
        out.update(_exact_norm(y, st))
    return out
