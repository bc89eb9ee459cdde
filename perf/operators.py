"""Cases of the softmax-attention operators that sit beside the gated delta rule in a hybrid
decoder: rotary positions, the (quantised) paged key-value cache, and attention of new tokens
over that cache.

`run(state)` computes a case either in its plain form (elementary torch operations in 32 bits,
rounded once at the end) or, where `own` is set, with the calls a user makes of the library.
`exact(case, seed)` computes the same from the definitions in 64 bits.
"""
import math

import torch

own = False

DEVICE = "cuda"
GOLDEN = 0.6180339887498949
ROPE_BASE = 1.0e6
QUANTISED = ("float8_e4m3fn", "int8")


# ---------------------------------------------------------------------------- cases

def listed():
    return [
        # One decode step of a batch of 64: launch latency is all of it.
        dict(name="rotary decode", kind="rotary", tokens=64, q_heads=32, k_heads=8, head_dim=128, rotary_dim=128,
             interleaved=False, inverse=False, dtype="float16", positions=32768),
        # A packed prompt batch of a layer that rotates a quarter of a 256-wide head, at long positions.
        dict(name="rotary prompt partial", kind="rotary", tokens=8192, q_heads=16, k_heads=2, head_dim=256,
             rotary_dim=64, interleaved=False, inverse=False, dtype="bfloat16", positions=262144),
        # The gradient of the interleaved form in a 32-bit training step, an odd number of tokens.
        dict(name="rotary gradient interleaved", kind="rotary", tokens=4111, q_heads=8, k_heads=8, head_dim=64,
             rotary_dim=64, interleaved=True, inverse=True, dtype="float32", positions=8192),
        # Short prompts written to an 8-bit floating cache and read back as the next chunk's prefix.
        dict(name="cache fp8 short prompts", kind="cache", seqs=4, lo=0, hi=60, new=17, kv_heads=8, head_dim=128,
             rotary_dim=128, page=16, heads_first=False, cache="float8_e4m3fn", dtype="float16"),
        # A chunk of 512 tokens of each of 8 prompts written to an 8-bit integer cache, the contexts read back.
        dict(name="cache int8 chunked prompt", kind="cache", seqs=8, lo=512, hi=8192, new=512, kv_heads=8,
             head_dim=128, rotary_dim=64, page=64, heads_first=True, cache="int8", dtype="bfloat16"),
        # One user, a short chat: the smallest attention call.
        dict(name="attention one short", kind="attention", seqs=1, lo=100, hi=100, new=1, q_heads=32, kv_heads=8,
             head_dim=128, page=16, heads_first=False, cache="float16", dtype="float16"),
        # One user, one very long document: the cache's length has to be split over the whole GPU.
        dict(name="attention one long", kind="attention", seqs=1, lo=131071, hi=131071, new=1, q_heads=32,
             kv_heads=8, head_dim=128, page=32, heads_first=False, cache="float16", dtype="float16"),
        # A serving batch of ragged long contexts, two wide key heads in an 8-bit floating cache.
        dict(name="attention ragged fp8 wide", kind="attention", seqs=64, lo=1, hi=16384, new=1, q_heads=16,
             kv_heads=2, head_dim=256, page=64, heads_first=True, cache="float8_e4m3fn", dtype="bfloat16"),
        # Verification of four drafted tokens a request (causal among themselves).
        dict(name="attention verify drafts", kind="attention", seqs=16, lo=1000, hi=8191, new=4, q_heads=32,
             kv_heads=4, head_dim=128, page=16, heads_first=False, cache="bfloat16", dtype="bfloat16"),
        # Many short requests, some with nothing cached yet, groups of seven, an 8-bit integer cache.
        dict(name="attention many int8", kind="attention", seqs=256, lo=0, hi=1024, new=1, q_heads=28, kv_heads=4,
             head_dim=128, page=16, heads_first=False, cache="int8", dtype="float16"),
        # Every query head with its own keys, 32-bit values, pages of seven tokens.
        dict(name="attention heads fp32", kind="attention", seqs=8, lo=17, hi=4099, new=1, q_heads=8, kv_heads=8,
             head_dim=64, page=7, heads_first=False, cache="float32", dtype="float32"),
        # A whole decode step: rotate q and k, write k and v, attend.
        dict(name="decode step", kind="step", seqs=64, lo=128, hi=2048, new=1, q_heads=32, kv_heads=8, head_dim=128,
             rotary_dim=128, page=16, heads_first=True, cache="float16", dtype="float16"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["rotary", "cache", "attention", "attention", "attention", "step"])
    d = rng.choice([64, 128, 256])
    dtype = rng.choice(["float16", "bfloat16"])
    if kind == "rotary":
        interleaved = rng.random() < 0.4
        kh = rng.choice([1, 2, 4, 8])
        dtype = rng.choice(["float16", "bfloat16", "float32"])
        tokens = _log_int(rng, 1, 8192)
        while tokens * kh * 5 * d > 8192 * 18 * 256:
            tokens //= 2
        return dict(kind=kind, tokens=tokens, q_heads=kh * rng.choice([1, 2, 4]), k_heads=kh, head_dim=d,
                    rotary_dim=rng.choice([d, d // 2, d // 4]), interleaved=interleaved,
                    inverse=rng.random() < 0.3, dtype=dtype, positions=_log_int(rng, 1024, 262144))
    page = rng.choice([5, 16, 16, 32, 64, 128])
    heads_first = rng.random() < 0.5
    kv_heads = rng.choice([1, 2, 3, 4, 8])
    if kind == "cache":
        seqs = _log_int(rng, 1, 32)
        budget = max(64, 32768 * 8 * 128 // (seqs * kv_heads * d))
        hi = _log_int(rng, 16, min(budget, 16384))
        return dict(kind=kind, seqs=seqs, lo=rng.choice([0, hi // 4, hi]), hi=hi, new=_log_int(rng, 1, min(budget, 512)),
                    kv_heads=kv_heads, head_dim=d, rotary_dim=rng.choice([d, d // 2, d // 4]), page=page,
                    heads_first=heads_first, cache=rng.choice([dtype, "float8_e4m3fn", "int8", "float8_e4m3fn", "int8"]),
                    dtype=dtype)
    group = rng.choice([1, 2, 4, 5, 6, 7, 8, 12, 16])
    seqs = _log_int(rng, 1, 256)
    if kind == "step":
        cache = dtype
    else:
        cache = rng.choice([dtype, "float8_e4m3fn", "int8"])
        if rng.random() < 0.1:
            dtype = cache = "float32"
    budget = (96 if seqs == 1 else 48) * 1024 * 1024 // (seqs * kv_heads * d) // (2 if dtype == "float32" else 1)
    hi = _log_int(rng, 1, max(1, min(budget, 131071)))
    new = 1 if kind == "step" or rng.random() < 0.6 else rng.randint(2, 8)
    lo = rng.choice([0, 1, hi // 2, hi])
    if kind == "step":
        lo, hi = max(1, lo), max(1, hi)
    c = dict(kind=kind, seqs=seqs, lo=lo, hi=hi, new=new, q_heads=group * kv_heads, kv_heads=kv_heads, head_dim=d,
             page=page, heads_first=heads_first, cache=cache, dtype=dtype)
    if kind == "step":
        c["rotary_dim"] = rng.choice([d, d // 2, d // 4])
    return c


# ---------------------------------------------------------------------------- sizes

def _lens(case):
    """Each sequence's length: spread evenly over [lo, hi] in a scattered order (for "cache" the
    context before the new tokens, otherwise all that attention sees)."""
    lo, hi, n = case["lo"], case["hi"], case["seqs"]
    if n == 1:
        return [hi]
    return [lo + int((hi - lo + 1) * ((i + 1) * GOLDEN % 1.0)) for i in range(n)]


def _bytes(dtype):
    return {"float32": 4, "float16": 2, "bfloat16": 2, "float8_e4m3fn": 1, "int8": 1}[dtype]


def work(case):
    io = _bytes(case["dtype"])
    if case["kind"] == "rotary":
        t, heads, d, r = case["tokens"], case["q_heads"] + case["k_heads"], case["head_dim"], case["rotary_dim"]
        table = min(t, case["positions"]) * r * 4
        return {"bytes": 2 * t * heads * d * io + table + 4 * t, "flops": 3 * t * heads * r}
    h, d, n, seqs = case["kv_heads"], case["head_dim"], case["new"], case["seqs"]
    row = h * (d * _bytes(case["cache"]) + (4 if case["cache"] in QUANTISED else 0))  # one token's keys or values
    lens = _lens(case)
    if case["kind"] == "cache":
        new, total = seqs * n, sum(lens) + seqs * n
        moved = 2 * (new * h * d * io + new * row + sum(lens) * row + total * h * d * io)
        return {"bytes": moved + new * (case["rotary_dim"] * 4 + 8) + 4 * total // case["page"],
                "flops": 2 * h * d * (2 * total + 3 * new)}
    heads = case["q_heads"]
    seen = sum(lens)
    moved = 2 * seen * row + 2 * seqs * n * heads * d * io + 4 * seen // case["page"] + 4 * seqs
    pairs = sum(max(0, l - n + 1 + i) for l in lens for i in range(n))
    if case["kind"] == "step":
        moved += seqs * (2 * h * d * io + case["rotary_dim"] * 4 + 8)
    return {"bytes": moved, "flops": 4 * heads * d * pairs}


# ---------------------------------------------------------------------------- inputs

def _table(positions, rotary_dim):
    """cos | sin of every position's angles, [positions, rotary_dim] in 32 bits."""
    freq = ROPE_BASE ** (-torch.arange(0, rotary_dim, 2, dtype=torch.float64, device=DEVICE) / rotary_dim)
    angle = torch.arange(positions, dtype=torch.float64, device=DEVICE)[:, None] * freq
    return torch.cat([angle.cos(), angle.sin()], 1).float()


def _quantise(x, dtype):
    """Rows of x (32 bits) as 8-bit values and each row's scale: for e4m3 the smallest power of two
    that brings the row's largest magnitude to at most 448, for int8 that magnitude / 127."""
    top = x.abs().amax(-1)
    if dtype == "int8":
        scale = top / torch.full_like(top, 127.0)
        scale = torch.where(top > 0, scale, torch.ones_like(top))
        q = (x / scale[..., None]).round().clamp(-127, 127).to(torch.int8)
    else:
        mantissa, exponent = torch.frexp(top)
        exponent = (exponent - torch.where(mantissa > 0.875, 8, 9)).clamp(min=-120)
        scale = torch.where(top > 0, torch.ldexp(torch.ones_like(top), exponent), torch.ones_like(top))
        q = (x / scale[..., None]).to(torch.float8_e4m3fn)
    return q, scale


def _slots(table, positions, page):
    """Row index (page * page size + offset) of each sequence's given positions, [seqs, n]."""
    return table.long().gather(1, positions // page) * page + positions % page


def _block_table(lens, page, g):
    """Pages in no order; entries past a sequence's end are invalid.  Returns the table and the pool's pages."""
    need = torch.tensor([(l + page - 1) // page for l in lens])
    total, width = int(need.sum()), max(1, int(need.max()))
    table = torch.full((len(lens), width), -1, dtype=torch.int32, device=DEVICE)
    owned = (torch.arange(width)[None] < need[:, None]).to(DEVICE)
    table[owned] = torch.randperm(total + 3, generator=g, device=DEVICE)[:total].to(torch.int32)
    return table, total + 3


def _stored(x, heads_first):
    """[pages, page, heads, ...] with the same values, each head's page contiguous if asked."""
    return x.transpose(1, 2).contiguous().transpose(1, 2) if heads_first else x.contiguous()


def _pool(case, table, pages, lens, g):
    """One half (keys or values) of a paged cache that holds `lens` tokens of each sequence: values
    and scales (None unless quantised).  Rows that hold no token keep what was there before, which
    is NaN where the type has one."""
    page, h, d, dtype = case["page"], case["kv_heads"], case["head_dim"], case["cache"]
    gain = 0.5 + torch.rand(h, d, generator=g, device=DEVICE)
    gain[:, :: d // 4] *= 4.0  # a few channels stand out, as they do in trained keys
    x = torch.randn(pages, page, h, d, generator=g, device=DEVICE) * gain
    length = torch.tensor(lens, device=DEVICE)
    t = torch.arange(table.shape[1] * page, device=DEVICE)
    held = t[None] < length[:, None]
    free = torch.ones(pages * page, dtype=torch.bool, device=DEVICE)
    free[(table.long()[:, t // page] * page + t % page)[held]] = False
    x.view(pages * page, h, d)[free] = float("nan")
    scale = None
    if dtype in QUANTISED:
        x, scale = _quantise(x, dtype)
        scale.view(pages * page, h)[free] = float("nan")
        scale = _stored(scale, case["heads_first"])
    return _stored(x.to(getattr(torch, dtype)), case["heads_first"]), scale


def _normal(g, *shape, dtype):
    return torch.randn(*shape, generator=g, device=DEVICE).to(getattr(torch, dtype))


def prepare(case, seed):
    g = torch.Generator(DEVICE).manual_seed(seed)
    kind, d, dtype = case["kind"], case["head_dim"], case["dtype"]
    st = {"case": dict(case)}
    if kind == "rotary":
        t = case["tokens"]
        st["q"] = _normal(g, t, case["q_heads"], d, dtype=dtype)
        st["k"] = _normal(g, t, case["k_heads"], d, dtype=dtype)
        st["positions"] = torch.randint(0, case["positions"], (t,), generator=g, device=DEVICE, dtype=torch.int32)
        st["table"] = _table(case["positions"], case["rotary_dim"])
    else:
        n, seqs, h, page = case["new"], case["seqs"], case["kv_heads"], case["page"]
        lens = _lens(case)
        ends = [l + n for l in lens] if kind == "cache" else lens
        held = ends if kind == "attention" else [e - n for e in ends]
        st["block_table"], pages = _block_table(ends, page, g)
        st["k_cache"], st["k_scale"] = _pool(case, st["block_table"], pages, held, g)
        st["v_cache"], st["v_scale"] = _pool(case, st["block_table"], pages, held, g)
        st["kv_lens"] = torch.tensor(ends, dtype=torch.int32, device=DEVICE)
        if kind != "attention":
            at = st["kv_lens"].long()[:, None] - n + torch.arange(n, device=DEVICE)
            st["positions"] = at.flatten().to(torch.int32)
            st["slots"] = _slots(st["block_table"], at, page).flatten().to(torch.int32)
            st["table"] = _table(max(ends), case["rotary_dim"])
            st["k"] = _normal(g, seqs * n, h, d, dtype=dtype)
            st["v"] = _normal(g, seqs * n, h, d, dtype=dtype)
        if kind == "cache":
            st["total"] = sum(ends)
            st["cu_seqlens"] = torch.tensor([0] + ends, device=DEVICE).cumsum(0).to(torch.int32)
        else:
            st["q"] = _normal(g, seqs * n, case["q_heads"], d, dtype=dtype)
            st["cu_seqlens"] = torch.arange(0, seqs * n + 1, n, dtype=torch.int32, device=DEVICE) if n > 1 else None
    if own:
        _plan(st)
    return st


def _plan(st):
    """The call objects a serving program keeps for its fixed buffers (arguments checked and resolved once)."""
    import gated_delta_rule_gateddeltanet_gb300 as gdn

    case = st["case"]
    kind = case["kind"]
    if kind == "rotary":
        st["calls"] = [gdn.RotaryCall(st["q"], st["k"], st["positions"], st["table"],
                                      interleaved=case["interleaved"], inverse=case["inverse"])]
        return
    cache = gdn.PagedKVCache(st["k_cache"], st["v_cache"], st["k_scale"], st["v_scale"])
    if kind == "cache":
        st["calls"] = [gdn.KVCacheWriteCall(st["k"], st["v"], cache, st["slots"], positions=st["positions"],
                                            table=st["table"]),
                       gdn.KVCacheReadCall(cache, st["block_table"], st["cu_seqlens"], st["total"],
                                           dtype=getattr(torch, case["dtype"]))]
        return
    q, st["calls"] = st["q"], []
    if kind == "step":
        write = gdn.KVCacheWriteCall(st["k"], st["v"], cache, st["slots"], positions=st["positions"],
                                     table=st["table"], q=q)
        q = st["q_rotated"] = write.outputs
        st["calls"].append(write)
    st["calls"].append(gdn.PagedAttentionCall(q, cache, st["block_table"], st["kv_lens"],
                                              cu_seqlens=st["cu_seqlens"]))


# ---------------------------------------------------------------------------- plain form

def _rotate(x, table, positions, interleaved, inverse):
    """x [tokens, heads, d] in 32 bits with its first rotary_dim channels turned by the positions' angles."""
    r = table.shape[1]
    row = table[positions.long()][:, None]
    c, s = row[..., : r // 2], row[..., r // 2:]
    s = -s if inverse else s
    a, b = (x[..., 0:r:2], x[..., 1:r:2]) if interleaved else (x[..., : r // 2], x[..., r // 2: r])
    y = (a * c - b * s, b * c + a * s)
    y = torch.stack(y, -1).flatten(-2) if interleaved else torch.cat(y, -1)
    return torch.cat([y, x[..., r:]], -1)


def _write(cache, scale, x, slots):
    """Rows x (32 bits) into the cache at `slots`, quantised where the cache has scales."""
    page = cache.shape[1]
    at = (slots.long() // page, slots.long() % page)
    if scale is None:
        cache[at] = x.to(cache.dtype)
        return
    q, s = _quantise(x, str(cache.dtype).replace("torch.", ""))
    cache.view(torch.uint8)[at] = q.view(torch.uint8)
    scale[at] = s


def _rows(cache, scale, pages, offsets):
    """Cache rows at (pages, offsets) in 32 bits."""
    if scale is None:
        return cache[pages, offsets].float()
    return cache.view(torch.uint8)[pages, offsets].view(cache.dtype).float() * scale[pages, offsets][..., None]


def _attend(st, q):
    case = st["case"]
    n, h, d, page = case["new"], case["kv_heads"], case["head_dim"], case["page"]
    table, lens = st["block_table"], st["kv_lens"].long()
    seqs, group = table.shape[0], case["q_heads"] // h
    t = torch.arange(table.shape[1] * page, device=q.device)
    pages = table.long().clamp(min=0)[:, t // page]
    offsets = (t % page).expand_as(pages)
    inside = (t < lens[:, None])[..., None, None]
    k = torch.where(inside, _rows(st["k_cache"], st["k_scale"], pages, offsets), 0.0)
    v = torch.where(inside, _rows(st["v_cache"], st["v_scale"], pages, offsets), 0.0)
    q = q.float().view(seqs, n, h, group, d).transpose(1, 2).reshape(seqs, h, n * group, d)
    score = (q @ k.permute(0, 2, 3, 1)) * d ** -0.5
    last = lens[:, None] - n + torch.arange(n, device=q.device)  # a query sees positions up to its own
    seen = (t <= last[..., None]).repeat_interleave(group, 1)[:, None]
    score = torch.where(seen, score, -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.where(seen, (score - top).exp(), 0.0)
    total = p.sum(-1, keepdim=True)
    out = torch.where(total > 0, (p @ v.transpose(1, 2)) / total, 0.0)
    return out.view(seqs, h, n, group, d).transpose(1, 2).reshape(seqs * n, h * group, d).to(st["q"].dtype)


def _plain(st):
    case = st["case"]
    kind = case["kind"]
    if kind == "rotary":
        turn = (st["table"], st["positions"], case["interleaved"], case["inverse"])
        return {"q": _rotate(st["q"].float(), *turn).to(st["q"].dtype),
                "k": _rotate(st["k"].float(), *turn).to(st["k"].dtype)}
    if kind == "attention":
        return {"out": _attend(st, st["q"])}
    turn = (st["table"], st["positions"], False, False)
    _write(st["k_cache"], st["k_scale"], _rotate(st["k"].float(), *turn), st["slots"])
    _write(st["v_cache"], st["v_scale"], st["v"].float(), st["slots"])
    if kind == "step":
        q = _rotate(st["q"].float(), *turn).to(st["q"].dtype)
        return {"out": _attend(st, q), "q": q, "k_cache": st["k_cache"], "v_cache": st["v_cache"]}
    page, cu = case["page"], st["cu_seqlens"].long()
    row = torch.arange(st["total"], device=cu.device)
    seq = torch.searchsorted(cu, row, right=True) - 1
    t = row - cu[seq]
    pages, offsets = st["block_table"].long()[seq, t // page], t % page
    return {"k": _rows(st["k_cache"], st["k_scale"], pages, offsets).to(st["k"].dtype),
            "v": _rows(st["v_cache"], st["v_scale"], pages, offsets).to(st["v"].dtype)}


def run(state):
    if not own:
        return _plain(state)
    outputs = [call.launch() for call in state["calls"]]
    kind = state["case"]["kind"]
    if kind in ("rotary", "cache"):
        return {"q": outputs[-1][0], "k": outputs[-1][1]} if kind == "rotary" else dict(zip("kv", outputs[-1]))
    if kind == "attention":
        return {"out": outputs[-1]}
    return {"out": outputs[-1], "q": state["q_rotated"], "k_cache": state["k_cache"], "v_cache": state["v_cache"]}


# ---------------------------------------------------------------------------- in 64 bits

def _turned(x, st, interleaved=False, inverse=False):
    """Rotation in 64 bits: each channel pair is a complex number times e^(i angle)."""
    r = st["table"].shape[1]
    row = st["table"].double()[st["positions"].long()]
    turn = torch.complex(row[:, : r // 2], -row[:, r // 2:] if inverse else row[:, r // 2:])[:, None]
    x = x.double()
    head = x[..., :r].unflatten(-1, (r // 2, 2) if interleaved else (2, r // 2))
    pair = head if interleaved else head.transpose(-1, -2)
    y = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * turn)
    y = y if interleaved else y.transpose(-1, -2)
    return torch.cat([y.flatten(-2), x[..., r:]], -1)


def _held(x, dtype):
    """The values (64 bits) that a cache of `dtype` holds for rows x: what reading them back gives."""
    if dtype not in QUANTISED:
        return x.to(getattr(torch, dtype)).double()
    top = x.abs().amax(-1, keepdim=True)
    if dtype == "int8":
        scale = (top / 127).float().double()
        return (x / scale).round() * scale
    scale = torch.exp2(torch.ceil(torch.log2(top / 448)))
    y = x / scale
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    return (y / step).round() * step * scale


def _sequence(st, b, length, half):
    """Sequence b's cached rows in 64 bits, [length, heads, d]."""
    page = st["case"]["page"]
    t = torch.arange(length, device=DEVICE)
    at = (st["block_table"][b, t // page].long(), t % page)
    if st[half + "_scale"] is None:
        return st[half + "_cache"][at].double()
    x = st[half + "_cache"]
    return x.view(torch.uint8)[at].view(x.dtype).double() * st[half + "_scale"][at].double()[..., None]


def exact(case, seed):
    st = prepare(case, seed)
    kind, n, h = case["kind"], case.get("new"), case.get("kv_heads")
    if kind == "rotary":
        return {name: _turned(st[name], st, case["interleaved"], case["inverse"]) for name in ("q", "k")}
    ends = st["kv_lens"].tolist()
    fresh = {}
    if kind != "attention":
        fresh = {"k": _held(_turned(st["k"], st), case["cache"]), "v": _held(st["v"].double(), case["cache"])}
    rows = {half: [] for half in "kv"}
    outs = []
    q = st.get("q")
    if kind == "step":
        q = _turned(q, st).to(q.dtype)
    for b, end in enumerate(ends):
        both = {}
        for half in "kv":
            x = _sequence(st, b, end, half)
            if fresh:
                x[end - n:] = fresh[half][b * n:(b + 1) * n]
            both[half] = x
        if kind == "cache":
            for half in "kv":
                rows[half].append(both[half])
            continue
        for i in range(n):
            sees = end - n + 1 + i
            if sees <= 0:
                outs.append(torch.zeros(case["q_heads"], case["head_dim"], dtype=torch.float64, device=DEVICE))
                continue
            query = q[b * n + i].double().view(h, -1, case["head_dim"])
            score = torch.einsum("hgd,thd->hgt", query, both["k"][:sees]) / math.sqrt(case["head_dim"])
            outs.append(torch.einsum("hgt,thd->hgd", score.softmax(-1), both["v"][:sees]).flatten(0, 1))
    if kind == "cache":
        return {half: torch.cat(rows[half]) for half in "kv"}
    out = {"out": torch.stack(outs)}
    if kind == "step":
        page = case["page"]
        at = (st["slots"].long() // page, st["slots"].long() % page)
        for half in "kv":
            st[half + "_cache"][at] = fresh[half].to(st[half + "_cache"].dtype)
            out[half + "_cache"] = st[half + "_cache"].double()
        out["q"] = q.double()
    return out
