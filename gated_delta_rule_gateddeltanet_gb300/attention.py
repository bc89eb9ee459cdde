"""Python binding of the softmax-attention operators of include/gdn.h: rotary
positions, the paged key-value cache and attention of new tokens over it.

As in the package's ``__init__``, this only marshals arguments: it checks
types, devices and shapes, allocates outputs that the caller did not pass, and
calls the library on the current torch stream.

Every operator has a function (checks and launches) and a call object (checks
once; ``launch()`` is then one C-ABI call on the same buffers, for loops that
refill fixed inputs and for CUDA graphs):

    rotary_table(...)     -> table [P, rotary_dim]
    rotary(...)           / RotaryCall         -> (q_out, k_out)
    kv_cache_write(...)   / KVCacheWriteCall   -> q_out or None (the cache is written in place)
    kv_cache_read(...)    / KVCacheReadCall    -> (k, v)
    paged_attention(...)  / PagedAttentionCall -> output, or (output, lse)
"""
from __future__ import annotations

import ctypes

import torch

from . import DTYPE, GdnError, _check, _ptr, _shape, _token_stride, load_library

CACHE_DTYPE = {**DTYPE, torch.float8_e4m3fn: 3, torch.int8: 4}
ROPE_SCALING = {"none": 0, "linear": 1, "ntk": 2, "by_parts": 3, "yarn": 4}

_i32, _i64, _f32, _f64, _p = ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_double, ctypes.c_void_p


class RotaryTableArgs(ctypes.Structure):
    """Mirror of ``gdn_rotary_table_args``."""
    _fields_ = [("max_positions", _i32), ("rotary_dim", _i32), ("scaling", _i32), ("original_positions", _i32),
                ("base", _f64), ("factor", _f64), ("beta_fast", _f64), ("beta_slow", _f64),
                ("attention_factor", _f64), ("table", _p)]


class RotaryArgs(ctypes.Structure):
    """Mirror of ``gdn_rotary_args``."""
    _fields_ = [("total_tokens", _i32), ("num_q_heads", _i32), ("num_k_heads", _i32), ("head_dim", _i32),
                ("rotary_dim", _i32), ("max_positions", _i32), ("io_dtype", _i32), ("interleaved", _i32),
                ("inverse", _i32), ("q_stride", _i64), ("k_stride", _i64), ("q_out_stride", _i64),
                ("k_out_stride", _i64), ("q", _p), ("k", _p), ("q_out", _p), ("k_out", _p), ("positions", _p),
                ("table", _p), ("status", _p)]


class KVCacheArgs(ctypes.Structure):
    """Mirror of ``gdn_kv_cache``."""
    _fields_ = [("num_pages", _i32), ("page_size", _i32), ("num_kv_heads", _i32), ("head_dim", _i32),
                ("cache_dtype", _i32), ("page_stride", _i64), ("token_stride", _i64), ("head_stride", _i64),
                ("scale_page_stride", _i64), ("scale_token_stride", _i64), ("scale_head_stride", _i64),
                ("k", _p), ("v", _p), ("k_scale", _p), ("v_scale", _p)]


class KVWriteArgs(ctypes.Structure):
    """Mirror of ``gdn_kv_write_args``."""
    _fields_ = [("cache", KVCacheArgs), ("total_tokens", _i32), ("num_q_heads", _i32), ("rotary_dim", _i32),
                ("max_positions", _i32), ("io_dtype", _i32), ("interleaved", _i32), ("k_stride", _i64),
                ("v_stride", _i64), ("q_stride", _i64), ("q_out_stride", _i64), ("k", _p), ("v", _p), ("q", _p),
                ("q_out", _p), ("slots", _p), ("positions", _p), ("table", _p), ("status", _p)]


class KVReadArgs(ctypes.Structure):
    """Mirror of ``gdn_kv_read_args``."""
    _fields_ = [("cache", KVCacheArgs), ("num_seqs", _i32), ("total_tokens", _i32), ("pages_per_seq", _i32),
                ("io_dtype", _i32), ("block_table_stride", _i64), ("block_table", _p), ("cu_seqlens", _p),
                ("k_out", _p), ("v_out", _p), ("status", _p)]


class PagedAttentionArgs(ctypes.Structure):
    """Mirror of ``gdn_paged_attention_args``."""
    _fields_ = [("cache", KVCacheArgs), ("num_seqs", _i32), ("total_tokens", _i32), ("num_q_heads", _i32),
                ("pages_per_seq", _i32), ("window", _i32), ("max_seqlen", _i32), ("io_dtype", _i32),
                ("scale", _f32), ("block_table_stride", _i64), ("q_stride", _i64), ("q", _p), ("block_table", _p),
                ("kv_lens", _p), ("cu_seqlens", _p), ("output", _p), ("lse", _p), ("status", _p),
                ("workspace", _p), ("workspace_bytes", ctypes.c_size_t)]


ENTRY_POINTS = {"gdn_rotary_table": RotaryTableArgs, "gdn_rotary": RotaryArgs, "gdn_kv_cache_write": KVWriteArgs,
                "gdn_kv_cache_read": KVReadArgs, "gdn_paged_attention": PagedAttentionArgs}


def declare(lib):
    """Argument types of this module's entry points (called when the library is loaded)."""
    for name, args in ENTRY_POINTS.items():
        f = getattr(lib, name)
        f.restype, f.argtypes = _i32, [ctypes.POINTER(args), _p]
    f = lib.gdn_paged_attention_workspace_size
    f.restype, f.argtypes = _i32, [ctypes.POINTER(PagedAttentionArgs), ctypes.POINTER(ctypes.c_size_t)]


class _Call:
    """A C-ABI call with its arguments resolved; the tensors must stay alive and in place."""

    def _resolve(self, name, args, outputs, keep, device):
        self.args, self.outputs, self._name, self._keep, self._device = args, outputs, name, keep, device
        self._ref = ctypes.byref(args)
        self._fn, self._index = None, device.index

    def launch(self, stream=None):
        """Runs the call on ``stream`` (a torch.cuda.Stream; default: the current stream); returns ``outputs``."""
        if self._fn is None:
            if self._device.type != "cuda":
                raise ValueError(f"{self._name}: tensors must be on a GPU, got {self._device}")
            self._fn = getattr(load_library(), self._name)
        # (the raw handle of the current stream: building a Stream object takes 2 of a launch's 5 us)
        rc = self._fn(self._ref, torch._C._cuda_getCurrentRawStream(self._index) if stream is None else stream.cuda_stream)
        if rc != 0:
            raise GdnError(rc, self._name)
        return self.outputs


def _int32(x, name):
    """``x`` as the int32 of a C struct, which would take a larger number modulo 2^32."""
    x = int(x)
    if not -2 ** 31 <= x < 2 ** 31:
        raise ValueError(f"{name} must fit in 32 bits, got {x}")
    return x


def _io(t, name):
    if t.dtype not in DTYPE:
        raise TypeError(f"{name}: unsupported dtype {t.dtype}")
    return DTYPE[t.dtype]


def _index(t, name, shape, device):
    """An int32 index tensor of the given shape."""
    _check(t, name, dtype=torch.int32, device=device)
    _shape(t, name, shape)


def _status(t, device):
    _check(t, "status", dtype=torch.int32, device=device)
    if t is not None and t.numel() < 1:
        raise ValueError("status must hold one int32")


def _block_table(t, seqs, device):
    """(pages_per_seq, row stride) of a [seqs, pages] int32 block table whose rows may lie apart."""
    _check(t, "block_table", dtype=torch.int32, device=device, contiguous=False)
    if t.dim() != 2 or t.shape[0] != seqs:
        raise ValueError(f"block_table must be [{seqs}, pages], got {tuple(t.shape)}")
    if t.shape[1] > 1 and t.stride(1) != 1:
        raise ValueError("block_table: a row's entries must be contiguous")
    if seqs > 1 and t.shape[1] > 0 and t.stride(0) == 0:  # (0 is the C ABI's word for no gap)
        raise ValueError("block_table: rows must not share memory (an expanded view)")
    return t.shape[1], t.stride(0) if seqs > 1 and t.shape[1] > 0 else t.shape[1]


def _cu_seqlens(t, device):
    _check(t, "cu_seqlens", dtype=torch.int32, device=device)
    if t.dim() != 1 or t.shape[0] < 1:
        raise ValueError("cu_seqlens must be one-dimensional [B + 1]")
    return t.shape[0] - 1


def _table(t, device):
    """(max_positions, rotary_dim) of a rotary table."""
    _check(t, "table", dtype=torch.float32, device=device)
    if t.dim() != 2:
        raise ValueError("table must be [positions, rotary_dim]")
    return t.shape


def _heads_out(out, name, like, device):
    """An output shaped like ``like`` [T, heads, d], allocated if absent; its heads lie next to each other."""
    if out is None:
        out = torch.empty(tuple(like.shape), dtype=like.dtype, device=device)
    _check(out, name, dtype=like.dtype, device=device, contiguous=False)
    _shape(out, name, like.shape)
    return out


def rotary_table(max_positions, rotary_dim, *, base=10000.0, scaling="none", factor=1.0, original_positions=0,
                 beta_fast=32.0, beta_slow=1.0, attention_factor=0.0, device="cuda", table=None):
    """Cosines and sines of positions 0 .. max_positions - 1 (C ABI
    ``gdn_rotary_table``): [max_positions, rotary_dim] fp32, a row holding the
    cosines of its rotary_dim / 2 pairs and then their sines.  ``scaling``:
    "none", "linear", "ntk", "by_parts" or "yarn" (see ``GDN_ROPE_*``), with
    ``factor`` and, for the last two, ``original_positions``, ``beta_fast`` and
    ``beta_slow``."""
    if table is None:
        table = torch.empty((max_positions, rotary_dim), dtype=torch.float32, device=device)
    _check(table, "table", dtype=torch.float32)
    _shape(table, "table", (max_positions, rotary_dim))
    a = RotaryTableArgs(int(max_positions), int(rotary_dim), ROPE_SCALING[scaling],
                        _int32(original_positions, "original_positions"),
                        float(base), float(factor), float(beta_fast), float(beta_slow), float(attention_factor),
                        _ptr(table))
    call = _Call()
    call._resolve("gdn_rotary_table", a, table, (table,), table.device)
    return call.launch()


class RotaryCall(_Call):
    """Rotates the first ``table.shape[1]`` channels of every head of q and k
    by their token's position (C ABI ``gdn_rotary``).  q: [T, Hq, d], k:
    [T, Hk, d] or None, fp16 / bf16 / fp32, token strides free; positions: [T]
    int32.  ``interleaved``: pairs are channels (2i, 2i + 1) instead of (i, i +
    rotary_dim / 2).  ``inverse``: the gradient's direction.  Outputs may be
    the inputs (in place).  ``outputs`` is ``(q_out, k_out)``."""

    def __init__(self, q, k, positions, table, *, interleaved=False, inverse=False, q_out=None, k_out=None, status=None):
        dev = q.device
        T, Hq, d = q.shape
        a = RotaryArgs()
        a.io_dtype = _io(q, "q")
        a.max_positions, a.rotary_dim = _table(table, dev)
        _index(positions, "positions", (T,), dev)
        _status(status, dev)
        a.total_tokens, a.num_q_heads, a.head_dim = T, Hq, d
        a.interleaved, a.inverse = int(interleaved), int(inverse)
        q_out = _heads_out(q_out, "q_out", q, dev)
        a.q_stride, a.q_out_stride = _token_stride(q, "q", Hq * d), _token_stride(q_out, "q_out", Hq * d)
        a.q, a.q_out = _ptr(q), _ptr(q_out)
        if k is not None:
            _check(k, "k", dtype=q.dtype, device=dev, contiguous=False)
            if k.dim() != 3:
                raise ValueError("k must be [T, Hk, d]")
            Hk = k.shape[1]
            _shape(k, "k", (T, Hk, d))
            k_out = _heads_out(k_out, "k_out", k, dev)
            a.num_k_heads = Hk
            a.k_stride, a.k_out_stride = _token_stride(k, "k", Hk * d), _token_stride(k_out, "k_out", Hk * d)
            a.k, a.k_out = _ptr(k), _ptr(k_out)
        a.positions, a.table, a.status = _ptr(positions), _ptr(table), _ptr(status)
        self._resolve("gdn_rotary", a, (q_out, k_out), (q, k, positions, table, status), dev)


def rotary(q, k, positions, table, **kw):
    """``RotaryCall(...).launch()``: returns ``(q_out, k_out)``."""
    return RotaryCall(q, k, positions, table, **kw).launch()


class PagedKVCache:
    """A paged cache: ``k`` and ``v`` are [pages, page_size, heads, d] views
    with contiguous channels and the same strides (any order of pages, tokens
    and heads in memory), in fp16, bf16, fp32, float8_e4m3fn or int8; the 8-bit
    types come with ``k_scale`` and ``v_scale`` [pages, page_size, heads] fp32
    (one scale a row, any strides, the same for both; a cache whose rows share
    scales, a stride of 0, can be read but not written)."""

    def __init__(self, k, v, k_scale=None, v_scale=None):
        if k.dim() != 4:
            raise ValueError("k must be [pages, page_size, heads, d]")
        if k.dtype not in CACHE_DTYPE:
            raise TypeError(f"unsupported cache dtype {k.dtype}")
        _check(v, "v", dtype=k.dtype, device=k.device, contiguous=False)
        _shape(v, "v", k.shape)
        quantised = k.dtype in (torch.float8_e4m3fn, torch.int8)
        if quantised != (k_scale is not None) or quantised != (v_scale is not None):
            raise ValueError("k_scale and v_scale go with the 8-bit cache types, and only with them")
        a = KVCacheArgs()
        a.num_pages, a.page_size, a.num_kv_heads, a.head_dim = k.shape
        a.cache_dtype = CACHE_DTYPE[k.dtype]
        if k.numel() and (k.stride(3) != 1 or v.stride(3) != 1):
            raise ValueError("a cache row's channels must be contiguous")
        a.page_stride, a.token_stride, a.head_stride = self._strides(k, v, "k and v", k.shape[3])
        if quantised:
            for name, t in (("k_scale", k_scale), ("v_scale", v_scale)):
                _check(t, name, dtype=torch.float32, device=k.device, contiguous=False)
                _shape(t, name, k.shape[:3])
            a.scale_page_stride, a.scale_token_stride, a.scale_head_stride = self._strides(
                k_scale, v_scale, "k_scale and v_scale", 1)
        a.k, a.v, a.k_scale, a.v_scale = _ptr(k), _ptr(v), _ptr(k_scale), _ptr(v_scale)
        self.k, self.v, self.k_scale, self.v_scale, self.args, self.device = k, v, k_scale, v_scale, a, k.device

    @staticmethod
    def _strides(x, y, names, inner):
        """The common (page, token, head) strides; those of an extent of one are free and taken as if dense."""
        dense = (x.shape[1] * x.shape[2] * inner, x.shape[2] * inner, inner)
        of = lambda t: tuple(t.stride(i) if t.shape[i] > 1 else dense[i] for i in range(3))  # noqa: E731
        if of(x) != of(y):
            raise ValueError(f"{names} must have the same strides")
        if x.numel() and of(x) == (0, 0, 0):  # (the C ABI's word for no gaps)
            raise ValueError(f"{names}: one row for all pages, tokens and heads (an expanded view)")
        return of(x)

    @classmethod
    def allocate(cls, num_pages, page_size, num_kv_heads, head_dim, *, dtype=torch.float16, device="cuda",
                 heads_first=False):
        """An uninitialised cache; ``heads_first`` keeps each head's page contiguous."""
        shape = (num_pages, num_kv_heads, page_size) if heads_first else (num_pages, page_size, num_kv_heads)
        order = (lambda t: t.transpose(1, 2)) if heads_first else (lambda t: t)
        rows = [order(torch.empty(*shape, head_dim, dtype=dtype, device=device)) for _ in range(2)]
        scales = [None, None]
        if dtype in (torch.float8_e4m3fn, torch.int8):
            scales = [order(torch.empty(*shape, dtype=torch.float32, device=device)) for _ in range(2)]
        return cls(*rows, *scales)


class KVCacheWriteCall(_Call):
    """Writes new tokens' rows into a ``PagedKVCache`` (C ABI
    ``gdn_kv_cache_write``), quantising for the 8-bit types.  k, v: [T, heads,
    d], token strides free; slots: [T] int32, page * page_size + offset of each
    token, or -1 (not stored).  With ``table`` and ``positions`` the keys are
    rotated first, and queries ``q`` [T, Hq, d], if given, into ``q_out`` (may be
    q).  ``outputs`` is q_out or None."""

    def __init__(self, k, v, cache, slots, *, positions=None, table=None, interleaved=False, q=None, q_out=None,
                 status=None):
        dev = cache.device
        a = KVWriteArgs()
        a.cache = cache.args
        _, _, H, d = cache.k.shape
        a.io_dtype = _io(k, "k")
        T = k.shape[0]
        for name, t in (("k", k), ("v", v)):
            _check(t, name, dtype=k.dtype, device=dev, contiguous=False)
            _shape(t, name, (T, H, d))
        a.k_stride, a.v_stride = _token_stride(k, "k", H * d), _token_stride(v, "v", H * d)
        _index(slots, "slots", (T,), dev)
        _status(status, dev)
        a.total_tokens, a.interleaved = T, int(interleaved)
        if (positions is None) != (table is None):
            raise ValueError("positions and table go together")
        if table is not None:
            a.max_positions, a.rotary_dim = _table(table, dev)
            _index(positions, "positions", (T,), dev)
        if q is not None:
            if table is None:
                raise ValueError("q is rotated: it needs positions and table")
            _check(q, "q", dtype=k.dtype, device=dev, contiguous=False)
            if q.dim() != 3:
                raise ValueError("q must be [T, Hq, d]")
            Hq = q.shape[1]
            _shape(q, "q", (T, Hq, d))
            q_out = _heads_out(q_out, "q_out", q, dev)
            a.num_q_heads = Hq
            a.q_stride, a.q_out_stride = _token_stride(q, "q", Hq * d), _token_stride(q_out, "q_out", Hq * d)
            a.q, a.q_out = _ptr(q), _ptr(q_out)
        elif q_out is not None:
            raise ValueError("q_out without q")
        a.k, a.v, a.slots, a.positions = _ptr(k), _ptr(v), _ptr(slots), _ptr(positions)
        a.table, a.status = _ptr(table), _ptr(status)
        self._resolve("gdn_kv_cache_write", a, q_out, (k, v, cache, slots, positions, table, q, status), dev)


def kv_cache_write(k, v, cache, slots, **kw):
    """``KVCacheWriteCall(...).launch()``: returns the rotated queries, or None."""
    return KVCacheWriteCall(k, v, cache, slots, **kw).launch()


class KVCacheReadCall(_Call):
    """Reads the first ``cu_seqlens[b + 1] - cu_seqlens[b]`` cached tokens of
    every sequence, packed and dequantised (C ABI ``gdn_kv_cache_read``).
    block_table: [B, pages] int32; ``total_tokens`` = cu_seqlens[B].
    ``outputs`` is (k, v), [total_tokens, heads, d] in ``dtype``."""

    def __init__(self, cache, block_table, cu_seqlens, total_tokens, *, dtype=None, k_out=None, v_out=None, status=None):
        dev = cache.device
        _, _, H, d = cache.k.shape
        if dtype is None:
            dtype = k_out.dtype if k_out is not None else cache.k.dtype if cache.k_scale is None else torch.float16
        if dtype not in DTYPE:
            raise TypeError(f"unsupported dtype {dtype}")
        a = KVReadArgs()
        a.cache = cache.args
        B = _cu_seqlens(cu_seqlens, dev)
        a.pages_per_seq, a.block_table_stride = _block_table(block_table, B, dev)
        _status(status, dev)
        T = _int32(total_tokens, "total_tokens")
        outs = []
        for name, t in (("k_out", k_out), ("v_out", v_out)):
            if t is None:
                t = torch.empty((T, H, d), dtype=dtype, device=dev)
            _check(t, name, dtype=dtype, device=dev)
            _shape(t, name, (T, H, d), leading_at_least=True)
            outs.append(t)
        a.num_seqs, a.total_tokens, a.io_dtype = B, T, DTYPE[dtype]
        a.block_table, a.cu_seqlens, a.status = _ptr(block_table), _ptr(cu_seqlens), _ptr(status)
        a.k_out, a.v_out = _ptr(outs[0]), _ptr(outs[1])
        self._resolve("gdn_kv_cache_read", a, tuple(outs), (cache, block_table, cu_seqlens, status), dev)


def kv_cache_read(cache, block_table, cu_seqlens, total_tokens, **kw):
    """``KVCacheReadCall(...).launch()``: returns (k, v)."""
    return KVCacheReadCall(cache, block_table, cu_seqlens, total_tokens, **kw).launch()


class PagedAttentionCall(_Call):
    """Attention of each sequence's newest tokens over its cached keys and
    values (C ABI ``gdn_paged_attention``).  q: [T, Hq, d], token stride free;
    block_table: [B, pages] int32; kv_lens: [B] int32, new tokens included;
    ``cu_seqlens`` [B + 1] int32 packs several query tokens a sequence (None:
    one each, T = B), ``max_seqlen`` bounds them (a hint).  ``window`` > 0 limits
    each query to the newest ``window`` positions up to its own.  ``workspace``:
    see ``paged_attention_workspace``; one is allocated here if none is passed.
    ``outputs`` is output [T, Hq, d], or (output, lse [T, Hq] fp32) with
    ``return_lse``."""

    def __init__(self, q, cache, block_table, kv_lens, *, cu_seqlens=None, scale=0.0, window=0, max_seqlen=0,
                 output=None, lse=None, return_lse=False, workspace=None, status=None):
        dev = cache.device
        _, _, H, d = cache.k.shape
        a = PagedAttentionArgs()
        a.cache = cache.args
        a.io_dtype = _io(q, "q")
        _check(q, "q", device=dev, contiguous=False)
        if q.dim() != 3:
            raise ValueError("q must be [T, Hq, d]")
        T, Hq = q.shape[0], q.shape[1]
        _shape(q, "q", (T, Hq, d))
        B = T if cu_seqlens is None else _cu_seqlens(cu_seqlens, dev)
        a.pages_per_seq, a.block_table_stride = _block_table(block_table, B, dev)
        _index(kv_lens, "kv_lens", (B,), dev)
        _status(status, dev)
        if output is None:
            output = torch.empty((T, Hq, d), dtype=q.dtype, device=dev)
        _check(output, "output", dtype=q.dtype, device=dev)
        _shape(output, "output", (T, Hq, d), leading_at_least=True)
        if lse is None and return_lse:
            lse = torch.empty((T, Hq), dtype=torch.float32, device=dev)
        _check(lse, "lse", dtype=torch.float32, device=dev)
        _shape(lse, "lse", (T, Hq), leading_at_least=True)
        a.num_seqs, a.total_tokens, a.num_q_heads = B, T, Hq
        a.window, a.max_seqlen = _int32(window, "window"), _int32(max_seqlen or 0, "max_seqlen")
        a.scale = float(scale or 0.0)
        a.q_stride = _token_stride(q, "q", Hq * d)
        a.q, a.block_table, a.kv_lens, a.cu_seqlens = _ptr(q), _ptr(block_table), _ptr(kv_lens), _ptr(cu_seqlens)
        a.output, a.lse, a.status = _ptr(output), _ptr(lse), _ptr(status)
        if workspace is None:
            workspace = torch.empty(_workspace_size(a), dtype=torch.uint8, device=dev)
        _check(workspace, "workspace", device=dev)
        a.workspace, a.workspace_bytes = _ptr(workspace), workspace.numel() * workspace.element_size()
        self._resolve("gdn_paged_attention", a, (output, lse) if return_lse or lse is not None else output,
                      (q, cache, block_table, kv_lens, cu_seqlens, status, workspace), dev)


def _workspace_size(args):
    n = ctypes.c_size_t(0)
    rc = load_library().gdn_paged_attention_workspace_size(ctypes.byref(args), ctypes.byref(n))
    if rc != 0:
        raise GdnError(rc, "gdn_paged_attention_workspace_size")
    return int(n.value)


def paged_attention_workspace(cache, num_q_heads, *, dtype=torch.float16, max_seqlen=1):
    """A workspace for calls over ``cache`` with these query heads and at most
    ``max_seqlen`` query tokens a sequence; one serves any number of calls that
    do not overlap."""
    a = PagedAttentionArgs()
    a.cache = cache.args
    a.num_seqs = a.total_tokens = 1
    a.num_q_heads, a.max_seqlen = _int32(num_q_heads, "num_q_heads"), _int32(max_seqlen, "max_seqlen")
    a.io_dtype = DTYPE[dtype]
    return torch.empty(_workspace_size(a), dtype=torch.uint8, device=cache.device)


def paged_attention(q, cache, block_table, kv_lens, **kw):
    """``PagedAttentionCall(...).launch()``: returns output, or (output, lse)."""
    return PagedAttentionCall(q, cache, block_table, kv_lens, **kw).launch()
