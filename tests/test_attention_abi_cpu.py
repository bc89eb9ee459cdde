"""CPU checks of the softmax-attention operators' C ABI and binding: struct
layouts match the header, argument errors return before any launch, and the
binding refuses tensors whose types, shapes or strides do not fit.  No call here
reaches a kernel."""
import ctypes
import os
import subprocess

import pytest
import torch

import gated_delta_rule_gateddeltanet_gb300 as gdn
from gated_delta_rule_gateddeltanet_gb300 import attention as at

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
NULL, DTYPE, SHAPE, ALIGN, WORKSPACE, ARG = 1, 2, 3, 4, 5, 8


@pytest.fixture(scope="module")
def lib():
    from gated_delta_rule_gateddeltanet_gb300 import build
    build.build()
    return gdn.load_library()


STRUCTS = {"gdn_rotary_table_args": at.RotaryTableArgs, "gdn_rotary_args": at.RotaryArgs, "gdn_kv_cache": at.KVCacheArgs,
           "gdn_kv_write_args": at.KVWriteArgs, "gdn_kv_read_args": at.KVReadArgs,
           "gdn_paged_attention_args": at.PagedAttentionArgs}


def test_struct_layouts_match_c(tmp_path):
    body = ""
    for name, cls in STRUCTS.items():
        body += "".join(f'printf("{name}.{f} %zu\\n", offsetof({name}, {f}));' for f, _ in cls._fields_)
        body += f'printf("{name} %zu\\n", sizeof({name}));'
    src = tmp_path / "layout.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "gdn.h"\nint main(void){' + body + "return 0;}\n")
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-std=c11", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    got = dict(line.split() for line in subprocess.run([str(exe)], capture_output=True, text=True,
                                                       check=True).stdout.splitlines())
    for name, cls in STRUCTS.items():
        assert int(got[name]) == ctypes.sizeof(cls)
        for f, _ in cls._fields_:
            assert int(got[f"{name}.{f}"]) == getattr(cls, f).offset, (name, f)


FAKE = 0x1000  # never dereferenced: every case fails its host check first


def _set(a, kw):
    for k, v in kw.items():
        target = a
        while "." in k:
            head, k = k.split(".", 1)
            target = getattr(target, head)
        setattr(target, k, v)
    return a


def _cache(dtype=1):
    c = at.KVCacheArgs()
    c.num_pages, c.page_size, c.num_kv_heads, c.head_dim, c.cache_dtype = 8, 16, 2, 128, dtype
    c.k = c.v = FAKE
    if dtype >= 3:
        c.k_scale = c.v_scale = FAKE
    return c


@pytest.mark.parametrize("kw,code", [
    (dict(scaling=5), ARG), (dict(scaling=-1), ARG), (dict(base=1.0), ARG), (dict(base=float("nan")), ARG),
    (dict(rotary_dim=7), SHAPE), (dict(rotary_dim=0), SHAPE), (dict(max_positions=-1), SHAPE), (dict(table=None), NULL),
    (dict(scaling=1, factor=0.5), ARG), (dict(scaling=3, original_positions=0), ARG),
    (dict(scaling=4, beta_fast=1.0, beta_slow=2.0), ARG), (dict(scaling=2, rotary_dim=2), SHAPE),
    (dict(attention_factor=-1.0), ARG), (dict(max_positions=0, table=None), 0),
])
def test_rotary_table_refusals(lib, kw, code):
    a = at.RotaryTableArgs(64, 64, 0, 4096, 1e4, 4.0, 32.0, 1.0, 0.0, FAKE)
    assert lib.gdn_rotary_table(ctypes.byref(_set(a, kw)), None) == code


def test_null_argument_structs(lib):
    for name in at.ENTRY_POINTS:
        assert getattr(lib, name)(None, None) == NULL
    assert lib.gdn_paged_attention_workspace_size(ctypes.byref(at.PagedAttentionArgs()), None) == NULL


@pytest.mark.parametrize("kw,code", [
    (dict(io_dtype=3), DTYPE), (dict(io_dtype=9), DTYPE), (dict(interleaved=2), ARG), (dict(inverse=-1), ARG),
    (dict(head_dim=65), SHAPE), (dict(rotary_dim=130), SHAPE), (dict(rotary_dim=9), SHAPE), (dict(total_tokens=-1), SHAPE),
    (dict(q_stride=100), SHAPE), (dict(k_out_stride=1), SHAPE), (dict(q=None), NULL), (dict(k_out=None), NULL),
    (dict(positions=None), NULL), (dict(table=None), NULL), (dict(q_out=FAKE, q_out_stride=1024), ARG),
    (dict(total_tokens=0, q=None), 0),
])
def test_rotary_refusals(lib, kw, code):
    a = at.RotaryArgs()
    a.total_tokens, a.num_q_heads, a.num_k_heads, a.head_dim, a.rotary_dim, a.max_positions, a.io_dtype = 4, 4, 2, 128, 64, 99, 1
    a.q = a.k = a.positions = a.table = FAKE
    a.q_out = a.k_out = 2 * FAKE
    assert lib.gdn_rotary(ctypes.byref(_set(a, kw)), None) == code


CACHE_REFUSALS = [
    ({"cache.cache_dtype": 7}, DTYPE), ({"cache.head_dim": 96}, SHAPE), ({"cache.page_size": 0}, SHAPE),
    ({"cache.num_pages": 1 << 28}, SHAPE), ({"cache.num_kv_heads": 0}, SHAPE), ({"cache.num_kv_heads": 65536}, SHAPE),
    ({"cache.k": None}, NULL),
    ({"cache.v": FAKE + 8}, ALIGN), ({"cache.page_stride": 4096, "cache.token_stride": 260, "cache.head_stride": 128}, ALIGN),
    ({"cache.page_stride": 4096, "cache.token_stride": 0, "cache.head_stride": 128}, SHAPE),
    ({"cache.page_stride": 1 << 40, "cache.token_stride": 256, "cache.head_stride": 128}, SHAPE),
]


@pytest.mark.parametrize("kw,code", CACHE_REFUSALS + [
    (dict(io_dtype=2), DTYPE),                       # the cache is FP16
    (dict(io_dtype=4), DTYPE), (dict(total_tokens=-1), SHAPE), (dict(k=None), NULL), (dict(slots=None), NULL),
    (dict(rotary_dim=24), SHAPE), (dict(rotary_dim=144), SHAPE), (dict(positions=None), NULL), (dict(interleaved=3), ARG),
    (dict(table=None), ARG),                         # queries without a rotation
    (dict(q=None), NULL), (dict(k=FAKE + 2), ALIGN), (dict(v_stride=260), ALIGN), (dict(q_stride=100), SHAPE),
    (dict(q_out=FAKE, q_out_stride=1024), ARG), (dict(total_tokens=0, k=None), 0),
])
def test_cache_write_refusals(lib, kw, code):
    a = at.KVWriteArgs()
    a.cache = _cache()
    a.total_tokens, a.num_q_heads, a.rotary_dim, a.max_positions, a.io_dtype = 4, 4, 64, 100, 1
    a.k = a.v = a.q = a.slots = a.positions = a.table = FAKE
    a.q_out = 2 * FAKE
    assert lib.gdn_kv_cache_write(ctypes.byref(_set(a, kw)), None) == code


def test_eight_bit_caches_need_scales(lib):
    a = at.KVWriteArgs()
    a.cache = _cache(4)
    a.total_tokens, a.io_dtype = 1, 0
    a.k = a.v = a.slots = FAKE
    a.cache.v_scale = None
    assert lib.gdn_kv_cache_write(ctypes.byref(a), None) == NULL


@pytest.mark.parametrize("kw,code", CACHE_REFUSALS + [
    (dict(io_dtype=3), DTYPE), (dict(num_seqs=-1), SHAPE), (dict(num_seqs=65536), SHAPE), (dict(pages_per_seq=-1), SHAPE),
    (dict(block_table_stride=2), SHAPE), (dict(block_table=None), NULL), (dict(cu_seqlens=None), NULL),
    (dict(k_out=None), NULL), (dict(v_out=FAKE + 4), ALIGN), (dict(num_seqs=0, k_out=None), 0), (dict(total_tokens=0), 0),
])
def test_cache_read_refusals(lib, kw, code):
    a = at.KVReadArgs()
    a.cache = _cache()
    a.num_seqs, a.total_tokens, a.pages_per_seq, a.io_dtype = 2, 20, 4, 1
    a.block_table = a.cu_seqlens = a.k_out = a.v_out = FAKE
    assert lib.gdn_kv_cache_read(ctypes.byref(_set(a, kw)), None) == code


@pytest.mark.parametrize("kw,code", CACHE_REFUSALS + [
    (dict(io_dtype=2), DTYPE), (dict(io_dtype=0), DTYPE),
    ({"cache.cache_dtype": 3, "cache.k_scale": FAKE, "cache.v_scale": FAKE, "io_dtype": 0}, DTYPE),  # FP32 queries, 8-bit cache
    (dict(num_q_heads=5), SHAPE), (dict(num_q_heads=0), SHAPE), (dict(window=-1), SHAPE), (dict(max_seqlen=-1), SHAPE),
    (dict(scale=-1.0), SHAPE), (dict(scale=float("nan")), SHAPE), (dict(scale=float("inf")), SHAPE),
    (dict(total_tokens=4), SHAPE),                   # one token a sequence without cu_seqlens
    (dict(num_seqs=70000), SHAPE), (dict(q_stride=100), SHAPE), (dict(block_table_stride=1), SHAPE),
    (dict(q=None), NULL), (dict(kv_lens=None), NULL), (dict(output=None), NULL), (dict(block_table=None), NULL),
    (dict(q=FAKE + 8), ALIGN), (dict(q_stride=1028), ALIGN), (dict(workspace=None), WORKSPACE),
    (dict(workspace_bytes=100), WORKSPACE), (dict(workspace=FAKE + 4), ALIGN), (dict(num_seqs=0, total_tokens=0, q=None), 0),
])
def test_paged_attention_refusals(lib, kw, code):
    a = at.PagedAttentionArgs()
    a.cache = _cache()
    a.num_seqs = a.total_tokens = 3
    a.num_q_heads, a.pages_per_seq, a.io_dtype = 8, 4, 1
    a.q = a.block_table = a.kv_lens = a.output = a.workspace = FAKE
    a.workspace_bytes = 1 << 30
    assert lib.gdn_paged_attention(ctypes.byref(_set(a, kw)), None) == code


def test_workspace_size_does_not_depend_on_lengths(lib):
    sizes = set()
    for seqs, pages in ((1, 1), (1, 10000), (500, 64)):
        a = at.PagedAttentionArgs()
        a.cache = _cache()
        a.num_seqs = a.total_tokens = seqs
        a.num_q_heads, a.pages_per_seq, a.io_dtype = 8, pages, 1
        n = ctypes.c_size_t(0)
        assert lib.gdn_paged_attention_workspace_size(ctypes.byref(a), ctypes.byref(n)) == 0
        sizes.add(n.value)
    assert len(sizes) == 1 and 0 < sizes.pop() < 16 << 20


# ---------------------------------------------------------------- binding

def z(*shape, dtype=torch.float16):
    return torch.zeros(shape, dtype=dtype)


def _kv(dtype=torch.float16, heads=2, d=64):
    c = gdn.PagedKVCache.allocate(6, 16, heads, d, dtype=dtype, device="cpu")
    return c


def test_cache_object_refuses_what_does_not_fit():
    with pytest.raises(TypeError, match="cache dtype"):
        gdn.PagedKVCache(z(2, 16, 1, 64, dtype=torch.int16), z(2, 16, 1, 64, dtype=torch.int16))
    with pytest.raises(ValueError, match="scale"):
        gdn.PagedKVCache(z(2, 16, 1, 64, dtype=torch.int8), z(2, 16, 1, 64, dtype=torch.int8))
    with pytest.raises(ValueError, match="scale"):
        gdn.PagedKVCache(z(2, 16, 1, 64), z(2, 16, 1, 64), z(2, 16, 1, dtype=torch.float32), z(2, 16, 1, dtype=torch.float32))
    with pytest.raises(ValueError, match="same strides"):
        gdn.PagedKVCache(z(2, 16, 4, 64), z(2, 4, 16, 64).transpose(1, 2))
    with pytest.raises(ValueError, match="contiguous"):
        gdn.PagedKVCache(z(2, 16, 64, 4).transpose(2, 3), z(2, 16, 64, 4).transpose(2, 3))
    with pytest.raises(ValueError, match="v must have shape"):
        gdn.PagedKVCache(z(2, 16, 1, 64), z(3, 16, 1, 64))


def test_cache_object_takes_any_order_of_pages_tokens_and_heads():
    a = gdn.PagedKVCache.allocate(5, 16, 4, 64, device="cpu").args
    assert (a.page_stride, a.token_stride, a.head_stride) == (4096, 256, 64)
    b = gdn.PagedKVCache.allocate(5, 16, 4, 64, device="cpu", heads_first=True, dtype=torch.int8).args
    assert (b.page_stride, b.token_stride, b.head_stride) == (4096, 64, 1024)
    assert (b.scale_page_stride, b.scale_token_stride, b.scale_head_stride) == (64, 1, 16)
    both = z(5, 2, 16, 4, 64)
    c = gdn.PagedKVCache(both[:, 0], both[:, 1]).args
    assert (c.page_stride, c.token_stride, c.head_stride) == (8192, 256, 64)
    one = torch.zeros(5, 16, 1, 64).as_strided((5, 16, 1, 64), (1024, 64, 3, 1))  # the stride of one head is free
    assert gdn.PagedKVCache(one, one.clone()).args.head_stride == 64


@pytest.mark.parametrize("name,bad,error", [
    ("q", z(3, 4, 64, dtype=torch.float64), TypeError), ("k", z(3, 2, 32), ValueError), ("k", z(2, 2, 64), ValueError),
    ("k", z(3, 2, 64, dtype=torch.bfloat16), TypeError), ("positions", torch.zeros(3, dtype=torch.int64), TypeError),
    ("positions", torch.zeros(2, dtype=torch.int32), ValueError), ("table", z(9, 64), TypeError),
    ("table", torch.zeros(64), ValueError), ("q_out", z(3, 4, 32), ValueError), ("q", z(3, 64, 4).transpose(1, 2), ValueError),
])
def test_rotary_binding_refusals(name, bad, error):
    kw = dict(q=z(3, 4, 64), k=z(3, 2, 64), positions=torch.zeros(3, dtype=torch.int32), table=torch.zeros(9, 64))
    gdn.RotaryCall(**kw)
    with pytest.raises(error):
        gdn.RotaryCall(**{**kw, name: bad})


@pytest.mark.parametrize("name,bad,error", [
    ("k", z(3, 2, 128), ValueError), ("v", z(4, 2, 64), ValueError), ("v", z(3, 2, 64, dtype=torch.float32), TypeError),
    ("slots", torch.zeros(3, dtype=torch.int64), TypeError), ("slots", torch.zeros(4, dtype=torch.int32), ValueError),
    ("positions", None, ValueError), ("table", None, ValueError), ("q", z(3, 4, 32), ValueError),
])
def test_cache_write_binding_refusals(name, bad, error):
    i = torch.zeros(3, dtype=torch.int32)
    kw = dict(k=z(3, 2, 64), v=z(3, 2, 64), cache=_kv(), slots=i, positions=i, table=torch.zeros(9, 64), q=z(3, 4, 64))
    gdn.KVCacheWriteCall(**kw)
    with pytest.raises(error):
        gdn.KVCacheWriteCall(**{**kw, name: bad})


@pytest.mark.parametrize("name,bad,error", [
    ("block_table", torch.zeros(3, 2, dtype=torch.int32), ValueError), ("block_table", torch.zeros(2, 2), TypeError),
    ("cu_seqlens", torch.zeros(1, 3, dtype=torch.int32), ValueError), ("dtype", torch.int8, TypeError),
    ("k_out", z(9, 2, 64), ValueError), ("v_out", z(10, 2, 64, dtype=torch.float32), TypeError),
])
def test_cache_read_binding_refusals(name, bad, error):
    kw = dict(cache=_kv(), block_table=torch.zeros(2, 2, dtype=torch.int32), cu_seqlens=torch.zeros(3, dtype=torch.int32),
              total_tokens=10, dtype=torch.float16)
    gdn.KVCacheReadCall(**kw)
    with pytest.raises(error):
        gdn.KVCacheReadCall(**{**kw, name: bad})


@pytest.mark.parametrize("name,bad,error", [
    ("q", z(3, 8, 128), ValueError), ("q", z(3, 8, 64, dtype=torch.int8), TypeError),
    ("block_table", torch.zeros(2, 2, dtype=torch.int32), ValueError), ("kv_lens", torch.zeros(3, dtype=torch.int64), TypeError),
    ("kv_lens", torch.zeros(2, dtype=torch.int32), ValueError), ("cu_seqlens", torch.zeros(3, dtype=torch.int32), ValueError),
    ("output", z(3, 8, 32), ValueError), ("lse", z(3, 8), TypeError), ("q", z(3, 64, 8).transpose(1, 2), ValueError),
])
def test_paged_attention_binding_refusals(name, bad, error):
    kw = dict(q=z(3, 8, 64), cache=_kv(), block_table=torch.zeros(3, 2, dtype=torch.int32),
              kv_lens=torch.zeros(3, dtype=torch.int32), workspace=torch.zeros(16, dtype=torch.uint8))
    gdn.PagedAttentionCall(**kw)
    with pytest.raises(error):
        gdn.PagedAttentionCall(**{**kw, name: bad})
