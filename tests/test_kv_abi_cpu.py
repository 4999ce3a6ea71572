"""K/V cache entry points: sizes, and every refusal, before any device is touched."""

import ctypes

import pytest
import torch

from fp4_weight_only_gb300 import binding

A = 0x10000       # an aligned address that validation must never use
ODD = 0x10008
OK, INVALID, SHAPE, ALIGN, WORKSPACE = 0, 1, 2, 3, 4


@pytest.fixture(scope="module")
def lib():
    return binding.load()


def cache(lib, **k):
    d = dict(data=A, scales=None, num_pages=8, page_stride=None, page_size=32, num_kv_heads=4, head_dim=128, fmt=0)
    d.update(k)
    if d["page_stride"] is None:
        d["page_stride"] = lib.petit_kv_page_bytes(d["page_size"], d["num_kv_heads"], d["head_dim"], d["fmt"])
    return binding.KvCacheInfo(*d.values())


def attn(**k):
    r = binding.Rows(A, 1024, 128)
    d = dict(q=r, out=r, lse=None, block_table=A, seq_lens=A, q_offsets=None, batch=2, total_q=2, max_q=1, max_pages=4,
             table_stride=4, num_q_heads=8, dtype=0, scale=0.1, causal=1, window=0)
    d.update(k)
    return binding.KvAttentionArgs(*d.values())


def test_page_bytes(lib):
    f = lib.petit_kv_page_bytes
    assert f(64, 8, 128, 0) == 8 * 64 * (128 + 16)
    assert f(16, 1, 64, 1) == 16 * (64 + 4)
    for bad in ((8, 1, 64, 0), (48, 1, 64, 0), (512, 1, 64, 0), (64, 0, 64, 0), (64, 1025, 64, 0), (64, 1, 96, 0),
                (64, 1, 128, 2), (64, 1, 128, 7)):
        assert f(*bad) == 0, bad


@pytest.mark.parametrize("change,want", [
    (dict(data=None), INVALID), (dict(num_pages=0), INVALID), (dict(fmt=2), INVALID), (dict(fmt=9), INVALID),
    (dict(fmt=1, scales=A), INVALID), (dict(page_size=24, page_stride=1 << 20), SHAPE),
    (dict(head_dim=80, page_stride=1 << 20), SHAPE), (dict(num_kv_heads=2000, page_stride=1 << 30), SHAPE),
    (dict(page_stride=64), INVALID), (dict(page_stride=(1 << 20) + 8), ALIGN), (dict(data=ODD), ALIGN),
    (dict(scales=0x10002), ALIGN), (dict(num_pages=(1 << 31) + 1), SHAPE), (dict(page_stride=1 << 41), SHAPE)])
def test_cache_refusals(lib, change, want):
    c = cache(lib, **change)
    r = binding.Rows(A, 512, 128)
    p = [ctypes.addressof(x) for x in (c, r)]
    x = attn()
    assert lib.petit_kv_append(p[0], p[1], p[1], 0, A, 3, None, 0, None) == want
    assert lib.petit_kv_read(p[0], A, 3, p[1], p[1], 0, None, 0, None) == want
    assert lib.petit_kv_attention(p[0], ctypes.addressof(x), A, 1 << 40, None) == want


def test_copy_refusals(lib):
    c = cache(lib)
    pc = ctypes.addressof(c)

    def both(k=None, v=None, dtype=0, slots=A, n=3, ws=None, nbytes=0):
        rk, rv = k or binding.Rows(A, 512, 128), v or binding.Rows(A, 512, 128)
        st = lib.petit_kv_append(pc, ctypes.addressof(rk), ctypes.addressof(rv), dtype, slots, n, ws, nbytes, None)
        assert st == lib.petit_kv_read(pc, slots, n, ctypes.addressof(rk), ctypes.addressof(rv), dtype, ws, nbytes, None)
        return st

    assert both(n=0) == OK                                   # nothing to do, nothing touched
    assert both(n=-1) == INVALID
    assert both(dtype=2) == INVALID
    assert both(slots=None) == INVALID
    assert both(slots=0x10004) == ALIGN
    assert both(n=(1 << 24) + 1) == SHAPE
    assert both(k=binding.Rows(None, 512, 128)) == INVALID
    assert both(v=binding.Rows(ODD, 512, 128)) == ALIGN
    assert both(k=binding.Rows(A, 513, 128)) == ALIGN
    assert both(v=binding.Rows(A, 512, 132)) == ALIGN
    assert both(ws=A, nbytes=128) == WORKSPACE
    assert both(ws=ODD, nbytes=512) == ALIGN
    assert lib.petit_kv_append(None, A, A, 0, A, 3, None, 0, None) == INVALID
    assert lib.petit_kv_append(pc, None, A, 0, A, 3, None, 0, None) == INVALID


@pytest.mark.parametrize("change,want", [
    (dict(batch=0, total_q=0), OK), (dict(total_q=0, max_q=0), OK), (dict(batch=-1), INVALID), (dict(total_q=3), INVALID),
    (dict(max_q=-1), INVALID), (dict(max_pages=-1), INVALID), (dict(window=-1), INVALID), (dict(dtype=2), INVALID),
    (dict(window=4, causal=0), INVALID), (dict(causal=2), INVALID), (dict(scale=float("nan")), INVALID),
    (dict(scale=float("inf")), INVALID), (dict(num_q_heads=6), INVALID), (dict(num_q_heads=0), INVALID),
    (dict(table_stride=3), INVALID), (dict(seq_lens=None), INVALID), (dict(block_table=None), INVALID),
    (dict(q=binding.Rows(None, 1024, 128)), INVALID), (dict(q=binding.Rows(ODD, 1024, 128)), ALIGN),
    (dict(out=binding.Rows(A, 1020, 128)), ALIGN), (dict(q=binding.Rows(A, 1024, 4)), ALIGN),
    (dict(seq_lens=0x10002), ALIGN), (dict(lse=0x10002), ALIGN), (dict(q_offsets=0x10001), ALIGN),
    (dict(batch=(1 << 20) + 1, total_q=(1 << 20) + 1), SHAPE), (dict(max_pages=1 << 27, table_stride=1 << 27), SHAPE),
    (dict(num_q_heads=4 * 1025), SHAPE)])
def test_attention_refusals(lib, change, want):
    c, x = cache(lib), attn(**change)
    assert lib.petit_kv_attention(ctypes.addressof(c), ctypes.addressof(x), A, 1 << 40, None) == want


def test_attention_workspace_refusals(lib):
    c, x = cache(lib), attn()
    p = ctypes.addressof(c), ctypes.addressof(x)
    assert lib.petit_kv_attention(*p, None, 0, None) == WORKSPACE
    assert lib.petit_kv_attention(*p, ODD, 1 << 40, None) == ALIGN
    assert lib.petit_kv_attention(p[0], None, A, 1 << 40, None) == INVALID
    assert lib.petit_kv_attention_workspace_bytes(4, 96, 0) == 0
    assert lib.petit_kv_attention_workspace_bytes(4, 128, 2) == 0


def test_binding_refuses_host_tensors_and_bad_geometry(lib):
    with pytest.raises(ValueError, match="CUDA"):
        binding.KVCache(2, 16, 2, 64, data=torch.zeros((2, 16 * 2 * 72), dtype=torch.uint8))
    with pytest.raises(binding.PetitError):
        binding.KVCache(2, 20, 2, 64, data=torch.zeros((2, 4096), dtype=torch.uint8))
    with pytest.raises(ValueError, match="fmt"):
        binding.KVCache(2, 16, 2, 64, fmt="nvfp4_f16")
