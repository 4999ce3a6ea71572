"""Writing and reading the 4-bit K/V cache: bit for bit against the oracle."""

import numpy as np
import pytest
import torch

from oracle import kv
from tests.kv_util import rows

pytestmark = pytest.mark.gpu


def _scales(heads, fmt):
    return None if fmt == "mxfp4" else torch.tensor(
        [[0.01 + 0.003 * h for h in range(heads)], [0.7 / (h + 1) for h in range(heads)]], dtype=torch.float32)


def _expect(data, slots, page, k, v, fmt, g):
    gk, gv = (None, None) if g is None else (g[0].numpy(), g[1].numpy())
    pk = kv.quantize_rows(k.float().numpy(), fmt, gk)
    pv = kv.quantize_rows(v.float().numpy(), fmt, gv)
    kv.store(data, slots, page, pk, pv, fmt)
    return kv.values(*pk, fmt, gk), kv.values(*pv, fmt, gv)


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("heads,dim,page,n", [(1, 64, 16, 1), (8, 128, 64, 37), (3, 64, 32, 100), (5, 128, 128, 300),
                                              (2, 128, 256, 17)])
def test_append_and_read_bit_exact(cuda_lib, fmt, dtype, heads, dim, page, n):
    rng = np.random.default_rng(n + dim)
    pages = -(-n // page) + 2
    g = _scales(heads, fmt)
    cache = cuda_lib.KVCache(pages, page, heads, dim, fmt, scales=None if g is None else g.cuda())
    slots = rng.permutation(pages * page)[:n].astype(np.int64)
    k, v = rows(rng, n, heads, dim, dtype), rows(rng, n, heads, dim, dtype)
    cache.append(k.cuda(), v.cuda(), torch.from_numpy(slots).cuda())
    want = np.zeros(tuple(cache.data.shape), dtype=np.uint8)
    vk, vv = _expect(want, slots, page, k, v, fmt, g)
    np.testing.assert_array_equal(cache.data.cpu().numpy(), want)   # untouched tokens stay zero
    for out_dtype in (torch.bfloat16, torch.float16):
        rk, rv = cache.read(torch.from_numpy(slots).cuda(), out_dtype)
        for got, val, gs in ((rk, vk, None if g is None else g[0]), (rv, vv, None if g is None else g[1])):
            # code * scale is exact in FP32 and g rounds once: the FP32 product, rounded once more
            f = val if gs is None else (val / gs.numpy()[None, :, None].astype(np.float64)).astype(np.float32) * gs.numpy()[None, :, None]
            assert torch.equal(got.cpu(), torch.from_numpy(np.asarray(f, dtype=np.float32)).to(out_dtype))


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
def test_strided_rows(cuda_lib, fmt):
    """K and V as views of a fused projection, and outputs as views of a wider buffer."""
    rng = np.random.default_rng(5)
    n, heads, dim, page = 21, 4, 128, 16
    qkv = torch.from_numpy(rng.standard_normal((n, 6 * heads * dim)).astype(np.float32)).to(torch.bfloat16).cuda()
    k = qkv[:, 4 * heads * dim:5 * heads * dim].view(n, heads, dim)
    v = qkv.view(n, 6, heads, dim)[:, 5]
    slots = torch.arange(n, device="cuda") + 7
    a = cuda_lib.KVCache(3, page, heads, dim, fmt)
    b = cuda_lib.KVCache(3, page, heads, dim, fmt)
    a.append(k, v, slots)
    b.append(k.contiguous(), v.contiguous(), slots)
    assert torch.equal(a.data, b.data) and a.data.any()
    # head-major rows (a transposed view), and a zero head stride (one row for all heads)
    c = cuda_lib.KVCache(3, page, heads, dim, fmt)
    c.append(k.transpose(0, 1).contiguous().transpose(0, 1), v, slots)
    assert torch.equal(a.data, c.data)
    c.append(k[:, :1].expand(n, heads, dim), v, slots)
    assert torch.equal(c.read(slots)[0], a.read(slots)[0][:, :1].expand(n, heads, dim))
    wide = torch.full((n, 3, heads, dim), 9.0, dtype=torch.bfloat16, device="cuda")
    a.read(slots, out=(wide[:, 0], wide[:, 2]))
    rk, rv = a.read(slots)
    assert torch.equal(wide[:, 0], rk) and torch.equal(wide[:, 2], rv) and (wide[:, 1] == 9).all()


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
def test_slots_that_are_no_slots(cuda_lib, fmt):
    n, heads, dim, page, pages = 9, 2, 64, 16, 2
    cache = cuda_lib.KVCache(pages, page, heads, dim, fmt)
    guard = cache.data.clone()
    k = torch.randn(n, heads, dim, device="cuda").to(torch.bfloat16)
    ws = cuda_lib.Workspace()
    cache.append(k, k, torch.full((n,), -1, dtype=torch.int64, device="cuda"), workspace=ws)
    assert torch.equal(cache.data, guard) and ws.status() == 0          # padding, no error
    slots = torch.tensor([0, -1, 32, 5, 1 << 40, -(1 << 62), 31, (1 << 62), 7], device="cuda")
    cache.append(k, k, slots, workspace=ws)
    assert ws.status() == 8 and ws.status() == 0
    rk, rv = cache.read(slots, workspace=ws)
    assert ws.status() == 8
    good = torch.tensor([True, False, False, True, False, False, True, False, True])
    assert (rk[~good] == 0).all() and (rv[~good] == 0).all() and (rk[good] != 0).any(-1).all()
    cache.append(k, k, slots)                                            # no workspace: skipped all the same
    cache.append(k[:0], k[:0], slots[:0])
    assert cache.read(slots[:0])[0].shape == (0, heads, dim)
    ref = cuda_lib.KVCache(pages, page, heads, dim, fmt)
    ref.append(k[good.cuda()], k[good.cuda()], slots[good.cuda()])
    assert torch.equal(ref.data, cache.data)


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
def test_not_finite_rows_are_written_finite(cuda_lib, fmt):
    x = torch.zeros(4, 1, 64, device="cuda", dtype=torch.bfloat16)
    x[0, 0, :3] = torch.tensor([float("nan"), 1.0, -2.0])
    x[1, 0, :3] = torch.tensor([float("inf"), -float("inf"), 3.0])
    x[2, 0, :2] = torch.tensor([3.38e38, -3.38e38])
    x[3] = float("nan")
    cache = cuda_lib.KVCache(1, 16, 1, 64, fmt)
    slots = torch.arange(4, device="cuda")
    cache.append(x, x, slots)
    k, v = cache.read(slots)
    assert torch.isfinite(k).all() and torch.equal(k, v)
    assert k[0, 0, 0] == 0 and k[0, 0, 1] != 0 and (k[3] == 0).all()
    assert k[1, 0, 0] == k[1, 0].abs().max() and k[1, 0, 1] == -k[1, 0, 0] and k[1, 0, 0] > 1000
    assert k[2, 0, 0] > 1000 and k[2, 0, 1] == -k[2, 0, 0]


def test_cache_past_4_gb(cuda_lib):
    """Byte offsets past 32 bits, through a page stride wider than the page."""
    heads, dim, page, pages = 1, 64, 16, 70
    nbytes = 16 * 72
    data = torch.empty((pages, 1 << 26), dtype=torch.uint8, device="cuda")[:, :nbytes]   # 4.7 GB, hardly touched
    cache = cuda_lib.KVCache(pages, page, heads, dim, "nvfp4", data=data)
    k = torch.randn(3, heads, dim, device="cuda").to(torch.bfloat16)
    slots = torch.tensor([0, 69 * 16 + 15, 33 * 16], device="cuda")
    cache.append(k, k * 2, slots)
    small = cuda_lib.KVCache(pages, page, heads, dim, "nvfp4")
    small.append(k, k * 2, slots)
    for a, b in zip(cache.read(slots), small.read(slots)):
        assert torch.equal(a, b)
    out = [c.attention(k[:1], torch.tensor([[69, 0]], dtype=torch.int32, device="cuda"),
                       torch.tensor([16], dtype=torch.int32, device="cuda")) for c in (_only_last(cache), _only_last(small))]
    assert torch.equal(*out) and (out[0] != 0).any()


def _only_last(cache):
    """Page 69 wholly written."""
    k = torch.arange(16 * 64, device="cuda").view(16, 1, 64).to(torch.bfloat16) / 64
    cache.append(k, k, torch.arange(69 * 16, 70 * 16, device="cuda"))
    return cache


def test_runs_on_the_current_stream(cuda_lib):
    s = torch.cuda.Stream()
    cache = cuda_lib.KVCache(4, 64, 8, 128, "nvfp4")
    k = torch.randn(200, 8, 128, device="cuda").to(torch.bfloat16)
    slots = torch.arange(200, device="cuda")
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        cache.append(k, k, slots)
        a, b = cache.read(slots)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(a, b) and (a != 0).any()


def test_argument_refusals(cuda_lib):
    cache = cuda_lib.KVCache(2, 16, 2, 64, "nvfp4")
    k = torch.zeros(3, 2, 64, dtype=torch.bfloat16, device="cuda")
    slots = torch.arange(3, device="cuda")
    before = cache.data.clone()
    for bad, match in (((k.float(), k.float(), slots), "BF16"), ((k.cpu(), k, slots), "k:"), ((k, k[:2], slots), "v:"),
                       ((k, k.half(), slots), "v:"), ((k[:, :1], k, slots), "k:"), ((k, k, slots.int()), "slots"),
                       ((k, k, slots.cpu()), "slots"), ((k, k, slots[:2]), "slots"),
                       ((k.transpose(1, 2).contiguous().transpose(1, 2), k, slots), "k:")):
        with pytest.raises(ValueError, match=match):
            cache.append(*bad)
    odd = torch.zeros(3 * 129, dtype=torch.bfloat16, device="cuda")[1:385].view(3, 2, 64)
    with pytest.raises(cuda_lib.PetitError) as e:
        cache.append(odd, k, slots)
    assert e.value.status == 3
    with pytest.raises(ValueError, match="dtype"):
        cache.read(slots, torch.float32)
    with pytest.raises(ValueError, match="scales"):
        cuda_lib.KVCache(2, 16, 2, 64, "mxfp4", scales=torch.ones(2, 2, device="cuda"))
    with pytest.raises(ValueError, match="scales"):
        cuda_lib.KVCache(2, 16, 2, 64, "nvfp4", scales=torch.ones(2, 3, device="cuda"))
    with pytest.raises(ValueError, match="data"):
        cuda_lib.KVCache(2, 16, 2, 64, "nvfp4", data=torch.zeros((2, 100), dtype=torch.uint8, device="cuda"))
    assert torch.equal(cache.data, before)
