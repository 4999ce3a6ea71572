"""Where the K/V kernels change their way: codes decided by a product or a
division, the rows that choose a kernel, contexts joined from many parts."""

import numpy as np
import pytest
import torch

from oracle import kv
from tests.kv_util import Case
from tests.test_gpu_kv_attention import _run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_values_at_and_beside_the_middle_of_two_codes(cuda_lib, fmt, dtype):
    """Blocks whose largest value sets the scale and whose others are the
    midpoints between codes, exactly (scales that are powers of two) or rounded
    to the type, and their neighbours on both sides."""
    rng = np.random.default_rng(0)
    n, heads, dim = 256, 4, 128
    block = 16 if fmt == "nvfp4" else 32
    g = np.array([[2.0 ** -7, 0.0123, 1.0, 0.37]] * 2, dtype=np.float32)
    unit = 2.0 ** rng.integers(-3, 3, (n, heads, dim // block, 1)) * (1.0 if fmt == "mxfp4" else rng.choice(
        [1.0, 1.125, 1.625], (n, heads, dim // block, 1)))
    mid = rng.choice([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], (n, heads, dim // block, block))
    mid *= rng.choice([-1.0, 1.0], mid.shape)
    mid[..., 0] = 6.0
    x = mid * unit
    if fmt == "nvfp4":
        x *= g[0][None, :, None, None]
    x = torch.from_numpy(x.reshape(n, heads, dim).astype(np.float32)).to(dtype)
    step = torch.from_numpy(rng.integers(-1, 2, (n, heads, dim)).astype(np.int16))
    step[..., ::block] = 0
    k = (x.view(torch.int16) + step).view(dtype)
    cache = cuda_lib.KVCache(n // 16, 16, heads, dim, fmt, scales=torch.from_numpy(g).cuda() if fmt == "nvfp4" else None)
    cache.append(k.cuda(), x.cuda(), torch.arange(n, device="cuda"))
    want = np.zeros(tuple(cache.data.shape), dtype=np.uint8)
    pair = [kv.quantize_rows(r.float().numpy(), fmt, g[i] if fmt == "nvfp4" else None) for i, r in enumerate((k, x))]
    kv.store(want, np.arange(n), 16, *pair, fmt)
    np.testing.assert_array_equal(cache.data.cpu().numpy(), want)


@pytest.mark.parametrize("fmt,dim", [("nvfp4", 128), ("mxfp4", 64)])
@pytest.mark.parametrize("nq,group", [(1, 8), (9, 1), (2, 24), (7, 7), (16, 3), (17, 3), (1, 128), (1, 130), (3, 130), (256, 1), (257, 1)])
def test_rows_beside_the_limits_of_a_kernel(cuda_lib, fmt, dim, nq, group):
    case = Case(cuda_lib, [140 + nq, nq], 1, dim, fmt, 32, seed=nq + group)
    _run(case, cuda_lib, [nq, nq], group, torch.bfloat16)


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("nq,group,window", [(1, 4, 0), (16, 4, 0), (50, 4, 0), (16, 4, 30000)])
def test_context_joined_from_many_parts(cuda_lib, fmt, nq, group, window):
    """40000 keys of one head: every thread block has a part of one item."""
    case = Case(cuda_lib, [40000 + nq, 70 + nq], 1, 64, fmt, 256, seed=4)
    q, off, out, _, ws = _run(case, cuda_lib, [nq, nq], group, torch.bfloat16, window=window)
    assert torch.equal(out, case.cache.attention(q, case.d_table, case.d_lens, off, nq, window=window, workspace=ws))
    assert not ws.buf[:4352].any()


@pytest.mark.parametrize("nq", [1, 20])
def test_another_stream_and_its_workspace(cuda_lib, nq):
    """The same cache read on two streams, each with a workspace of its own."""
    case = Case(cuda_lib, [3000 + nq, 500], 2, 128, "nvfp4", 64, seed=3)
    q, off = case.queries([nq, nq], 8, torch.bfloat16)
    want = case.cache.attention(q, case.d_table, case.d_lens, off, nq)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    spaces = [cuda_lib.Workspace(nbytes=case.cache.workspace_bytes()) for _ in streams]
    torch.cuda.synchronize()
    outs = []
    for i in range(6):
        with torch.cuda.stream(streams[i % 2]):
            outs.append(case.cache.attention(q, case.d_table, case.d_lens, off, nq, workspace=spaces[i % 2]))
    torch.cuda.synchronize()
    for o in outs:
        assert torch.equal(o, want)
    assert [w.status() for w in spaces] == [0, 0]
