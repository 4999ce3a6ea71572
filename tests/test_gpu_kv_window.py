"""What lies before a sliding window is not seen: pages given back (no table
entry), tokens overwritten, scales that are NaN or huge."""

import numpy as np
import pytest
import torch

from tests.kv_tight import Pool

pytestmark = pytest.mark.gpu

FORMATS = [("nvfp4", 128), ("mxfp4", 128), ("nvfp4", 64), ("mxfp4", 64)]
# query tokens and heads a K/V head: a token, a draft, a prompt of one row tile, of two, of several items
ROWS = [(1, 8), (5, 3), (40, 3), (70, 3), (300, 2)]


def spoil(pool, slots, byte):
    """Every code and scale byte of the tokens in `slots` becomes `byte`."""
    block = 16 if pool.fmt == "nvfp4" else 32
    heads = pool.cache.data.view(pool.cache.num_pages, pool.heads, pool.page // 16, -1)
    page, tok = np.divmod(np.asarray(slots), pool.page)
    at = 0
    for n in (pool.dim // 2, pool.dim // block) * 2:
        part = heads[..., at:at + 16 * n].unflatten(-1, (16, n))
        part[torch.from_numpy(page).cuda(), :, torch.from_numpy(tok // 16).cuda(), torch.from_numpy(tok % 16).cuda()] = byte
        at += 16 * n


@pytest.mark.parametrize("fmt,dim", FORMATS)
@pytest.mark.parametrize("nq,group", ROWS)
@pytest.mark.parametrize("window", [1, 33, 200])
@pytest.mark.parametrize("page", [16, 64])
def test_pages_before_the_window_may_be_gone(cuda_lib, fmt, dim, nq, group, window, page):
    lens = [nq + 611, nq + 300, nq]
    need = [-(-n // page) for n in lens]
    pool = Pool(cuda_lib, sum(need), 2, dim, fmt, page, seed=nq)
    order = iter(pool.rng.permutation(sum(need)))
    table = [[int(next(order)) for _ in range(n)] for n in need]
    q = pool.queries(3 * nq, group, torch.float16)
    want = pool.run(q, [nq] * 3, table, lens, window=window)
    for row, n in zip(table, lens):
        gone = max(0, n - nq - window + 1) // page      # whole pages before the first query's window
        row[:gone] = [-1] * gone
    got = pool.run(q, [nq] * 3, table, lens, window=window)     # (checks that no status is set)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("fmt,dim", FORMATS)
@pytest.mark.parametrize("nq,group", ROWS)
@pytest.mark.parametrize("window", [1, 33, 200])
def test_tokens_before_the_window_may_hold_anything(cuda_lib, fmt, dim, nq, group, window):
    """NaN scales, the largest and small ones, up to the token beside the window: the same bits."""
    lens, page = [nq + 611, nq + 300], 64
    pool = Pool(cuda_lib, 40, 1, dim, fmt, page, seed=nq)
    order = [int(x) for x in pool.rng.permutation(40)]
    table = [order[:20], order[20:]]
    q = pool.queries(2 * nq, group, torch.bfloat16)
    before = []
    for row, n in zip(table, lens):
        j = np.arange(max(0, n - nq - window + 1))
        before.append(np.asarray(row)[j // page] * page + j % page)
    outs = [pool.run(q, [nq] * 2, table, lens, window=window)]
    for byte in (0xFF, 0x7E, 0xFD, 0x01):
        spoil(pool, np.concatenate(before), byte)
        outs.append(pool.run(q, [nq] * 2, table, lens, window=window))
    for o in outs[1:]:
        assert torch.equal(o[0], outs[0][0]) and torch.equal(o[1], outs[0][1])
