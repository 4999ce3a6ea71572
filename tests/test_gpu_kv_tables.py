"""Block tables placed by hand: pages whose order a copy of several groups
could mistake for consecutive ones."""

import pytest
import torch

from tests.kv_tight import Pool

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt,dim", [("nvfp4", 64), ("mxfp4", 64), ("nvfp4", 128), ("mxfp4", 128)])
@pytest.mark.parametrize("nqs,group", [([1, 1], 8), ([1, 1], 16), ([3, 2], 4), ([70, 64], 2), ([1, 1], 130)])
@pytest.mark.parametrize("heads,pad,rows", [
    (1, 0, [[5, 9, 2, 8], [3, 4, 9, 6]]),          # a page is a group: the last lies three after the first
    (3, 0, [[4, 9, 2, 5], [7, 7, 7, 8]]),          # a page of three heads: the next page lies three groups on
    (1, 1, [[6, 1, 9, 7], [2, 0, 5, 3]]),          # pages padded to three groups
    (2, 0, [[5, 6, 9, 6], [5, 5, 5, 6]])])         # (the nearest that cannot be mistaken)
def test_pages_that_look_consecutive(cuda_lib, fmt, dim, nqs, group, heads, pad, rows):
    page_bytes = cuda_lib.load().petit_kv_page_bytes(16, heads, dim, cuda_lib.FORMATS[fmt])
    pool = Pool(cuda_lib, 10, heads, dim, fmt, 16, seed=heads, pad=2 * page_bytes * pad)
    table = [r + [0, 1] for r in rows]
    lens = [90, 64]
    if max(nqs) * group > 48 and group <= 128:
        lens = [96, 70]
    for dtype in (torch.bfloat16, torch.float16):
        pool.run(pool.queries(sum(nqs), group, dtype), nqs, table, lens)
