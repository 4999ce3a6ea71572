"""Contexts that many thread blocks share, with a bound for every element: the
parts' sums, their joins, and MXFP4 scales that differ from part to part."""

import numpy as np
import pytest
import torch

from tests.kv_tight import Pool

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt,dim", [("nvfp4", 64), ("mxfp4", 64), ("nvfp4", 128), ("mxfp4", 128)])
@pytest.mark.parametrize("nq,group,window", [(1, 4, 0), (16, 3, 0), (50, 4, 0), (16, 4, 30000), (100, 2, 9000)])
@pytest.mark.parametrize("lens", [(40000,), (9000, 70, 20000)])
def test_parts_of_a_long_context(cuda_lib, fmt, dim, nq, group, window, lens):
    page = 256
    lens = [n + nq for n in lens]
    need = [-(-n // page) for n in lens]
    pages = sum(need)
    rng = np.random.default_rng(nq)
    k, v = rng.standard_normal((2, pages * page, 1, dim))
    # sizes of V that change along the context and between blocks
    v *= 2.0 ** rng.integers(-3, 4, (pages * 4, 1, dim // 32)).repeat(page // 4, 0).repeat(32, 2)
    pool = Pool(cuda_lib, pages, 1, dim, fmt, page, rows=[k, v])
    order = iter(rng.permutation(pages))
    table = [[int(next(order)) for _ in range(n)] for n in need]
    for dtype in (torch.bfloat16, torch.float16):
        pool.run(pool.queries(len(lens) * nq, group, dtype, 2.0), [nq] * len(lens), table, lens, window=window)
