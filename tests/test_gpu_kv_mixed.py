"""Batches that mix prompt pieces with single tokens: which kernel takes them
goes by the rows of all sequences."""

import pytest
import torch

from tests.kv_tight import Pool

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt,dim", [("nvfp4", 128), ("mxfp4", 128), ("nvfp4", 64), ("mxfp4", 64)])
@pytest.mark.parametrize("window", [0, 90])
@pytest.mark.parametrize("pieces,single,group", [([100], 39, 8), ([300], 39, 8), ([60, 0, 33], 7, 4), ([0, 0, 200], 0, 1)])
def test_pieces_among_single_tokens(cuda_lib, fmt, dim, window, pieces, single, group):
    page, heads = 32, 4
    nqs = pieces + [1] * single
    lens = [n + 50 if n else 20 for n in pieces] + [3 + 11 * i for i in range(single)]
    need = [-(-n // page) for n in lens]
    pool = Pool(cuda_lib, sum(need), heads, dim, fmt, page, seed=len(nqs))
    order = iter(pool.rng.permutation(sum(need)))
    table = [[int(next(order)) for _ in range(n)] for n in need]
    pool.run(pool.queries(sum(nqs), group, torch.bfloat16), nqs, table, lens, window=window)
