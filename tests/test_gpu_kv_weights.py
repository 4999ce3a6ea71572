"""Softmax weights far below a row's largest, and rows whose maximum rises."""

import numpy as np
import pytest
import torch

from tests.kv_tight import Pool

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("nq,group,batch", [(1, 1, 500), (1, 16, 500), (2, 30, 300), (200, 2, 100)])
@pytest.mark.parametrize("bits", [21.0, 24.2, 26.0, 28.5])
def test_many_small_weights_beside_a_large_one(cuda_lib, fmt, nq, group, batch, bits):
    """One key takes nearly all of the weight, as the first token of a context
    often does, and 1500 others 2^-bits of it each: the output is theirs alone,
    as the large one's value is zero.  So many sequences that few are cut (the
    parts of one that is have maxima of their own)."""
    n, page, dim = 1500 + nq, 256, 64
    pages = -(-n // page)
    k, v = np.zeros((pages * page, 1, dim)), np.full((pages * page, 1, dim), -6.0)
    k[0, 0, 0], v[0] = 6.0, 0.0
    pool = Pool(cuda_lib, pages, 1, dim, fmt, page, rows=[k, v])
    q = torch.zeros((batch * nq, group, dim), dtype=torch.float16, device="cuda")
    q[..., 0] = 1.0
    scale = bits * np.log(2.0) / pool.k[0, 0, 0]
    pool.run(q, [nq] * batch, [list(range(pages))] * batch, [n] * batch, scale=float(scale))
