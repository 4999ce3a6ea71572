"""Rows whose maximum rises, in either half of a 128-key tile and in many tiles
on end: what has been weighed by the old maximum is scaled again."""

import numpy as np
import pytest
import torch

from tests.kv_tight import Pool

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt,dim", [("nvfp4", 128), ("mxfp4", 128), ("nvfp4", 64), ("mxfp4", 64)])
@pytest.mark.parametrize("nq,group", [(1, 8), (3, 5), (50, 1), (64, 2), (90, 2), (256, 1), (400, 1)])
@pytest.mark.parametrize("step", [33, 64, 100])
def test_maxima_that_rise_on_and_on(cuda_lib, fmt, dim, nq, group, step):
    """A score of 9 log2 units more every `step` keys; rows with a fraction of
    that, and with its opposite, stand between them."""
    n, page = 770, 64
    pages = -(-n // page)
    rng = np.random.default_rng(step)
    k, v = rng.standard_normal((2, pages * page, 1, dim))
    k[:, 0, 0] = 9.0 * (np.arange(pages * page) // step)
    # MXFP4: values whose scale rises too, so that the reference for V moves
    v *= 2.0 ** (np.arange(pages * page) // 150)[:, None, None]
    pool = Pool(cuda_lib, pages, 1, dim, fmt, page, rows=[k, v])
    top = pool.k[:n, 0, 0].max() / (9.0 * ((n - 1) // step))
    q = pool.queries(nq, group, torch.float16, 0.02)
    q[..., 0] = torch.from_numpy(rng.choice([1.0, 1.0, 0.25, 0.9, -1.0], (nq, group))).to(q)
    for causal in (False, True):
        pool.run(q, [nq], [list(range(pages))], [n], causal=causal, scale=float(np.log(2.0) / top))
