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


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("nq", [64, 130])
@pytest.mark.parametrize("at", [64, 100])
@pytest.mark.parametrize("bits", [9.3, 17.3, 21.7, 26.0, 28.5])
def test_weights_made_before_the_maximum_rose(cuda_lib, fmt, nq, at, bits):
    """A key in the middle of a tile has 2^bits of the weight of those before
    it, and a value of zero: the output is what they had."""
    n, page, dim = 128 + nq, 64, 64
    pages = -(-n // page)
    k, v = np.zeros((2, pages * page, 1, dim))
    k[at, 0, 0], v[:at], k[at + 1:, 0, 0] = 6.0, -6.0, -6.0
    pool = Pool(cuda_lib, pages, 1, dim, fmt, page, rows=[k, v])
    q = torch.zeros((nq, 1, dim), dtype=torch.float16, device="cuda")
    q[..., 0] = 1.0
    pool.run(q, [nq], [list(range(pages))], [n], scale=float(bits * np.log(2.0) / pool.k[at, 0, 0]))


@pytest.mark.parametrize("fmt,dim", [("nvfp4", 128), ("mxfp4", 128), ("nvfp4", 64), ("mxfp4", 64)])
@pytest.mark.parametrize("nq,group", [(1, 8), (3, 4), (64, 1), (90, 4)])
def test_a_query_that_sees_one_key_gets_its_value(cuda_lib, fmt, dim, nq, group):
    """Whatever its weight is rounded to, it is the sum too.  FP16: rounded once
    (2^-11), after a division and a product in FP32 (2^-24 each, and g's)."""
    pool = Pool(cuda_lib, 3, 2, dim, fmt, 64, seed=nq)
    q = pool.queries(nq, group, torch.float16)
    out, _ = pool.run(q, [nq], [[0, 1, 2]], [100 + nq - 10], window=1)
    want = np.repeat(pool.v[90:90 + nq], group, axis=1)
    assert (np.abs(out.double().cpu().numpy() - want) <= np.abs(want) * (2.0 ** -11 + 2.0 ** -22)).all()
