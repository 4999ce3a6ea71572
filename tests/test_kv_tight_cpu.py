"""The element-wise bound of kv_tight turns down wrong attention outputs."""

import numpy as np
import pytest
import torch

from oracle import kv
from tests.kv_tight import bounds, expect, outside

SHAPES = [(1, 40), (1, 500), (1, 6000), (1, 40001), (16, 40016), (50, 700), (300, 300)]


@pytest.mark.parametrize("nq,n", SHAPES)
@pytest.mark.parametrize("window", [0, 3000])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_wrong_outputs_are_turned_down(nq, n, window, dtype):
    rng = np.random.default_rng(n)
    dim = 64
    q = rng.standard_normal((nq, 2, dim))
    k, v = rng.standard_normal((n, 1, dim)), rng.standard_normal((n, 1, dim))
    want, lse, *rest = expect(q, k, v, dim ** -0.5, window=window)
    out, lb = bounds(want, lse, *rest, dim, dtype)
    assert not outside(want, want, out).any() and not outside(lse, lse, lb).any()
    # a vector of outputs is told from nothing, from its opposite and from half of its keys
    half = expect(q, k[n // 2:], v[n // 2:], dim ** -0.5, window=window)
    for wrong in (np.zeros_like(want), -want, np.full_like(want, np.nan)):
        assert (outside(wrong, want, out).any(-1) | (rest[-1] == 0)[:, None]).all()
    cut = (rest[-1] > (half[-1] + 1))[:, None]
    assert (outside(half[0], want, out).any(-1) | ~cut).all()
    assert (outside(half[1], lse, lb) | ~cut).all()


@pytest.mark.parametrize("nq,n,causal,window", [(1, 30, True, 0), (5, 3, True, 0), (9, 40, True, 7), (4, 20, False, 0)])
def test_same_attention_as_the_oracle(nq, n, causal, window):
    rng = np.random.default_rng(n)
    q = rng.standard_normal((nq, 4, 64))
    k, v = rng.standard_normal((n, 2, 64)), rng.standard_normal((n, 2, 64))
    a, b = expect(q, k, v, 0.1, causal, window), kv.attention(q, k, v, 0.1, causal, window)
    np.testing.assert_allclose(a[0], b[0], atol=1e-12)
    np.testing.assert_allclose(a[1], b[1], atol=1e-12)
    np.testing.assert_allclose(a[2], b[2], atol=1e-12)
