"""Pins of the K/V cache oracle: hand-worked cases, brute force, torch."""

import numpy as np
import pytest
import torch

from oracle import gemm, kv, quantize


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
def test_rows_quantise_like_weights_per_head(fmt):
    rng = np.random.default_rng(1)
    x = (rng.standard_normal((5, 3, 64)) * 4).astype(np.float32)
    g = np.array([0.5, 1.0, 0.03], dtype=np.float32) if fmt == "nvfp4" else None
    codes, scales = kv.quantize_rows(x, fmt, g)
    for h in range(3):
        c, s = quantize.nvfp4_quantize(x[:, h], g[h]) if fmt == "nvfp4" else quantize.mxfp4_quantize(x[:, h])
        np.testing.assert_array_equal(codes[:, h], c)
        np.testing.assert_array_equal(scales[:, h], s)
    v = kv.values(codes, scales, fmt, g)
    # an element is within half a grid step (at most scale) of its value; the
    # steps at the top are 2 scales wide, and a scale rounded down saturates
    assert np.abs(v - x).max() <= np.abs(x).max() / 4


def test_mxfp4_scale_cap_keeps_values_finite():
    x = np.zeros((1, 1, 32), dtype=np.float32)
    x[0, 0, :4] = [3.3e38, -3.3e38, 2.0 ** 125, 1.0]
    codes, scales = kv.quantize_rows(x, "mxfp4")
    assert scales[0, 0, 0] == 252
    assert list(codes[0, 0, :4]) == [7, 15, 2, 0]
    assert np.isfinite(kv.values(codes, scales, "mxfp4").astype(np.float32)).all()


def test_store_order_by_hand():
    """Token 17 of a 32-token page, head 1 of 2, D = 64, NVFP4: group 1, row 1."""
    heads, d, page = 2, 64, 32
    group = 16 * (32 + 4 + 32 + 4)
    data = np.zeros((3, heads * 2 * group), dtype=np.uint8)
    kc = np.zeros((1, heads, d), dtype=np.uint8)
    kc[0, 1, 0], kc[0, 1, 1] = 3, 9
    ks = np.zeros((1, heads, 4), dtype=np.uint8)
    ks[0, 1, 2] = 77
    vc = np.zeros_like(kc)
    vc[0, 1, 63] = 5
    vs = np.zeros_like(ks)
    vs[0, 1, 3] = 88
    kv.store(data, [2 * page + 17], page, (kc, ks), (vc, vs), "nvfp4")
    base = 3 * group   # head 1's second group
    row = np.zeros(heads * 2 * group, dtype=np.uint8)
    row[base + 32] = 3 | 9 << 4
    row[base + 16 * 32 + 4 + 2] = 77
    row[base + 16 * 36 + 32 + 31] = 5 << 4
    row[base + 16 * 68 + 4 + 3] = 88
    np.testing.assert_array_equal(data[2], row)
    assert not data[:2].any()


@pytest.mark.parametrize("causal,window", [(True, 0), (True, 3), (False, 0)])
def test_attention_matches_brute_force(causal, window):
    rng = np.random.default_rng(2)
    nq, n, hq, hk, d = 4, 9, 4, 2, 8
    q, k, v = rng.standard_normal((nq, hq, d)), rng.standard_normal((n, hk, d)), rng.standard_normal((n, hk, d))
    out, lse, _, _ = kv.attention(q, k, v, 0.3, causal, window)
    for i in range(nq):
        for a in range(hq):
            p = n - nq + i
            js = [j for j in range(n) if (not causal or j <= p) and (not window or j > p - window)]
            e = [np.exp(0.3 * sum(q[i, a, x] * k[j, a // 2, x] for x in range(d))) for j in js]
            want = sum(w * v[j, a // 2] for w, j in zip(e, js)) / sum(e)
            np.testing.assert_allclose(out[i, a], want, rtol=1e-12)
            np.testing.assert_allclose(lse[i, a], np.log(sum(e)), rtol=1e-12)


def test_attention_matches_torch_and_empty_rows_are_zero():
    rng = np.random.default_rng(3)
    q, k, v = rng.standard_normal((3, 2, 16)), rng.standard_normal((7, 2, 16)), rng.standard_normal((7, 2, 16))
    out, _, _, _ = kv.attention(q, k, v, 0.25, causal=False)
    t = [torch.from_numpy(x).transpose(0, 1) for x in (q, k, v)]
    want = torch.softmax(0.25 * t[0] @ t[1].transpose(1, 2), -1) @ t[2]
    np.testing.assert_allclose(out, want.transpose(0, 1).numpy(), rtol=1e-10)
    out, lse, _, _ = kv.attention(q, k[:2], v[:2], 0.25, causal=True)   # more queries than keys
    assert (out[0] == 0).all() and np.isneginf(lse[0]).all() and np.isfinite(lse[1:]).all()
    out, lse, _, _ = kv.attention(q, k[:0], v[:0], 0.25)
    assert (out == 0).all() and np.isneginf(lse).all()
