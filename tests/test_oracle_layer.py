"""Pins of the oracle's norm, rotary positions and gated projections."""

import math

import numpy as np
import pytest
import torch

from oracle import layer


def test_rms_norm_by_hand():
    y, s = layer.rms_norm([[3.0, 4.0]], [1.0, 2.0], 0.0, [[0.0, -8.0]])
    np.testing.assert_allclose(s, [[3.0, -4.0]])
    np.testing.assert_allclose(y, [[3.0 / math.sqrt(12.5), -8.0 / math.sqrt(12.5)]])
    # the scale of a row cancels but for eps
    x = np.random.default_rng(0).normal(size=(3, 40))
    np.testing.assert_allclose(layer.rms_norm(x, None, 0.0)[0], layer.rms_norm(x * 1e6, None, 0.0)[0])
    assert (layer.rms_norm(np.zeros((1, 8)))[0] == 0).all()


def test_e4m3_groups_reach_the_top_and_err_by_half_a_step():
    y = np.random.default_rng(1).normal(size=(5, 64))
    v, s = layer.e4m3_groups(y, 16)
    assert s.shape == (5, 4) and (np.abs(v).reshape(5, 4, 16).max(-1) == 448.0).all()
    err = np.abs(v.reshape(5, 4, 16) * s[..., None] - y.reshape(5, 4, 16))
    assert (err <= np.abs(y.reshape(5, 4, 16)) * 2.0 ** -4 + s[..., None] * 2.0 ** -10 * (1 + 1e-12)).all()
    assert (layer.e4m3_groups(np.zeros((1, 16)), 16)[1] == 1e-8 / 448).all()


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotary_is_a_turn_of_pairs(interleaved):
    x = np.random.default_rng(2).normal(size=(3, 2, 10))
    f = [1.0, 0.25, 0.01]
    y = layer.rotary(x, [0, 7, -3], f, interleaved, 1.5)
    np.testing.assert_allclose(y[0, :, :6], 1.5 * x[0, :, :6])
    np.testing.assert_array_equal(y[..., 6:], x[..., 6:])
    pair = (lambda t, i: t[..., 2 * i] + 1j * t[..., 2 * i + 1]) if interleaved else (lambda t, i: t[..., i] + 1j * t[..., i + 3])
    for t, p in enumerate((0, 7, -3)):
        for i in range(3):
            np.testing.assert_allclose(pair(y[t], i), 1.5 * pair(x[t], i) * np.exp(1j * p * f[i]))


def test_rotary_at_far_positions():
    # 2^20 turns more change nothing: a frequency of a 64th of a turn, positions 5 and 5 + 2^26
    c, s = layer.turned([5, 5 + (1 << 26)], [2.0 * math.pi / 64])
    # (the double frequency is 2^-53 of itself off, 2^26 positions on)
    np.testing.assert_allclose([c[0], s[0]], [c[1], s[1]], atol=2.0 ** 26 * 0.1 * 2.0 ** -52)


@pytest.mark.parametrize("name,f", [("silu", torch.nn.functional.silu), ("gelu", torch.nn.functional.gelu),
                                    ("gelu_tanh", lambda x: torch.nn.functional.gelu(x, approximate="tanh"))])
def test_activations_against_library(name, f):
    x = torch.linspace(-12, 12, 4001, dtype=torch.float64)
    np.testing.assert_allclose(layer.act(x.numpy(), name), f(x).numpy(), rtol=1e-9, atol=1e-14)


def test_gated_by_hand():
    h, g, u = layer.gated([[1.0, 2.0]], [[1.0, 1.0]], [[3.0, -1.0]], 2.0, 0.5)
    assert g[0, 0] == 6.0 and u[0, 0] == 0.5
    np.testing.assert_allclose(h, [[6.0 / (1 + math.exp(-6.0)) * 0.5]])
