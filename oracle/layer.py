"""The operators around a decoder layer's products in float64: the
root-mean-square norm with its 8-bit output, rotary positions and the gated
feed-forward projections.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__.py``).
"""

import math
from fractions import Fraction

import numpy as np

from . import formats

_PI = Fraction(31415926535897932384626433832795028841971, 10 ** 40)


def rms_norm(x, weight=None, eps=1e-6, residual=None):
    """(y, s) of rows x [rows, dim]: s = x + residual, y = s / sqrt(mean(s^2) + eps) * weight."""
    s = np.asarray(x, np.float64) + (0.0 if residual is None else np.asarray(residual, np.float64))
    y = s / np.sqrt((s * s).mean(-1, keepdims=True) + eps)
    return (y if weight is None else y * np.asarray(weight, np.float64)), s


def e4m3_groups(y, group):
    """(values of the codes, scales) of rows y: a scale per `group` elements."""
    b = y.reshape(y.shape[0], -1, group)
    scale = np.maximum(np.abs(b).max(-1), 1e-8) / 448.0
    return formats.e4m3_decode(formats.e4m3_encode(b / scale[..., None])).reshape(y.shape), scale


def turned(angle_positions, frequencies):
    """(cos, sin) [tokens, pairs] of position * frequency, the angle taken
    modulo a turn in exact fractions: right at any position."""
    out = np.empty((2, len(angle_positions), len(frequencies)))
    for i, p in enumerate(angle_positions):
        for j, f in enumerate(frequencies):
            t = Fraction(int(p)) * Fraction(float(f)) / (2 * _PI)
            t = float(t - round(t)) * 2.0 * math.pi
            out[:, i, j] = math.cos(t), math.sin(t)
    return out


def rotary(x, positions, frequencies, interleaved=False, magnitude=1.0):
    """Rows x [tokens, heads, D] with the first 2 len(frequencies) elements of every head turned."""
    y = np.array(x, np.float64)
    half = len(frequencies)
    c, s = magnitude * turned(positions, frequencies)[:, :, None, :]
    a, b = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if interleaved else (slice(0, half), slice(half, 2 * half))
    p, q = y[..., a].copy(), y[..., b].copy()
    y[..., a], y[..., b] = p * c - q * s, q * c + p * s
    return y


def act(x, name):
    """silu x / (1 + e^-x), gelu x Phi(x), or gelu_tanh, the latter with tanh in Phi's place."""
    x = np.asarray(x, np.float64)
    if name == "silu":
        return x * np.where(x >= 0, 1.0, np.exp(np.minimum(x, 0.0))) / (1.0 + np.exp(-np.abs(x)))
    if name == "gelu":
        return x * 0.5 * np.vectorize(math.erfc, otypes=[np.float64])(-x / math.sqrt(2.0))
    if name == "gelu_tanh":
        z = 2.0 * math.sqrt(2.0 / math.pi) * (x + 0.044715 * x ** 3)
        return x * np.where(z >= 0, 1.0, np.exp(np.minimum(z, 0.0))) / (1.0 + np.exp(-np.abs(z)))
    raise ValueError(name)


def gated(a, w_gate, w_up, g_gate=1.0, g_up=1.0, name="silu"):
    """(h, gate, up) of rows a [m, k]: h = act(gate) * up, gate = g_gate a w_gate^T, up = g_up a w_up^T."""
    a = np.asarray(a, np.float64)
    gate, up = g_gate * (a @ np.asarray(w_gate, np.float64).T), g_up * (a @ np.asarray(w_up, np.float64).T)
    return act(gate, name) * up, gate, up
