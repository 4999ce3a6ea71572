"""Norm and rotary entry points: every refusal, before any device is touched,
and the host arithmetic of frequencies."""

import ctypes
import math
from fractions import Fraction

import pytest
import torch

from fp4_weight_only_gb300 import binding

A, B, C = 0x10000, 0x20000, 0x30000   # aligned addresses that validation must never use
ODD = 0x10008
OK, INVALID, SHAPE, ALIGN = 0, 1, 2, 3
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    return binding.load()


def norm(**k):
    d = dict(x=A, residual=B, weight=C, sum=0x40000, out=0x50000, scales=None, rows=3, dim=64, x_stride=64, residual_stride=64,
             sum_stride=64, out_stride=64, scale_stride=1, dtype=0, weight_f32=0, eps=1e-6, group=0)
    d.update(k)
    return binding.RmsNormArgs(*d.values())


@pytest.mark.parametrize("change,want", [
    (dict(rows=0), OK), (dict(rows=0, x=None, out=None), OK), (dict(rows=-1), INVALID), (dict(dim=0), INVALID),
    (dict(dtype=2), INVALID), (dict(weight_f32=2), INVALID), (dict(eps=-1.0), INVALID), (dict(eps=NAN), INVALID),
    (dict(eps=INF), INVALID), (dict(dim=60), SHAPE), (dict(dim=32776), SHAPE), (dict(rows=(1 << 24) + 1), SHAPE),
    (dict(x=None), INVALID), (dict(out=None), INVALID), (dict(x=ODD), ALIGN), (dict(residual=ODD), ALIGN),
    (dict(weight=ODD), ALIGN), (dict(sum=ODD), ALIGN), (dict(out=ODD), ALIGN), (dict(x_stride=68), ALIGN),
    (dict(residual_stride=65), ALIGN), (dict(sum_stride=65), ALIGN), (dict(out_stride=68), ALIGN),
    (dict(out_stride=56), INVALID), (dict(sum_stride=0), INVALID),                       # rows that share memory
    (dict(group=16), INVALID),                                                           # a group without scales
    (dict(scales=C, group=48), SHAPE), (dict(scales=C, group=8), SHAPE), (dict(scales=C, group=512, dim=512), SHAPE),
    (dict(scales=C, group=128), SHAPE), (dict(scales=C, group=-16), SHAPE), (dict(scales=C + 2, group=16, scale_stride=4), ALIGN),
    (dict(scales=C, group=16, scale_stride=3), INVALID), (dict(scales=C, scale_stride=0), INVALID),
    (dict(sum=0x50000), INVALID),                                                        # two outputs in one place
    (dict(rows=1, x_stride=3, out_stride=0, sum_stride=1, eps=NAN), INVALID), (dict(sum=B, sum_stride=72), INVALID), (dict(out=A, out_stride=72), INVALID), (dict(out=A, scales=C), INVALID)])
def test_norm_refusals(lib, change, want):
    a = norm(**change)
    assert lib.petit_rms_norm(ctypes.addressof(a), None) == want


def test_norm_without_arguments(lib):
    assert lib.petit_rms_norm(None, None) == INVALID
    assert lib.petit_rotary(None, None) == INVALID


def rotary(**k):
    r, o = (A, 512, 64), (B, 512, 64)
    d = dict(q=r, k=r, q_out=o, k_out=o, turns=A, positions=A, num_tokens=3, num_q_heads=6, num_k_heads=2, head_dim=64,
             rot_dim=64, dtype=0, interleaved=0, positions_32=0, magnitude=1.0)
    d.update(k)
    return binding.RotaryArgs(*(v for x in d.values() for v in (x if isinstance(x, tuple) else (x,))))


def R(*rows):
    return rows


@pytest.mark.parametrize("change,want", [
    (dict(num_tokens=0), OK), (dict(num_tokens=0, turns=None), OK), (dict(num_tokens=-1), INVALID),
    (dict(num_q_heads=-1), INVALID), (dict(num_k_heads=-1), INVALID), (dict(num_q_heads=0, num_k_heads=0), SHAPE),
    (dict(num_q_heads=4096), SHAPE), (dict(head_dim=60), SHAPE), (dict(head_dim=0), SHAPE), (dict(head_dim=1032), SHAPE),
    (dict(rot_dim=0), SHAPE), (dict(rot_dim=7), SHAPE), (dict(rot_dim=66), SHAPE), (dict(num_tokens=(1 << 24) + 1), SHAPE),
    (dict(num_tokens=1 << 24, num_q_heads=126), SHAPE), (dict(num_tokens=1 << 24, head_dim=1024, rot_dim=64), SHAPE),
    (dict(dtype=2), INVALID), (dict(interleaved=2), INVALID), (dict(positions_32=2), INVALID), (dict(magnitude=NAN), INVALID),
    (dict(turns=None), INVALID), (dict(positions=None), INVALID), (dict(turns=A + 4), ALIGN), (dict(positions=A + 4), ALIGN),
    (dict(positions=A + 2, positions_32=1), ALIGN), (dict(q=R(None, 512, 64)), INVALID), (dict(k_out=R(None, 512, 64)), INVALID),
    (dict(q=R(ODD, 512, 64)), ALIGN), (dict(k=R(A, 516, 64)), ALIGN), (dict(q_out=R(B, 512, 68)), ALIGN),
    (dict(q_out=R(B, 0, 64)), INVALID), (dict(k_out=R(B, 512, 0)), INVALID), (dict(k_out=R(B, 512, 56)), INVALID),
    (dict(q_out=R(A, 1024, 64)), INVALID), (dict(q_out=R(A, 512, 72)), INVALID),
    (dict(num_tokens=1, num_q_heads=1, q=R(A, 3, 5), q_out=R(B, 1, 0), positions=None), INVALID)])   # (strides of one row)
def test_rotary_refusals(lib, change, want):
    a = rotary(**change)
    assert lib.petit_rotary(ctypes.addressof(a), None) == want


def test_turns(lib):
    pi = Fraction(31415926535897932384626433832795028841971, 10 ** 40)
    for f in (1.0, 0.5, 1e-4, 1e-9, 3.0, math.pi, 6.5, -0.75, 100.0, 0.0):
        got = lib.petit_rotary_turns(f)
        want = Fraction(f) / (2 * pi) * (1 << 64)
        off = (Fraction(got) - want) % (1 << 64)
        # two roundings of 2^-53 of the turns
        assert min(off, (1 << 64) - off) <= abs(want) * Fraction(1, 1 << 52) + 1, f
    for bad in (NAN, INF, -INF):
        assert lib.petit_rotary_turns(bad) == 0


def test_frequencies():
    plain = binding.rotary_frequencies(8, 16.0)
    assert plain == pytest.approx([1.0, 0.5, 0.25, 0.125])
    assert binding.rotary_frequencies(8, 16.0, 4.0) == pytest.approx([f / 4 for f in plain])
    # 2 pi / 64 positions a turn: frequencies that turn 64 f / (2 pi) times in 64 positions
    f = binding.rotary_frequencies(64, 10000.0, 8.0, "bands", 2048, 1.0, 4.0)
    p = binding.rotary_frequencies(64, 10000.0)
    for a, b in zip(f, p):
        turns = 2048 * b / (2 * math.pi)
        assert a == b if turns >= 4 else a == pytest.approx(b / 8) if turns <= 1 else b / 8 < a < b
    f = binding.rotary_frequencies(64, 10000.0, 8.0, "ramp", 2048, 1.0, 32.0)
    ratio = [a / b for a, b in zip(f, p)]
    assert ratio[0] == 1.0 and ratio[-1] == pytest.approx(1 / 8) and ratio == sorted(ratio, reverse=True)
    inside = [r for r in ratio if 1 / 8 < r < 1]
    steps = [a - b for a, b in zip(inside, inside[1:])]   # linear in the pair's index
    assert len(inside) > 5 and steps == pytest.approx([steps[0]] * len(steps))
    for bad in (dict(rot_dim=7), dict(rot_dim=0), dict(rot_dim=8, base=1.0), dict(rot_dim=8, factor=0.0), dict(rot_dim=8, kind="x"),
                dict(rot_dim=8, kind="bands", low=4.0, high=4.0), dict(rot_dim=8, kind="ramp", context=0)):
        with pytest.raises(ValueError, match="rotary_frequencies"):
            binding.rotary_frequencies(**bad)


def test_binding_refuses_before_the_library(lib):
    x = torch.zeros((2, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="x:"):
        binding.rms_norm(x)                                     # a host tensor
    with pytest.raises(ValueError, match="group"):
        binding.rms_norm_e4m3(x, group=48)
    with pytest.raises(ValueError, match="frequencies"):
        binding.Rotary(64, frequencies=[1.0] * 31, device="cpu")
    with pytest.raises(ValueError, match="finite"):
        binding.Rotary(4, frequencies=[1.0, INF], device="cpu")
    rope = binding.Rotary(64, device="cpu")
    assert rope.turns.shape == (32,)
    q = torch.zeros((2, 3, 64), dtype=torch.bfloat16)
    for bad in (dict(q=q.float()), dict(q=q[0]), dict(q=q.transpose(1, 2)), dict(k=q[:1]), dict(k=q.half()),
                dict(positions=torch.zeros(3, dtype=torch.int64)), dict(positions=torch.zeros(2)), dict(out=(q[:, :2], q))):
        with pytest.raises(ValueError):
            binding.rotary(rope, **{**dict(q=q, k=q, positions=torch.zeros(2, dtype=torch.int64)), **bad})
    with pytest.raises(ValueError, match="CUDA"):
        binding.rotary(rope, q, q, torch.zeros(2, dtype=torch.int64))
