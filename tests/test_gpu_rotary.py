"""Rotary positions against the float64 oracle, whose angles are exact.

Bounds, for every element: cos and sin of the angle are 2^-20.4 off at most (the
hardware's 2^-20.9, and the angle's rounding to FP32, 2^-23), products and sum
2^-22 of |a| + |b|, so 2^-20 of |a| + |b| and the magnitude; a frequency is held
to 2^-52 of its turns, so its angle at position p is p f 2^-51 off at most; then
half a step of the output (2^-8, 2^-11, or 2^-25 where FP16 is subnormal)."""

import numpy as np
import pytest
import torch

from oracle import layer
from tests.test_gpu_norm import HALF, _f64

pytestmark = pytest.mark.gpu


def check(got, x, positions, freq, interleaved, magnitude):
    rel, least = HALF[got.dtype]
    xs = _f64(x)
    want = layer.rotary(xs, positions, freq, interleaved, magnitude)
    half = len(freq)
    size = np.zeros_like(xs)                             # |a| + |b| of an element's pair
    a, b = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if interleaved else (slice(0, half), slice(half, 2 * half))
    size[..., a] = size[..., b] = np.abs(xs[..., a]) + np.abs(xs[..., b])
    angle = np.zeros((len(positions), 1, xs.shape[2]))
    angle[..., a] = angle[..., b] = np.abs(np.asarray(positions, np.float64)[:, None, None] * np.asarray(freq))
    off = size * abs(magnitude) * (2.0 ** -20 + angle * 2.0 ** -51)
    err = np.abs(_f64(got) - want)
    assert (err <= np.abs(want) * rel + off * (1 + rel) + least).all(), err.max()
    assert torch.equal(got[..., 2 * half:], x[..., 2 * half:])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("tokens,hq,hk,dim,rot,interleaved", [
    (1, 1, 1, 8, 2, False), (1, 8, 1, 128, 128, False), (3, 5, 2, 64, 64, True), (5, 4, 4, 64, 32, False), (7, 3, 1, 96, 24, True),
    (2, 9, 3, 80, 80, False), (11, 6, 2, 80, 20, False), (4, 7, 1, 256, 64, True), (3, 2, 0, 48, 10, False), (3, 2, 1, 48, 10, True),
    (2, 3, 1, 1024, 1024, False), (70, 16, 2, 64, 16, False), (129, 10, 2, 128, 128, False)])
def test_rotary(cuda_lib, tokens, hq, hk, dim, rot, interleaved, dtype):
    g = torch.Generator().manual_seed(tokens + dim + rot)
    qkv = torch.randn((tokens, hq + 2 * hk, dim), generator=g).to(dtype).cuda()
    q, k, _ = qkv.split((hq, hk, hk), dim=1)
    k = k if hk else None
    freq = cuda_lib.rotary_frequencies(rot, 10000.0, 4.0, "bands")
    rope = cuda_lib.Rotary(rot, frequencies=freq, interleaved=interleaved, magnitude=1.25)
    pos = torch.randint(-50, 9000, (tokens,), generator=g)
    for positions in (pos.cuda(), pos.int().cuda()):
        before = qkv.clone()
        yq, yk = rope(q, k, positions)
        assert torch.equal(qkv, before)
        check(yq, q, pos.tolist(), freq, interleaved, 1.25)
        if hk:
            check(yk, k, pos.tolist(), freq, interleaved, 1.25)
    # in place, in the fused product; what is not turned stays
    rope(q, k, positions, out=(q, k))
    assert torch.equal(q, yq) and (not hk or torch.equal(k, yk))
    assert torch.equal(qkv[:, hq + hk:], before[:, hq + hk:])


def test_far_positions(cuda_lib):
    pos = [0, 1, -1, 131071, 1000003, (1 << 24) + 1, (1 << 31) - 1, -(1 << 31), 1 << 40, -(1 << 40) + 5]
    g = torch.Generator().manual_seed(3)
    x = torch.randn((len(pos), 2, 64), generator=g).half().cuda()
    freq = cuda_lib.rotary_frequencies(64, 500000.0)
    rope = cuda_lib.Rotary(64, 500000.0)
    check(rope(x, None, torch.tensor(pos).cuda())[0], x, pos, freq, False, 1.0)
    short = [p for p in pos if -(1 << 31) <= p < 1 << 31]
    x = x[:len(short)]
    check(rope(x, None, torch.tensor(short, dtype=torch.int32).cuda())[0], x, short, freq, False, 1.0)


def test_other_frequencies(cuda_lib):
    """Whole turns, zero, negative and large frequencies."""
    freq = [0.0, np.pi, 2 * np.pi, 100.0, -0.3, 1e-9, np.pi / 2, 3.0]
    g = torch.Generator().manual_seed(4)
    x = torch.randn((6, 3, 24), generator=g).cuda().bfloat16()
    pos = [0, 1, 2, 77, 1000, -9]
    for inter in (False, True):
        rope = cuda_lib.Rotary(16, frequencies=torch.tensor(freq), interleaved=inter, magnitude=-2.0)
        fr = torch.tensor(freq).double().tolist()
        check(rope(x, None, torch.tensor(pos).cuda())[0], x, pos, fr, inter, -2.0)


def test_orders_strides_and_values(cuda_lib):
    g = torch.Generator().manual_seed(5)
    rope = cuda_lib.Rotary(64)
    pos = torch.arange(9, device="cuda")
    x = torch.randn((9, 4, 64), generator=g).bfloat16().cuda()
    want = rope(x, None, pos)[0]
    # heads before tokens, rows with gaps
    t = x.transpose(0, 1).contiguous().transpose(0, 1)
    assert torch.equal(rope(t, None, pos)[0], want)
    wide = torch.zeros((9, 4, 72), dtype=x.dtype, device="cuda")
    wide[..., :64] = x
    out = torch.full((12, 6, 80), 5.0, dtype=x.dtype, device="cuda")
    rope(wide[..., :64], None, pos, out=(out[:9, 1:5, :64], None))
    assert torch.equal(out[:9, 1:5, :64], want)
    out[:9, 1:5, :64] = 5.0
    assert (out == 5).all()
    # one head for all: a stride of zero is fine for what is read
    one = x[:, :1].expand(9, 4, 64)
    assert torch.equal(rope(one, None, pos)[0], rope(one.contiguous(), None, pos)[0])
    # NaN and infinities stay in their pairs
    y = x.clone()
    y[2, 1, 3], y[4, 0, 40] = float("inf"), float("nan")
    z = rope(y, None, pos)[0]
    bad = ~torch.isfinite(z)
    assert bad[2, 1, [3, 35]].all() and bad[4, 0, [8, 40]].all() and bad.sum() == 4
    assert torch.equal(z[~bad], want[~bad])
    assert rope(x[:0], x[:0], pos[:0])[0].shape == (0, 4, 64)


def test_refusals(cuda_lib):
    rope = cuda_lib.Rotary(64)
    x = torch.zeros((3, 2, 64), dtype=torch.bfloat16, device="cuda")
    pos = torch.arange(3, device="cuda")
    for bad in (dict(q=x.cpu()), dict(q=x.float()), dict(k=x.half()), dict(k=x[:2]), dict(positions=pos.float()), dict(positions=pos[:2]),
                dict(positions=pos.cpu()), dict(positions=torch.arange(6, device="cuda")[::2]), dict(out=(x, x[:, :1])), dict(q=x.transpose(1, 2))):
        with pytest.raises(ValueError):
            cuda_lib.rotary(rope, **{**dict(q=x, k=x.clone(), positions=pos), **bad})
    with pytest.raises(cuda_lib.PetitError):
        rope(x[..., :32], None, pos)                       # rot_dim past the head
    with pytest.raises(cuda_lib.PetitError):
        rope(x, None, pos, out=(x[:, :1].expand(3, 2, 64), None))
    with pytest.raises(cuda_lib.PetitError):
        cuda_lib.Rotary(32)(torch.zeros((3, 2, 68), dtype=x.dtype, device="cuda")[..., 4:], None, pos)


def test_graph_follows_positions(cuda_lib):
    rope = cuda_lib.Rotary(128, 500000.0)
    g = torch.Generator().manual_seed(6)
    qkv = torch.randn((5, 12, 128), generator=g).bfloat16().cuda()
    q, k, _ = qkv.split((8, 2, 2), dim=1)
    pos = torch.zeros(5, dtype=torch.int32, device="cuda")
    rope(q, k, pos)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pos.add_(3)
        y = rope(q, k, pos)
    for step in (3, 6):
        graph.replay()
        at = torch.full((5,), step, dtype=torch.int64, device="cuda")
        assert all(torch.equal(a, b) for a, b in zip(y, rope(q, k, at)))
