"""The root-mean-square norm against the float64 oracle.

Bounds, for every element.  In FP32 the sum x + r is rounded once (2^-24 of
itself), a sum of squares of at most 32768 positive terms in a tree with at most
32 + 12 steps a path, the mean, the root (2 units) and two products are below
2^-18 of y together; the last rounding is half a step: 2^-8 of y in BF16, 2^-11
in FP16 (or 2^-25 where FP16 is subnormal), 2^-4 of a code's value in E4M3 (or
2^-10 where it is subnormal).  The rounded sum has one value only."""

import numpy as np
import pytest
import torch

from oracle import formats, layer

pytestmark = pytest.mark.gpu

F32 = 2.0 ** -18
HALF = {torch.bfloat16: (2.0 ** -8, 2.0 ** -134), torch.float16: (2.0 ** -11, 2.0 ** -25)}


def _rows(gen, rows, dim, dtype, pad=0, scale=1.0):
    """A view of rows with `pad` elements between them."""
    t = torch.randn((rows, dim + pad), generator=gen) * scale
    t[:, ::17] *= 9.0
    return t.to(dtype).cuda()[:, :dim]


def _f64(t):
    return t.float().cpu().numpy().astype(np.float64)


def check16(got, want, dtype):
    rel, least = HALF[dtype]
    err = np.abs(_f64(got) - want)
    assert (err <= np.abs(want) * (rel * (1 + F32) + F32) + least).all(), err.max()


def check8(codes, scales, want, group):
    top = np.maximum(np.abs(want).reshape(want.shape[0], -1, group).max(-1), 1e-8)
    s = _f64(scales)
    assert s.shape == top.shape and (np.abs(s - top / 448.0) <= top / 448.0 * F32).all()
    v = formats.e4m3_decode(codes.view(torch.uint8).cpu().numpy()) * np.repeat(s, group, axis=1)
    err = np.abs(v - want)
    assert (err <= np.abs(want) * (2.0 ** -4 * (1 + F32) + F32) + np.repeat(s, group, axis=1) * 2.0 ** -10).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("rows,dim", [(1, 8), (3, 16), (5, 64), (9, 248), (1, 256), (4, 264), (7, 1024), (2, 1032), (3, 2048), (1, 4104),
                                      (2, 8192), (3, 8200), (2, 16384), (2, 32768), (600, 1088), (1300, 264), (300, 8192)])
def test_norm(cuda_lib, rows, dim, dtype):
    g = torch.Generator().manual_seed(rows * 7 + dim)
    x, r = _rows(g, rows, dim, dtype, 8), _rows(g, rows, dim, dtype, 24, 3.0)
    w = torch.randn(dim, generator=g)
    for weight in (w.to(dtype).cuda(), w.cuda(), None):
        wn = None if weight is None else _f64(weight)
        y, s = cuda_lib.rms_norm(x, weight, 1e-5, r)
        assert y.shape == x.shape and y.dtype == dtype
        assert torch.equal(s, (x.float() + r.float()).to(dtype))
        check16(y, layer.rms_norm(_f64(x), wn, 1e-5, _f64(r))[0], dtype)
    # without a residual, without a weight
    check16(cuda_lib.rms_norm(x), layer.rms_norm(_f64(x))[0], dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("rows,dim,group", [(1, 16, 16), (3, 128, 16), (2, 96, 32), (5, 448, 64), (2, 1152, 128), (700, 512, 256), (3, 128, 128),
                                            (1, 8192, 128), (40, 2560, 128), (1, 32768, 256), (3, 8, 0), (2, 264, 0), (5, 2568, 0),
                                            (300, 4096, 0), (2, 8192, 0), (1, 24000, 0)])
def test_norm_e4m3(cuda_lib, rows, dim, group, dtype):
    g = torch.Generator().manual_seed(rows + dim + group)
    x, r = _rows(g, rows, dim, dtype, 8), _rows(g, rows, dim, dtype)
    w = torch.randn(dim, generator=g).to(dtype).cuda()
    codes, scales, s = cuda_lib.rms_norm_e4m3(x, w, 1e-6, r, group)
    assert codes.dtype == torch.float8_e4m3fn
    assert torch.equal(s, (x.float() + r.float()).to(dtype))
    check8(codes, scales, layer.rms_norm(_f64(x), _f64(w), 1e-6, _f64(r))[0], group or dim)
    check8(*cuda_lib.rms_norm_e4m3(x, group=group), layer.rms_norm(_f64(x))[0], group or dim)


def test_rows_of_zeros_and_of_extremes(cuda_lib):
    x = torch.zeros((6, 64), dtype=torch.bfloat16)
    x[1] = 2.0 ** -100          # squares below FP32: eps decides
    x[2] = 2.0 ** 60            # squares within it
    x[3, 5] = float("inf")      # as the arithmetic has it: 0 for finite elements, NaN for the infinite one
    x[4, 7] = float("nan")
    x[5, 0] = -1.0
    x = x.cuda()
    y = cuda_lib.rms_norm(x, None, 1e-6).float().cpu()
    assert (y[0] == 0).all()
    check16(y[1:3].to(torch.bfloat16), layer.rms_norm(_f64(x[1:3]))[0], torch.bfloat16)
    assert torch.isnan(y[3, 5]) and (y[3, torch.arange(64) != 5] == 0).all()
    assert torch.isnan(y[4]).all()
    check16(y[5:].to(torch.bfloat16), layer.rms_norm(_f64(x[5:]))[0], torch.bfloat16)
    codes, scales = cuda_lib.rms_norm_e4m3(x, None, 1e-6, group=32)
    raw, s = codes.view(torch.uint8).cpu(), scales.cpu()
    least = torch.tensor(1e-8) / 448
    assert (raw[0] == 0).all() and (s[0] == least).all()
    assert raw[3, 5] & 0x7F == 0x7F and (raw[3, torch.arange(64) != 5] == 0).all() and (s[3] == least).all()
    assert ((raw[4] & 0x7F) == 0x7F).all() and (s[4] == least).all()
    assert s[5, 1] == least
    # eps 0 and a row of zeros: 0 / 0
    assert torch.isnan(cuda_lib.rms_norm(x[:1], None, 0.0)).all()


def test_in_place_broadcast_rows_and_empty(cuda_lib):
    g = torch.Generator().manual_seed(5)
    x, r = _rows(g, 33, 512, torch.bfloat16, 16), _rows(g, 33, 512, torch.bfloat16)
    y, s = cuda_lib.rms_norm(x, None, 1e-6, r)
    x2, r2 = x.clone(), r.clone()
    a, b = cuda_lib.rms_norm(x2, None, 1e-6, r2, out=x2, sum_out=r2)
    assert a is x2 and b is r2 and torch.equal(a, y) and torch.equal(b, s)
    x3, r3 = x.clone(), r.clone()
    cuda_lib.rms_norm(x3, None, 1e-6, r3, out=r3, sum_out=x3)
    assert torch.equal(r3, y) and torch.equal(x3, s)
    # one row for all: a stride of zero is fine for inputs
    one = cuda_lib.rms_norm(x, None, 1e-6, r[:1].expand(33, 512))[0]
    assert torch.equal(one, cuda_lib.rms_norm(x, None, 1e-6, r[:1].expand(33, 512).contiguous())[0])
    assert cuda_lib.rms_norm(x[:0]).shape == (0, 512)
    assert [t.shape for t in cuda_lib.rms_norm_e4m3(x[:0], residual=r[:0])] == [(0, 512), (0, 4), (0, 512)]
    # what lies between and behind the rows stays
    out = torch.full((40, 544), 7.0, dtype=torch.bfloat16, device="cuda")
    cuda_lib.rms_norm(x, None, 1e-6, r, out=out[:33, :512])
    assert torch.equal(out[:33, :512], y) and (out[33:] == 7).all() and (out[:, 512:] == 7).all()
    out8 = torch.full((40, 544), 1.0, device="cuda").to(torch.float8_e4m3fn)
    sc = torch.full((40, 9), 3.0, device="cuda")
    codes, scales = cuda_lib.rms_norm_e4m3(x, group=64, out=out8[:33, :512], scales=sc[:33, :8])
    want = cuda_lib.rms_norm_e4m3(x, group=64)
    assert torch.equal(codes.view(torch.uint8), want[0].view(torch.uint8)) and torch.equal(scales, want[1])
    assert (out8.float()[33:] == 1).all() and (out8.float()[:, 512:] == 1).all() and (sc[33:] == 3).all() and (sc[:, 8] == 3).all()


def test_refusals(cuda_lib):
    x = torch.zeros((4, 64), dtype=torch.bfloat16, device="cuda")
    for bad in (dict(x=x.float()), dict(x=x.t()), dict(x=x[0]), dict(x=x, weight=x[0].half()), dict(x=x, weight=x[0, :32]),
                dict(x=x, residual=x[:2]), dict(x=x, residual=x.half()), dict(x=x, out=x[:, :32]), dict(x=x, residual=x, sum_out=x.cpu())):
        with pytest.raises(ValueError):
            cuda_lib.rms_norm(**bad)
    for bad in (dict(x=x[:, :60]), dict(x=x[:, 4:36]), dict(x=x, out=x[:1].expand(4, 64)), dict(x=x, residual=x, out=x, sum_out=x),
                dict(x=x, eps=-1.0), dict(x=torch.zeros((1, 32776), dtype=torch.bfloat16, device="cuda"))):
        with pytest.raises(cuda_lib.PetitError):
            cuda_lib.rms_norm(**bad)
    with pytest.raises(cuda_lib.PetitError):
        cuda_lib.rms_norm_e4m3(x, group=8)


def test_streams_and_graphs(cuda_lib):
    g = torch.Generator().manual_seed(6)
    x, r = _rows(g, 65, 2048, torch.bfloat16), _rows(g, 65, 2048, torch.bfloat16)
    w = torch.ones(2048, dtype=torch.bfloat16, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        cuda_lib.rms_norm(x, w, 1e-6, r)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a = x + 1.0                                   # a kernel before, whose output the norm reads
        y, s = cuda_lib.rms_norm(a, w, 1e-6, r)
        y2, s2 = cuda_lib.rms_norm(y, w, 1e-6, s)     # and one that reads what the norm wrote
    for seed in (1, 2):
        x.copy_(_rows(torch.Generator().manual_seed(seed), 65, 2048, torch.bfloat16))
        graph.replay()
        e, es = cuda_lib.rms_norm(x + 1.0, w, 1e-6, r)
        e2, es2 = cuda_lib.rms_norm(e, w, 1e-6, es)
        assert torch.equal(y, e) and torch.equal(s, es) and torch.equal(y2, e2) and torch.equal(s2, es2)
