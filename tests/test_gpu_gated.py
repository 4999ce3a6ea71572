"""Gated products against the float64 oracle.

Bounds, for every element.  A sum of k products (exact in FP32's 24 bits) is
taken in steps of 16 whose terms are cut to 24 bits of the largest: at most
(k / 16 + parts) * 17 * 2^-24 of the sum S of the products' magnitudes, so
1.25 * k * 2^-24 * S covers it for k >= 128 (parts of a split tile, at most k /
128, and the factor's rounding among it).  The derivatives of the three
activations are below 1.13; evaluating one costs 2^-15 of it at most (e^x at |x| <
88 has its argument rounded to 2^-24: 2^-17 of it, three roundings of z; below
that the value is under 2^-120), and the output's rounding half a step."""

import numpy as np
import pytest
import torch

from fp4_weight_only_gb300 import synth
from oracle import gemm, layer
from tests.gpu_util import oracle_quantize, to_device_packed
from tests.test_gpu_norm import HALF, _f64

pytestmark = pytest.mark.gpu


def matrices(cuda_lib, n, k, fmt, seed, scales):
    """(repacked, dequantised gate, dequantised up) of an oracle-quantised pair."""
    packed, values = [], []
    base = "mxfp4" if fmt == "mxfp4" else "nvfp4"
    for i in (0, 1):
        codes, s = oracle_quantize(synth.weights(n, k, seed=seed + i), base, scales[i])
        packed.extend(to_device_packed(codes, s))
        values.append(gemm.dequantize(codes, s, base))
    return cuda_lib.gated_repack(*packed, fmt), *values


def check(got, a, wg, wu, scales, act, what=""):
    x = _f64(a)
    h, g, u = layer.gated(x, wg, wu, *scales, act)
    step = 1.25 * x.shape[1] * 2.0 ** -24
    dg, du = (step * s * (np.abs(x) @ np.abs(w).T) for s, w in zip(scales, (wg, wu)))
    rel, least = HALF[got.dtype]
    t = np.abs(layer.act(g, act))
    off = (1.13 * dg + t * 2.0 ** -15 + 2.0 ** -120) * (np.abs(u) + du) + t * du
    err = np.abs(_f64(got) - h)
    worst = (err - (np.abs(h) * rel + off * (1 + rel) + least)).max()
    assert worst <= 0, f"{what}: {worst} over"


def activations(m, k, fmt, seed):
    a = synth.activations(m, k, seed=seed)
    return (a.half() if fmt == "nvfp4_f16" else a).cuda()


SCALES = {"nvfp4": (0.0009, 0.0013), "nvfp4_f16": (0.0013, 0.0009), "mxfp4": (1.0, 1.0)}


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4", "nvfp4_f16"])
@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
def test_rows_of_every_tile_height(cuda_lib, fmt, act):
    n, k = 192, 640            # three weight tiles, five 128-k chunks: pairs do not apply, tiles are split
    rep, wg, wu = matrices(cuda_lib, n, k, fmt, 5, SCALES[fmt])
    ws = cuda_lib.Workspace()
    for m in (1, 2, 15, 16, 17, 33, 64, 65, 128, 129, 250, 257, 600):
        a = activations(m, k, fmt, m)
        got = cuda_lib.gated_gemm(a, rep, n, fmt, SCALES[fmt], act, ws)
        check(got, a, wg, wu, SCALES[fmt], act, f"m = {m}")
        assert torch.equal(got, cuda_lib.gated_gemm(a, rep, n, fmt, SCALES[fmt], act, ws))
    assert ws.status() == 0


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4", "nvfp4_f16"])
@pytest.mark.parametrize("m,n,k", [(1, 64, 128), (3, 64, 4096), (16, 2112, 256), (40, 512, 4096), (130, 1024, 1024), (256, 128, 2048),
                                   (300, 64, 3968), (520, 1088, 512)])
def test_shapes(cuda_lib, fmt, m, n, k):
    rep, wg, wu = matrices(cuda_lib, n, k, fmt, n + k, SCALES[fmt])
    a = activations(m, k, fmt, m)
    ws = cuda_lib.Workspace()
    check(cuda_lib.gated_gemm(a, rep, n, fmt, SCALES[fmt], "silu", ws), a, wg, wu, SCALES[fmt], "silu")
    assert ws.status() == 0


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4", "nvfp4_f16"])
def test_tile_shapes_and_pairs(cuda_lib, fmt):
    """Every kernel, forced, with split and with whole tiles."""
    scales = SCALES[fmt]
    try:
        for n, k in ((256, 1024), (20480, 128)):
            rep, wg, wu = matrices(cuda_lib, n, k, fmt, 11, scales)
            for bn, ku, pair in ((16, 1, 0), (16, 2, 0), (32, 1, 0), (32, 2, 0), (64, 1, 0), (64, 2, 0), (128, 1, 1), (256, 1, 1),
                                 (128, 1, 2), (256, 1, 2)):
                cuda_lib.set_tile_config(bn, ku)
                cuda_lib.set_pair_mode(pair)
                m = 37 if n > 1000 else 300
                a = activations(m, k, fmt, bn)
                ws = cuda_lib.Workspace()
                check(cuda_lib.gated_gemm(a, rep, n, fmt, scales, "gelu_tanh", ws), a, wg, wu, scales, "gelu_tanh", f"{n} {bn} {ku} {pair}")
                assert ws.status() == 0
    finally:
        cuda_lib.set_tile_config()
        cuda_lib.set_pair_mode()


@pytest.mark.parametrize("m", [5, 40, 200, 300])
def test_bounds_checking_build(cuda_lib, m):
    """No index of the gated epilogue leaves its buffer; with C's extent cut the
    check, and nothing else, answers."""
    n, k = 256, 1024
    rep, wg, wu = matrices(cuda_lib, n, k, "nvfp4", 3, SCALES["nvfp4"])
    a = activations(m, k, "nvfp4", m)
    want = cuda_lib.gated_gemm(a, rep, n, "nvfp4", SCALES["nvfp4"])
    with cuda_lib.bounds_checked() as chk:
        ws = cuda_lib.Workspace()
        got = cuda_lib.gated_gemm(a, rep, n, "nvfp4", SCALES["nvfp4"], workspace=ws)
        assert ws.status() == 0 and torch.equal(got, want)
        try:
            assert chk.petit_check_set_limits(-1, m * n - 1) == 0
            cuda_lib.gated_gemm(a, rep, n, "nvfp4", SCALES["nvfp4"], workspace=ws)
            assert ws.status() == 8
        finally:
            chk.petit_check_set_limits(-1, -1)
        assert torch.equal(cuda_lib.gated_gemm(a, rep, n, "nvfp4", SCALES["nvfp4"], workspace=ws), want) and ws.status() == 0


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
def test_experts(cuda_lib, fmt):
    n, k, E = 320, 768, 5
    scales = [(0.001 * (1 + i), 0.002 / (1 + i)) if fmt == "nvfp4" else (1.0, 1.0) for i in range(E)]
    mats = [matrices(cuda_lib, n, k, fmt, 20 + 2 * i, scales[i]) for i in range(E)]
    rep = torch.cat([m[0] for m in mats])
    torch.cuda.synchronize()
    ws = cuda_lib.Workspace()
    for off in ([0, 1, 1, 4, 5, 5], [0, 0, 70, 70, 200, 210], [0, 300, 301, 301, 301, 330], [0, 0, 0, 0, 0, 17]):
        a = activations(off[-1], k, fmt, off[-1])
        out = torch.full((off[-1] + 3, n), 9.0, dtype=torch.bfloat16, device="cuda")
        got = cuda_lib.moe_gated_gemm(a, rep, off, n, fmt, scales, "silu", ws, out=out[:off[-1]])
        for e in range(E):
            if off[e + 1] > off[e]:
                rows = slice(off[e], off[e + 1])
                check(got[rows], a[rows], *mats[e][1:], scales[e], "silu", f"{off} expert {e}")
        assert (out[off[-1]:] == 9).all()
    none = cuda_lib.moe_gated_gemm(a[:0], rep, [0] * 6, n, fmt, scales, workspace=ws)
    assert none.shape == (0, n) and ws.status() == 0


def test_weight_class_and_unfused_product(cuda_lib):
    """GatedWeight against two FP4Weight products of the same matrices."""
    wg, wu = synth.weights(256, 512, seed=1, device="cuda"), synth.weights(256, 512, seed=2, device="cuda", std=0.05)
    a = activations(33, 512, "nvfp4", 3)
    for fmt in ("nvfp4", "mxfp4", "nvfp4_f16"):
        x = a.half() if fmt == "nvfp4_f16" else a
        both = cuda_lib.GatedWeight(wg, wu, fmt, "amax")
        g, u = (cuda_lib.FP4Weight(w, fmt, "amax")(x).float() for w in (wg, wu))
        want = torch.nn.functional.silu(g) * u
        # g and u rounded to 16 bits on the way: half a step each, g's through a derivative below 1.13 silu'/silu
        assert ((both(x).float() - want).norm() / want.norm()).item() < 2.0 ** -7
        assert both(x, out=torch.empty((33, 256), dtype=x.dtype, device="cuda")).shape == (33, 256)


def test_extremes(cuda_lib):
    """Rows of zeros, large sums of either sign, infinities and NaN."""
    n, k = 64, 128
    w = torch.zeros((n, k)).bfloat16()
    w[:, 0] = 6.0
    w = w.cuda()
    one = cuda_lib.GatedWeight(w, w, "mxfp4")
    a = torch.zeros((8, k), dtype=torch.bfloat16)
    for i, v in enumerate((0.0, 1e4, -1e4, 1e30, -1e30, float("inf"), float("nan"), -3.0)):
        a[i, 0] = v
    for act in ("silu", "gelu", "gelu_tanh"):
        h = one(a.cuda(), act).float().cpu()
        z = 6.0 * a[:, 0].double().numpy()
        want = float(layer.act(z[7], act) * z[7])
        assert (h[0] == 0).all() and (h[2] == 0).all() and (h[4] == 0).all()
        assert ((h[1] - 3.6e9).abs() <= 3.6e9 * 2.0 ** -7).all()        # (1e4 itself is rounded to BF16)
        assert torch.isinf(h[3]).all() and not torch.isfinite(h[5]).any() and torch.isnan(h[6]).all()
        assert ((h[7] - want).abs() <= abs(want) * 2.0 ** -7 + 2.0 ** -120).all()


def test_graph_and_streams(cuda_lib):
    """Two graphs and an eager call share a workspace, one after the other; the norm before feeds the product."""
    n, k = 256, 512
    rep, wg, wu = matrices(cuda_lib, n, k, "nvfp4", 7, SCALES["nvfp4"])
    ws = cuda_lib.Workspace()
    x = activations(20, k, "nvfp4", 1)
    run = lambda: cuda_lib.gated_gemm(cuda_lib.rms_norm(x), rep, n, "nvfp4", SCALES["nvfp4"], workspace=ws)  # noqa: E731
    run()
    graphs, outs = [], []
    for _ in range(2):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append(run())
    for seed in (2, 3):
        x.copy_(activations(20, k, "nvfp4", seed))
        graphs[0].replay()
        eager = run()
        graphs[1].replay()
        check(eager, cuda_lib.rms_norm(x), wg, wu, SCALES["nvfp4"], "silu")
        assert torch.equal(outs[0], eager) and torch.equal(outs[1], eager)
    assert ws.status() == 0


def test_refusals(cuda_lib):
    w = synth.weights(64, 128, device="cuda")
    one = cuda_lib.GatedWeight(w, w, "mxfp4")
    x = activations(3, 128, "mxfp4", 1)
    for bad in (dict(A=x.half()), dict(A=x.cpu()), dict(A=x[:, ::2]), dict(act="relu"), dict(rep=one.rep[:-16]), dict(n=128),
                dict(out=x[:, :64]), dict(out=torch.empty((4, 64), dtype=x.dtype, device="cuda"))):
        with pytest.raises(ValueError):
            cuda_lib.gated_gemm(**{**dict(A=x, rep=one.rep, n=64, fmt="mxfp4"), **bad})
    for bad in (dict(n=32), dict(global_scales=(0.0, 1.0)), dict(A=x[:0])):
        with pytest.raises(cuda_lib.PetitError):
            cuda_lib.gated_gemm(**{**dict(A=x, rep=one.rep, n=64, fmt="mxfp4"), **bad})
    with pytest.raises(ValueError, match="pairs"):
        cuda_lib.moe_gated_gemm(x, one.rep, [0, 3], 64, "mxfp4", [])
    with pytest.raises(ValueError, match="rep"):
        cuda_lib.moe_gated_gemm(x, one.rep, [0, 1, 3], 64, "mxfp4")
