"""Gated products whose tiles are lower than their kernel's, with every kernel that
the planner has, alone and in groups of different sizes; bounds as in
test_gpu_gated."""

import pytest
import torch

from tests.test_gpu_gated import SCALES, activations, check, matrices

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4", "nvfp4_f16"])
@pytest.mark.parametrize("n,k", [(1024, 1024), (320, 896)])      # (pairs and two chunks a unit; neither)
def test_rows_between_tile_heights(cuda_lib, fmt, n, k):
    rep, wg, wu = matrices(cuda_lib, n, k, fmt, n, SCALES[fmt])
    ws = cuda_lib.Workspace()
    seen = set()
    for m in (63, 66, 70, 81, 95, 97, 112, 113, 127, 130, 145, 161, 177, 193, 210, 225, 241, 255, 258, 275, 321, 385, 513, 700):
        a = activations(m, k, fmt, m)
        out = torch.full((m + 40, n), 3.0, dtype=a.dtype, device="cuda")
        check(cuda_lib.gated_gemm(a, rep, n, fmt, SCALES[fmt], "silu", ws, out=out[:m]), a, wg, wu, SCALES[fmt], "silu", f"m = {m}")
        assert (out[m:] == 3).all()                        # rows behind the last one stay
        p = cuda_lib.gated_plan([0, m], n, k, fmt)
        seen.add((p["bn"], p["ku"], p["cta_pairs"]))
    assert ws.status() == 0 and (n != 1024 or len(seen) > 1)   # (the forced shapes below cover the rest)


@pytest.mark.parametrize("bn,ku,pair", [(128, 1, 1), (128, 1, 2), (256, 1, 1), (256, 1, 2), (64, 2, 0), (32, 2, 0)])
def test_forced_tiles_and_few_rows(cuda_lib, bn, ku, pair):
    n, k = 512, 2048
    rep, wg, wu = matrices(cuda_lib, n, k, "nvfp4", 9, SCALES["nvfp4"])
    ws = cuda_lib.Workspace()
    try:
        cuda_lib.set_tile_config(bn, ku)
        cuda_lib.set_pair_mode(pair)
        for m in (1, 16, 17, 33, 50, 129, 257, 290):
            a = activations(m, k, "nvfp4", m)
            check(cuda_lib.gated_gemm(a, rep, n, "nvfp4", SCALES["nvfp4"], "gelu", ws), a, wg, wu, SCALES["nvfp4"], "gelu", f"m = {m}")
    finally:
        cuda_lib.set_tile_config()
        cuda_lib.set_pair_mode()
    assert ws.status() == 0


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("bn,pair", [(0, 0), (64, 0), (128, 1), (128, 2), (256, 1), (256, 2)])
def test_groups_of_different_heights(cuda_lib, fmt, bn, pair):
    n, k, E = 256, 1024, 7
    scales = [(0.001 * (1 + i), 0.002 / (1 + i)) if fmt == "nvfp4" else (1.0, 1.0) for i in range(E)]
    mats = [matrices(cuda_lib, n, k, fmt, 40 + 2 * i, scales[i]) for i in range(E)]
    rep = torch.cat([m[0] for m in mats])
    torch.cuda.synchronize()
    ws = cuda_lib.Workspace()
    try:
        if bn:
            cuda_lib.set_tile_config(bn, 2 if bn <= 64 else 1)
        cuda_lib.set_pair_mode(pair)
        for sizes in ([3, 0, 100, 17, 0, 260, 1], [130, 131, 64, 65, 33, 16, 200], [0, 0, 0, 0, 0, 0, 300], [1, 1, 1, 1, 1, 1, 1]):
            off = [0]
            for s in sizes:
                off.append(off[-1] + s)
            a = activations(off[-1], k, fmt, off[-1])
            out = torch.full((off[-1] + 9, n), 5.0, dtype=torch.bfloat16, device="cuda")
            got = cuda_lib.moe_gated_gemm(a, rep, off, n, fmt, scales, "silu", ws, out=out[:off[-1]])
            assert torch.equal(got, cuda_lib.moe_gated_gemm(a, rep, off, n, fmt, scales, "silu", ws))
            for e in range(E):
                if sizes[e]:
                    rows = slice(off[e], off[e + 1])
                    check(got[rows], a[rows], *mats[e][1:], scales[e], "silu", f"{sizes} expert {e}")
            assert (out[off[-1]:] == 5).all()
    finally:
        cuda_lib.set_tile_config()
        cuda_lib.set_pair_mode()
    assert ws.status() == 0


@pytest.mark.parametrize("m", [100, 150, 290])
def test_bounds_checking_build(cuda_lib, m):
    n, k = 256, 1024
    rep, _, _ = matrices(cuda_lib, n, k, "mxfp4", 3, SCALES["mxfp4"])
    a = activations(m, k, "mxfp4", m)
    off = [0, 5, 5, m]
    many = torch.cat([rep] * 3)
    torch.cuda.synchronize()
    want = cuda_lib.gated_gemm(a, rep, n, "mxfp4"), cuda_lib.moe_gated_gemm(a, many, off, n, "mxfp4")
    with cuda_lib.bounds_checked() as chk:
        ws = cuda_lib.Workspace()
        got = cuda_lib.gated_gemm(a, rep, n, "mxfp4", workspace=ws), cuda_lib.moe_gated_gemm(a, many, off, n, "mxfp4", workspace=ws)
        assert ws.status() == 0 and all(torch.equal(x, y) for x, y in zip(got, want))
        try:
            assert chk.petit_check_set_limits(-1, m * n - 1) == 0
            cuda_lib.moe_gated_gemm(a, many, off, n, "mxfp4", workspace=ws)
            assert ws.status() == 8
        finally:
            chk.petit_check_set_limits(-1, -1)


@pytest.mark.parametrize("fmt,m,k", [("nvfp4", 300, 5120), ("nvfp4", 2100, 4096), ("mxfp4", 700, 5120)])
def test_tiles_dealt_out_to_ranges(cuda_lib, fmt, m, k):
    """Weights past what L2 holds and several activation tiles: ranges take tiles
    that lie apart.  Every column against products of the dequantised weights in 64
    bits; no index leaves its buffer."""
    n = 14336
    g = torch.Generator(device="cuda").manual_seed(m)
    wg, wu = ((torch.randn((n, k), generator=g, device="cuda") * k ** -0.5).bfloat16() for _ in range(2))
    one = cuda_lib.GatedWeight(wg, wu, fmt, "amax")
    a = activations(m, k, fmt, m)
    got = one(a, "silu").double()
    both = cuda_lib.dequant(one.rep, 2 * n, k, fmt).unflatten(0, (-1, 2, 8)).transpose(0, 1).flatten(1, 2).double()
    x = a.double()
    gate, up = (s * (x @ w.T) for s, w in zip(one.global_scales, both))
    step = 1.25 * k * 2.0 ** -24
    dg, du = (step * s * (x.abs() @ w.abs().T) for s, w in zip(one.global_scales, both))
    act = gate * torch.sigmoid(gate)
    want = act * up
    off = (1.13 * dg + act.abs() * 2.0 ** -15 + 2.0 ** -120) * (up.abs() + du) + act.abs() * du
    assert ((got - want).abs() <= want.abs() * 2.0 ** -8 + off * (1 + 2.0 ** -8) + 2.0 ** -134).all()
    if m == 300:
        with cuda_lib.bounds_checked():
            ws = cuda_lib.Workspace()
            checked = one(a, "silu", workspace=ws)
            assert ws.status() == 0 and torch.equal(checked.double(), got)


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("n,sizes", [(2048, [100, 0, 128, 33, 97, 100, 64, 128, 120]),    # pairs, many tiles a range
                                     (7168, [90]), (1088, [100, 128, 100, 0, 96, 128])])  # pairs, few; no pairs
def test_accumulators_in_turn(cuda_lib, fmt, n, sizes):
    k, scales = 1024, SCALES[fmt]
    mats = [matrices(cuda_lib, n, k, fmt, 90 + 2 * i, scales) for i in range(2)]   # (experts take one of two in turn)
    rep = torch.cat([mats[e % 2][0] for e in range(len(sizes))])
    off = [0]
    for s in sizes:
        off.append(off[-1] + s)
    a = activations(off[-1], k, fmt, 3)
    ws = cuda_lib.Workspace()
    torch.cuda.synchronize()
    call = lambda: cuda_lib.moe_gated_gemm(a, rep, off, n, fmt, [scales] * len(sizes), "silu", ws)  # noqa: E731
    y = call()
    for e, (lo, hi) in enumerate(zip(off, off[1:])):
        if lo < hi:
            check(y[lo:hi], a[lo:hi], *mats[e % 2][1:], scales, "silu", f"expert {e}")
    assert all(torch.equal(call(), y) for _ in range(20)) and ws.status() == 0
    with cuda_lib.bounds_checked():
        ws = cuda_lib.Workspace()
        assert torch.equal(call(), y) and ws.status() == 0
