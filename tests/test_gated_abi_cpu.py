"""Gated products: every refusal, before any device is touched."""

import ctypes

import pytest
import torch

from fp4_weight_only_gb300 import binding

A, ODD = 0x10000, 0x10008   # addresses that validation must never use
OK, INVALID, SHAPE, ALIGN, WORKSPACE = 0, 1, 2, 3, 4


@pytest.fixture(scope="module")
def lib():
    return binding.load()


BAD = [(dict(fmt=3), INVALID), (dict(fmt=-1), INVALID), (dict(A=None), INVALID), (dict(rep=None), INVALID), (dict(C=None), INVALID),
       (dict(act=3), INVALID), (dict(act=-1), INVALID), (dict(g=0.0), INVALID), (dict(u=-1.0), INVALID), (dict(g=float("nan")), INVALID),
       (dict(u=float("inf")), INVALID), (dict(n=96), SHAPE), (dict(n=0), SHAPE), (dict(n=-64), SHAPE), (dict(k=192), SHAPE),
       (dict(k=0), SHAPE), (dict(n=1 << 24), SHAPE), (dict(n=1 << 62), SHAPE), (dict(k=1 << 25), SHAPE), (dict(A=ODD), ALIGN),
       (dict(rep=ODD), ALIGN), (dict(C=ODD), ALIGN), (dict(ws=None), WORKSPACE), (dict(ws=ODD), ALIGN)]


def _args(change):
    d = dict(fmt=0, A=A, rep=A, g=1.0, u=1.0, act=0, C=A, n=128, k=256, ws=A)
    d.update(change)
    return d


@pytest.mark.parametrize("change,want", BAD + [(dict(m=0), INVALID), (dict(m=-1), INVALID), (dict(m=(1 << 24) + 1), SHAPE)])
def test_dense(lib, change, want):
    d = _args({"m": 4, **change})
    assert lib.petit_gated_gemm(d["fmt"], d["A"], d["rep"], d["g"], d["u"], d["act"], d["C"], d["m"], d["n"], d["k"], d["ws"],
                                1 << 40, None) == want


@pytest.mark.parametrize("change,want", BAD + [
    (dict(fmt=2), INVALID), (dict(off=None), INVALID), (dict(off=[1, 2]), INVALID), (dict(off=[0, 3, 2]), INVALID),
    (dict(off=[0] * 66), SHAPE), (dict(off=[0]), INVALID), (dict(off=[0, (1 << 24) + 1]), SHAPE), (dict(off=[0, 0, 0]), OK),
    (dict(g=None), INVALID), (dict(u=None), INVALID)])
def test_grouped(lib, change, want):
    d = _args({"off": [0, 3, 4], **change})
    off = d["off"] or [0, 3]
    e = len(off) - 1
    scales = [None if s is None else (ctypes.c_float * max(e, 1))(*[s] * max(e, 1)) for s in (d["g"], d["u"])]
    arr = None if d["off"] is None else (ctypes.c_int64 * len(off))(*off)
    assert lib.petit_moe_gated_gemm(d["fmt"], d["A"], d["rep"], *scales, arr, e, d["act"], d["C"], d["n"], d["k"], d["ws"], 1 << 40,
                                    None) == want


def test_binding(lib):
    x = torch.zeros((2, 128), dtype=torch.bfloat16)
    rep = torch.zeros(1 << 16, dtype=torch.uint8)
    with pytest.raises(ValueError, match="CUDA"):
        binding.gated_gemm(x, rep, 64)
    with pytest.raises(ValueError, match="CUDA"):
        binding.moe_gated_gemm(x, rep, [0, 2], 64)
    with pytest.raises(ValueError, match="must equal"):
        binding.moe_gated_gemm(x, rep, [0, 1], 64)
    with pytest.raises(ValueError, match="shape"):
        binding.gated_repack(rep.view(-1, 64), rep.view(-1, 8), rep.view(-1, 32), rep.view(-1, 8))
    with pytest.raises(ValueError, match="shape"):
        binding.GatedWeight(x, x[:1])
