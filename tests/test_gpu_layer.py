"""The decoder layer: every stage against the float64 oracle on the stage's own
inputs, with that operator's bound, and the layer against the stages bit for bit."""

import types

import numpy as np
import pytest
import torch

from fp4_weight_only_gb300 import attend, layer, synth
from oracle import gemm
from oracle import layer as olayer
from tests.gpu_util import assert_parity, oracle_quantize
from tests.kv_util import Case
from tests.test_gpu_attend import _values
from tests.test_gpu_gated import check as check_gated
from tests.test_gpu_norm import _f64, check16
from tests.test_gpu_rotary import check as check_rotary

pytestmark = pytest.mark.gpu


def _dequantized(w, fmt, g):
    codes, scales = oracle_quantize(w.cpu(), fmt, g)
    return gemm.dequantize(codes, scales, fmt)


@pytest.mark.parametrize("fmt,act,interleaved,rot", [("nvfp4", "silu", False, 64), ("mxfp4", "gelu_tanh", True, 32), ("nvfp4", "gelu", False, 24)])
def test_stages(cuda_lib, fmt, act, interleaved, rot):
    hidden, inter, hq, hk, dim, page = 256, 384, 4, 2, 64, 16
    w = lambda n, k, j: synth.weights(n, k, seed=j, device="cuda", std=k ** -0.5)  # noqa: E731
    wq, wo = w((hq + 2 * hk) * dim, hidden, 1), w(hidden, hq * dim, 2)
    wg, wu, wd = w(inter, hidden, 3), w(inter, hidden, 4), w(hidden, inter, 5)
    n1, n2 = (1.0 + 0.1 * synth.activations(1, hidden, seed=s, device="cuda")[0].float() for s in (6, 7))
    scales = torch.full((2, hk), 0.002, device="cuda") if fmt == "nvfp4" else None
    freq = cuda_lib.rotary_frequencies(rot, 10000.0, 2.0, "ramp", 64, 1.0, 4.0)
    rope = cuda_lib.Rotary(rot, frequencies=freq, interleaved=interleaved, magnitude=1.125)
    one = layer.DecoderLayer(wq, wo, wg, wu, wd, n1, n2, hq, hk, dim, 24, rope, 1e-5, act, page, fmt, scales)
    table = torch.randperm(24, generator=torch.Generator().manual_seed(0)).view(3, 8).int().cuda()
    ks, vs, lens = [[], [], []], [[], [], []], [0, 0, 0]
    gs = [None, None] if scales is None else list(scales.cpu().numpy())
    # prompts of three sequences, then a token of each, then two of one
    for i, nqs in enumerate(([17, 1, 40], [1, 1, 1], [0, 2, 0])):
        total = sum(nqs)
        pos = torch.cat([torch.arange(n) + lens[b] for b, n in enumerate(nqs)]).cuda()
        seq = torch.repeat_interleave(torch.arange(3), torch.tensor(nqs)).cuda()
        lens = [n + m for n, m in zip(lens, nqs)]
        x = synth.activations(total, hidden, seed=20 + i, device="cuda")
        residual = synth.activations(total, hidden, seed=30 + i, device="cuda") if i else None
        args = (attend.slots_of(table, seq, pos, page), table, torch.tensor(lens, dtype=torch.int32, device="cuda"),
                torch.tensor(np.cumsum([0] + nqs), dtype=torch.int32, device="cuda"), max(nqs))
        kept = x.clone(), None if residual is None else residual.clone()
        y, stream = one(x, residual, pos, *args)
        assert torch.equal(x, kept[0]) and (residual is None or torch.equal(residual, kept[1]))

        # the stages, each from what the one before gave
        h = cuda_lib.rms_norm(x, n1, 1e-5, residual)
        h, r1 = (h, x) if residual is None else h
        check16(h, olayer.rms_norm(_f64(x), _f64(n1), 1e-5, None if residual is None else _f64(residual))[0], torch.bfloat16)
        att = one.attention
        q0, k0, v = (t.clone() for t in att.project(h))
        assert_parity(att.qkv(h, one.workspace), gemm.gemm(_f64(h), _dequantized(wq, fmt, att.qkv.global_scale), att.qkv.global_scale))
        q, k = rope(q0, k0, pos)
        check_rotary(q, q0, pos.tolist(), freq, interleaved, 1.125)
        check_rotary(k, k0, pos.tolist(), freq, interleaved, 1.125)
        heads = att.attend(h, *args, position=lambda a, b: (q, k))
        at = 0
        for b, n in enumerate(nqs):
            for dst, rows, s in ((ks, k, gs[0]), (vs, v, gs[1])):
                dst[b].append(_values(_f64(rows[at:at + n]).astype(np.float32), fmt, s))
            at += n
        Case.check(types.SimpleNamespace(dim=dim, lens=lens, k=[np.concatenate(z) for z in ks], v=[np.concatenate(z) for z in vs]),
                   q, nqs, heads)
        a = att.o(heads.reshape(total, -1), one.workspace)
        assert_parity(a, gemm.gemm(_f64(heads.reshape(total, -1)), _dequantized(wo, fmt, att.o.global_scale), att.o.global_scale))
        h2, r2 = cuda_lib.rms_norm(a, n2, 1e-5, r1)
        check16(h2, olayer.rms_norm(_f64(a), _f64(n2), 1e-5, _f64(r1))[0], torch.bfloat16)
        m = one.gated(h2, act, one.workspace)
        sc = one.gated.global_scales
        check_gated(m, h2, _dequantized(wg, fmt, sc[0]), _dequantized(wu, fmt, sc[1]), sc, act)
        want = one.down(m, one.workspace)
        assert torch.equal(y, want) and torch.equal(stream, r2)
    assert one.workspace.status() == 0


def test_without_positions_and_stack(cuda_lib):
    """No rope: the attention block's own positions-free form; a stack adds its last output to the stream."""
    hidden = 256
    w = lambda n, k, j: synth.weights(n, k, seed=j, device="cuda", std=k ** -0.5)  # noqa: E731
    norm = torch.ones(hidden, dtype=torch.bfloat16, device="cuda")
    ws = cuda_lib.Workspace()
    stack = [layer.DecoderLayer(w(512, hidden, 1 + 9 * i), w(hidden, 256, 2), w(128, hidden, 3), w(128, hidden, 4), w(hidden, 128, 5), norm,
                                norm, 4, 2, 64, 4, page_size=16, fmt="mxfp4", workspace=ws) for i in (0, 1)]
    x = synth.activations(5, hidden, seed=8, device="cuda")
    table = torch.arange(4, dtype=torch.int32, device="cuda").view(1, 4)
    args = (torch.arange(5, device="cuda"), torch.arange(5, device="cuda"), table, torch.tensor([5], dtype=torch.int32, device="cuda"),
            torch.tensor([0, 5], dtype=torch.int32, device="cuda"), 5)
    y = layer.run(stack, x, *args)
    a, r = stack[0](x, None, *args)
    a, r = stack[1](a, r, *args)
    assert torch.equal(y, a + r) and ws.status() == 0


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
def test_command(cuda_lib, fmt, capsys):
    import json
    assert layer.main(["--layers", "2", "--batch", "3", "--prompt", "70", "--steps", "5", "--hidden", "512", "--intermediate", "896",
                       "--q-heads", "8", "--kv-heads", "2", "--head-dim", "64", "--page", "16", "--fmt", fmt]) == 0
    r = json.loads(capsys.readouterr().out)
    # 23 + 46 + 70 prompt tokens and eight steps of three sequences
    assert r["prompt_tokens"] == 139 and r["cached_tokens"] == 139 + 3 * (2 + 1 + 5) and r["layers"] == 2


def test_refusals(cuda_lib):
    w = lambda n, k: synth.weights(n, k, device="cuda")  # noqa: E731
    good = dict(w_qkv=w(512, 256), w_o=w(256, 256), w_gate=w(128, 256), w_up=w(128, 256), w_down=w(256, 128),
                norm_attention=torch.ones(256, device="cuda"), norm_mlp=torch.ones(256, device="cuda"), num_q_heads=4, num_kv_heads=2,
                head_dim=64, num_pages=2)
    layer.DecoderLayer(**good)
    for bad in (dict(w_up=w(64, 256)), dict(w_down=w(256, 256)), dict(w_gate=w(128, 128), w_up=w(128, 128)), dict(norm_mlp=torch.ones(64, device="cuda")),
                dict(act="relu"), dict(w_o=w(256, 128))):
        with pytest.raises(ValueError):
            layer.DecoderLayer(**{**good, **bad})
