"""The attention block (QKV product, cache, attention, O product) against the
float64 oracle: K and V of the device's QKV product are quantised and attended
on the CPU; error bounds as in kv_util.Case.check."""

import types

import numpy as np
import pytest
import torch

from fp4_weight_only_gb300 import attend, synth
from oracle import kv
from tests.kv_util import Case

pytestmark = pytest.mark.gpu


def _values(x, fmt, scales):
    return kv.values(*kv.quantize_rows(x, fmt, scales), fmt, scales)


@pytest.mark.parametrize("fmt,dim,group,window", [("nvfp4", 128, 4, 0), ("mxfp4", 64, 3, 0), ("nvfp4", 64, 8, 20)])
def test_prompt_pieces_then_single_tokens(cuda_lib, fmt, dim, group, window):
    kvh, hidden, page, batch = 2, 512, 16, 3
    heads = kvh * group
    scales = torch.full((2, kvh), 0.002, device="cuda") if fmt == "nvfp4" else None
    w_qkv = synth.weights((heads + 2 * kvh) * dim, hidden, seed=1, device="cuda", std=hidden ** -0.5)
    w_o = synth.weights(hidden, heads * dim, seed=2, device="cuda")
    block = attend.AttentionBlock(w_qkv, w_o, heads, kvh, dim, 24, page, fmt, scales)
    g = torch.Generator().manual_seed(0)
    table = torch.randperm(24, generator=g).view(batch, 8).int().cuda()
    ks, vs = [[] for _ in range(batch)], [[] for _ in range(batch)]
    lens = [0] * batch
    gs = [None, None] if scales is None else list(scales.cpu().numpy())
    # ragged prompts, a second piece for one of them, then single tokens
    for i, nqs in enumerate(([17, 1, 60], [0, 40, 0], [1, 1, 1], [1, 1, 1], [2, 1, 3])):
        pos = torch.cat([torch.arange(n) + lens[b] for b, n in enumerate(nqs)]).cuda()
        seq = torch.repeat_interleave(torch.arange(batch), torch.tensor(nqs)).cuda()
        lens = [n + m for n, m in zip(lens, nqs)]
        x = synth.activations(sum(nqs), hidden, seed=10 + i, device="cuda")
        args = (attend.slots_of(table, seq, pos, page), table, torch.tensor(lens, dtype=torch.int32, device="cuda"),
                torch.tensor(np.cumsum([0] + nqs), dtype=torch.int32, device="cuda"), max(nqs), window)
        y = block(x, *args)
        out = block.attend(x, *args)
        assert torch.equal(y, block.o(out.view(sum(nqs), -1), block.workspace)) and y.shape == x.shape
        q, k, v = block.project(x)
        at = 0
        for b, n in enumerate(nqs):
            for dst, rows, s in ((ks, k, gs[0]), (vs, v, gs[1])):
                dst[b].append(_values(rows[at:at + n].float().cpu().numpy(), fmt, s))
            at += n
        want = types.SimpleNamespace(dim=dim, lens=lens, k=[np.concatenate(z) for z in ks],
                                     v=[np.concatenate(z) for z in vs])
        Case.check(want, q, nqs, out, window=window)
    assert block.workspace.status() == 0


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
def test_command(cuda_lib, fmt, capsys):
    import json
    assert attend.main(["--batch", "3", "--prompt", "70", "--steps", "5", "--hidden", "512", "--q-heads", "8",
                        "--kv-heads", "2", "--head-dim", "64", "--page", "16", "--fmt", fmt]) == 0
    r = json.loads(capsys.readouterr().out)
    # 23 + 46 + 70 prompt tokens and eight steps of three sequences
    assert r["prompt_tokens"] == 139 and r["cached_tokens"] == 139 + 3 * (2 + 1 + 5)
    assert r["cache_bytes_per_token"] == 2 * 2 * (32 + (4 if fmt == "nvfp4" else 2))
    # BF16 outputs (2^-9 on average at most), weights of 11 bits
    assert r["relative_error"] < 2.0 ** -8


def test_weights_that_do_not_fit(cuda_lib):
    w = synth.weights(768, 512, device="cuda")
    o = synth.weights(512, 512, device="cuda")
    for bad in ((w[:700], o, 8, 2, 64), (w, o[:, :256], 8, 2, 64), (w, o[:100], 8, 2, 64)):
        with pytest.raises(ValueError, match="w_"):
            attend.AttentionBlock(*bad, num_pages=2)
    with pytest.raises(cuda_lib.PetitError):
        attend.AttentionBlock(w, o, 8, 2, 64, num_pages=2, page_size=24)
