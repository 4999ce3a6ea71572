"""Position encoding in the attention block: q and k are rotated between the
QKV product and the cache, by the caller's function."""

import numpy as np
import pytest
import torch

from fp4_weight_only_gb300 import attend, synth
from oracle import kv
from tests.kv_tight import bounds, expect, outside

pytestmark = pytest.mark.gpu


def rotate(x, pos):
    """Rotary encoding of x [tokens, heads, dim] at positions `pos`."""
    half = x.shape[-1] // 2
    angle = pos[:, None, None].float() * 10000.0 ** (-torch.arange(half, device=x.device) / half)
    a, b = x[..., :half].float(), x[..., half:].float()
    return torch.cat((a * angle.cos() - b * angle.sin(), a * angle.sin() + b * angle.cos()), -1).to(x.dtype)


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
def test_rotated_queries_and_keys(cuda_lib, fmt):
    heads, kvh, dim, hidden, page = 6, 2, 64, 512, 16
    scales = torch.full((2, kvh), 0.002, device="cuda") if fmt == "nvfp4" else None
    block = attend.AttentionBlock(synth.weights((heads + 2 * kvh) * dim, hidden, seed=1, device="cuda", std=hidden ** -0.5),
                                  synth.weights(hidden, heads * dim, seed=2, device="cuda"), heads, kvh, dim, 8, page,
                                  fmt, scales)
    table = torch.tensor([[5, 2, 7, 0]], dtype=torch.int32, device="cuda")
    gs = [None, None] if scales is None else list(scales.cpu().numpy())
    held, n = [[], []], 0
    for m in (20, 1, 9, 1):
        pos = torch.arange(n, n + m, device="cuda")
        n += m
        x = synth.activations(m, hidden, seed=n, device="cuda")
        args = (attend.slots_of(table, torch.zeros_like(pos), pos, page), table,
                torch.tensor([n], dtype=torch.int32, device="cuda"), None, m)

        def position(q, k):
            assert q.shape == (m, heads, dim) and k.shape == (m, kvh, dim)
            return rotate(q, pos), rotate(k, pos)

        y = block(x, *args, position=position)
        out = block.attend(x, *args, position=position)
        assert torch.equal(y, block.o(out.view(m, -1), block.workspace))
        q, k, v = block.project(x)
        q = rotate(q, pos)
        for dst, rows, g in zip(held, (rotate(k, pos), v), gs):
            dst.append(kv.values(*kv.quantize_rows(rows.float().cpu().numpy(), fmt, g), fmt, g))
        k, v = (np.concatenate(z) for z in held)
        want, *rest = expect(q.float().cpu().numpy(), k, v, dim ** -0.5)
        assert not outside(out.float().cpu().numpy(), want, bounds(want, *rest, dim, out.dtype)[0]).any()
    assert block.workspace.status() == 0
