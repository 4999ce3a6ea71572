"""Errors that K/V calls record in a workspace, when the workspace grows."""

import pytest
import torch

pytestmark = pytest.mark.gpu


def _one_token(cuda_lib):
    cache = cuda_lib.KVCache(2, 16, 1, 64, "nvfp4")
    k = torch.ones((1, 1, 64), dtype=torch.bfloat16, device="cuda")
    table = torch.zeros((1, 1), dtype=torch.int32, device="cuda")
    return cache, k, table, torch.ones(1, dtype=torch.int32, device="cuda")


def test_a_recorded_slot_outlives_the_workspace_it_was_recorded_in(cuda_lib):
    """The workspace grows between the call that records an error and the question for it."""
    cache, k, table, lens = _one_token(cuda_lib)
    ws = cuda_lib.Workspace()
    cache.append(k, k, torch.tensor([32], device="cuda"), ws)
    cache.attention(k, table, lens, workspace=ws)
    assert ws.status() == 8
    assert ws.status() == 0


def test_a_captured_call_keeps_its_workspace(cuda_lib):
    """A graph holds the workspace as it was when the call was captured: it
    records there, and nobody else's tensor takes its place."""
    cache, k, table, lens = _one_token(cuda_lib)
    ws = cuda_lib.Workspace()
    slot = torch.zeros(1, dtype=torch.int64, device="cuda")
    cache.append(k, k, slot, ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        cache.append(k, k, slot, ws)
    cache.attention(k, table, lens, workspace=ws)
    others = [torch.zeros(256, dtype=torch.uint8, device="cuda") for _ in range(64)]
    slot.fill_(99)
    g.replay()
    torch.cuda.synchronize()
    assert not any(o.any() for o in others)
    assert ws.status() == 8 and ws.status() == 0
    slot.fill_(1)
    g.replay()
    assert ws.status() == 0
