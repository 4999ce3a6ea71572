"""Arguments that the K/V binding builds or refuses, seen without a device: the
library's entry point is replaced by one that records them."""

import ctypes
import types

import pytest
import torch

from fp4_weight_only_gb300 import binding


@pytest.fixture
def calls(monkeypatch):
    made = []

    def attention(cache, args, *rest):
        args = ctypes.cast(args, ctypes.POINTER(binding.KvAttentionArgs)).contents
        made.append({n: getattr(args, n) for n, _ in args._fields_})
        return 0

    monkeypatch.setattr(binding, "load", lambda: types.SimpleNamespace(petit_kv_attention=attention))
    monkeypatch.setattr(binding, "_stream", lambda: 0)
    return made


def _call(table, batch=None, **k):
    cache = types.SimpleNamespace(num_kv_heads=1, head_dim=64, device=torch.device("cpu"), device_index=-1, _ref=None,
                                  workspace_bytes=lambda: 256)
    batch = table.shape[0] if batch is None else batch
    q = torch.zeros((batch, 2, 64), dtype=torch.bfloat16)
    return binding.kv_attention(cache, q, table, torch.ones(batch, dtype=torch.int32), **k)


def test_rows_of_a_table_that_share_memory_are_refused(calls):
    """A row of pages given to every sequence by expand() has a stride of zero;
    the kernels would read batch rows of memory that holds one."""
    row = torch.arange(7, dtype=torch.int32)
    for table in (row.expand(5, 7), row.as_strided((3, 4), (1, 1)), row.as_strided((2, 4), (3, 1))):
        with pytest.raises(ValueError, match="block_table"):
            _call(table)
    assert calls == []


@pytest.mark.parametrize("table,stride", [
    (torch.zeros((5, 7), dtype=torch.int32), 7), (torch.zeros((5, 9), dtype=torch.int32)[:, :7], 9),
    (torch.zeros((6, 9), dtype=torch.int32)[::2, 2:5], 18), (torch.zeros(7, dtype=torch.int32).expand(1, 7), 7),
    (torch.zeros((4, 0), dtype=torch.int32), 1), (torch.zeros((3, 1), dtype=torch.int32), 1),
    (torch.zeros((7, 3), dtype=torch.int32).t()[:, :1], 1)])
def test_strides_of_a_table(calls, table, stride):
    _call(table)
    assert len(calls) == 1
    assert calls[0]["batch"] == table.shape[0] and calls[0]["max_pages"] == table.shape[1]
    assert calls[0]["table_stride"] == stride and calls[0]["block_table"] in (table.data_ptr(), None)
