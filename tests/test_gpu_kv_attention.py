"""Attention over the 4-bit K/V cache against the float64 oracle, row by row,
with error bounds derived from the formats (kv_util.Case.check)."""

import numpy as np
import pytest
import torch

from tests.kv_util import Case

pytestmark = pytest.mark.gpu


def _run(case, cuda_lib, nqs, group, dtype, causal=True, window=0, scale=None, qscale=1.0, offsets=True):
    q, off = case.queries(nqs, group, dtype, qscale)
    ws = cuda_lib.Workspace()
    lse = torch.full((q.shape[0], q.shape[1]), 7.0, device="cuda")
    out = torch.full(q.shape, float("nan"), dtype=dtype, device="cuda")
    r = case.cache.attention(q, case.d_table, case.d_lens, off if offsets else None, max(nqs), scale=scale,
                             causal=causal, window=window, workspace=ws, out=out, lse=lse)
    assert r is out and ws.status() == 0
    case.check(q, nqs, out, lse, causal, window, scale)
    return q, off, out, lse, ws


FORMATS = [("nvfp4", 128), ("mxfp4", 128), ("nvfp4", 64), ("mxfp4", 64)]


@pytest.mark.parametrize("fmt,dim", FORMATS)
@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
def test_single_tokens_ragged_lengths(cuda_lib, fmt, dim, page):
    lens = [1, 2, 15, 16, 17, 31, 32, 33, 0, 63, 64, 65, 127, 200, 500]
    case = Case(cuda_lib, lens, 2, dim, fmt, page, seed=page)
    _run(case, cuda_lib, [1] * len(lens), 8, torch.bfloat16, offsets=page > 32)


@pytest.mark.parametrize("fmt,dim", FORMATS)
@pytest.mark.parametrize("heads,group", [(1, 1), (1, 2), (3, 3), (2, 5), (1, 7), (8, 8), (1, 9), (2, 16), (1, 24), (1, 40)])
def test_head_layouts(cuda_lib, fmt, dim, heads, group):
    case = Case(cuda_lib, [70, 5], heads, dim, fmt, 16, seed=group)
    _run(case, cuda_lib, [1, 1], group, torch.float16)


@pytest.mark.parametrize("fmt,dim", FORMATS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("nqs,lens,group", [
    ([1, 2, 3, 4, 5], [10, 100, 3, 40, 333], 8), ([6, 0, 1], [50, 20, 1], 3), ([17, 40], [17, 130], 4),
    ([130], [257], 1), ([33, 200, 1], [33, 700, 90], 8), ([300], [300], 2)])
def test_several_query_tokens(cuda_lib, fmt, dim, dtype, nqs, lens, group):
    case = Case(cuda_lib, lens, 2, dim, fmt, 32, seed=len(lens))
    _run(case, cuda_lib, nqs, group, dtype)


@pytest.mark.parametrize("fmt,dim", FORMATS)
@pytest.mark.parametrize("nq", [1, 3, 70])
@pytest.mark.parametrize("causal,window", [(False, 0), (True, 1), (True, 33), (True, 100), (True, 1 << 40)])
def test_masks(cuda_lib, fmt, dim, nq, causal, window):
    lens = [400, nq, 90]
    case = Case(cuda_lib, lens, 1, dim, fmt, 16, seed=nq)
    _run(case, cuda_lib, [nq] * 3, 4, torch.bfloat16, causal, window, offsets=False)


@pytest.mark.parametrize("fmt,dim", FORMATS)
@pytest.mark.parametrize("nq,group", [(1, 8), (4, 8), (60, 4), (200, 1)])
def test_rows_that_see_nothing(cuda_lib, fmt, dim, nq, group):
    """No cached token, and more queries than tokens: zeros and -inf, beside rows that see something."""
    lens = [0, 1, max(1, nq - 3), nq + 30]
    case = Case(cuda_lib, lens, 2, dim, fmt, 16, seed=3)
    _, _, out, lse, _ = _run(case, cuda_lib, [nq] * 4, group, torch.bfloat16)
    assert (out[:nq] == 0).all() and torch.isneginf(lse[:nq]).all()


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("nq", [1, 50])
@pytest.mark.parametrize("fill", [0x00, 0x7F, 0xFF])
def test_what_lies_past_a_sequence_is_not_seen(cuda_lib, fmt, nq, fill):
    """The rest of the last page holds NaN scales, largest scales or zeros: results are the same bits."""
    lens = [5 + nq, 47 + nq, 161 + nq]
    outs = []
    for f in (fill, 0x11):
        case = Case(cuda_lib, lens, 2, 128, fmt, 64, seed=9, fill=f)
        outs.append(_run(case, cuda_lib, [nq] * 3, 8, torch.bfloat16)[2])
    assert torch.equal(*outs)


@pytest.mark.parametrize("nq", [1, 100])
def test_split_long_context(cuda_lib, nq):
    """A long axis cut over many thread blocks and joined; equal bits on every run, and the workspace is left as it was."""
    case = Case(cuda_lib, [6000 + nq, 3, 1000 + nq], 1, 128, "nvfp4", 64, seed=4)
    q, off, out, lse, ws = _run(case, cuda_lib, [nq, 1, nq], 8, torch.bfloat16)
    for _ in range(3):
        again = case.cache.attention(q, case.d_table, case.d_lens, off, nq, workspace=ws)
        assert torch.equal(again, out)
    assert not ws.buf[:4352].any()


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("nq", [1, 64])
def test_scales_and_magnitudes(cuda_lib, fmt, nq):
    """Sharp softmax, negative scale, zero scale, tiny and large queries."""
    case = Case(cuda_lib, [150 + nq], 2, 128, fmt, 32, seed=6)
    for scale, qs in ((1.0, 1.0), (-0.3, 1.0), (0.0, 1.0), (0.05, 1e-6), (1e-30, 1e30), (0.01, 30.0)):
        _run(case, cuda_lib, [nq], 4, torch.bfloat16, scale=scale, qscale=qs)
    _run(case, cuda_lib, [nq], 4, torch.float16, scale=1000.0, qscale=1e-4)


@pytest.mark.parametrize("nq", [1, 40])
def test_mxfp4_scales_of_any_size(cuda_lib, nq):
    """Blocks whose scales lie 2^30 apart, within a token and between tokens."""
    n, heads, dim = 120 + nq, 2, 128
    rng = np.random.default_rng(8)
    k = rng.standard_normal((n, heads, dim)).astype(np.float32)
    v = rng.standard_normal((n, heads, dim)).astype(np.float32)
    k[..., 32:64] *= 2.0 ** -28
    k[::3, :, 96:] *= 2.0 ** -20
    v[::2] *= 2.0 ** 15
    v[1::2, :, :32] *= 2.0 ** -15
    case = Case(cuda_lib, [n], heads, dim, "mxfp4", 64, seed=2)
    slots = torch.from_numpy(case.table[0][np.arange(n) // 64].astype(np.int64) * 64 + np.arange(n) % 64).cuda()
    case.cache.append(torch.from_numpy(k).bfloat16().cuda(), torch.from_numpy(v).bfloat16().cuda(), slots)
    from oracle import kv
    for x, dst in ((k, case.k), (v, case.v)):
        dst[0] = kv.values(*kv.quantize_rows(torch.from_numpy(x).bfloat16().float().numpy(), "mxfp4"), "mxfp4")
    _run(case, cuda_lib, [nq], 4, torch.bfloat16)


@pytest.mark.parametrize("nq", [1, 48])
def test_not_finite_queries_stay_in_their_rows(cuda_lib, nq):
    case = Case(cuda_lib, [100 + nq], 2, 128, "nvfp4", 64, seed=6)
    q, off = case.queries([nq], 8, torch.bfloat16)
    q[0, 3, 5] = float("nan")
    q[0, 9, 0] = float("inf")
    out = case.cache.attention(q, case.d_table, case.d_lens, off, nq)
    bad = torch.zeros(q.shape[:2], dtype=torch.bool, device="cuda")
    bad[0, 3] = bad[0, 9] = True
    assert torch.isnan(out[bad]).all()
    clean = q.clone()
    clean[0, 3] = clean[0, 9] = 0
    want = case.cache.attention(clean, case.d_table, case.d_lens, off, nq)
    assert torch.equal(out[~bad], want[~bad])


@pytest.mark.parametrize("nq", [1, 64])
def test_strided_queries_and_outputs(cuda_lib, nq):
    """q as a view of a fused projection; the output inside a wider buffer whose rest stays."""
    case = Case(cuda_lib, [64 + nq, nq + 7], 2, 64, "nvfp4", 16, seed=1, stride_extra=48)
    heads = 8
    q, off = case.queries([nq, nq], 4, torch.bfloat16)
    wide = torch.randn(2 * nq, heads + 4, 64, device="cuda").to(torch.bfloat16)
    wide[:, :heads] = q
    buf = torch.full((heads, 2 * nq, 72), 5.0, dtype=torch.bfloat16, device="cuda")
    out = buf[:, :, :64].transpose(0, 1)
    case.cache.attention(wide[:, :heads], case.d_table, case.d_lens, off, nq, out=out)
    case.check(q, [nq, nq], out)
    assert (buf[:, :, 64:] == 5).all()


def test_pages_lengths_and_offsets_outside_their_range(cuda_lib):
    """Recorded, and nothing outside is read or written: other sequences keep
    their results (not their bits: how the work is cut depends on the whole batch)."""
    for nq in (1, 50):
        case = Case(cuda_lib, [100, 100, 100, 100], 2, 128, "nvfp4", 16, seed=5)
        nqs = [nq] * 4
        q, off = case.queries(nqs, 4, torch.bfloat16)
        ws = cuda_lib.Workspace()
        case.check(q, nqs, case.cache.attention(q, case.d_table, case.d_lens, off, nq, workspace=ws))
        assert ws.status() == 0
        for change in ("page", "negative page", "length", "negative length"):
            table, lens = case.d_table.clone(), case.d_lens.clone()
            if change == "page":
                table[1, 2] = case.cache.num_pages
            elif change == "negative page":
                table[1, 0] = -1
            elif change == "length":
                lens[1] = 1 << 30
            else:
                lens[1] = -5
            out = case.cache.attention(q, table, lens, off, nq, workspace=ws)
            assert ws.status() == 8, change
            case.check(q, nqs, out, only=[0, 2, 3])
            # (a cut length reaches tokens nobody wrote: what they hold is the caller's)
            assert change == "length" or torch.isfinite(out).all()
        # offsets: sequence 1 has impossible ones and is left out
        bad = torch.tensor([0, nq, 10 ** 9, 3 * nq, 4 * nq], dtype=torch.int32, device="cuda")
        out = torch.full_like(q, 3.0)
        case.cache.attention(q, case.d_table, case.d_lens, bad, nq, workspace=ws, out=out)
        assert ws.status() == 8
        case.check(q, nqs, out, only=[0, 3])
        assert (out[nq:3 * nq] == 3).all()


def test_left_out_page_equals_a_shorter_context(cuda_lib):
    case = Case(cuda_lib, [64], 1, 128, "nvfp4", 16, seed=5)
    q, _ = case.queries([1], 8, torch.bfloat16)
    table = case.d_table.clone()
    table[0, 3] = -1
    ws = cuda_lib.Workspace()
    out = case.cache.attention(q, table, case.d_lens, workspace=ws, causal=False)
    assert ws.status() == 8
    case.lens, case.k, case.v = [48], [case.k[0][:48]], [case.v[0][:48]]
    case.check(q, [1], out, causal=False)


@pytest.mark.parametrize("nq", [1, 3, 64])
def test_graph_follows_changed_lengths(cuda_lib, nq):
    case = Case(cuda_lib, [300, 200], 2, 128, "nvfp4", 32, seed=7)
    q, off = case.queries([nq, nq], 8, torch.bfloat16)
    ws = cuda_lib.Workspace()
    out = torch.empty_like(q)
    lens = case.d_lens.clone()
    case.cache.attention(q, case.d_table, lens, off, nq, workspace=ws, out=out)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        case.cache.attention(q, case.d_table, lens, off, nq, workspace=ws, out=out)
    for n in ([300, 200], [77, 200], [nq, 123]):
        lens.copy_(torch.tensor(n, dtype=torch.int32))
        g.replay()
        want = case.cache.attention(q, case.d_table, torch.tensor(n, dtype=torch.int32, device="cuda"), off, nq)
        assert torch.equal(out, want)
    assert ws.status() == 0


def test_many_sequences(cuda_lib):
    """More sequences than a thread block has threads, empty ones and ones without queries among them."""
    rng = np.random.default_rng(0)
    lens = [int(x) for x in rng.integers(0, 40, 700)]
    nqs = [int(x) for x in rng.integers(0, 3, 700)]
    case = Case(cuda_lib, lens, 1, 64, "mxfp4", 16, seed=11)
    _run(case, cuda_lib, nqs, 2, torch.float16)


def test_max_q_may_be_too_small(cuda_lib):
    case = Case(cuda_lib, [90, 300], 1, 128, "nvfp4", 16, seed=12)
    q, off = case.queries([5, 150], 2, torch.bfloat16)
    out = case.cache.attention(q, case.d_table, case.d_lens, off, 1)
    case.check(q, [5, 150], out)


def test_workspace_shared_with_gemms(cuda_lib):
    from fp4_weight_only_gb300 import synth
    case = Case(cuda_lib, [900], 2, 128, "nvfp4", 64, seed=13)
    q, off = case.queries([1], 8, torch.bfloat16)
    ws = cuda_lib.Workspace()
    w = cuda_lib.FP4Weight(synth.weights(1024, 2048, seed=1, device="cuda"), "nvfp4")
    a = synth.activations(1, 2048, seed=2, device="cuda")
    want = w(a), case.cache.attention(q, case.d_table, case.d_lens)
    for _ in range(4):
        c = w(a, workspace=ws)
        o = case.cache.attention(q, case.d_table, case.d_lens, workspace=ws)
        assert torch.equal(c, want[0]) and torch.equal(o, want[1])
    assert ws.status() == 0


def test_empty_calls_and_refusals(cuda_lib):
    case = Case(cuda_lib, [20, 30], 2, 64, "nvfp4", 16, seed=1)
    q, off = case.queries([2, 3], 3, torch.bfloat16)
    at = case.cache.attention
    assert at(q[:0], case.d_table, case.d_lens, off.clone().zero_(), 0).shape == (0, 6, 64)
    assert at(q[:0], case.d_table[:0], case.d_lens[:0]).shape == (0, 6, 64)
    ok = dict(q_offsets=off, max_q=3)
    for bad, match in ((dict(q=q.float()), "q:"), (dict(q=q[:, :5]), "heads"), (dict(q=q[..., :32]), "q:"),
                       (dict(seq_lens=case.d_lens.long()), "seq_lens"), (dict(seq_lens=case.d_lens[:1]), "seq_lens"),
                       (dict(block_table=case.d_table.long()), "block_table"), (dict(block_table=case.d_table[0]), "block_table"),
                       (dict(q_offsets=off[:2]), "q_offsets"), (dict(out=q[:1]), "out"), (dict(out=q.half()), "out"),
                       (dict(lse=torch.zeros(5, device="cuda")), "lse")):
        args = dict(q=q, block_table=case.d_table, seq_lens=case.d_lens, **ok)
        args.update(bad)
        with pytest.raises(ValueError, match=match):
            at(**args)
    for bad, status in ((dict(window=-1), 1), (dict(window=3, causal=False), 1), (dict(scale=float("nan")), 1),
                        (dict(q_offsets=None), 1)):
        args = dict(q=q, block_table=case.d_table, seq_lens=case.d_lens, **ok)
        args.update(bad)
        with pytest.raises(cuda_lib.PetitError) as e:
            at(**args)
        assert e.value.status == status
