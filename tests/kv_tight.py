"""Attention over hand-made block tables, against float64 with a bound of its
own for every element.

``Pool`` fills every token of a cache with rows of its own, so that a table may
name any pages in any order and a key taken from a wrong place shows.
"""

import numpy as np
import torch

from oracle import kv
from tests.kv_util import NP


def expect(q, k, v, scale, causal=True, window=0):
    """One sequence in float64: q [nq, Hq, D], k and v [len, Hkv, D] -> (out, lse, spread, total, score, seen).

    For every row: ``spread`` [.., D] the softmax average of |v|, ``total``
    [.., D] the sum of |v|, ``score`` the largest sum of |q k| * scale and
    ``seen`` the number of keys, all over the keys that the row sees.
    """
    nq, hq, d = q.shape
    n, hk = k.shape[0], k.shape[1]
    pos = n - nq + np.arange(nq)[:, None] if causal else np.full((nq, 1), n - 1)
    keys = np.arange(n)[None, :]
    see = keys <= pos
    if window:
        see = see & (keys > pos - window)
    out, spread, total = (np.zeros((nq, hq, d)) for _ in range(3))
    lse, score = np.full((nq, hq), -np.inf), np.zeros((nq, hq))
    has = see.any(1)
    for a in range(hq):
        h = a // (hq // hk)
        # (a key that no row sees may hold anything, NaN among it)
        kh, vh = (np.where(see.any(0)[:, None], x[:, h], 0.0) for x in (k, v))
        qa = q[:, a].astype(np.float64)
        x = np.where(see, scale * (qa @ kh.T), -np.inf)
        m = np.where(has, x.max(1, initial=-np.inf), 0.0)[:, None]
        p = np.exp(x - m)
        s = p.sum(1)
        w = p / np.where(has, s, 1.0)[:, None]
        out[:, a], spread[:, a], total[:, a] = w @ vh, w @ np.abs(vh), see @ np.abs(vh)
        lse[has, a] = m[has, 0] + np.log(s[has])
        if n:
            score[:, a] = abs(scale) * np.where(see, np.abs(qa) @ np.abs(kh).T, 0.0).max(1)
    return out, lse, spread, total, score, see.sum(1)


def bounds(want, lse, spread, total, score, seen, dim, dtype):
    """How far out and lse may lie from float64, element by element.

    A weight p_j of the softmax is rounded to 11 bits (2^-11), or, 2^-21 and
    more below the row's largest, to a multiple of 2^-31 of that; its score is
    an FP32 sum of dim products whose absolute values sum to at most `score`,
    with an exponential good to 2^-22: d, and e^d - 1 <= 2 d.  These enter the
    sum over v and the sum of weights, hence |v| + |out| each time.  The FP32
    sums add one product of 16 keys, or two weights, at a time: at most seen /
    8 steps of 2^-22, and the joins.  The output is rounded once.
    """
    d = (dim + 16) * 2.0 ** -23 * score + 2.0 ** -22
    steps = (seen / 8 + 64)[:, None] * 2.0 ** -22
    rel = (2.0 ** -11 + 2 * d + steps)[..., None]
    n = seen[:, None, None]
    least = 2.0 ** -25 if dtype is torch.float16 else 2.0 ** -133
    out = (spread + np.abs(want)) * rel + 2.0 ** -31 * (total + n * np.abs(want)) + NP[dtype] * np.abs(want) + least
    finite = np.where(np.isneginf(lse), 0.0, lse)
    return out, 2 * d + steps + 2.0 ** -11 + seen[:, None] * 2.0 ** -31 + 2.0 ** -20 * np.abs(finite)


def outside(got, want, bound):
    """Elements beyond their bound (NaN among them)."""
    return ~(np.abs(got - want) <= bound)


class Pool:
    """`pages` pages, every token a row of its own; `k` and `v` hold their float64 values by slot."""

    def __init__(self, binding, pages, heads, dim, fmt, page=16, seed=0, rows=None, pad=0):
        rng = self.rng = np.random.default_rng(seed)
        self.binding, self.heads, self.dim, self.fmt, self.page = binding, heads, dim, fmt, page
        self.g = (0.02 * (0.5 + rng.random((2, heads)))).astype(np.float32) if fmt == "nvfp4" else None
        nbytes = binding.load().petit_kv_page_bytes(page, heads, dim, binding.FORMATS[fmt])
        data = torch.full((pages, nbytes + pad), 0xEE, dtype=torch.uint8, device="cuda")
        self.cache = binding.KVCache(pages, page, heads, dim, fmt, data=data,
                                     scales=None if self.g is None else torch.from_numpy(self.g).cuda())
        n = pages * page
        x = rows or [rng.standard_normal((n, heads, dim)) for _ in range(2)]
        x = [torch.from_numpy(np.asarray(r, dtype=np.float32)).bfloat16() for r in x]
        self.cache.append(x[0].cuda(), x[1].cuda(), torch.arange(n, device="cuda"))
        self.k, self.v = (kv.values(*kv.quantize_rows(r.float().numpy(), fmt, g), fmt, g)
                          for r, g in zip(x, [None, None] if self.g is None else self.g))

    def queries(self, n, group, dtype, scale=1.0):
        q = self.rng.standard_normal((n, self.heads * group, self.dim)).astype(np.float32) * scale
        return torch.from_numpy(q).to(dtype).cuda()

    def run(self, q, nqs, table, lens, causal=True, window=0, scale=None, workspace=None):
        """Sequences of `table` (lists of pages; -1 fills them up) with nqs queries each, checked; (out, lse)."""
        width = max(len(t) for t in table)
        t = torch.tensor([list(r) + [-1] * (width - len(r)) for r in table], dtype=torch.int32, device="cuda")
        n = torch.tensor(lens, dtype=torch.int32, device="cuda")
        off = torch.tensor(np.cumsum([0] + list(nqs)), dtype=torch.int32, device="cuda")
        ws = workspace or self.binding.Workspace()
        lse = torch.full(q.shape[:2], 7.0, device="cuda")
        out = self.cache.attention(q, t, n, off, max(nqs), causal=causal, window=window, scale=scale, workspace=ws,
                                   lse=lse)
        assert ws.status() == 0
        self.check(q, nqs, table, lens, out, lse, causal, window, scale)
        return out, lse

    def check(self, q, nqs, table, lens, out, lse, causal=True, window=0, scale=None):
        scale = self.dim ** -0.5 if scale is None else float(np.float32(scale))
        qf, of, lf = (x.float().cpu().numpy().astype(np.float64) for x in (q, out, lse))
        at, known = 0, {}
        for b, (nq, n) in enumerate(zip(nqs, lens)):
            same = tuple(table[b]), n, qf[at:at + nq].tobytes()
            if same not in known:
                j = np.arange(n)
                slots = np.asarray(table[b])[j // self.page] * self.page + j % self.page
                here = slots >= 0
                slots = np.where(here, slots, 0)
                k, v = (np.where(here[:, None, None], x[slots], np.nan) for x in (self.k, self.v))
                r = expect(qf[at:at + nq], k, v, scale, causal, window)
                known[same] = r, *bounds(*r, self.dim, q.dtype)
            r, ob, lb = known[same]
            bad = outside(of[at:at + nq], r[0], ob)
            assert not bad.any(), (b, np.argwhere(bad)[:4], of[at:at + nq][bad][:4], r[0][bad][:4], ob[bad][:4])
            empty = np.isneginf(r[1])
            assert np.array_equal(np.isneginf(lf[at:at + nq]), empty)
            bad = outside(lf[at:at + nq][~empty], r[1][~empty], lb[~empty])
            assert not bad.any(), (b, lf[at:at + nq][~empty][bad][:4], r[1][~empty][bad][:4], lb[~empty][bad][:4])
            at += nq
