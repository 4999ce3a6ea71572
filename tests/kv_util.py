"""Building caches for the K/V tests: the oracle quantises and stores, the
device gets the bytes."""

import numpy as np
import torch

from oracle import kv

NP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}   # unit roundoff of the outputs


def rows(rng, n, heads, dim, dtype):
    """Rows representable in `dtype`: unit normals with strong channels, a zero block, a huge and a tiny one."""
    x = rng.standard_normal((n, heads, dim)).astype(np.float32)
    x[..., ::29] *= 6.0
    if n > 2:
        x[1, 0, :32] = 0.0
        x[2, 0, 32:64] *= 1000.0
        x[0, -1, :32] *= 1e-5
    return torch.from_numpy(x).to(dtype)


class Case:
    """Sequences of cached tokens on shuffled pages; everything no sequence owns is filled with `fill`."""

    def __init__(self, binding, lens, heads, dim, fmt, page=16, seed=0, fill=0xFF, pad_pages=1, stride_extra=0):
        rng = np.random.default_rng(seed)
        self.binding, self.lens, self.heads, self.dim, self.fmt, self.page = binding, lens, heads, dim, fmt, page
        self.g = None
        if fmt == "nvfp4":
            self.g = (0.02 * (0.5 + rng.random((2, heads)))).astype(np.float32)
        need = [-(-n // page) for n in lens]
        pages = sum(need) + pad_pages
        nbytes = binding.load().petit_kv_page_bytes(page, heads, dim, binding.FORMATS[fmt])
        data = np.full((pages, nbytes), fill, dtype=np.uint8)
        order = rng.permutation(pages)
        self.table = np.full((len(lens), max(max(need), 1)), -7, dtype=np.int32)   # unused entries are no pages
        self.k, self.v = [], []
        at = 0
        for b, n in enumerate(lens):
            self.table[b, :need[b]] = order[at:at + need[b]]
            at += need[b]
            x = [rows(rng, n, heads, dim, torch.bfloat16).float().numpy() for _ in range(2)]
            pair = [kv.quantize_rows(x[i], fmt, None if self.g is None else self.g[i]) for i in range(2)]
            slots = self.table[b][np.arange(n) // page].astype(np.int64) * page + np.arange(n) % page
            kv.store(data, slots, page, pair[0], pair[1], fmt)
            for i, dst in enumerate((self.k, self.v)):
                dst.append(kv.values(*pair[i], fmt, None if self.g is None else self.g[i]))
        full = torch.full((pages, nbytes + stride_extra), 0xEE, dtype=torch.uint8, device="cuda")
        full[:, :nbytes] = torch.from_numpy(data).cuda()
        scales = None if self.g is None else torch.from_numpy(self.g).cuda()
        self.cache = binding.KVCache(pages, page, heads, dim, fmt, scales=scales, data=full)
        self.d_table = torch.from_numpy(self.table).cuda()
        self.d_lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
        self.rng = rng

    def queries(self, nqs, group, dtype, scale=1.0):
        q = self.rng.standard_normal((sum(nqs), self.heads * group, self.dim)).astype(np.float32) * scale
        off = torch.tensor([0] + list(np.cumsum(nqs)), dtype=torch.int32, device="cuda")
        return torch.from_numpy(q).to(dtype).cuda(), off

    def check(self, q, nqs, out, lse=None, causal=True, window=0, scale=None, only=None):
        """Every row (of the sequences `only`) against the oracle, element by element.

        Error bound: with A the softmax average of |v|, each p_j is rounded to
        11 bits and carries its score's error d,
        e^d - 1 <= 2 d; FP32 sums over the keys add len * 2^-23; p below FP16's
        normal range have an absolute error of 2^-25 of the largest; the output
        is rounded once.  A score is an FP32 sum of dim products whose absolute
        values sum to at most `score`, scaled once (and ex2 has 2^-22).
        """
        scale = self.dim ** -0.5 if scale is None else scale
        u = NP[q.dtype]
        at = 0
        qf, of = q.float().cpu().numpy().astype(np.float64), out.float().cpu().numpy().astype(np.float64)
        for b, (nq, n) in enumerate(zip(nqs, self.lens)):
            if only is not None and b not in only:
                at += nq
                continue
            want, wl, spread, score = kv.attention(qf[at:at + nq], self.k[b], self.v[b], scale, causal, window)
            got = of[at:at + nq]
            assert np.isfinite(got).all(), f"sequence {b}"
            d = ((self.dim + 16) * 2.0 ** -23 * score + 2.0 ** -22)[..., None]
            pu = 2.0 ** -11
            vmax = np.abs(self.v[b]).max(initial=0.0)
            bound = spread * (pu + 2 * d + (n + 64) * 2.0 ** -23) + u * np.abs(want) + n * 2.0 ** -25 * vmax + 1e-7
            bad = np.abs(got - want) > bound
            assert not bad.any(), (b, np.argwhere(bad)[:4], np.abs(got - want)[bad][:4], bound[bad][:4])
            if lse is not None:
                gl = lse[at:at + nq].cpu().numpy().astype(np.float64)
                empty = np.isneginf(wl)
                assert np.array_equal(np.isneginf(gl), empty)
                tol = d[..., 0] + (n + 64) * 2.0 ** -23 + 2.0 ** -20 * np.abs(np.where(empty, 0, wl)) + pu
                assert (np.abs(gl[~empty] - wl[~empty]) <= tol[~empty]).all()
            at += nq
