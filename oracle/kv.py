"""The 4-bit K/V cache and attention over it, in float64.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__.py``).

The cache's rows are quantised by ``quantize`` (binary32 steps, one global
scale per head); MXFP4 scale codes stop at 252, so that 6 * 2^125 stays a
finite BF16 number.  Storage order: per page, per head, groups of 16 tokens,
each ``K codes | K scales | V codes | V scales``.
"""

import numpy as np

from . import formats, gemm, quantize

GROUP = 16
MXFP4_MAX_CODE = 252


def quantize_rows(x, fmt, g=None):
    """Rows x [tokens, heads, D] -> codes [.., D], scale bytes [.., D/B]; g: a scale per head (NVFP4)."""
    x = np.asarray(x, dtype=np.float32)
    codes, scales = [], []
    for h in range(x.shape[1]):
        if fmt == "nvfp4":
            c, s = quantize.nvfp4_quantize(x[:, h], 1.0 if g is None else g[h])
        else:
            c, s = quantize.mxfp4_quantize(x[:, h])
            if s.max(initial=0) > MXFP4_MAX_CODE:   # a capped scale, and the codes it gives
                s = np.minimum(s, MXFP4_MAX_CODE).astype(np.uint8)
                d = np.exp2(s.astype(np.float64) - 127)
                y = x[:, h].astype(np.float64).reshape(x.shape[0], -1, quantize.MXFP4_GROUP) / d[..., None]
                c = formats.e2m1_encode(y.astype(np.float32)).reshape(c.shape)
        codes.append(c)
        scales.append(s)
    return np.stack(codes, 1), np.stack(scales, 1)


def values(codes, scales, fmt, g=None):
    """float64 values of codes [tokens, heads, D]."""
    t, h, d = codes.shape
    v = gemm.dequantize(codes.reshape(t * h, d), scales.reshape(t * h, scales.shape[2]), fmt).astype(np.float64)
    v = v.reshape(t, h, d)
    return v if g is None else v * np.asarray(g, dtype=np.float64)[None, :, None]


def store(data, slots, page_size, k, v, fmt):
    """Put (codes, scales) pairs k and v into the uint8 cache data [pages, page bytes] (in place)."""
    (kc, ks), (vc, vs) = k, v
    heads = kc.shape[1]
    view = data.reshape(data.shape[0], heads, page_size // GROUP, -1)
    for i, slot in enumerate(slots):
        if slot < 0 or slot >= data.shape[0] * page_size:
            continue
        page, tok = divmod(int(slot), page_size)
        for h in range(heads):
            at = 0
            for row in (quantize.pack_codes(kc[i, h][None])[0], ks[i, h], quantize.pack_codes(vc[i, h][None])[0],
                        vs[i, h]):
                n = row.size
                start = at + (tok % GROUP) * n
                view[page, h, tok // GROUP, start:start + n] = row
                at += GROUP * n


def attention(q, k, v, scale, causal=True, window=0):
    """One sequence: q [nq, Hq, D], k and v [len, Hkv, D] -> (out, lse, spread, score).

    ``spread`` is the softmax average of |v| (what rounding of the weights is
    relative to) and ``score`` the largest sum of |q k| * scale of a row (what
    rounding inside a score is relative to); both bound errors in the tests.
    """
    nq, hq, d = q.shape
    n, hk = k.shape[0], k.shape[1]
    out = np.zeros((nq, hq, d))
    spread = np.zeros((nq, hq, d))
    lse = np.full((nq, hq), -np.inf)
    score = np.zeros((nq, hq))
    pos = n - nq + np.arange(nq)[:, None] if causal else np.full((nq, 1), n - 1)
    keys = np.arange(n)[None, :]
    seen = keys <= pos
    if window:
        seen = seen & (keys > pos - window)
    for a in range(hq):
        h = a // (hq // hk)
        x = scale * (q[:, a].astype(np.float64) @ k[:, h].T)
        x = np.where(seen, x, -np.inf)
        m = np.where(seen.any(1), x.max(1, initial=-np.inf), 0.0)
        p = np.where(seen, np.exp(np.where(seen, x - m[:, None], 0.0)), 0.0)
        s = p.sum(1)
        has = s > 0
        div = np.where(has, s, 1.0)[:, None]
        out[:, a] = p @ v[:, h] / div
        spread[:, a] = p @ np.abs(v[:, h]) / div
        lse[has, a] = m[has] + np.log(s[has])
        if n:
            score[:, a] = abs(scale) * (np.abs(q[:, a].astype(np.float64)) @ np.abs(k[:, h].T)).max(1)
    return out, lse, spread, score
