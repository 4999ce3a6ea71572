"""The operators of the 4-bit K/V cache, as cases to time and compare.

A paged cache holds K and V in E2M1 codes with block scales (NVFP4: an E4M3
scale per 16 elements and an FP32 scale per head; MXFP4: an E8M0 scale per
32).  A head's part of a page is a run of 16-token groups, each
``K codes | K scales | V codes | V scales``; a token's D elements are D/2
bytes, element 2j in the low nibble of byte j.

Three operators: writing rows into the cache (``write_read`` cases, which read
the rows back, so that the outputs are what the cache then holds), reading rows
(``read``), and attention over it (``attend``).  ``run`` computes them in plain
torch operations in 32 bits, or, where ``own`` is true, through the package.
"""

import math
import random

import numpy as np
import torch

own = False

GROUP = 16                                   # tokens per storage group
BLOCK = {"nvfp4": 16, "mxfp4": 32}           # elements per scale
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------- cases
def _case(kind, name=None, **k):
    c = {"kind": kind, "heads": 8, "dim": 128, "fmt": "nvfp4", "dtype": "bf16", "page": 64}
    c.update(k)
    if name:
        c["name"] = name
    return c


def _attend(name=None, **k):
    c = {"batch": 1, "group": 8, "len_lo": 1, "len_hi": 1, "q_lo": 1, "q_hi": 1, "window": 0, "lengths": 1}
    c.update(k)
    return _case("attend", name, **c)


def listed():
    return [
        # one user's next token: the smallest write, all latency
        _case("write_read", "write_read_one", tokens=1),
        # the next token of a few hundred users, small heads, small pages
        _case("write_read", "write_read_batch", tokens=333, heads=4, dim=64, fmt="mxfp4", dtype="fp16", page=16),
        # a prompt's rows out of a fused QKV product (a view of its output)
        _case("write_read", "write_read_prompt", tokens=8192),
        # one turn of a conversation read back
        _case("read", "read_turn", tokens=1501, fmt="mxfp4", page=32),
        # a whole long context read back
        _case("read", "read_context", tokens=131071),
        # one user, a short context: latency
        _attend("decode_one", len_lo=1000, len_hi=1000),
        # one user, a long context: few rows, one long axis
        _attend("decode_long", len_lo=131071, len_hi=131071),
        # a serving batch of ragged contexts, the heads of the benchmark's model
        _attend("decode_batch", batch=64, len_lo=1, len_hi=8192),
        # a large serving batch, other format, type, group and page
        _attend("decode_wide", batch=160, len_lo=200, len_hi=16000, fmt="mxfp4", dtype="fp16", group=4, page=16),
        # checking a few drafted tokens a sequence
        _attend("verify", batch=24, len_lo=40, len_hi=6000, q_lo=1, q_hi=6, dim=64, page=32),
        # a ragged batch of prompt pieces with a sliding window, small heads
        _attend("prompt_ragged", batch=5, len_lo=700, len_hi=5000, q_lo=3, q_hi=1100, window=1024, dim=64,
                fmt="mxfp4", dtype="fp16", group=4, page=32),
        # a piece of a long prompt behind what is cached of it: the largest
        _attend("prompt_chunk", len_lo=16384, len_hi=16384, q_lo=4096, q_hi=4096),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    common = {"dim": rng.choice((64, 128)), "fmt": rng.choice(("nvfp4", "mxfp4")), "dtype": rng.choice(("bf16", "fp16")),
              "page": rng.choice((16, 32, 64, 128)), "heads": rng.choice((1, 2, 4, 8))}
    kind = rng.choice(("write_read", "read", "decode", "decode", "verify", "prompt", "prompt"))
    if kind == "write_read":
        return _case(kind, tokens=_log_int(rng, 1, 8192), **common)
    if kind == "read":
        return _case(kind, tokens=_log_int(rng, 1, 131071), **common)
    common |= {"group": rng.choice((1, 2, 3, 4, 5, 7, 8, 16)), "lengths": rng.randrange(1 << 20)}
    if kind == "decode":
        batch = _log_int(rng, 1, 160)
        hi = _log_int(rng, 16, min(131071, 1300000 // batch))
        return _attend(batch=batch, len_lo=max(1, hi // rng.choice((1, 4, 100))), len_hi=hi,
                       window=rng.choice((0, 0, 0, max(1, hi // 3))), **common)
    if kind == "verify":
        batch, hi = _log_int(rng, 1, 32), _log_int(rng, 16, 8000)
        return _attend(batch=batch, len_lo=min(hi, 16), len_hi=hi, q_lo=1, q_hi=rng.randint(2, 12), **common)
    batch, q = rng.choice((1, 1, 2, 3, 5)), _log_int(rng, 20, 2000)
    hi = _log_int(rng, q, 8000)
    return _attend(batch=batch, len_lo=max(1, hi // rng.choice((1, 3))), len_hi=hi, q_lo=max(1, q // rng.choice((1, 10))), q_hi=q,
                   window=rng.choice((0, 0, rng.randint(64, 2000))), **common)


def _lengths(case):
    """(query tokens, context length) of each sequence; a context holds its own queries."""
    r = random.Random(case["lengths"])
    nq = [r.randint(case["q_lo"], case["q_hi"]) for _ in range(case["batch"])]
    ln = [max(q, r.randint(case["len_lo"], case["len_hi"])) for q in nq]
    ln[0] = max(nq[0], case["len_hi"])
    return nq, ln


def _token_bytes(case):
    return case["heads"] * (case["dim"] + 2 * case["dim"] // BLOCK[case["fmt"]])


def work(case):
    h, d = case["heads"], case["dim"]
    if case["kind"] == "read":
        return {"bytes": case["tokens"] * (_token_bytes(case) + 4 * h * d + 8), "flops": case["tokens"] * 4 * h * d}
    if case["kind"] == "write_read":
        # rows in, codes and scales out and in again, rows out
        return {"bytes": case["tokens"] * (2 * _token_bytes(case) + 8 * h * d + 8), "flops": case["tokens"] * 16 * h * d}
    w, pairs, keys = case["window"], 0, 0
    nq, ln = _lengths(case)
    for q, n in zip(nq, ln):
        keys += min(n, q - 1 + w) if w else n
        seen = np.arange(n - q + 1, n + 1, dtype=np.int64)
        pairs += int((np.minimum(seen, w) if w else seen).sum())
    hq = h * case["group"]
    return {"bytes": keys * _token_bytes(case) + 4 * sum(nq) * hq * d, "flops": 4 * d * hq * pairs}


# ------------------------------------------------------------------ inputs
def _power(e):
    """2^e in FP32, exactly, for int32 e in -126..127."""
    return ((e + 127) << 23).view(torch.float32)


def _encode(x, g, fmt):
    """Codes 0..15 and scale bytes of rows x [..., D] (FP32); g divides NVFP4 scales (broadcast over blocks)."""
    b = x.unflatten(-1, (-1, BLOCK[fmt]))
    amax = b.abs().amax(-1).clamp_min(1e-8)
    if fmt == "nvfp4":
        s = (amax / (6.0 * g)).clamp_max(448.0).to(torch.float8_e4m3fn).view(torch.uint8).clamp_min(1)
        y = b / (s.view(torch.float8_e4m3fn).float() * g).unsqueeze(-1)
    else:
        m, e = torch.frexp(amax / 6.0)
        e = (e - (m == 0.5).int()).clamp(-127, 125)
        s = (e + 127).to(torch.uint8)
        y = b * _power(-e).unsqueeze(-1)
    a = y.abs()
    c = (a > 0.25).byte() + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0)
    c = c + 8 * ((y < 0) & (c > 0)).byte()
    return c.flatten(-2), s


def _pack(c):
    return c[..., 0::2] | (c[..., 1::2] << 4)


def _views(case, data):
    """K codes, K scales, V codes, V scales as views [pages, heads, groups, 16, bytes] of the cache."""
    d = case["dim"]
    g = data.view(data.shape[0], case["heads"], case["page"] // GROUP, -1)
    out, at = [], 0
    for n in (d // 2, d // BLOCK[case["fmt"]]) * 2:
        out.append(g[..., at:at + GROUP * n].unflatten(-1, (GROUP, n)))
        at += GROUP * n
    return out


def _rows(gen, n, h, d):
    """Rows of K or V: unit normals with a few strong channels, as models have them."""
    x = torch.randn((n, h, d), generator=gen, device="cuda", dtype=torch.float32)
    x[..., ::37] *= 4.0
    return x


def _fill(case, data, gen):
    """Every token of the cache gets rows of its own, a run of pages at a time."""
    kc, ks, vc, vs = _views(case, data)
    step = max(1, (1 << 26) // (case["heads"] * case["dim"] * case["page"]))
    for at in range(0, data.shape[0], step):
        n = min(step, data.shape[0] - at)
        for codes, scales, g in ((kc, ks, 0.02), (vc, vs, 0.01)):
            x = _rows(gen, n * case["page"], case["heads"], case["dim"])
            c, s = _encode(x, g if case["fmt"] == "nvfp4" else 1.0, case["fmt"])
            shape = (n, case["page"] // GROUP, GROUP, case["heads"], -1)
            codes[at:at + n] = _pack(c).view(shape).permute(0, 3, 1, 2, 4)
            scales[at:at + n] = s.view(shape).permute(0, 3, 1, 2, 4)


def _cache(case, pages, gen, fill=True):
    data = torch.zeros((pages, case["page"] * _token_bytes(case)), dtype=torch.uint8, device="cuda")
    if fill:
        _fill(case, data, gen)
    scales = None
    if case["fmt"] == "nvfp4":   # what calibration gives: a scale per head, for K and for V
        scales = 0.02 * (0.75 + 0.5 * torch.rand((2, case["heads"]), generator=gen, device="cuda"))
        scales[1] *= 0.5
    return data, scales


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    h, d, dt = case["heads"], case["dim"], DTYPES[case["dtype"]]
    state = {"case": case, "handle": {}}
    if case["kind"] != "attend":
        n = case["tokens"]
        pages = -(-n // case["page"]) + 3
        state["data"], state["scales"] = _cache(case, pages, gen, fill=case["kind"] == "read")
        slots = torch.randperm(pages, generator=gen, device="cuda")[:, None] * case["page"]
        slots = (slots + torch.arange(case["page"], device="cuda")).flatten()
        state["slots"] = slots[3:3 + n].contiguous()
        if case["kind"] == "write_read":
            # q, k and v side by side, as the fused projection leaves them (8 query heads a head)
            qkv = torch.empty((n, 10 * h * d), dtype=dt, device="cuda")
            state["k"] = qkv[:, 8 * h * d:9 * h * d].view(n, h, d)
            state["v"] = qkv[:, 9 * h * d:].view(n, h, d)
            state["k"].copy_(_rows(gen, n, h, d))
            state["v"].copy_(_rows(gen, n, h, d))
        return state
    nq, ln = _lengths(case)
    most = -(-max(ln) // case["page"])
    need = [-(-n // case["page"]) for n in ln]
    state["data"], state["scales"] = _cache(case, sum(need) + 2, gen)
    order = torch.randperm(sum(need) + 2, generator=gen, device="cuda").int()
    table = torch.zeros((len(ln), most), dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    state["table"] = table
    state["lens"] = torch.tensor(ln, dtype=torch.int32, device="cuda")
    state["offsets"] = torch.tensor([0] + list(np.cumsum(nq)), dtype=torch.int32, device="cuda")
    state["max_q"], state["max_len"] = max(nq), max(ln)
    q = torch.randn((sum(nq), h * case["group"], d), generator=gen, device="cuda")
    q *= 0.5 + 1.5 * torch.rand((1, h * case["group"], 1), generator=gen, device="cuda")
    state["q"] = q.to(dt)
    return state


# --------------------------------------------------------------- plain form
def _decode(codes, scales, g, fmt):
    """FP32 values of packed codes [..., D/2] with scale bytes [..., D/BLOCK]; g broadcasts over the row."""
    level = torch.tensor(LEVELS + tuple(-v for v in LEVELS), dtype=torch.float32, device=codes.device)
    v = torch.stack((level[(codes & 15).int()], level[(codes >> 4).int()]), -1).flatten(-2)
    if fmt == "nvfp4":
        s = scales.view(torch.float8_e4m3fn).float()
    else:
        s = _power(scales.int() - 127)
    v = (v.unflatten(-1, (-1, BLOCK[fmt])) * s.unsqueeze(-1)).flatten(-2)
    return v if g is None else v * g


def _gather(state, slots):
    """K and V [*slots.shape, heads, D] of the cache in FP32."""
    case = state["case"]
    page, tok = slots // case["page"], slots % case["page"]
    kc, ks, vc, vs = (x[page, :, tok // GROUP, tok % GROUP] for x in _views(case, state["data"]))
    s = state["scales"]
    gk, gv = (None, None) if s is None else (s[0, :, None], s[1, :, None])
    return _decode(kc, ks, gk, case["fmt"]), _decode(vc, vs, gv, case["fmt"])


def _plain_write(state):
    case, slots = state["case"], state["slots"]
    page, tok = slots // case["page"], slots % case["page"]
    kc, ks, vc, vs = _views(case, state["data"])
    for x, codes, scales, i in ((state["k"], kc, ks, 0), (state["v"], vc, vs, 1)):
        g = 1.0 if state["scales"] is None else state["scales"][i, :, None]
        c, s = _encode(x.float(), g, case["fmt"])
        codes[page, :, tok // GROUP, tok % GROUP] = _pack(c)
        scales[page, :, tok // GROUP, tok % GROUP] = s


def _plain_attend(state):
    case, q, lens, off = state["case"], state["q"], state["lens"].long(), state["offsets"].long()
    h, g, d = case["heads"], case["group"], case["dim"]
    keys = torch.arange(state["max_len"], device="cuda")
    slots = state["table"].long()[:, keys // case["page"]] * case["page"] + keys % case["page"]
    k, v = _gather(state, slots)                                      # [B, L, h, D]
    held = keys < lens[:, None]
    v = v * held[..., None, None]
    token = torch.arange(q.shape[0], device="cuda")
    seq = torch.searchsorted(off, token, right=True) - 1
    nq = off[1:] - off[:-1]
    row = torch.arange(state["max_q"], device="cuda")
    index = (off[:-1, None] + row).clamp_max(q.shape[0] - 1)
    qp = q.float()[index].view(len(lens), -1, h, g, d).permute(0, 2, 1, 3, 4).flatten(2, 3)   # [B, h, Q*g, D]
    x = qp @ k.permute(0, 2, 3, 1) / math.sqrt(d)                     # [B, h, Q*g, L]
    del k, qp
    last = (lens - nq)[:, None] + row                                 # the last key each query sees
    seen = held[:, None] & (keys <= last[..., None])
    if case["window"]:
        seen = seen & (keys > last[..., None] - case["window"])
    x = x.unflatten(2, (-1, g)).masked_fill_(~seen[:, None, :, None], -math.inf)
    m = x.amax(-1, keepdim=True).clamp_min(-3e38)
    x = x.sub_(m).exp_()
    total = x.sum(-1, keepdim=True)
    o = (x.flatten(2, 3) @ v.permute(0, 2, 1, 3)).unflatten(2, (-1, g)) / total.clamp_min(1e-38)
    o = o.permute(0, 2, 1, 3, 4)[seq, token - off[seq]]
    return o.reshape(q.shape).to(q.dtype)


def run(state):
    case = state["case"]
    if own:
        return _run_own(state)
    if case["kind"] == "attend":
        return _plain_attend(state)
    if case["kind"] == "write_read":
        _plain_write(state)
    dt = DTYPES[case["dtype"]]
    k, v = _gather(state, state["slots"])
    return k.to(dt), v.to(dt)


# --------------------------------------------------------- the package's form
def _run_own(state):
    case, handle = state["case"], state["handle"]
    if not handle:   # what a program keeps: the cache around its memory, and a workspace
        from fp4_weight_only_gb300 import binding
        handle["cache"] = binding.KVCache(state["data"].shape[0], case["page"], case["heads"], case["dim"], case["fmt"],
                                          scales=state["scales"], data=state["data"])
        handle["workspace"] = binding.Workspace()
    cache = handle["cache"]
    if case["kind"] == "attend":
        one = case["q_hi"] == 1
        return cache.attention(state["q"], state["table"], state["lens"], None if one else state["offsets"], state["max_q"],
                               window=case["window"], workspace=handle["workspace"])
    if case["kind"] == "write_read":
        cache.append(state["k"], state["v"], state["slots"])
    return cache.read(state["slots"], DTYPES[case["dtype"]])


# -------------------------------------------------------------- in 64 bits
def _e4m3_64(t):
    """Nearest E4M3 value to t >= 0 in 64 bits, ties to even, saturating."""
    e = np.clip(np.floor(np.log2(np.maximum(t, 2.0 ** -12))), -6, 8)
    e = np.where(t >= 2.0 ** (e + 1), e + 1, np.where(t < 2.0 ** e, e - 1, e)).clip(-6, 8)
    step = 2.0 ** (e - 3)
    return np.minimum(np.rint(t / step) * step, 448.0)


def _round_64(x, fmt, g):
    """Rows [..., D] to what the cache holds of them, block by block."""
    b = x.reshape(*x.shape[:-1], -1, BLOCK[fmt])
    amax = np.maximum(np.abs(b).max(-1, keepdims=True), 1e-8)
    if fmt == "nvfp4":
        s = np.maximum(_e4m3_64(amax / (6.0 * g)), 2.0 ** -9) * g
    else:
        s = 2.0 ** np.minimum(np.ceil(np.log2(amax / 6.0)), 125)
    level = np.array(LEVELS)
    a = np.abs(b) / s
    i = np.searchsorted((level[1:] + level[:-1]) / 2, a, side="left")
    up = np.searchsorted((level[1:] + level[:-1]) / 2, a, side="right")
    i = np.where(i % 2 == 0, i, up)          # a tie goes to the even code
    return (np.sign(b) * level[i] * s).reshape(x.shape)


def _values_64(bytes_, scale_bytes, fmt, g):
    """Values of codes [..., D/2] and scale bytes by their bit fields, in 64 bits on the GPU."""
    c = torch.stack((bytes_ & 15, bytes_ >> 4), -1).flatten(-2).long()
    exp, man = (c >> 1) & 3, c & 1
    mag = torch.where(exp == 0, 0.5 * man.double(), (1.0 + 0.5 * man.double()) * 2.0 ** (exp - 1).double())
    val = torch.where(c >= 8, -mag, mag)
    s = scale_bytes.long()
    if fmt == "nvfp4":
        se, sm = (s >> 3) & 15, (s & 7).double() / 8.0
        sv = torch.where(se == 0, sm * 2.0 ** -6, (1.0 + sm) * 2.0 ** (se - 7).double())
    else:
        sv = 2.0 ** (s - 127).double()
    return val * sv.repeat_interleave(BLOCK[fmt], -1) * g


def exact(case, seed):
    state = prepare(case, seed)
    h, d, fmt = case["heads"], case["dim"], case["fmt"]
    kc, ks, vc, vs = _views(case, state["data"])
    g = [1.0, 1.0]
    if state["scales"] is not None:
        g = [state["scales"][i].double() for i in (0, 1)]
    if case["kind"] == "write_read":
        out = []
        for x, gi in ((state["k"], g[0]), (state["v"], g[1])):
            gi = gi.cpu().numpy()[:, None, None] if isinstance(gi, torch.Tensor) else gi
            out.append(_round_64(x.double().cpu().numpy(), fmt, gi))
        return tuple(out)
    if case["kind"] == "read":
        page, tok = state["slots"] // case["page"], state["slots"] % case["page"]
        out = []
        for codes, scales, gi in ((kc, ks, g[0]), (vc, vs, g[1])):
            gi = gi[:, None] if isinstance(gi, torch.Tensor) else gi
            at = (page, slice(None), tok // GROUP, tok % GROUP)
            out.append(_values_64(codes[at], scales[at], fmt, gi))
        return tuple(out)
    nq, ln = _lengths(case)
    result = torch.zeros(state["q"].shape, dtype=torch.float64, device="cuda")
    at = 0
    for b, (n, length) in enumerate(zip(nq, ln)):
        keys = torch.arange(length, device="cuda")
        page = state["table"][b].long()[keys // case["page"]]
        last = torch.arange(length - n, length, device="cuda")[:, None]
        hide = keys > last
        if case["window"]:
            hide = hide | (keys <= last - case["window"])
        for head in range(h):
            where = (page, head, (keys % case["page"]) // GROUP, keys % GROUP)
            gk, gv = (gi[head] if isinstance(gi, torch.Tensor) else gi for gi in g)
            k = _values_64(kc[where], ks[where], fmt, gk)
            v = _values_64(vc[where], vs[where], fmt, gv)
            for i in range(head * case["group"], (head + 1) * case["group"]):
                x = state["q"][at:at + n, i].double() @ k.T / math.sqrt(d)
                x[hide] = -math.inf
                result[at:at + n, i] = torch.softmax(x, -1) @ v
        at += n
    return result
