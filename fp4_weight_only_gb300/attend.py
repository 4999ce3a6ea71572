"""The attention block of a decoder layer with FP4 weights and an FP4 K/V cache.

    python -m fp4_weight_only_gb300.attend [--batch 8] [--prompt 1000] [--steps 32] [--fmt nvfp4]

``AttentionBlock`` strings the library's calls together as a server does: the
fused QKV product, `kv_append` of its K and V columns (views, nothing is
copied), `kv_attention` over the paged cache, and the O product.  The command
serves a batch of random prompts of different lengths: one call for all
prompts, then token after token through one CUDA graph, whose lengths and
slots the device advances.  It prints the times, and how far the attention
lies from one in FP32 over the tokens that `kv_read` gives back.  Weights and
inputs are random and carry no positions; norms and the MLP are the caller's,
and so is position encoding, which enters between the product and the cache
(`position`); ``layer.DecoderLayer`` brings all three.
"""

import argparse
import json

import torch

from . import binding


class AttentionBlock:
    """`w_qkv` [(num_q_heads + 2 num_kv_heads) * head_dim, hidden] and `w_o`
    [hidden, num_q_heads * head_dim], BF16 CUDA tensors, are quantised once;
    the cache has room for `num_pages` pages of `page_size` tokens.  `fmt` is
    the format of weights and cache.  `kv_scales` (NVFP4): FP32 [2,
    num_kv_heads], see :class:`binding.KVCache`."""

    def __init__(self, w_qkv, w_o, num_q_heads, num_kv_heads, head_dim, num_pages, page_size=64, fmt="nvfp4",
                 kv_scales=None, workspace=None):
        if w_qkv.shape[0] != (num_q_heads + 2 * num_kv_heads) * head_dim:
            raise ValueError(f"w_qkv: need {(num_q_heads + 2 * num_kv_heads) * head_dim} rows")
        if w_o.shape != (w_qkv.shape[1], num_q_heads * head_dim):
            raise ValueError(f"w_o: need shape ({w_qkv.shape[1]}, {num_q_heads * head_dim})")
        self.heads = (num_q_heads, num_kv_heads, num_kv_heads)
        self.head_dim = head_dim
        self.qkv = binding.FP4Weight(w_qkv, fmt, "amax")
        self.o = binding.FP4Weight(w_o, fmt, "amax")
        self.cache = binding.KVCache(num_pages, page_size, num_kv_heads, head_dim, fmt, scales=kv_scales,
                                     device=w_qkv.device)
        self.workspace = workspace or binding.Workspace(w_qkv.device)

    def project(self, x):
        """q, k and v of x [tokens, hidden], as views [tokens, heads, head_dim] of one product."""
        return self.qkv(x, self.workspace).view(x.shape[0], sum(self.heads), self.head_dim).split(self.heads, dim=1)

    def attend(self, x, slots, block_table, seq_lens, q_offsets=None, max_q=1, window=0, position=None):
        """The heads' outputs [tokens, num_q_heads, head_dim]; x's K and V enter
        the cache at `slots`.  `position`, if given, is called with q and k
        ([tokens, heads, head_dim], views that it may change in place) and
        returns them with their positions encoded."""
        q, k, v = self.project(x)
        if position is not None:
            q, k = position(q, k)
        self.cache.append(k, v, slots, self.workspace)
        return self.cache.attention(q, block_table, seq_lens, q_offsets, max_q, window=window,
                                    workspace=self.workspace)

    def __call__(self, x, slots, block_table, seq_lens, q_offsets=None, max_q=1, window=0, position=None):
        """Attention over the cached tokens and x's own, [tokens, hidden].
        Arguments as :func:`binding.kv_attention`; `seq_lens` counts x's
        tokens; `position` as :meth:`attend`."""
        heads = self.attend(x, slots, block_table, seq_lens, q_offsets, max_q, window, position)
        return self.o(heads.view(x.shape[0], -1), self.workspace)


def slots_of(block_table, sequences, positions, page_size):
    """Cache slots of tokens: token i is position positions[i] of sequence sequences[i] (int64 tensors)."""
    return block_table[sequences, positions // page_size].long() * page_size + positions % page_size


def serve(batch=8, prompt=1000, steps=32, hidden=8192, num_q_heads=64, num_kv_heads=8, head_dim=128, page_size=64,
          fmt="nvfp4", seed=0):
    """Serves a batch on the current GPU; returns the figures that the command prints."""
    from . import synth
    dev = torch.device("cuda", torch.cuda.current_device())
    rng = torch.Generator().manual_seed(seed)
    lens = [max(1, prompt * (b + 1) // batch) for b in range(batch)]
    per = -(-(max(lens) + steps + 3) // page_size)   # pages a sequence (3: the uncounted steps)
    table = torch.randperm(batch * per, generator=rng).view(batch, per).int().to(dev)
    dims = (num_q_heads + 2 * num_kv_heads) * head_dim
    # NVFP4's scales per head: what the largest of a unit normal's values asks for
    scales = torch.full((2, num_kv_heads), 5.0 / (6 * 448), device=dev) if fmt == "nvfp4" else None
    block = AttentionBlock(synth.weights(dims, hidden, seed=1, device=dev, std=hidden ** -0.5),
                           synth.weights(hidden, num_q_heads * head_dim, seed=2, device=dev), num_q_heads,
                           num_kv_heads, head_dim, batch * per, page_size, fmt, scales)
    page = block.cache.page_size

    def timed(f, n=1):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        for _ in range(n):
            r = f()
        b.record()
        torch.cuda.synchronize()
        return a.elapsed_time(b) * 1e3 / n, r

    # all prompts in one call
    seq = torch.repeat_interleave(torch.arange(batch), torch.tensor(lens))
    pos = torch.cat([torch.arange(n) for n in lens])
    slots = slots_of(table, seq.to(dev), pos.to(dev), page)
    offsets = torch.tensor([0] + lens).cumsum(0).int().to(dev)
    seq_lens = torch.tensor(lens, dtype=torch.int32, device=dev)
    x = synth.activations(sum(lens), hidden, seed=3, device=dev)
    run = lambda: block(x, slots, table, seq_lens, offsets, max(lens))  # noqa: E731
    run()
    prompt_us, y = timed(run)

    # how far the first sequence's heads are from FP32 attention over the cached values
    heads = block.attend(x, slots, table, seq_lens, offsets, max(lens))
    n = lens[0]
    q = block.project(x[:n])[0].float().transpose(0, 1)
    k, v = (t.float().repeat_interleave(num_q_heads // num_kv_heads, 1).transpose(0, 1)
            for t in block.cache.read(slots[:n]))
    s = (q @ k.transpose(1, 2)) * head_dim ** -0.5
    s = s.masked_fill(torch.ones(n, n, dtype=torch.bool, device=dev).triu(1), -torch.inf)
    want = (s.softmax(-1) @ v).transpose(0, 1)
    error = ((heads[:n].float() - want).norm() / want.norm()).item()

    # token after token: the graph advances lengths and slots by itself
    tok = synth.activations(batch, hidden, seed=4, device=dev)
    every = torch.arange(batch, device=dev)

    def step():
        slot = slots_of(table, every, seq_lens.long(), page)
        seq_lens.add_(1)
        return block(tok, slot, table, seq_lens)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    graph.replay()
    step_us, _ = timed(graph.replay, steps)
    status = block.workspace.status()
    if status != 0:
        raise RuntimeError(f"device status {binding.STATUS.get(status, status)} while serving")
    if not torch.isfinite(y.float()).all():
        raise RuntimeError("outputs are not finite")
    return {"fmt": fmt, "batch": batch, "prompt_tokens": sum(lens), "prompt_us": round(prompt_us, 1), "steps": steps,
            "step_us": round(step_us, 1), "cached_tokens": int(seq_lens.sum()),
            "cache_bytes_per_token": block.cache.page_bytes // page, "relative_error": float(f"{error:.3g}")}


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    ap.add_argument("--batch", type=int, default=8)
    ap.add_argument("--prompt", type=int, default=1000, help="tokens of the longest prompt")
    ap.add_argument("--steps", type=int, default=32, help="timed decode steps")
    ap.add_argument("--hidden", type=int, default=8192)
    ap.add_argument("--q-heads", type=int, default=64)
    ap.add_argument("--kv-heads", type=int, default=8)
    ap.add_argument("--head-dim", type=int, default=128, choices=(64, 128))
    ap.add_argument("--page", type=int, default=64)
    ap.add_argument("--fmt", default="nvfp4", choices=("nvfp4", "mxfp4"))
    a = ap.parse_args(argv)
    print(json.dumps(serve(a.batch, a.prompt, a.steps, a.hidden, a.q_heads, a.kv_heads, a.head_dim, a.page, a.fmt)))
    return 0


if __name__ == "__main__":
    raise SystemExit(main())
