"""A decoder layer with FP4 weights and an FP4 K/V cache.

    python -m fp4_weight_only_gb300.layer [--layers 2] [--batch 8] [--prompt 1000] [--steps 32] [--fmt nvfp4]

``DecoderLayer`` puts the norms, the rotary positions and the gated feed-forward
block around :class:`attend.AttentionBlock`: norm with the residual's addition,
QKV product, positions (in place), cache and attention, O product, norm, gated
projections in one kernel, down product.  A layer hands on its output and the
residual stream; the next layer's first norm adds them.  The command serves a
batch of random prompts through a stack of layers, all prompts in one call, then
token after token through one CUDA graph, and prints the times and how far the
last prompt's last token lies from the same token fed by itself behind the
others.  Weights and inputs are random; embeddings and the output head are the
caller's.
"""

import argparse
import json

import torch

from . import attend, binding


class DecoderLayer:
    """`w_qkv` and `w_o` as :class:`attend.AttentionBlock`'s; `w_gate`, `w_up`
    [intermediate, hidden] and `w_down` [hidden, intermediate], BF16 CUDA tensors
    that are quantised once; `norm_attention` and `norm_mlp` [hidden], the norms'
    weights.  `rope`: a :class:`binding.Rotary`, or None for no positions."""

    def __init__(self, w_qkv, w_o, w_gate, w_up, w_down, norm_attention, norm_mlp, num_q_heads, num_kv_heads, head_dim,
                 num_pages, rope=None, eps=1e-5, act="silu", page_size=64, fmt="nvfp4", kv_scales=None, workspace=None):
        hidden = w_qkv.shape[1]
        if w_gate.shape != w_up.shape or w_gate.shape[1] != hidden or w_down.shape != (hidden, w_gate.shape[0]):
            raise ValueError(f"w_gate, w_up, w_down: need [intermediate, {hidden}] twice and [{hidden}, intermediate]")
        if norm_attention.shape != (hidden,) or norm_mlp.shape != (hidden,):
            raise ValueError(f"norm_attention, norm_mlp: need shape ({hidden},)")
        if act not in binding.ACTIVATIONS:
            raise ValueError(f"act: need one of {', '.join(binding.ACTIVATIONS)}")
        self.attention = attend.AttentionBlock(w_qkv, w_o, num_q_heads, num_kv_heads, head_dim, num_pages, page_size, fmt,
                                               kv_scales, workspace)
        self.workspace = self.attention.workspace
        self.gated = binding.GatedWeight(w_gate, w_up, fmt, "amax")
        self.down = binding.FP4Weight(w_down, fmt, "amax")
        self.norm_attention, self.norm_mlp = norm_attention, norm_mlp
        self.rope, self.eps, self.act = rope, eps, act

    def __call__(self, x, residual, positions, slots, block_table, seq_lens, q_offsets=None, max_q=1, window=0):
        """(output, residual) of tokens x [tokens, hidden]; `residual` is what the
        layer before handed on, or None for the first layer (x is then the
        stream).  `positions`: int64 or int32 [tokens]; the other arguments as
        :meth:`attend.AttentionBlock.attend`.  x and residual are left as they are."""
        if residual is None:
            h, residual = binding.rms_norm(x, self.norm_attention, self.eps), x
        else:
            h, residual = binding.rms_norm(x, self.norm_attention, self.eps, residual)
        turn = None if self.rope is None else lambda q, k: self.rope(q, k, positions, out=(q, k))
        a = self.attention(h, slots, block_table, seq_lens, q_offsets, max_q, window, turn)
        h, residual = binding.rms_norm(a, self.norm_mlp, self.eps, residual, out=a)
        return self.down(self.gated(h, self.act, self.workspace), self.workspace), residual


def run(layers, x, *args, **kwargs):
    """The residual stream after a stack of layers, before the last norm."""
    residual = None
    for layer in layers:
        x, residual = layer(x, residual, *args, **kwargs)
    return x + residual


def serve(layers=2, batch=8, prompt=1000, steps=32, hidden=8192, intermediate=28672, num_q_heads=64, num_kv_heads=8,
          head_dim=128, page_size=64, fmt="nvfp4", act="silu", seed=0):
    """Serves a batch on the current GPU; returns the figures that the command prints."""
    from . import synth
    dev = torch.device("cuda", torch.cuda.current_device())
    rng = torch.Generator().manual_seed(seed)
    lens = [max(2, prompt * (b + 1) // batch) for b in range(batch)]
    per = -(-(max(lens) + steps + 3) // page_size)   # pages a sequence (3: the uncounted steps)
    table = torch.randperm(batch * per, generator=rng).view(batch, per).int().to(dev)
    dims = (num_q_heads + 2 * num_kv_heads) * head_dim
    # NVFP4's scales per head: what the largest of a unit normal's values asks for
    scales = torch.full((2, num_kv_heads), 5.0 / (6 * 448), device=dev) if fmt == "nvfp4" else None
    rope = binding.Rotary(head_dim, 500000.0, device=dev)
    ones = torch.ones(hidden, dtype=torch.bfloat16, device=dev)
    ws = binding.Workspace(dev)
    stack = []
    for i in range(layers):
        w = lambda n, k, j: synth.weights(n, k, seed=10 * i + j, device=dev, std=k ** -0.5)  # noqa: E731,B023
        stack.append(DecoderLayer(w(dims, hidden, 1), w(hidden, num_q_heads * head_dim, 2), w(intermediate, hidden, 3),
                                  w(intermediate, hidden, 4), w(hidden, intermediate, 5), ones, ones, num_q_heads,
                                  num_kv_heads, head_dim, batch * per, rope, act=act, page_size=page_size, fmt=fmt,
                                  kv_scales=scales, workspace=ws))

    def timed(f, n=1):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        for _ in range(n):
            r = f()
        b.record()
        torch.cuda.synchronize()
        return a.elapsed_time(b) * 1e3 / n, r

    # all prompts in one call
    seq = torch.repeat_interleave(torch.arange(batch), torch.tensor(lens)).to(dev)
    pos = torch.cat([torch.arange(n) for n in lens]).to(dev)
    slots = attend.slots_of(table, seq, pos, page_size)
    offsets = torch.tensor([0] + lens).cumsum(0).int().to(dev)
    seq_lens = torch.tensor(lens, dtype=torch.int32, device=dev)
    x = synth.activations(sum(lens), hidden, seed=3, device=dev)
    prompts = lambda: run(stack, x, pos, slots, table, seq_lens, offsets, max(lens))  # noqa: E731
    prompts()
    prompt_us, y = timed(prompts)

    # the last sequence's last token by itself, behind what is cached of the others
    last = run(stack, x[-1:], pos[-1:], slots[-1:], table[-1:], seq_lens[-1:]).float()
    difference = ((y[-1:].float() - last).norm() / last.norm()).item()

    # token after token: the graph advances lengths, positions and slots by itself
    tok = synth.activations(batch, hidden, seed=4, device=dev)
    every = torch.arange(batch, device=dev)

    def step():
        at = seq_lens.long()
        seq_lens.add_(1)
        return run(stack, tok, at, attend.slots_of(table, every, at, page_size), table, seq_lens)

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
    status = ws.status()
    if status != 0:
        raise RuntimeError(f"device status {binding.STATUS.get(status, status)} while serving")
    if not torch.isfinite(y.float()).all():
        raise RuntimeError("outputs are not finite")
    return {"fmt": fmt, "layers": layers, "batch": batch, "prompt_tokens": sum(lens),
            "prompt_us_per_layer": round(prompt_us / layers, 1), "steps": steps, "step_us_per_layer": round(step_us / layers, 1),
            "cached_tokens": int(seq_lens.sum()), "single_token_difference": float(f"{difference:.3g}")}


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    ap.add_argument("--layers", type=int, default=2)
    ap.add_argument("--batch", type=int, default=8)
    ap.add_argument("--prompt", type=int, default=1000, help="tokens of the longest prompt")
    ap.add_argument("--steps", type=int, default=32, help="timed decode steps")
    ap.add_argument("--hidden", type=int, default=8192)
    ap.add_argument("--intermediate", type=int, default=28672)
    ap.add_argument("--q-heads", type=int, default=64)
    ap.add_argument("--kv-heads", type=int, default=8)
    ap.add_argument("--head-dim", type=int, default=128, choices=(64, 128))
    ap.add_argument("--page", type=int, default=64)
    ap.add_argument("--fmt", default="nvfp4", choices=("nvfp4", "mxfp4"))
    ap.add_argument("--act", default="silu", choices=tuple(binding.ACTIVATIONS))
    a = ap.parse_args(argv)
    print(json.dumps(serve(a.layers, a.batch, a.prompt, a.steps, a.hidden, a.intermediate, a.q_heads, a.kv_heads, a.head_dim,
                           a.page, a.fmt, a.act)))
    return 0


if __name__ == "__main__":
    raise SystemExit(main())
