"""The softmax-attention layer of a hybrid stack in serving, from the library's calls.

    q, k, v  = h W_q, h W_k, h W_v                    (one product, one buffer)
    blocks, positions, slots of the step's tokens     (kda_cache_plan)
    q, k     turned by their positions, in place      (kda_rotary)
    k, v     into the paged cache, in 8 bits          (kda_cache_write)
    o        = softmax attention over the cache       (kda_cache_attention)
    y        = o W_o

Requests enter with prompts of any lengths, are answered token by token, and leave; a decode
step is one CUDA graph, replayed while lengths, blocks and slots move on by themselves.

    python examples/softmax_layer.py [--heads 32] [--kv-heads 8] [--dim 128] [--new 16]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))
import kimi_delta_attention_12_gb300 as kda  # noqa: E402


class SoftmaxLayer:
    def __init__(self, width, heads, kv_heads, dim, requests, tokens, block=64, device="cuda",
                 seed=0):
        g = torch.Generator(device=device).manual_seed(seed)
        self.heads, self.kv_heads, self.dim, self.block = heads, kv_heads, dim, block
        inner = (heads + 2 * kv_heads) * dim
        self.w_in = (torch.randn(width, inner, generator=g, device=device) * width ** -0.5).bfloat16()
        self.w_out = (torch.randn(heads * dim, width, generator=g, device=device)
                      * (heads * dim) ** -0.5).bfloat16()
        self.inv_freq, self.magnitude = kda.rotary_frequencies(dim // 2, scaling="by_parts",
                                                               factor=8.0, device=device)
        per = -(-tokens // block)
        pool = requests * per
        i32 = dict(dtype=torch.int32, device=device)
        self.cache = [torch.empty(pool, kv_heads, block, dim, dtype=torch.float8_e4m3fn,
                                  device=device) for _ in range(2)]
        self.scale = [torch.ones(pool, kv_heads, device=device) for _ in range(2)]
        self.table = torch.zeros(requests, per, **i32)
        self.free, self.n_free = torch.arange(pool, **i32), torch.tensor([pool], **i32)
        self.past = torch.zeros(requests, **i32)

    def step(self, h, new, max_new):
        """h [rows, width] of the requests' new tokens, new [requests] how many each has (-1: the
        request ends).  Returns y [rows, width] and the plan; the rows of a request whose status in
        it is not 0 are zero and to be given again."""
        plan = kda.kda_cache_plan(self.past, new, self.table, self.free, self.n_free, self.block,
                                  h.shape[0], n_free_out=self.n_free)
        # a request that is not served this time (no free block, say) waits where it is
        served = plan["status"] == kda.KDA_PLAN_OK
        self.past.copy_(torch.where(served, plan["context_lens"], self.past))
        qkv = (h @ self.w_in).view(h.shape[0], self.heads + 2 * self.kv_heads, self.dim)
        q, k = qkv[:, :self.heads], qkv[:, self.heads:self.heads + self.kv_heads]
        v = qkv[:, self.heads + self.kv_heads:]
        kda.kda_rotary(q, k, plan["positions"], self.inv_freq, first=self.dim // 2,
                       magnitude=self.magnitude, q_out=q, k_out=k)
        kda.kda_cache_write(k, v, plan["slots"], *self.cache, *self.scale)
        o = kda.kda_cache_attention(q, *self.cache, *self.scale, self.table, plan["context_lens"],
                                    plan["cu_seqlens"], max_new=max_new)
        return o.view(h.shape[0], self.heads * self.dim) @ self.w_out, plan

    def capture(self, h, new):
        """A decode step on the buffers h [requests, width] and new [requests] as a graph.
        Returns (graph, y)."""
        before = [t.clone() for t in (self.past, self.table, self.free, self.n_free)]
        kept = [t.clone() for t in (*self.cache, *self.scale)]
        self.step(h, new, 1)                         # once outside, so that all is set up
        for t, b in zip((self.past, self.table, self.free, self.n_free, *self.cache, *self.scale),
                        before + kept):
            t.copy_(b)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            y, _ = self.step(h, new, 1)
        return graph, y


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--heads", type=int, default=32)
    ap.add_argument("--kv-heads", type=int, default=8)
    ap.add_argument("--dim", type=int, default=128)
    ap.add_argument("--prompts", default="1000,37,2049,515")
    ap.add_argument("--new", type=int, default=16, help="tokens decoded after the prompts")
    a = ap.parse_args(argv)
    lens = [int(x) for x in a.prompts.split(",")]
    width, n, longest = a.heads * a.dim // 2, len(lens), max(lens) + a.new
    gen = torch.Generator(device="cuda").manual_seed(1)
    tokens = [torch.randn(x + a.new, width, generator=gen, device="cuda").bfloat16() for x in lens]

    def layer():
        return SoftmaxLayer(width, a.heads, a.kv_heads, a.dim, n, longest)

    def i32(x):
        return torch.tensor(x, dtype=torch.int32, device="cuda")

    # every request's tokens at once, and its prompt and then one token at a time
    whole, _ = layer().step(torch.cat(tokens), i32([len(t) for t in tokens]), longest)
    whole = whole.split([len(t) for t in tokens])
    served = layer()
    served.step(torch.cat([t[:x] for t, x in zip(tokens, lens)]), i32(lens), max(lens))
    h, one = torch.empty(n, width, dtype=torch.bfloat16, device="cuda"), i32([1] * n)
    graph, y = served.capture(h, one)
    off = 0.0
    for i in range(a.new):
        h.copy_(torch.stack([t[x + i] for t, x in zip(tokens, lens)]))
        graph.replay()
        want = torch.stack([w[x + i] for w, x in zip(whole, lens)]).float()
        off = max(off, float((y.float() - want).norm() / want.norm()))
    _, plan = served.step(h[:0], i32([-1] * n), 0)
    left = int(plan["n_free"])
    print(f"prompts of {a.prompts} tokens, {a.new} more one at a time: off the whole's by {off:.1e}; "
          f"{left} of {served.free.shape[0]} blocks free after the requests have ended")
    return off, left == served.free.shape[0]


if __name__ == "__main__":
    main()
