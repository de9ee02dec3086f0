"""One decayed linear-attention block of a hybrid stack, from the library's calls.

    q, k, v, t = h W_q, h W_k, h W_v, h W_t          (h: the normed stream)
    o          = linear attention with one decay per head (kda_lin_prefill / _decode_step)
    u          = RMSNorm per head(o) * sigmoid(t)     (kda_block_norm over heads)
    y          = u W_o
    x', h'     = x + res_scale * RMSNorm(y), RMSNorm(x')   (kda_block_norm over rows)

The prompt pass, single tokens on a state pool, and the training backward of the
block; the projections are plain matrix products.

    python examples/hybrid_block.py [--tokens 4096] [--heads 32] [--dim 128]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))
import kimi_delta_attention_12_gb300 as kda  # noqa: E402


class HybridBlock:
    def __init__(self, width, heads, dim, dtype, device="cuda", seed=0):
        g = torch.Generator(device=device).manual_seed(seed)

        def normal(*shape):
            return torch.randn(*shape, generator=g, device=device)

        inner = heads * dim
        self.heads, self.dim, self.scale = heads, dim, dim ** -0.5
        self.proj = {n: (normal(width, inner) * width ** -0.5).to(dtype) for n in "qkvt"}
        self.out = (normal(inner, width) * inner ** -0.5).to(dtype)
        self.log_decay = -torch.exp2(-8.0 * torch.arange(1, heads + 1, device=device) / heads)
        self.w_head = 1.0 + 0.1 * normal(dim)
        self.w_post, self.w_next = 1.0 + 0.1 * normal(width), 1.0 + 0.1 * normal(width)
        self.res_scale = 0.5 + 0.1 * normal(width)

    def _project(self, h):
        q, k, v, t = (h @ self.proj[n] for n in "qkvt")
        return (*(a.view(-1, self.heads, self.dim) for a in (q, k, v)), t)

    def _after(self, x, o, t):
        u, _ = kda.kda_block_norm(o.view(t.shape), self.w_head, gate=t)
        y = u @ self.out
        x_out, h_out = kda.kda_block_norm(y, self.w_post, x=x, res_scale=self.res_scale,
                                          w_pre=self.w_next)
        return u, y, x_out, h_out

    def prefill(self, x, h, cu=None, cu_host=None, state=None):
        """x, h [tokens, width] of packed prompts.  Returns (x', h', the states after the
        prompts, what the backward needs)."""
        q, k, v, t = self._project(h)
        o, last = kda.kda_lin_prefill(q, k, v, self.log_decay, state, cu, cu_host,
                                      scale=self.scale)
        u, y, x_out, h_out = self._after(x, o, t)
        return x_out, h_out, last, (h, q, k, v, t, o, u, y, x_out, cu, cu_host, state)

    def decode(self, x, h, pool, slots=None):
        """One token per row; the rows' states in `pool` move on in place."""
        q, k, v, t = self._project(h)
        o = kda.kda_lin_decode_step(q, k, v, self.log_decay, pool, slots, scale=self.scale)
        return self._after(x, o, t)[2:]

    def backward(self, saved, dx_out, dh_out):
        """Gradients of the stream, its norm, the initial states and every weight."""
        h, q, k, v, t, o, u, y, x_out, cu, cu_host, state = saved
        row = kda.kda_block_norm_backward(y, self.w_post, dx_out, x_out=x_out,
                                          res_scale=self.res_scale, w_pre=self.w_next, dh=dh_out)
        du = row["dy"] @ self.out.t()
        head = kda.kda_block_norm_backward(o.view(t.shape), self.w_head, du, gate=t,
                                           residual=False)
        att = kda.kda_lin_backward(q, k, v, self.log_decay, head["dy"].view(o.shape), state, cu,
                                   cu_host, scale=self.scale)
        inner = {"q": att["dq"], "k": att["dk"], "v": att["dv"], "t": head["dgate"]}
        inner = {n: a.reshape(t.shape) for n, a in inner.items()}
        dh = sum(inner[n] @ self.proj[n].t() for n in "qkvt")
        grads = {"d" + n: h.t() @ inner[n] for n in "qkvt"}
        grads.update(dout=u.t() @ row["dy"], dw_head=head["dw_post"], dw_post=row["dw_post"],
                     dw_next=row["dw_pre"], dres_scale=row["dres_scale"], dS0=att["dS0"])
        return row["dx"], dh, grads


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--tokens", type=int, default=4096)
    ap.add_argument("--heads", type=int, default=32)
    ap.add_argument("--dim", type=int, default=128)
    ap.add_argument("--new", type=int, default=8, help="tokens decoded after the prompt")
    a = ap.parse_args(argv)
    width, dt = a.heads * a.dim, torch.bfloat16
    block = HybridBlock(width, a.heads, a.dim, dt)
    gen = torch.Generator(device="cuda").manual_seed(1)
    x, h = (torch.randn(a.tokens + a.new, width, generator=gen, device="cuda").to(dt)
            for _ in range(2))
    whole = block.prefill(x, h)
    _, _, pool, _ = block.prefill(x[:a.tokens], h[:a.tokens])
    off = 0.0
    for i in range(a.tokens, a.tokens + a.new):
        x1, _ = block.decode(x[i:i + 1], h[i:i + 1], pool)
        want = whole[0][i:i + 1].float()
        off = max(off, float((x1.float() - want).norm() / want.norm()))
    dx, dh, grads = block.backward(whole[3], torch.randn_like(x), torch.randn_like(x))
    torch.cuda.synchronize()
    finite = all(bool(torch.isfinite(t).all()) for t in (dx, dh, *grads.values()))
    print(f"prompt of {a.tokens} tokens, {a.new} more one at a time: off the whole prompt's by "
          f"{off:.1e}; state after them off by "
          f"{float((pool - whole[2]).norm() / whole[2].norm()):.1e}; gradients finite: {finite}")
    return off, finite


if __name__ == "__main__":
    main()
