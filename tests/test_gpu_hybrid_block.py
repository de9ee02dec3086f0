"""The example block: its calls together, against 64-bit autograd of the formulas and, prompt
against single tokens, against itself."""
import os
import sys

import pytest
import torch

from conftest import ROOT

import lin_reference as R

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(ROOT, "examples"))


def plain(block, x, h, lens, state, eps=1e-6):
    """The block in 64 bits, token by token; returns (x', h')."""
    H, d = block.heads, block.dim
    q, k, v, t = (h @ block.p64[n] for n in "qkvt")
    q, k, v = (a.view(-1, H, d) for a in (q, k, v))
    a = torch.exp(block.log_decay.double())[:, None, None]
    o, at = [], 0
    for n, m in enumerate(lens):
        S = state[n]
        for i in range(at, at + m):
            S = a * S + k[i][:, :, None] * v[i][:, None, :]
            o.append(block.scale * torch.einsum("hij,hi->hj", S, q[i]))
        at += m
    o = torch.stack(o).reshape(t.shape)
    u = R.rms(o, block.f64["w_head"].repeat(H), d, eps) * torch.sigmoid(t)
    x = x + block.f64["res_scale"] * R.rms(u @ block.p64["out"], block.f64["w_post"],
                                           x.shape[1], eps)
    return x, R.rms(x, block.f64["w_next"], x.shape[1], eps)


def test_block_gradients_against_autograd():
    from hybrid_block import HybridBlock
    lens, H, d, width = [37, 0, 70], 2, 32, 48
    block = HybridBlock(width, H, d, torch.float32)
    gen = torch.Generator(device="cuda").manual_seed(3)
    x, h, dx, dh = (torch.randn(sum(lens), width, generator=gen, device="cuda")
                    for _ in range(4))
    state = 0.3 * torch.randn(len(lens), H, d, d, generator=gen, device="cuda")
    cu_host = torch.tensor(R.bounds_of(lens), dtype=torch.int32)
    x_out, h_out, _, saved = block.prefill(x, h, cu_host.cuda(), cu_host, state)
    gx, gh, grads = block.backward(saved, dx, dh)
    leaf = lambda t: t.double().requires_grad_(True)  # noqa: E731
    block.p64 = {**{n: leaf(w) for n, w in block.proj.items()}, "out": leaf(block.out)}
    block.f64 = {n: leaf(getattr(block, n)) for n in ("w_head", "w_post", "w_next", "res_scale")}
    x64, h64, s64 = leaf(x), leaf(h), leaf(state)
    wx, wh = plain(block, x64, h64, lens, s64)
    # fp32 through some 20 operations and sums of up to 107 terms: 1e-5 is 170 roundings
    assert R.rel_fro(x_out, R.f64(wx)) <= 1e-5 and R.rel_fro(h_out, R.f64(wh)) <= 1e-5
    ((wx * dx).sum() + (wh * dh).sum()).backward()
    want = {"d" + n: w.grad for n, w in block.p64.items()}
    want.update({"d" + n: w.grad for n, w in block.f64.items()}, dS0=s64.grad)
    assert set(want) == set(grads)
    for n, t in [("x", gx), ("h", gh), *grads.items()]:
        w = {"x": x64.grad, "h": h64.grad}.get(n, want.get(n))
        assert R.rel_fro(t, R.f64(w)) <= 1e-5, n


def test_example_runs():
    import hybrid_block
    off, finite = hybrid_block.main(["--tokens", "300", "--heads", "2", "--new", "5"])
    # bf16 rows: o, u, y and x' are rounded once each on both ways
    assert finite and off <= 4 * R.U16
