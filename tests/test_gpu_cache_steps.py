"""Serving steps of one softmax-attention layer: plan, rotary, write and attention together,
from prompts to the last token, in a pool that requests enter and leave."""
import numpy as np
import pytest
import torch

import cache_reference as R
import kimi_delta_attention_12_gb300 as kda

pytestmark = pytest.mark.gpu


def test_steps_of_a_layer():
    dev, block, H, G, d, N, W = "cuda", 16, 2, 3, 64, 3, 8
    nb = 14
    i32 = dict(dtype=torch.int32, device=dev)
    cache = [torch.zeros(nb, H, block, d, device=dev).to(torch.float8_e4m3fn) for _ in range(2)]
    scales = [torch.ones(nb, H, device=dev) for _ in range(2)]
    table = torch.full((N, W), -1, **i32)
    free, n_free = torch.arange(nb, **i32), torch.tensor([nb], **i32)
    past = torch.zeros(N, **i32)
    f, m = kda.rotary_frequencies(32, scaling="by_parts", factor=4.0)
    g = torch.Generator(device=dev).manual_seed(0)
    kept = [[] for _ in range(N)]               # the exact turned k and v of each request
    steps = [[37, 20, 5], [1, 1, 1], [1, 1, 11], [1, -1, 1], [1, 70, 1], [1, 1, -1], [20, 1, 3]]
    for new in steps:
        rows = sum(max(x, 0) for x in new)
        wide = torch.randn(rows, (G * H + 2 * H) * d, generator=g, device=dev).bfloat16()
        q = wide[:, :G * H * d].view(rows, G * H, d)
        k = wide[:, G * H * d:(G + 1) * H * d].view(rows, H, d)
        v = wide[:, (G + 1) * H * d:].view(rows, H, d)
        p = kda.kda_cache_plan(past, torch.tensor(new, **i32), table, free, n_free, block, rows,
                               n_free_out=n_free)
        assert not p["status"].any()
        kda.kda_rotary(q, k, p["positions"], f, first=16, magnitude=m, q_out=q, k_out=k)
        kda.kda_cache_write(k, v, p["slots"], *cache, *scales)
        o = kda.kda_cache_attention(q, *cache, *scales, table, p["context_lens"], p["cu_seqlens"],
                                    max_new=max(new))
        past = p["context_lens"]
        cu, context = p["cu_seqlens"].tolist(), past.tolist()
        # what the cache stands for, against the definition
        want, *sizes = R.attention(
            q, cache[0].view(torch.uint8).cpu().numpy(), cache[1].view(torch.uint8).cpu().numpy(),
            scales[0].cpu().numpy(), scales[1].cpu().numpy(), table.tolist(), context, cu,
            d ** -0.5, block)
        off = np.abs(o.double().cpu().numpy() - want)
        assert (off <= R.attention_bound(want, *sizes, d, max(context), True)).all()
        # and against the keys and values themselves: every cached number is within 2^-4 of its
        # own, or 2^-10 of its block's scale
        for i, n in enumerate(new):
            if n < 0:
                kept[i] = []
                continue
            kept[i] += [(k[t].double().cpu(), v[t].double().cpu()) for t in range(cu[i], cu[i + 1])]
            assert len(kept[i]) == context[i]
            for x, pair in enumerate(kept[i]):
                b, at = int(table[i, x // block]), x % block
                for c, s, y in zip(cache, scales, pair):
                    got = c[b, :, at].double().cpu() * s[b].double().cpu()[:, None]
                    slack = s[b].double().cpu()[:, None] * 2.0 ** -9
                    assert bool(((got - y).abs() <= 2.0 ** -4 * y.abs() + slack).all())
    held = sum(-(-c // block) for c in past.tolist())
    assert int(n_free) == nb - held
    assert sorted(free[:int(n_free)].tolist() + [int(table[i, j]) for i, c in enumerate(past.tolist())
                                                 for j in range(-(-c // block))]) == list(range(nb))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_a_step_without_tokens(dtype):
    """Requests end or wait, and no row comes: every call takes empty tensors."""
    i32 = dict(dtype=torch.int32, device="cuda")
    table, free, n_free = torch.tensor([[0, 1], [2, 0]], **i32), torch.zeros(4, **i32), \
        torch.tensor([0], **i32)
    p = kda.kda_cache_plan(torch.tensor([20, 3], **i32), torch.tensor([-1, 0], **i32), table, free,
                           n_free, 16, 0, n_free_out=n_free)
    assert p["context_lens"].tolist() == [0, 3] and n_free.tolist() == [2]
    assert p["slots"].shape == p["positions"].shape == (0,)
    wide = torch.empty(0, 6, 32, dtype=dtype, device="cuda")
    q, k, v = wide[:, :4], wide[:, 4:5], wide[:, 5:]
    f, _ = kda.rotary_frequencies(32)
    assert kda.kda_rotary(q, k, p["positions"], f, q_out=q, k_out=k)[0].shape == (0, 4, 32)
    assert kda.kda_rotary_backward(q, None, p["positions"], f)[0].shape == (0, 4, 32)
    cache = [torch.zeros(4, 1, 16, 32, device="cuda").to(torch.float8_e4m3fn) for _ in range(2)]
    scales = [torch.ones(4, 1, device="cuda") for _ in range(2)]
    kda.kda_cache_write(k, v, p["slots"], *cache, *scales)
    o = kda.kda_cache_attention(q, *cache, *scales, table, p["context_lens"], p["cu_seqlens"])
    assert o.shape == (0, 4, 32)
    torch.cuda.synchronize()
