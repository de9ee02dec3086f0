"""The example layer request by request: one that cannot be served for a step goes on where it
was, tokens one at a time are the whole's, and the outputs are those of the unrounded keys and
values."""
import pytest
import torch

import cache_reference as R
from test_gpu_softmax_layer import _example

pytestmark = pytest.mark.gpu


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _tokens(n, width, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(n, width, generator=g, device="cuda").bfloat16()


@pytest.mark.parametrize("captured", [False, True])
def test_a_request_that_waits_for_a_block_goes_on_where_it_was(captured):
    """Three blocks are free.  Two prompts take them, then one request needs a block that is not
    there; when the other has ended, it goes on.  The same tokens with blocks to spare are the
    measure."""
    width, block = 128, 64
    prompts, more, last = (_tokens(n, width, 5 + n) for n in (100 + block, 2, 1))

    def layer(blocks):
        x = _example().SoftmaxLayer(width, 4, 2, 64, requests=2, tokens=256, block=block)
        x.n_free.fill_(blocks)
        return x

    def blocks_of(x):
        held = [-(-c // block) for c in x.past.tolist()]
        rows = [x.table[i, :n].tolist() for i, n in enumerate(held)]
        return sorted(sum(rows, x.free[:int(x.n_free)].tolist()))

    short, plenty = layer(3), layer(8)
    for x in (short, plenty):
        x.step(prompts, _i32([100, block]), 100)
    assert short.past.tolist() == [100, block] and int(short.n_free) == 0
    assert blocks_of(short) == [0, 1, 2]
    if captured:
        graph, _ = short.capture(more, _i32([1, 1]))
        graph.replay()
    else:
        _, plan = short.step(more, _i32([1, 1]), 1)
        assert plan["status"].tolist() == [0, 3]
    assert short.past.tolist() == [101, block]
    assert blocks_of(short) == [0, 1, 2]
    y, plan = short.step(last, _i32([-1, 1]), 1)
    assert plan["status"].tolist() == [0, 0] and plan["positions"].tolist() == [block]
    assert short.past.tolist() == [0, block + 1] and blocks_of(short) == [0, 1, 2]
    want, _ = plenty.step(last, _i32([-1, 1]), 1)
    assert torch.equal(y, want)


def test_tokens_one_at_a_time_are_the_whole_for_each_request():
    """A block that grows keeps the larger scale, a power of two: what is rounded twice differs only
    below 2^-6 of the scale, by 2^-10 of it, where the block's largest is 224 scales or more.  What
    is left is the rounding of k and v before (products of other shapes), of weights, o and y to
    bf16, 2^-9 each on both sides, sums of many each: 2^-4 / 10 in all."""
    lens, new, width = [70, 3, 1, 129], 5, 128
    tokens = [_tokens(n + new, width, n) for n in lens]
    whole_layer, layer = (_example().SoftmaxLayer(width, 4, 2, 64, 4, 140) for _ in range(2))
    whole, _ = whole_layer.step(torch.cat(tokens), _i32([n + new for n in lens]), 134)
    whole = whole.float().split([n + new for n in lens])
    layer.step(torch.cat([t[:n] for t, n in zip(tokens, lens)]), _i32(lens), max(lens))
    for i in range(new):
        y, _ = layer.step(torch.stack([t[n + i] for t, n in zip(tokens, lens)]), _i32([1] * 4), 1)
        for r, n in enumerate(lens):
            want = whole[r][n + i]
            assert float((y[r].float() - want).norm() / want.norm()) < 2.0 ** -4 / 10


def test_outputs_are_those_of_the_unrounded_keys_and_values():
    """One prompt against softmax attention in 64 bits over k and v as they were before their
    rounding to 8 bits.  An e4m3 number is off by up to 2^-4 of itself, evenly spread: 0.026 rms
    over a binade.  That is a row's error from the values, as they and their errors are independent;
    a score's is 0.026 |magnitude^2 sum q k| / 8 = 0.034 or so, and a row's from it the same: 0.043
    together, and a row of the few tokens at the start may have twice as much.  A wrong head, row or
    position is off by 1."""
    n, heads, kv, d = 150, 4, 2, 64
    width = heads * d
    layer = _example().SoftmaxLayer(width, heads, kv, d, 1, 192)
    layer.w_out = torch.eye(width, device="cuda").bfloat16()         # y is o
    h = _tokens(n, width, 3)
    y, plan = layer.step(h, _i32([n]), n)
    qkv = (h @ layer.w_in).view(n, heads + 2 * kv, d)
    turned = R.rotary(qkv[:, :heads + kv], plan["positions"], layer.inv_freq, False, d // 2,
                      layer.magnitude)
    v = qkv[:, heads + kv:].double().cpu()
    got = y.view(n, heads, d).double().cpu()
    seen = torch.ones(n, n).tril().bool()
    for hq in range(heads):
        s = (turned[:, hq] @ turned[:, heads + hq // (heads // kv)].T) * d ** -0.5
        want = torch.softmax(s.masked_fill(~seen, float("-inf")), -1) @ v[:, hq // (heads // kv)]
        off = (got[:, hq] - want).norm(dim=-1) / want.norm(dim=-1)
        assert float((got[:, hq] - want).norm() / want.norm()) < 2 * 0.043
        assert float(off.max()) < 0.25
