"""The example layer request by request: one that cannot be served for a step goes on where it
was."""
import pytest
import torch

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
