"""A step's bookkeeping on the GPU against an allocator that takes the requests one by one."""
import random

import pytest
import torch

import cache_reference as R
import kimi_delta_attention_12_gb300 as kda

pytestmark = pytest.mark.gpu


def _i32(x):
    return torch.tensor(x, dtype=torch.int32).cuda()


def _setup(past, block, W, spare, seed, capacity=None):
    """A table whose rows hold the past tokens' blocks, and a free list of `spare` blocks."""
    rng = random.Random(seed)
    have = [min(max(0, -(-p // block)), W) for p in past]
    ids = list(range(sum(have) + spare))
    rng.shuffle(ids)
    table = []
    for h in have:
        table.append(ids[:h] + [-9] * (W - h))
        ids = ids[h:]
    free = ids + [-7] * ((capacity or len(ids) + sum(have)) - len(ids))
    return table, free or [-7], spare


def _check(past, new, table, free, n_free, block, rows):
    want = R.plan(past, new, table, free, n_free, block, rows)
    t, f = _i32(table), _i32(free)
    got = kda.kda_cache_plan(_i32(past), _i32(new), t, f, _i32([n_free]), block, rows)
    got = dict(got, block_table=t, free_blocks=f)
    for name, value in want.items():
        assert got[name].cpu().tolist() == value, name
    return want


@pytest.mark.parametrize("block", [16, 32, 64, 128])
@pytest.mark.parametrize("N", [1, 2, 33, 300, 1024, 1025, 2500])
def test_decode_steps(N, block):
    rng = random.Random(N * block)
    past = [rng.choice([0, 1, block - 1, block, block + 1, rng.randint(0, 1000)]) for _ in range(N)]
    table, free, spare = _setup(past, block, 1002 // block + 2, N, 1)
    _check(past, [1] * N, table, free, spare, block, N)


@pytest.mark.parametrize("seed", range(12))
def test_ragged_batches_with_ends(seed):
    rng = random.Random(seed)
    N, block = rng.choice([1, 3, 17, 70]), rng.choice([16, 64])
    past = [rng.choice([0, 0, rng.randint(0, 300)]) for _ in range(N)]
    new = [rng.choice([-1, 0, 1, rng.randint(0, 200)]) for _ in range(N)]
    table, free, spare = _setup(past, block, 600 // block + 1, rng.choice([0, 2, 40, 2000]), seed)
    total = sum(max(x, 0) for x in new)
    _check(past, new, table, free, spare, block, total + rng.choice([0, 5, 300]))


def test_requests_that_are_not_served():
    past, new = [0, -3, 5, 0, 32, 16, 10, 0], [16, 4, -2, 200, 40, 1, 6, 3]
    table, free, spare = _setup(past, 16, 5, 3, 2)
    want = _check(past, new, table, free, spare, 16, 400)
    assert want["status"] == [0, 1, 1, 2, 3, 3, 0, 3]
    want = _check(past, new, table, free, spare, 16, 20)      # rows run out
    assert want["status"][4:] == [4, 4, 4, 4] and want["cu_seqlens"][-1] == 20


def test_requests_without_tokens_behind_the_last_row():
    past, new = [0, 40, 7, 0], [30, -1, 0, 5]
    table, free, spare = _setup(past, 16, 4, 6, 8)
    want = _check(past, new, table, free, spare, 16, 20)
    assert want["status"] == [4, 0, 0, 4] and want["context_lens"] == [0, 0, 7, 0]
    assert want["n_free"] == [9]


def test_lengths_near_the_largest_whole_number():
    most = 0x7fffffff
    past, new = [most, most - 3, most, 2], [most, 3, -1, most]
    table, free, spare = _setup([0, 0, 0, 2], 128, 3, 2, 9)
    want = _check(past, new, table, free, spare, 128, 4)
    assert want["status"] == [2, 2, 2, 2]


def test_returned_blocks_are_taken_in_the_same_step():
    past, new = [40, 0, 33], [-1, 48, -1]
    table, free, spare = _setup(past, 16, 4, 0, 3)
    want = _check(past, new, table, free, spare, 16, 48)
    assert want["status"] == [0, 0, 0] and want["n_free"] == [3]


def test_free_list_that_is_full_or_says_nonsense():
    past, new = [40, 40], [-1, -1]
    table, free, _ = _setup(past, 16, 4, 1, 4, capacity=3)
    assert _check(past, new, table, free, 1, 16, 0)["n_free"] == [3]
    for n_free in (-5, 1000):
        _check([0, 20], [3, 30], *_setup([0, 20], 16, 4, 4, 5)[:2], n_free, 16, 40)


def test_no_rows_and_a_padded_batch():
    _check([3, 4], [0, 0], *_setup([3, 4], 16, 2, 2, 6), 16, 0)
    _check([3, 4], [0, 0], *_setup([3, 4], 16, 2, 2, 6), 16, 7)


def test_values_that_make_no_slot():
    t = _i32([[(1 << 30), 2], [-4, 3]])
    got = kda.kda_cache_plan(_i32([3, 3]), _i32([1, 1]), t, _i32([0]), _i32([1]), 16, 2)
    assert got["slots"].tolist() == [-1, -1] and got["status"].tolist() == [0, 0]


def test_steps_captured_in_a_graph_move_on():
    """Lengths, table and free list advance in place from replay to replay."""
    block, N = 16, 5
    past = [0, 15, 16, 31, 3]
    table, free, spare = _setup(past, block, 8, 30, 7)
    t, f, n, p = _i32(table), _i32(free), _i32([spare]), _i32(past)
    new = _i32([1, 1, 0, 1, 1])
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        kda.kda_cache_plan(p.clone(), new, t.clone(), f.clone(), n.clone(), block, 6)
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = kda.kda_cache_plan(p, new, t, f, n, block, 6, n_free_out=n)
        p.copy_(got["context_lens"])
    for _ in range(40):
        want = R.plan(past, [1, 1, 0, 1, 1], table, free, spare, block, 6)
        g.replay()
        torch.cuda.synchronize()
        for name in ("cu_seqlens", "context_lens", "positions", "slots", "status"):
            assert got[name].tolist() == want[name], name
        table, free, spare = want["block_table"], want["free_blocks"], want["n_free"][0]
        past = want["context_lens"]
        assert n.tolist() == [spare] and t.tolist() == table and f.tolist() == free


def test_binding_refusals():
    p, t, f, n = _i32([1, 2]), _i32([[0, 1], [2, 3]]), _i32([4, 5]), _i32([2])
    for bad in (lambda: kda.kda_cache_plan(p, p[:1], t, f, n, 16, 4),
                lambda: kda.kda_cache_plan(p.long(), p, t, f, n, 16, 4),
                lambda: kda.kda_cache_plan(p, p.clone(), t[:1], f, n, 16, 4),
                lambda: kda.kda_cache_plan(p, p.clone(), t, f, f, 16, 4),
                lambda: kda.kda_cache_plan(p, p.clone(), t, f, n, 20, 4),
                lambda: kda.kda_cache_plan(p, p.clone(), t, f, n, 16, -1),
                lambda: kda.kda_cache_plan(p, p.clone(), t.t(), f, n, 16, 4),
                lambda: kda.kda_cache_plan(p, p.clone(), t, f, n, 16, 4, n_free_out=f[:1])):
        with pytest.raises((ValueError, TypeError, kda.KDAError)):
            bad()
