"""Softmax attention over the paged 8-bit cache on the GPU against sums in 64 bits."""
import random

import numpy as np
import pytest
import torch

import cache_reference as R
import kimi_delta_attention_12_gb300 as kda

pytestmark = pytest.mark.gpu


class Batch:
    """Requests with `past` cached and `new` new tokens, in a pool with blocks in no order."""

    def __init__(self, past, new, block, Hq, H, d, dtype, seed=0, spread=2, q_size=1.0):
        g = torch.Generator().manual_seed(seed)
        self.past, self.new, self.block, self.d = past, new, block, d
        self.context = [p + n for p, n in zip(past, new)]
        need = [-(-max(c, 0) // block) for c in self.context]
        nb, W = sum(need) + 2, max(need) + 1
        ids = list(range(nb))
        random.Random(seed).shuffle(ids)
        self.table = [[ids.pop() for _ in range(n)] + [nb + 5] * (W - n) for n in need]
        self.cu = [0]
        for n in new:
            self.cu.append(self.cu[-1] + n)
        raw = [(torch.randn(nb, H, block, d, generator=g) * 90).clamp(-448, 448)
               .to(torch.float8_e4m3fn).view(torch.uint8) for _ in range(2)]
        for i, c in enumerate(self.context):       # what lies behind a request is NaN
            if c > 0 and c % block:
                for r in raw:
                    r[self.table[i][c // block], :, c % block:] = 0x7f
        self.k, self.v = raw
        self.ks, self.vs = (torch.exp2(torch.randint(-6 - spread, -6 + spread + 1, (nb, H),
                                                     generator=g).float()) for _ in range(2))
        self.q = (q_size * torch.randn(self.cu[-1], Hq, d, generator=g)).to(dtype)
        self.scale = d ** -0.5

    def args(self):
        i32 = dict(dtype=torch.int32, device="cuda")
        return (self.q.cuda(), self.k.cuda().view(torch.float8_e4m3fn),
                self.v.cuda().view(torch.float8_e4m3fn), self.ks.cuda(), self.vs.cuda(),
                torch.tensor(self.table, **i32), torch.tensor(self.context, **i32),
                torch.tensor(self.cu, **i32))

    def wide(self):
        """A table too wide for the clusters, which would leave a warp too many tokens."""
        t = torch.full((len(self.table), (1 << 16) // self.block), -1, dtype=torch.int32)
        t[:, :len(self.table[0])] = torch.tensor(self.table, dtype=torch.int32)
        return t.cuda()

    def check(self, got):
        o, *sizes = R.attention(self.q, self.k.numpy(), self.v.numpy(), self.ks.numpy(),
                                self.vs.numpy(), self.table, self.context, self.cu, self.scale,
                                self.block)
        bound = R.attention_bound(o, *sizes, self.d, max(self.context + [1]),
                                  self.q.dtype == torch.bfloat16)
        got, nan = got.double().cpu().numpy(), np.isnan(o)
        assert np.array_equal(np.isnan(got), nan)
        off = np.abs(got - o)
        worst = np.argwhere(~(off <= bound) & ~nan)[:4].tolist()
        assert not worst, (worst, [float(off[tuple(w)] / bound[tuple(w)]) for w in worst])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("G", [1, 4, 5, 8, 16])
def test_single_tokens(G, d, dtype):
    block = {32: 16, 64: 32, 128: 64}[d]
    past = [0, 1, 14, 15, 16, 17, 63, 64, 200, 701]
    b = Batch(past, [1] * len(past), block, 2 * G, 2, d, dtype, seed=G)
    args = b.args()
    b.check(kda.kda_cache_attention(*args[:-1]))        # few items: clusters
    b.check(kda.kda_cache_attention(*args, max_new=1))
    b.check(kda.kda_cache_attention(*args[:5], b.wide(), args[6]))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("N,H,G,d,new", [(1, 1, 4, 128, 1), (1, 3, 8, 64, 2), (2, 8, 2, 128, 3),
                                         (5, 7, 1, 32, 5), (3, 25, 16, 64, 1), (1, 9, 7, 128, 2),
                                         (1, 1, 64, 32, 1)])
def test_few_items(N, H, G, d, new, dtype):
    """Clusters of every size, tiles of one and two columns of eight, and the even stretches."""
    past = [random.Random(i).choice([0, 5, 300, 1500, 4000]) for i in range(N)]
    b = Batch(past, [new] * N, 32, G * H, H, d, dtype, seed=N + H)
    args = b.args()
    b.check(kda.kda_cache_attention(*args, max_new=new))
    b.check(kda.kda_cache_attention(*args[:5], b.wide(), *args[6:], max_new=new))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("block", [16, 32, 64, 128])
@pytest.mark.parametrize("Hq,H,d", [(3, 3, 64), (10, 2, 32), (8, 1, 128)])
def test_prompts_and_pieces(Hq, H, d, block, dtype):
    b = Batch([0, 100, 0, 37, 300, 5], [33, 7, 1, 0, 20, 130], block, Hq, H, d, dtype, seed=block)
    args = b.args()
    whole = kda.kda_cache_attention(*args)
    b.check(whole)
    for most in (1, 130):        # says which kernels, not what
        b.check(kda.kda_cache_attention(*args, max_new=most))


def _tensor_cores(b):
    """The batch's arguments with a table that can hold so much that its prompts go to the tensor
    cores' kernel, and the most new tokens."""
    rows, H = b.q.shape[0] * b.q.shape[1], b.ks.shape[1]
    assert rows >= 1024 and max(b.new) * b.q.shape[1] // H >= 64 and rows << 16 >= 1 << 24
    args = b.args()
    return (*args[:5], b.wide(), *args[6:]), max(b.new)


@pytest.mark.parametrize("past,new,block,Hq,H,d", [
    ([0], [130], 16, 32, 8, 128),               # one request: nothing for the other kernel
    ([0], [257], 64, 16, 16, 64),
    ([1000], [90], 128, 64, 4, 128),
    ([5, 300, 0, 77], [140, 1, 0, 129], 32, 32, 8, 128),      # prompts and single tokens
    ([40, 0, 900], [333, 64, 15], 16, 20, 4, 64),
    ([0, 0, 0], [1, 600, 2], 64, 7, 1, 128),
    ([127, 128, 129], [128, 127, 129], 16, 12, 2, 64),
])
def test_prompts_on_the_tensor_cores(past, new, block, Hq, H, d):
    b = Batch(past, new, block, Hq, H, d, torch.bfloat16, seed=sum(new))
    args, most = _tensor_cores(b)
    room = kda.cache_attention_workspace_bytes(b.q.shape[0], max(new), Hq, H, d, torch.bfloat16)
    ws = torch.full((room,), 255, dtype=torch.uint8, device="cuda")
    got = kda.kda_cache_attention(*args, max_new=most, workspace=ws)
    b.check(got)
    assert kda.workspace_status(ws) == kda.KDA_OK
    assert torch.equal(got, kda.kda_cache_attention(*args, max_new=most))
    b.check(kda.kda_cache_attention(*args, max_new=1))    # the other kernel, all rows


@pytest.mark.parametrize("d", [64, 128])
def test_extremes_on_the_tensor_cores(d):
    b = Batch([60, 0], [130, 100], 16, 32, 8, d, torch.bfloat16, seed=d)
    b.vs = torch.exp2(torch.randint(-60, 61, b.vs.shape,
                                    generator=torch.Generator().manual_seed(7)).float())
    args, most = _tensor_cores(b)
    b.check(kda.kda_cache_attention(*args, max_new=most))
    b.vs.fill_(1.0)
    b.q[::3] *= 1e30
    b.q[1::3] *= 1e-30
    b.q[2, 0] = 0.0
    for scale in (1e-30, 0.0, -0.3, 3.0):
        if scale in (-0.3, 3.0):
            b.q = torch.randn(b.q.shape, generator=torch.Generator().manual_seed(1)).bfloat16()
        b.scale = scale
        b.check(kda.kda_cache_attention(*_tensor_cores(b)[0], max_new=most, scale=scale))


@pytest.mark.parametrize("past,new,Hq,H,d", [
    ([900] * 30 + [0], [1] * 30 + [150], 32, 8, 128),           # singles beside a short prompt
    ([0, 300, 5, 70, 1200], [400, 1, 7, 0, 1], 16, 2, 64),      # the prompt first
    ([100, 200, 300], [90, 200, 130], 8, 4, 128),               # prompts alone
    ([0] * 4 + [40], [3, 15, 2, 1, 200], 16, 1, 64),
])
def test_both_kernels_of_a_batch_back_to_back(past, new, Hq, H, d):
    """The kernels of a call overlap; calls that share a workspace, eager and in a graph, do not."""
    b = Batch(past, new, 32, Hq, H, d, torch.bfloat16, seed=sum(new))
    c = Batch(past[::-1], new[::-1], 32, Hq, H, d, torch.bfloat16, seed=1 + sum(new))
    (x, most), (y, _) = _tensor_cores(b), _tensor_cores(c)
    room = kda.cache_attention_workspace_bytes(b.q.shape[0], most, Hq, H, d, torch.bfloat16)
    ws = torch.full((room,), 255, dtype=torch.uint8, device="cuda")
    outs = [[torch.full_like(x[0], 7) for _ in range(2)] for _ in range(6)]

    def calls(pair):
        kda.kda_cache_attention(*x, max_new=most, workspace=ws, o=pair[0])
        kda.kda_cache_attention(*y, max_new=most, workspace=ws, o=pair[1])

    for pair in outs[:5]:
        calls(pair)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls(outs[5])
        calls(outs[5])
    graph.replay()
    graph.replay()
    b.check(outs[0][0])
    c.check(outs[0][1])
    for pair in outs[1:]:
        assert torch.equal(pair[0], outs[0][0]) and torch.equal(pair[1], outs[0][1])
    assert kda.workspace_status(ws) == kda.KDA_OK


def test_growing_scores_on_the_tensor_cores():
    """Scores that rise along the keys: the running maximum moves at every step."""
    b = Batch([900], [128], 64, 32, 8, 128, torch.bfloat16, seed=3)
    for p in range(1028):
        b.k[b.table[0][p // 64], :, p % 64, :8] = int(p / 1028 * 120)
    b.q[:, :, :8] = b.q[:, :, :8].abs() + 1.0
    b.scale = 0.5
    b.check(kda.kda_cache_attention(*_tensor_cores(b)[0], max_new=128, scale=0.5))


def test_rows_without_keys_on_the_tensor_cores():
    b = Batch([0, 200, 0], [130, 140, 70], 16, 16, 4, 64, torch.bfloat16, seed=8)
    b.context = [0, 100, 30]           # fewer tokens than new ones
    b.table[1][2] = -1
    got = kda.kda_cache_attention(*_tensor_cores(b)[0], max_new=140)
    assert not got[:130].any()
    b.check(got)


def test_a_query_that_is_not_finite_on_the_tensor_cores():
    b = Batch([70, 9], [140, 130], 16, 16, 8, 64, torch.bfloat16, seed=10)
    args, _ = _tensor_cores(b)
    want = kda.kda_cache_attention(*args, max_new=140)
    q = args[0].clone()
    q[1, 2, 5], q[200, 0, 0] = float("nan"), float("inf")
    got = kda.kda_cache_attention(q, *args[1:], max_new=140)
    assert torch.isnan(got[1, 2]).all() and not torch.isfinite(got[200, 0]).any()
    got[1, 2], got[200, 0] = want[1, 2], want[200, 0]
    assert torch.equal(got, want)


def test_long_context_and_many_requests():
    b = Batch([20000, 3], [1, 1], 64, 4, 1, 32, torch.float32, seed=1)
    b.check(kda.kda_cache_attention(*b.args()[:-1]))
    past = [random.Random(2).randint(0, 40) for _ in range(700)]
    b = Batch(past, [1] * 700, 16, 2, 1, 32, torch.bfloat16, seed=3)
    b.check(kda.kda_cache_attention(*b.args()[:-1]))


def test_rows_without_keys_and_rows_behind():
    b = Batch([0, 40, 0, 3], [2, 3, 1, 0], 16, 4, 2, 64, torch.float32, seed=4)
    args = list(b.args())
    b.context[0], b.context[1] = 0, 2         # fewer tokens than new ones: two see none
    args[6] = torch.tensor(b.context, dtype=torch.int32).cuda()
    o = torch.full((9, 4, 64), 7.0, device="cuda")
    b.q = torch.cat((b.q, torch.zeros(3, 4, 64)))
    args[0] = b.q.cuda()
    got = kda.kda_cache_attention(*args, o=o)
    assert got.data_ptr() == o.data_ptr()
    assert bool((o[6:] == 7.0).all())
    assert not o[:2].any() and not o[2].any() and bool(o[3].any())
    b.q = b.q[:6]
    b.check(o[:6])


def test_table_entries_outside_the_pool_are_not_there():
    b = Batch([100, 47], [1, 2], 16, 4, 2, 32, torch.float32, seed=5)
    for row, at, value in ((0, 1, -1), (0, 4, 1 << 30), (1, 0, -7), (1, 1, 10 ** 6)):
        b.table[row][at] = value
    b.check(kda.kda_cache_attention(*b.args()))
    b.table = [[-1] * len(r) for r in b.table]
    assert not kda.kda_cache_attention(*b.args()).any()


def test_lengths_beyond_the_table_and_the_rows():
    b = Batch([60, 10], [1, 1], 16, 2, 1, 32, torch.float32, seed=6)
    args = list(b.args())
    W = len(b.table[0])
    args[6] = torch.tensor([10 ** 9, -4], dtype=torch.int32).cuda()
    args[7] = torch.tensor([0, 1, 50], dtype=torch.int32).cuda()
    got = kda.kda_cache_attention(*args)
    b.context = [W * 16, 0]
    b.check(got)
    args[7] = torch.tensor([2, -9, 1], dtype=torch.int32).cuda()      # nonsense stays inside
    kda.kda_cache_attention(*args)
    torch.cuda.synchronize()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_scales_far_apart(dtype):
    b = Batch([200, 90], [1, 3], 16, 4, 1, 64, dtype, seed=7)
    b.vs = torch.exp2(torch.randint(-60, 61, b.vs.shape,
                                    generator=torch.Generator().manual_seed(7)).float())
    b.check(kda.kda_cache_attention(*b.args()))
    b.vs.fill_(1.7)
    b.ks.fill_(2.0 ** -60)
    b.check(kda.kda_cache_attention(*b.args()))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_large_and_small_queries(dtype):
    b = Batch([150], [3], 32, 4, 2, 64, dtype, seed=8)
    b.q[0] *= 1e30
    b.q[1] *= 1e-30
    b.q[2, 0] = 0.0
    b.scale = 1e-30                      # scores of the first row near 1, of the others near 0
    b.check(kda.kda_cache_attention(*b.args(), scale=b.scale))
    b.scale = 0.0
    b.check(kda.kda_cache_attention(*b.args(), scale=0.0))
    b.q = torch.randn(3, 4, 64, generator=torch.Generator().manual_seed(8)).to(dtype)
    b.scale = -0.3
    b.check(kda.kda_cache_attention(*b.args(), scale=-0.3))


def test_peaked_scores():
    b = Batch([500], [1], 16, 2, 1, 32, torch.float32, seed=9, q_size=8.0)
    b.scale = 1.0
    b.check(kda.kda_cache_attention(*b.args(), scale=1.0))


def test_a_query_that_is_not_finite_spoils_its_own_row():
    b = Batch([70, 9], [2, 1], 16, 4, 2, 64, torch.bfloat16, seed=10)
    args = b.args()
    want = kda.kda_cache_attention(*args)
    q = args[0].clone()
    q[1, 2, 5], q[2, 0, 0] = float("nan"), float("inf")
    got = kda.kda_cache_attention(q, *args[1:])
    assert torch.isnan(got[1, 2]).all() and not torch.isfinite(got[2, 0]).any()
    got[1, 2], got[2, 0] = want[1, 2], want[2, 0]
    assert torch.equal(got, want)


def test_a_strided_query_and_the_same_bits_each_time():
    b = Batch([300, 2, 900], [4, 1, 9], 64, 8, 2, 64, torch.bfloat16, seed=11)
    args = b.args()
    T = b.q.shape[0]
    wide = torch.randn(T, 12 * 64, device="cuda").bfloat16()
    wide[:, 128:128 + 512] = args[0].view(T, 512)
    strided = wide[:, 128:128 + 512].view(T, 8, 64)
    first = kda.kda_cache_attention(*args)
    for _ in range(3):
        assert torch.equal(first, kda.kda_cache_attention(strided, *args[1:]))


def test_streams_and_graphs_with_one_workspace():
    a = Batch([300, 20, 77], [1, 1, 1], 16, 8, 2, 64, torch.bfloat16, seed=12)
    b = Batch([10, 200, 400], [1, 3, 9], 16, 8, 2, 64, torch.bfloat16, seed=13)
    ws = torch.empty(kda.cache_attention_workspace_bytes(13, 13, 8, 2, 64, torch.bfloat16),
                     dtype=torch.uint8, device="cuda")
    xs = [a.args(), b.args()]
    want = [kda.kda_cache_attention(*x) for x in xs]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = kda.kda_cache_attention(*xs[0], stream=s)
    s.synchronize()
    assert torch.equal(got, want[0])
    graphs = []
    for x in xs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = kda.kda_cache_attention(*x, workspace=ws)
        graphs.append((g, out))
    for _ in range(3):
        for g, out in graphs:
            out.zero_()
            g.replay()
    torch.cuda.synchronize()
    for (g, out), w in zip(graphs, want):
        assert torch.equal(out, w)


def test_lengths_change_between_replays():
    b = Batch([500, 40], [1, 1], 16, 4, 1, 32, torch.float32, seed=14)
    args = b.args()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = kda.kda_cache_attention(*args)
    for context in ([501, 41], [1, 1], [37, 0], [480, 16]):
        args[6].copy_(torch.tensor(context, dtype=torch.int32))
        g.replay()
        torch.cuda.synchronize()
        b.context = context
        b.check(out)


def test_binding_refusals():
    b = Batch([30, 4], [1, 1], 16, 4, 2, 64, torch.float32, seed=15)
    q, k, v, ks, vs, t, c, cu = b.args()
    f = kda.kda_cache_attention
    for bad in (lambda: f(q, k, v, ks, vs, t, c[:1], cu), lambda: f(q[:1], k, v, ks, vs, t, c),
                lambda: f(q, k, v, ks, vs, t, c, cu[:2]), lambda: f(q, k, v, ks, vs, t.long(), c),
                lambda: f(q, k.float(), v, ks, vs, t, c), lambda: f(q, k, v, ks[:1], vs, t, c),
                lambda: f(q[:, :3], k, v, ks, vs, t, c), lambda: f(q[..., :32], k, v, ks, vs, t, c),
                lambda: f(q.half(), k, v, ks, vs, t, c), lambda: f(q.cpu(), k, v, ks, vs, t, c),
                lambda: f(q, k, v, ks, vs, t, c, o=q), lambda: f(q, k, v, ks, vs, t, c, max_new=-1),
                lambda: f(q, k, v, ks, vs, t, c, workspace=torch.empty(16, device="cuda")),
                lambda: f(q, k, v, ks, vs, t, c, o=torch.empty_like(q).bfloat16())):
        with pytest.raises((ValueError, TypeError, kda.KDAError)):
            bad()
