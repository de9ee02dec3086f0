"""A pool whose bytes pass 32 bits, and prompts captured in graphs that share a workspace."""
import pytest
import torch

import cache_reference as R
import kimi_delta_attention_12_gb300 as kda

pytestmark = pytest.mark.gpu


def test_blocks_beyond_four_gigabytes():
    """Keys and values written to and read from the last blocks of a pool of 5 GB each, by every
    kernel: a lone token, a prompt, few and many requests."""
    H, block, d, dev = 8, 64, 128, "cuda"
    nb = 82_000
    if torch.cuda.mem_get_info()[0] < 14 << 30:
        pytest.skip("needs 14 GB")
    assert nb * H * block * d > 1 << 32
    k_cache, v_cache = (torch.empty(nb, H, block, d, dtype=torch.float8_e4m3fn, device=dev)
                        for _ in range(2))
    k_scale, v_scale = torch.ones(nb, H, device=dev), torch.ones(nb, H, device=dev)
    i32 = dict(dtype=torch.int32, device=dev)
    table = torch.tensor([[nb - 1, nb - 7, 0], [nb - 3, 1, nb - 2]], **i32)
    g = torch.Generator(device=dev).manual_seed(0)
    past, steps = [0, 0], [[130, 150], [1, 1]]
    kept = [[], []]
    for new in steps:
        rows = sum(new)
        q = torch.randn(rows, 32, d, generator=g, device=dev).bfloat16()
        k, v = (torch.randn(rows, H, d, generator=g, device=dev).bfloat16() for _ in range(2))
        cu = [0, new[0], rows]
        slots = [int(table[i, x // block]) * block + x % block
                 for i in range(2) for x in range(past[i], past[i] + new[i])]
        kda.kda_cache_write(k, v, torch.tensor(slots, **i32), k_cache, v_cache, k_scale, v_scale)
        past = [p + n for p, n in zip(past, new)]
        used = table.flatten().long()
        small = [t[used].view(torch.uint8).cpu().numpy() for t in (k_cache, v_cache)]
        scales = [t[used].cpu().numpy() for t in (k_scale, v_scale)]
        for i in range(2):
            kept[i] += [(k[t].float().cpu(), v[t].float().cpu()) for t in range(cu[i], cu[i + 1])]
            for x, pair in enumerate(kept[i]):
                for c, s, y in zip(small, scales, pair):
                    at = 3 * i + x // block
                    got = torch.from_numpy(R.e4m3_values(c[at, :, x % block]) * s[at][:, None])
                    assert bool(((got - y).abs() <= 2.0 ** -4 * y.abs() + 2.0 ** -9).all())
        want, *sizes = R.attention(q, *small, *scales, [[0, 1, 2], [3, 4, 5]], past, cu, d ** -0.5,
                                   block)
        bound = R.attention_bound(want, *sizes, d, max(past), True)
        wide = torch.cat((table, table.expand(2, 3).repeat(1, 200)), 1)    # other kernels' share
        for most, t in ((max(new), table), (1, table), (max(new), wide), (1, wide)):
            o = kda.kda_cache_attention(q, k_cache, v_cache, k_scale, v_scale, t.contiguous(),
                                        torch.tensor(past, **i32), torch.tensor(cu, **i32),
                                        max_new=most)
            off = abs(o.double().cpu().numpy() - want)
            assert (off <= bound).all()


def test_prompts_in_graphs_that_share_a_workspace():
    from test_gpu_cache_attention import Batch, _tensor_cores
    a = Batch([0, 70], [150, 90], 16, 32, 8, 64, torch.bfloat16, seed=1)
    b = Batch([300], [130], 32, 32, 8, 64, torch.bfloat16, seed=2)
    ws = torch.empty(max(kda.cache_attention_workspace_bytes(x.q.shape[0], max(x.new), 32, 8, 64,
                                                             torch.bfloat16) for x in (a, b)),
                     dtype=torch.uint8, device="cuda")
    graphs = []
    for x in (a, b):
        args, _ = _tensor_cores(x)
        kda.kda_cache_attention(*args, max_new=max(x.new), workspace=ws)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = kda.kda_cache_attention(*args, max_new=max(x.new), workspace=ws)
        graphs.append((g, out, args, x))
    for shorter in (0, 37, 149):
        for g, out, args, x in graphs:
            x.context = [max(p + n - shorter, 0) for p, n in zip(x.past, x.new)]
            args[6].copy_(torch.tensor(x.context, dtype=torch.int32))
            out.zero_()
            g.replay()
        for g, out, args, x in graphs:
            torch.cuda.synchronize()
            x.check(out)
    assert kda.workspace_status(ws) == kda.KDA_OK


def test_many_pieces_of_prompts():
    """More items than blocks, items across blocks, and tiles that do not need all of their steps."""
    from test_gpu_cache_attention import Batch, _tensor_cores
    b = Batch([0, 600], [700, 40], 64, 64, 16, 64, torch.bfloat16, seed=3)
    b.check(kda.kda_cache_attention(*_tensor_cores(b)[0], max_new=700))
    b = Batch([2000], [260], 128, 32, 2, 128, torch.bfloat16, seed=4)
    b.check(kda.kda_cache_attention(*_tensor_cores(b)[0], max_new=260))
