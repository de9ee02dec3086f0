"""Writing the 8-bit cache on the GPU, byte for byte against the definition in 64 bits."""
import random

import numpy as np
import pytest
import torch

import cache_reference as R
import kimi_delta_attention_12_gb300 as kda

pytestmark = pytest.mark.gpu


def _cache(nb, H, block, d, seed):
    g = torch.Generator().manual_seed(seed)
    c = [(torch.randn(nb, H, block, d, generator=g) * 100).clamp(-448, 448)
         .to(torch.float8_e4m3fn).cuda() for _ in range(2)]
    s = [torch.exp2(torch.randint(-9, -4, (nb, H), generator=g).float()).cuda() for _ in range(2)]
    return c, s


def _slots(past, new, block, nb, seed):
    ids = list(range(nb))
    random.Random(seed).shuffle(ids)
    out, rows = [], []
    for p, n in zip(past, new):
        mine = [ids.pop() for _ in range(-(-(p + n) // block))]
        rows += [mine[x // block] * block + x % block for x in range(p, p + n)]
    return rows


def _check(k, v, slots, c, s, block):
    before = [(a.view(torch.uint8).cpu().numpy(), b.cpu().numpy()) for a, b in zip(c, s)]
    kda.kda_cache_write(k, v, torch.tensor(slots, dtype=torch.int32).cuda(), *c, *s)
    for x, a, b, (ca, sc) in zip((k, v), c, s, before):
        want, scales = R.write(x, slots, ca, sc, block)
        got = a.view(torch.uint8).cpu().numpy()
        # a NaN's sign says nothing
        same = (got == want) | (((got & 127) == 127) & ((want & 127) == 127))
        assert same.all(), np.argwhere(~same)[:5]
        assert np.array_equal(b.cpu().numpy().astype(np.float64), scales)


def _data(T, H, d, dtype, seed, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    x = [torch.randn(T, H, d, generator=g) * torch.exp(spread * torch.randn(T, 1, 1, generator=g))
         for _ in range(2)]
    return [t.to(dtype).cuda() for t in x]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("block", [16, 32, 64, 128])
def test_ragged_prompts(block, d, dtype):
    past, new = [0, 5, block, 2 * block - 1, 7, 0], [3 * block + 1, 1, 17, block + 2, 0, 9]
    nb = sum(-(-(p + n) // block) for p, n in zip(past, new)) + 3
    c, s = _cache(nb, 3, block, d, 1)
    _check(*_data(sum(new), 3, d, dtype, 2), _slots(past, new, block, nb, 3), c, s, block)


@pytest.mark.parametrize("N", [1, 7, 130])
def test_decode_tokens(N):
    rng = random.Random(N)
    past, block = [rng.randint(0, 200) for _ in range(N)], 32
    nb = sum(-(-(p + 1) // block) for p in past) + 1
    c, s = _cache(nb, 2, block, 64, N)
    _check(*_data(N, 2, 64, torch.bfloat16, N, 2.0), _slots(past, [1] * N, block, nb, N), c, s,
           block)


def test_many_rows():
    """More rows than one tile of either kind takes, runs across tile borders."""
    past, new, block = [3, 50, 0, 0], [4000, 700, 1, 1500], 64
    nb = sum(-(-(p + n) // block) for p, n in zip(past, new))
    c, s = _cache(nb, 1, block, 32, 0)
    _check(*_data(sum(new), 1, 32, torch.bfloat16, 1), _slots(past, new, block, nb, 2), c, s, block)


def test_a_block_filled_token_by_token():
    """The scale grows with the values; earlier tokens move to it."""
    block, d = 16, 32
    c, s = _cache(2, 1, block, d, 5)
    g = torch.Generator().manual_seed(6)
    for t in range(block):
        k, v = (torch.randn(1, 1, d, generator=g).cuda() * 3.0 ** (t % 7 - 3) for _ in range(2))
        _check(k, v, [16 + t], c, s, block)


def test_extreme_values():
    block, d, H = 16, 32, 1
    c, s = _cache(8, H, block, d, 7)
    k, v = _data(96, H, d, torch.float32, 8)
    k[0:16] = 0.0                                       # a block of zeros
    k[16:32] *= 1e-30                                   # below the least scale
    k[32:48] *= 1e37
    k[48, 0, 3], k[49, 0, 4], k[50, 0, 5] = float("inf"), float("-inf"), float("nan")
    k[64:80] = float("inf")                             # nothing finite
    v[0, 0, 0], v[0:16, 0, 1] = 448.0, -0.0
    v[16:32] = 448.0 * 2.0 ** -3
    v[32:48] = torch.nextafter(torch.tensor(448.0), torch.tensor(500.0))
    _check(k, v, list(range(96)), c, s, block)


def test_scales_that_are_no_powers_of_two():
    """A cache that another program filled: quotients by any scale, rounded once."""
    block, d = 16, 64
    c, s = _cache(4, 2, block, d, 9)
    for t in s:
        t.mul_(1.3)
    k, v = _data(6, 2, d, torch.float32, 10, 1.5)
    slots = [3, 4, 5, 20, 50, 51]
    before = [(a.view(torch.uint8).cpu(), b.cpu()) for a, b in zip(c, s)]
    kda.kda_cache_write(k, v, torch.tensor(slots, dtype=torch.int32).cuda(), *c, *s)
    for x, a, b, (ca, sc) in zip((k, v), c, s, before):
        x = x.cpu()
        for rows, blk, off in ((range(0, 3), 0, 3), (range(3, 4), 1, 4), (range(4, 6), 3, 2)):
            for h in range(2):
                need = R.scale_of(float(x[list(rows), h].abs().max()))
                now = torch.tensor(max(need, float(sc[blk, h])), dtype=torch.float32)
                assert float(b[blk, h]) == float(now)
                new = (x[list(rows), h] / now).clamp(-448, 448).to(torch.float8_e4m3fn)
                got = a[blk, h, off:off + len(rows)].cpu()
                assert torch.equal(got.view(torch.uint8), new.view(torch.uint8))
                old = (ca[blk, h, :off].view(torch.float8_e4m3fn).float() * (sc[blk, h] / now))
                assert torch.equal(a[blk, h, :off].cpu().view(torch.uint8),
                                   old.to(torch.float8_e4m3fn).view(torch.uint8))


def test_slots_left_out():
    c, s = _cache(3, 2, 16, 32, 11)
    k, v = _data(7, 2, 32, torch.float32, 12)
    _check(k, v, [-1, 47, 48, 1 << 30, -5, 16, 17], c, s, 16)


def test_parts_of_one_projection():
    H, d, T = 2, 64, 21
    wide = _data(T, 1, 4 * H * d, torch.bfloat16, 13)[0].view(T, -1)
    k, v = wide[:, H * d:2 * H * d].view(T, H, d), wide[:, 2 * H * d:3 * H * d].view(T, H, d)
    c, s = _cache(2, H, 16, d, 14)
    _check(k, v, list(range(5, 5 + T)), c, s, 16)


def test_streams_and_graph():
    c, s = _cache(4, 2, 16, 32, 15)
    k, v = _data(9, 2, 32, torch.bfloat16, 16)
    slots = torch.arange(10, 19, dtype=torch.int32).cuda()
    c2, s2 = [x.clone() for x in c], [x.clone() for x in s]
    kda.kda_cache_write(k, v, slots, *c, *s)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    kda.kda_cache_write(k, v, slots, *c2, *s2, stream=st)
    st.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kda.kda_cache_write(k, v, slots, *c2, *s2)
    k.mul_(64)
    g.replay()
    kda.kda_cache_write(k, v, slots, *c, *s)
    torch.cuda.synchronize()
    for a, b in zip(c + s, c2 + s2):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_binding_refusals():
    c, s = _cache(2, 2, 16, 32, 17)
    k, v = _data(3, 2, 32, torch.float32, 18)
    i = torch.arange(3, dtype=torch.int32).cuda()
    for bad in (lambda: kda.kda_cache_write(k, v[:2], i, *c, *s),
                lambda: kda.kda_cache_write(k, v, i[:2], *c, *s),
                lambda: kda.kda_cache_write(k, v, i.long(), *c, *s),
                lambda: kda.kda_cache_write(k, v.bfloat16(), i, *c, *s),
                lambda: kda.kda_cache_write(k[:, :1], v[:, :1], i, *c, *s),
                lambda: kda.kda_cache_write(k, v, i, c[0], c[0], *s),
                lambda: kda.kda_cache_write(k, v, i, c[0].float(), c[1], *s),
                lambda: kda.kda_cache_write(k, v, i, *c, s[0], s[1][:1]),
                lambda: kda.kda_cache_write(k.cpu(), v, i, *c, *s),
                lambda: kda.kda_cache_write(k.half(), v.half(), i, *c, *s)):
        with pytest.raises((ValueError, TypeError, kda.KDAError)):
            bad()
