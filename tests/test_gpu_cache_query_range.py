"""Queries whose channels differ far in size: a row's small channels count as they should beside
one that is 2^8 to 2^24 times as large, in every form of the attention over the cache."""
import numpy as np
import pytest
import torch

import cache_reference as R
import kimi_delta_attention_12_gb300 as kda
from test_gpu_cache_attention import Batch, _tensor_cores

pytestmark = pytest.mark.gpu

LARGE = 5       # the channel


def _batch(past, new, block, Hq, H, d, dtype, k, keys):
    """Channel LARGE of every query is 2^k or -2^k; the keys there are 0, or 0 and the smallest
    e4m3 numbers."""
    b = Batch(past, new, block, Hq, H, d, dtype, seed=k)
    g = torch.Generator().manual_seed(k)
    sign = torch.randint(0, 2, b.q.shape[:2], generator=g).float() * 2 - 1
    b.q[..., LARGE] = (sign * 2.0 ** k).to(dtype)
    small = torch.zeros(b.k.shape[:-1], dtype=torch.uint8)
    if keys == "small":
        small = torch.randint(0, 2, small.shape, generator=g).to(torch.uint8)
    b.k[..., LARGE] = torch.where(b.k[..., LARGE] == 0x7f, b.k[..., LARGE], small)
    return b


def _check(b, got):
    """R.attention_bound allows 2^-22 of each product, which does not grow with the large channel
    where its keys are 0.  Beyond it, a channel of an fp32 query is held to 2^-39 of its row's
    largest: that comes to [2^14, 2^15), and the second half of a channel, an fp16 number, is off by
    2^-25 at most.  A score is then off by scale 2^-39 2^k sum |key|, a weight by that and the sum
    of weights by that again.  A channel of a bf16 query is exact: 8 bits, the last of them 2^-24 or
    more for what is at least 2^-31 of the largest.  (Smaller channels than that are below 2^-7 here:
    they are off by 2^-25, as those of fp32 queries are.)"""
    o, mass, size, least = R.attention(b.q, b.k.numpy(), b.v.numpy(), b.ks.numpy(), b.vs.numpy(),
                                       b.table, b.context, b.cu, b.scale, b.block)
    bound = R.attention_bound(o, mass, size, least, b.d, max(b.context + [1]),
                              b.q.dtype == torch.bfloat16)
    bytes_ = b.k.numpy()
    most_key = np.nan_to_num(np.abs(R.e4m3_values(bytes_))).sum(-1) * b.ks.numpy()[..., None]
    top = b.q.double().abs().amax(-1, keepdim=True).numpy()
    bound = bound + mass * 2 * b.scale * 2.0 ** -39 * top * most_key.max()
    off = np.abs(got.double().cpu().numpy() - o)
    worst = np.argwhere(~(off <= bound))[:4].tolist()
    assert not worst, (worst, [float(off[tuple(w)] / bound[tuple(w)]) for w in worst])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("k,keys", [(8, "none"), (12, "none"), (16, "none"), (20, "none"),
                                    (24, "none"), (8, "small"), (12, "small")])
def test_one_large_channel_among_few_rows(k, keys, d, dtype):
    b = _batch([200, 40, 0], [1, 3, 2], 32, 8, 2, d, dtype, k, keys)
    args = b.args()
    _check(b, kda.kda_cache_attention(*args, max_new=1))                         # clusters
    _check(b, kda.kda_cache_attention(*args[:5], b.wide(), *args[6:], max_new=3))  # stretches


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("k,keys", [(8, "none"), (12, "none"), (16, "none"), (20, "none"),
                                    (24, "none"), (8, "small"), (12, "small")])
def test_one_large_channel_on_the_tensor_cores(k, keys, d):
    b = _batch([60, 3], [90, 130], 16, 16, 4, d, torch.bfloat16, k, keys)
    args, most = _tensor_cores(b)
    _check(b, kda.kda_cache_attention(*args, max_new=most))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_the_largest_and_the_smallest_queries(dtype):
    """Exponents at both ends of the type's range, whole rows and single channels."""
    b = Batch([90], [4], 32, 4, 2, 64, dtype, seed=2)
    most = torch.finfo(dtype).max
    b.q[0] = b.q[0].sign() * most                 # every channel the largest number
    b.q[1] *= 2.0 ** -126                         # and around the smallest normal ones
    b.q[2] = 0.0
    b.q[2, :, LARGE] = most
    b.q[3] *= 2.0 ** -112
    b.scale = 2.0 ** -130
    _check(b, kda.kda_cache_attention(*b.args(), scale=b.scale))
    b.scale = 2.0 ** 100
    b.q[0] = 0.0
    b.q[2] = 0.0
    _check(b, kda.kda_cache_attention(*b.args(), scale=b.scale))
    c = Batch([90], [140], 16, 16, 4, 64, torch.bfloat16, seed=3)
    c.q[0] = c.q[0].sign() * torch.finfo(torch.bfloat16).max
    c.q[1:100] *= 2.0 ** -126
    c.scale = 2.0 ** -130
    _check(c, kda.kda_cache_attention(*_tensor_cores(c)[0], max_new=140, scale=c.scale))
