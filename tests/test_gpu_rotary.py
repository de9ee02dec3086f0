"""Rotary positions on the GPU against complex numbers in 64 bits: layouts, parts of the head,
far positions, strides, in place, the backward, streams and graphs."""
import pytest
import torch

import cache_reference as R
import kimi_delta_attention_12_gb300 as kda

pytestmark = pytest.mark.gpu

# An angle carries half a step of a 24-bit half turn (pi 2^-25 = 9.4e-8) and 2^-32 of a turn; its
# cosine and sine 2 steps of 2^-24, the magnitude one, the products and their sum three: in all
# less than 5e-7 of |u| + |w|.
TOL = 5e-7


def _check(got, x, pos, f, inter, first, mag, inverse=False):
    want = R.rotary(x, pos, f, inter, first, mag, inverse)
    bound = TOL * mag * R.rotary_size(x, f, inter, first)
    if x.dtype == torch.bfloat16:
        bound = bound + 2.0 ** -8 * want.abs()
    off = (got.double().cpu() - want).abs()
    assert bool((off <= bound).all()), float((off - bound).max())


def _data(T, H, d, dtype, seed=0):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(T, H, d, generator=g).to(dtype).cuda()


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,Hq,Hk,d,rot,first", [
    (1, 1, 0, 16, 16, 0), (1, 32, 8, 128, 128, 0), (77, 3, 1, 64, 32, 8), (300, 5, 2, 96, 48, 40),
    (1031, 1, 0, 32, 16, 16), (64, 96, 8, 128, 64, 64), (3, 2, 2, 512, 512, 0),
    (2100, 1, 1, 512, 256, 0), (9, 2, 1, 40, 16, 24),
])
def test_sizes(inter, dtype, T, Hq, Hk, d, rot, first):
    q, k = _data(T, Hq, d, dtype), _data(T, Hk, d, dtype, 1) if Hk else None
    pos = torch.randint(0, 1 << 20, (T,), dtype=torch.int32,
                        generator=torch.Generator().manual_seed(T))
    f, _ = kda.rotary_frequencies(rot)
    for call, inverse in ((kda.kda_rotary, False), (kda.kda_rotary_backward, True)):
        qo, ko = call(q, k, pos.cuda(), f, interleaved=inter, first=first, magnitude=1.25)
        _check(qo, q, pos, f, inter, first, 1.25, inverse)
        assert (ko is None) == (k is None)
        if k is not None:
            _check(ko, k, pos, f, inter, first, 1.25, inverse)


def test_far_and_negative_positions_and_odd_frequencies():
    # the reference's product of a 31-bit and a 24-bit number is rounded to 53 bits: 2^-22 of a
    # turn at most where the frequency is 1, less below
    pos = torch.tensor([0, 1, -1, -12345, (1 << 23) + 1, (1 << 24) - 1], dtype=torch.int32)
    f = torch.tensor([1.0, 0.5, 0.1, 3.0, -0.7, 0.0, 1e-30, 1e-38])
    x = _data(len(pos), 2, 16, torch.float32)
    got, _ = kda.kda_rotary(x, None, pos.cuda(), f.cuda())
    _check(got, x, pos, f, False, 0, 1.0)


def test_largest_position_in_exact_arithmetic():
    from fractions import Fraction
    import math
    p, f = (1 << 31) - 1, torch.tensor([0.7, 1.0, 1e-3, 0.33, 2.5, 0.011, 1e-5, 0.9])
    x = torch.zeros(1, 1, 16)
    x[0, 0, :8] = 1.0
    got, _ = kda.kda_rotary(x.cuda(), None, torch.tensor([p], dtype=torch.int32).cuda(), f.cuda())
    two_pi = Fraction(6283185307179586476925286766559005768394338798750211641949889, 10 ** 60)
    for j in range(8):
        turns = Fraction(float(f[j])) * p / two_pi
        a = float(turns - math.floor(turns)) * 2 * math.pi
        # the 64-bit fraction of a turn is off by at most 2^-64 a position
        assert abs(float(got[0, 0, j]) - math.cos(a)) < 1e-6
        assert abs(float(got[0, 0, 8 + j]) - math.sin(a)) < 1e-6


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_parts_of_one_projection_in_place(inter, dtype):
    T, Hq, Hk, d = 133, 6, 2, 64
    wide = _data(T, 1, (Hq + 2 * Hk) * d, dtype).view(T, -1)
    before = wide.clone()
    q = wide[:, :Hq * d].view(T, Hq, d)
    k = wide[:, Hq * d:(Hq + Hk) * d].view(T, Hk, d)
    pos = torch.arange(7, 7 + T, dtype=torch.int32)
    f, _ = kda.rotary_frequencies(32)
    q0, k0 = q.clone(), k.clone()
    apart, apart_k = kda.kda_rotary(q, k, pos.cuda(), f, interleaved=inter, first=16)
    qo, ko = kda.kda_rotary(q, k, pos.cuda(), f, interleaved=inter, first=16, q_out=q, k_out=k)
    assert qo.data_ptr() == q.data_ptr() and ko.data_ptr() == k.data_ptr()
    assert torch.equal(q, apart) and torch.equal(k, apart_k)
    _check(q, q0, pos, f, inter, 16, 1.0)
    _check(k, k0, pos, f, inter, 16, 1.0)
    assert torch.equal(wide[:, (Hq + Hk) * d:], before[:, (Hq + Hk) * d:])
    back, back_k = kda.kda_rotary_backward(q, k, pos.cuda(), f, interleaved=inter, first=16)
    if dtype == torch.float32:
        assert (back - q0).abs().max() < 4 * TOL * float(q0.abs().max())


def test_batch_of_four_dimensions():
    q = _data(12, 3, 32, torch.bfloat16).view(2, 6, 3, 32)
    pos = torch.arange(12, dtype=torch.int32).view(2, 6)
    f, _ = kda.rotary_frequencies(32)
    got, none = kda.kda_rotary(q, None, pos.cuda(), f)
    flat, _ = kda.kda_rotary(q.view(12, 3, 32), None, pos.view(12).cuda(), f)
    assert none is None and torch.equal(got.view(12, 3, 32), flat)


def test_copied_channels_keep_their_bits():
    x = _data(10, 2, 128, torch.float32)
    x[0, 0, 0], x[1, 1, 100] = float("nan"), float("inf")
    f, _ = kda.rotary_frequencies(32)
    got, _ = kda.kda_rotary(x, None, torch.arange(10, dtype=torch.int32).cuda(), f, first=32)
    for part in (slice(0, 32), slice(64, 128)):
        assert torch.equal(got[..., part].view(torch.int32), x[..., part].view(torch.int32))
    assert torch.isfinite(got[..., 32:64]).all()


def test_the_backward_is_the_gradient():
    """Against differences of the 64-bit forward along random directions."""
    x, w = _data(9, 2, 64, torch.float32), _data(9, 2, 64, torch.float32, 5)
    pos = torch.randint(0, 5000, (9,), dtype=torch.int32,
                        generator=torch.Generator().manual_seed(2))
    f, m = kda.rotary_frequencies(32, scaling="by_parts", factor=4.0)
    dx, _ = kda.kda_rotary_backward(w, None, pos.cuda(), f, first=16, magnitude=m)
    for seed in range(3):
        v = _data(9, 2, 64, torch.float32, 10 + seed).double().cpu()
        h = 1e-4

        def loss(t):
            return float((R.rotary(t, pos, f, False, 16, m) * w.double().cpu()).sum())
        want = (loss(x.double().cpu() + h * v) - loss(x.double().cpu() - h * v)) / (2 * h)
        assert abs(float((dx.double().cpu() * v).sum()) - want) < 1e-4 * abs(v).sum()


def test_streams_and_graph():
    q, k = _data(50, 4, 64, torch.bfloat16), _data(50, 1, 64, torch.bfloat16, 1)
    pos = torch.arange(50, dtype=torch.int32).cuda()
    f, _ = kda.rotary_frequencies(64)
    want = kda.kda_rotary(q, k, pos, f)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = kda.kda_rotary(q, k, pos, f, stream=s)
    s.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = kda.kda_rotary(q, k, pos, f)
    q.mul_(2)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out[0].float(), 2 * want[0].float()) and torch.equal(out[1], want[1])


def test_binding_refusals():
    q, k = _data(4, 4, 64, torch.float32), _data(4, 2, 64, torch.float32)
    pos = torch.arange(4, dtype=torch.int32).cuda()
    f, _ = kda.rotary_frequencies(64)
    for bad in (lambda: kda.kda_rotary(q, k[:3], pos, f), lambda: kda.kda_rotary(q, k, pos[:3], f),
                lambda: kda.kda_rotary(q, k, pos.long(), f),
                lambda: kda.kda_rotary(q, k.bfloat16(), pos, f),
                lambda: kda.kda_rotary(q, k, pos, f.double()),
                lambda: kda.kda_rotary(q.transpose(1, 2), None, pos, f),
                lambda: kda.kda_rotary(q[:1].expand(4, 4, 64), None, pos, f),
                lambda: kda.kda_rotary(q, None, pos, f, k_out=k),
                lambda: kda.kda_rotary(q, k, pos, f, q_out=k),
                lambda: kda.kda_rotary(q.cpu(), None, pos, f),
                lambda: kda.kda_rotary(q.half(), None, pos, f),
                lambda: kda.kda_rotary(q, None, pos, f, first=8),
                lambda: kda.kda_rotary(q, None, pos, f[:3]),
                lambda: kda.kda_rotary(q, None, pos, f, q_out=q[:, :, :64].clone().bfloat16())):
        with pytest.raises((ValueError, TypeError, kda.KDAError)):
            bad()
