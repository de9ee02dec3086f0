"""Host-side checks of the rotary positions and the paged 8-bit cache: the refusals of the C ABI
(nothing is launched) and of the binding, the frequencies, and the references against closed
forms and torch's own e4m3."""
import ctypes
import math

import numpy as np
import pytest
import torch

import cache_reference as R
import kimi_delta_attention_12_gb300 as kda

BASE = 0x7f0000000000   # an aligned fake device address; nothing dereferences it
M = 0x1000000
INV, UNS, ALI, WS = (kda.KDA_ERR_INVALID_ARG, kda.KDA_ERR_UNSUPPORTED, kda.KDA_ERR_ALIGNMENT,
                     kda.KDA_ERR_WORKSPACE)


@pytest.fixture(scope="module")
def L():
    from kimi_delta_attention_12_gb300 import build
    build.build()
    return kda.lib()


def _rotary(L, **over):
    a = dict(q=BASE, qs=256, k=BASE + M, ks=128, pos=BASE + 2 * M, f=BASE + 3 * M, T=8, Hq=4,
             Hk=2, d=64, rot=32, first=16, dt=kda.KDA_F32, flags=0, mag=1.0, qo=BASE + 4 * M,
             qos=256, ko=BASE + 5 * M, kos=128)
    a.update(over)
    return L.kda_rotary(a["q"], a["qs"], a["k"], a["ks"], a["pos"], a["f"], a["T"], a["Hq"],
                        a["Hk"], a["d"], a["rot"], a["first"], a["dt"], a["flags"], a["mag"],
                        a["qo"], a["qos"], a["ko"], a["kos"], None)


@pytest.mark.parametrize("over,expect", [
    (dict(dt=2), UNS), (dict(d=60), UNS), (dict(d=520), UNS), (dict(d=0), UNS),
    (dict(rot=8), UNS), (dict(rot=24), UNS), (dict(rot=64), UNS), (dict(first=4), UNS),
    (dict(first=-8), UNS), (dict(first=40), UNS),
    (dict(first=0x7ffffff8, rot=16), UNS), (dict(first=16, rot=0x7ffffff0), UNS),
    (dict(T=-1), INV), (dict(Hq=0), INV), (dict(Hk=-1), INV), (dict(flags=1), INV),
    (dict(flags=128), INV), (dict(mag=float("nan")), INV), (dict(mag=float("inf")), INV),
    (dict(f=None), INV), (dict(pos=None), INV), (dict(q=None), INV), (dict(qo=None), INV),
    (dict(k=None), INV), (dict(ko=None), INV), (dict(k=None, ko=None), INV), (dict(Hk=0), INV),
    (dict(qs=252), INV), (dict(qs=258), INV), (dict(qos=255), INV), (dict(ks=127), INV),
    (dict(kos=0), INV), (dict(dt=kda.KDA_BF16, qs=260), INV),
    (dict(q=BASE + 8), ALI), (dict(k=BASE + M + 4), ALI), (dict(qo=BASE + 4 * M + 2), ALI),
    (dict(pos=BASE + 2 * M + 2), ALI), (dict(f=BASE + 3 * M + 1), ALI),
    (dict(qo=BASE + 16), INV), (dict(qo=BASE + M), INV), (dict(ko=BASE), INV),
    (dict(qo=BASE, qos=512), INV),                      # in place with another stride
    (dict(ko=BASE + 4 * M + 512), INV),                 # k_out inside q_out
    (dict(qo=BASE + 2 * M), INV), (dict(ko=BASE + 3 * M), INV),
    # parts of one buffer of 384 a row: k_out reaches into q's columns
    (dict(qs=384, k=BASE + 1024, ks=384, qo=BASE, qos=384, ko=BASE + 1008, kos=384), INV),
])
def test_rotary_refusals(L, over, expect):
    assert _rotary(L, **over) == expect


def test_rotary_without_rows_launches_nothing(L):
    assert _rotary(L, T=0) == kda.KDA_OK
    assert _rotary(L, T=0, q=None, qo=None, pos=None) == kda.KDA_OK
    assert _rotary(L, T=0, q=None, qo=None, pos=None, k=None, ko=None) == kda.KDA_OK


def _plan(L, **over):
    a = dict(past=BASE, new=BASE + M, N=4, table=BASE + 2 * M, W=8, free=BASE + 3 * M, F=32,
             nf=BASE + 4 * M, nfo=BASE + 5 * M, block=16, T=64, cu=BASE + 6 * M, ctx=BASE + 7 * M,
             pos=BASE + 8 * M, slots=BASE + 9 * M, st=BASE + 10 * M)
    a.update(over)
    return L.kda_cache_plan(a["past"], a["new"], a["N"], a["table"], a["W"], a["free"], a["F"],
                            a["nf"], a["nfo"], a["block"], a["T"], a["cu"], a["ctx"], a["pos"],
                            a["slots"], a["st"], None)


@pytest.mark.parametrize("over,expect", [
    (dict(block=8), UNS), (dict(block=48), UNS), (dict(block=256), UNS),
    (dict(N=0), INV), (dict(T=-1), INV), (dict(W=0), INV), (dict(F=0), INV),
    (dict(N=0x7fff0001), UNS), (dict(T=0x7fff0001), UNS),
    (dict(past=None), INV), (dict(new=None), INV), (dict(table=None), INV), (dict(free=None), INV),
    (dict(nf=None), INV), (dict(nfo=None), INV), (dict(cu=None), INV), (dict(ctx=None), INV),
    (dict(pos=None), INV), (dict(slots=None), INV), (dict(st=None), INV),
    (dict(past=BASE + 2), ALI), (dict(slots=BASE + 9 * M + 1), ALI),
    (dict(table=BASE), INV), (dict(free=BASE + 2 * M + 64), INV), (dict(cu=BASE + 6 * M - M), INV),
    (dict(slots=BASE + 8 * M + 252), INV), (dict(ctx=BASE), INV), (dict(st=BASE + M), INV),
    (dict(nfo=BASE + 3 * M), INV), (dict(pos=BASE + 4 * M), INV),
])
def test_plan_refusals(L, over, expect):
    assert _plan(L, **over) == expect


def _write(L, **over):
    a = dict(k=BASE, ks=128, v=BASE + M, vs=128, slots=BASE + 2 * M, T=8, H=2, d=64,
             dt=kda.KDA_F32, kc=BASE + 3 * M, vc=BASE + 4 * M, ksc=BASE + 5 * M, vsc=BASE + 6 * M,
             nb=16, block=16)
    a.update(over)
    return L.kda_cache_write(a["k"], a["ks"], a["v"], a["vs"], a["slots"], a["T"], a["H"], a["d"],
                             a["dt"], a["kc"], a["vc"], a["ksc"], a["vsc"], a["nb"], a["block"],
                             None)


@pytest.mark.parametrize("over,expect", [
    (dict(dt=3), UNS), (dict(d=48), UNS), (dict(d=256), UNS), (dict(block=24), UNS),
    (dict(H=0), INV), (dict(nb=0), INV), (dict(T=-1), INV), (dict(nb=1 << 27), INV),
    (dict(T=0x7fff0001), UNS),
    (dict(k=None), INV), (dict(v=None), INV), (dict(slots=None), INV), (dict(kc=None), INV),
    (dict(vc=None), INV), (dict(ksc=None), INV), (dict(vsc=None), INV),
    (dict(ks=124), INV), (dict(vs=130), INV),
    (dict(k=BASE + 4), ALI), (dict(vc=BASE + 4 * M + 8), ALI), (dict(slots=BASE + 2 * M + 2), ALI),
    (dict(vsc=BASE + 6 * M + 2), ALI),
    (dict(kc=BASE), INV), (dict(vc=BASE + 3 * M + 16), INV), (dict(ksc=BASE + 3 * M + 32), INV),
    (dict(vsc=BASE + 5 * M), INV), (dict(kc=BASE + 2 * M), INV),
])
def test_write_refusals(L, over, expect):
    assert _write(L, **over) == expect


def test_write_without_rows_launches_nothing(L):
    assert _write(L, T=0, k=None, v=None, slots=None) == kda.KDA_OK


def _attention(L, **over):
    a = dict(q=BASE, qs=256, kc=BASE + M, vc=BASE + 2 * M, ksc=BASE + 3 * M, vsc=BASE + 4 * M,
             nb=16, block=16, table=BASE + 5 * M, W=4, ctx=BASE + 6 * M, cu=None, N=4, T=4, most=1,
             Hq=4, H=2, d=64, dt=kda.KDA_F32, scale=0.125, o=BASE + 7 * M, ws=BASE + 8 * M,
             ws_bytes=0x1000000)
    a.update(over)
    return L.kda_cache_attention(a["q"], a["qs"], a["kc"], a["vc"], a["ksc"], a["vsc"], a["nb"],
                                 a["block"], a["table"], a["W"], a["ctx"], a["cu"], a["N"], a["T"],
                                 a["most"], a["Hq"], a["H"], a["d"], a["dt"], a["scale"], a["o"],
                                 a["ws"], a["ws_bytes"], None)


@pytest.mark.parametrize("over,expect", [
    (dict(dt=2), UNS), (dict(d=96), UNS), (dict(block=8), UNS),
    (dict(Hq=130, qs=130 * 64), UNS), (dict(N=0x7fff0001, T=0x7fff0001), UNS),
    (dict(N=0x7fff0001, cu=BASE + 9 * M), UNS),
    (dict(H=0), INV), (dict(Hq=5, qs=320), INV), (dict(Hq=1, qs=64), INV), (dict(N=0), INV),
    (dict(T=-1), INV), (dict(T=5), INV), (dict(most=-1), INV), (dict(W=0), INV),
    (dict(nb=0), INV), (dict(nb=1 << 28), INV), (dict(scale=float("nan")), INV),
    (dict(scale=float("inf")), INV), (dict(q=None), INV), (dict(o=None), INV),
    (dict(kc=None), INV), (dict(vsc=None), INV), (dict(table=None), INV), (dict(ctx=None), INV),
    (dict(qs=252), INV), (dict(qs=258), INV),
    (dict(ws=None), WS), (dict(ws_bytes=255), WS),
    (dict(q=BASE + 8), ALI), (dict(o=BASE + 7 * M + 8), ALI), (dict(ws=BASE + 8 * M + 128), ALI),
    (dict(table=BASE + 5 * M + 2), ALI), (dict(ctx=BASE + 6 * M + 1), ALI),
    (dict(cu=BASE + 9 * M + 2), ALI),
    (dict(o=BASE), INV), (dict(o=BASE + M), INV), (dict(o=BASE + 4 * M), INV),
    (dict(ws=BASE + 5 * M), INV), (dict(ws=BASE + 7 * M), INV), (dict(ws=BASE + 2 * M), INV),
])
def test_attention_refusals(L, over, expect):
    assert _attention(L, **over) == expect


def test_workspace_size_is_zero_for_bad_sizes(L):
    size = L.kda_cache_attention_workspace_bytes
    assert size(4, 1, 8, 2, 64, kda.KDA_BF16) > 0
    for a in ((4, 1, 8, 3, 64, 1), (4, 1, 1, 2, 64, 1), (4, 1, 8, 0, 64, 1), (4, 1, 8, 2, 48, 1),
              (4, 1, 8, 2, 64, 2), (4, 1, 130, 2, 64, 1), (-1, 1, 8, 2, 64, 1),
              (4, -1, 8, 2, 64, 1)):
        assert size(*a) == 0


@pytest.mark.parametrize("scaling,factor", [(None, 1.0), ("linear", 8.0), ("by_parts", 8.0),
                                            ("by_parts", 1.0)])
def test_frequencies(L, scaling, factor):
    rot, base, length = 64, 1e4, 4096.0
    f, m = kda.rotary_frequencies(rot, base, scaling, factor, length, device="cpu")
    for j in range(rot // 2):
        want = base ** (-2 * j / rot)
        if scaling == "linear":
            want /= factor
        elif scaling == "by_parts":
            turns = length * want / (2 * math.pi)
            w = min(1.0, max(0.0, (turns - 1.0) / 31.0))
            want = want * w + (1 - w) * want / factor
        assert abs(float(f[j]) - want) <= 2.0 ** -23 * want
    assert abs(m - (0.1 * math.log(factor) + 1.0 if scaling == "by_parts" else 1.0)) < 1e-6


@pytest.mark.parametrize("args", [
    (0, 1e4, 0, 1.0, 1.0, 32.0, 1.0), (3, 1e4, 0, 1.0, 1.0, 32.0, 1.0),
    (70000, 1e4, 0, 1.0, 1.0, 32.0, 1.0), (16, 0.0, 0, 1.0, 1.0, 32.0, 1.0),
    (16, float("nan"), 0, 1.0, 1.0, 32.0, 1.0), (16, 1e4, 3, 1.0, 1.0, 32.0, 1.0),
    (16, 1e4, 1, 0.0, 1.0, 32.0, 1.0), (16, 1e4, 2, 8.0, 0.0, 32.0, 1.0),
    (16, 1e4, 2, 8.0, 4096.0, 1.0, 1.0), (16, 1e4, 2, 8.0, 4096.0, 32.0, 0.0),
])
def test_frequencies_refusals(L, args):
    out, m = (ctypes.c_float * 64)(), ctypes.c_float()
    assert L.kda_rotary_frequencies(*args, ctypes.addressof(out), ctypes.addressof(m)) == INV


def test_frequencies_binding_refuses_an_unknown_scaling():
    with pytest.raises(ValueError):
        kda.rotary_frequencies(64, scaling="other", device="cpu")


def test_binding_refuses_host_tensors():
    x = torch.zeros(2, 4, 64)
    i = torch.zeros(2, dtype=torch.int32)
    c = torch.zeros(2, 4, 16, 64).to(torch.float8_e4m3fn)
    s = torch.ones(2, 4)
    with pytest.raises(ValueError):
        kda.kda_rotary(x, None, i, torch.zeros(32))
    with pytest.raises(ValueError):
        kda.kda_cache_plan(i, i, i[None].expand(2, 2).contiguous(), i, i[:1], 16, 4)
    with pytest.raises(ValueError):
        kda.kda_cache_write(x, x, i, c, c.clone(), s, s.clone())
    with pytest.raises(ValueError):
        kda.kda_cache_attention(x, c, c, s, s, i[None].expand(2, 2).contiguous(), i)


# ------------------------------------------------------------- the references themselves
def test_reference_bytes_are_torchs_e4m3():
    every = np.arange(256, dtype=np.uint8)
    mine = R.e4m3_values(every)
    torchs = torch.from_numpy(every).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(mine, torchs, equal_nan=True)
    x = np.concatenate([np.linspace(-460, 460, 4001), R.E4M3, (R.E4M3[1:] + R.E4M3[:-1]) / 2,
                        2.0 ** -np.arange(4, 14), [0.0, 2.0 ** -10, 3 * 2.0 ** -11]])
    t = torch.from_numpy(x.astype(np.float32)).clamp(-448, 448).to(torch.float8_e4m3fn)
    assert np.array_equal(R.e4m3_values(R.e4m3_bytes(x.astype(np.float32).astype(np.float64))),
                          t.double().numpy())


def test_reference_rotary_is_a_rotation():
    g = torch.Generator().manual_seed(0)
    x = torch.randn(5, 2, 64, generator=g, dtype=torch.float64)
    pos = torch.tensor([0, 1, 7, 1 << 20, 99], dtype=torch.int32)
    f = torch.tensor([10000.0 ** (-j / 16) for j in range(16)])
    for inter in (False, True):
        y = R.rotary(x, pos, f, inter, 16, 1.0)
        assert torch.equal(y[0], x[0])
        assert (y.norm(dim=-1) - x.norm(dim=-1)).abs().max() < 1e-12
        assert (R.rotary(y, pos, f, inter, 16, 1.0, inverse=True) - x).abs().max() < 1e-12
        # neighbours in the definition: channel 16 and its partner by hand at position 7
        a = 7.0 * float(f[0])
        w = x[2, 0, 17] if inter else x[2, 0, 32]
        assert abs(float(y[2, 0, 16] - (x[2, 0, 16] * math.cos(a) - w * math.sin(a)))) < 1e-12


def test_reference_attention_of_one_key_is_its_value():
    k = np.zeros((1, 1, 16, 32), np.uint8)
    v = np.arange(16 * 32, dtype=np.uint8).reshape(1, 1, 16, 32) % 120
    one = np.ones((1, 1))
    o, *_ = R.attention(torch.ones(1, 2, 32), k, v, one, one * 2.0, [[0]], [1], [0, 1], 1.0, 16)
    assert np.array_equal(o[0, 0], 2.0 * R.e4m3_values(v[0, 0, 0]))
    o, *_ = R.attention(torch.ones(1, 2, 32), k, v, one, one, [[5]], [3], [0, 1], 1.0, 16)
    assert not o.any()
