"""Host-side checks of the decayed linear attention and the block norms: every
refusal of the C ABI (nothing is launched), the binding's refusals, and the
64-bit references against differences and closed forms."""
import ctypes

import numpy as np
import pytest
import torch

import kimi_delta_attention_12_gb300 as kda
import lin_reference as R

BASE = 0x7f0000000000   # an aligned fake device address; nothing dereferences it
M = 0x100000
INV, UNS, ALI, WS = (kda.KDA_ERR_INVALID_ARG, kda.KDA_ERR_UNSUPPORTED, kda.KDA_ERR_ALIGNMENT,
                     kda.KDA_ERR_WORKSPACE)


@pytest.fixture(scope="module")
def L():
    from kimi_delta_attention_12_gb300 import build
    build.build()
    return kda.lib()


def _prefill(L, **over):
    a = dict(q=BASE, k=BASE + M, v=BASE + 2 * M, g=BASE + 3 * M, S0=None, cu=None, cu_host=None,
             N=1, T=64, H=2, dk=32, dv=32, dt=kda.KDA_F32, scale=1.0, flags=0, o=BASE + 4 * M,
             Sf=BASE + 5 * M, ws=BASE + 6 * M, ws_bytes=16 * M)
    a.update(over)
    return L.kda_lin_prefill(a["q"], a["k"], a["v"], a["g"], a["S0"], a["cu"], a["cu_host"],
                             a["N"], a["T"], a["H"], a["dk"], a["dv"], a["dt"], a["scale"],
                             a["flags"], a["o"], a["Sf"], a["ws"], a["ws_bytes"], None)


@pytest.mark.parametrize("over,expect", [
    (dict(dk=48), UNS), (dict(dv=256), UNS), (dict(dt=2), UNS),
    (dict(N=0), INV), (dict(H=0), INV), (dict(T=-1), INV), (dict(q=None), INV),
    (dict(v=None), INV), (dict(o=None), INV), (dict(g=None), INV),
    (dict(flags=1), INV), (dict(flags=4), INV), (dict(scale=float("inf")), INV),
    (dict(scale=float("nan")), INV), (dict(N=3), INV),
    (dict(ws=None), WS), (dict(ws_bytes=255), WS),
    (dict(q=BASE + 8), ALI), (dict(o=BASE + 4 * M + 4), ALI), (dict(Sf=BASE + 5 * M + 8), ALI),
    (dict(S0=BASE + 7 * M + 4), ALI), (dict(g=BASE + 3 * M + 2), ALI),
    (dict(cu=BASE + 7 * M + 2), ALI), (dict(ws=BASE + 6 * M + 128), ALI),
    (dict(o=BASE), INV), (dict(o=BASE + 2 * M + 16), INV),          # o on q, o inside v
    (dict(Sf=BASE + 4 * M), INV),                                   # final state on o
    (dict(S0=BASE + 5 * M + 256), INV),                             # the two states half apart
    (dict(ws=BASE + M), INV), (dict(ws=BASE + 4 * M), INV),         # workspace on k, on o
])
def test_prefill_refusals(L, over, expect):
    assert _prefill(L, **over) == expect


@pytest.mark.parametrize("cu", [[1, 64], [0, 63], [0, 40, 30, 64]])
def test_prefill_refuses_bad_host_seqlens(L, cu):
    arr = (ctypes.c_int32 * len(cu))(*cu)
    assert _prefill(L, N=len(cu) - 1, cu=BASE + 7 * M, cu_host=arr) == INV


def test_prefill_of_nothing(L):
    assert _prefill(L, T=0, Sf=None) == kda.KDA_OK      # nothing is launched


def _decode(L, **over):
    a = dict(q=BASE, k=BASE + M, v=BASE + 2 * M, g=BASE + 3 * M, state=BASE + 16 * M, slots=None,
             pool=4, B=4, H=2, dk=128, dv=128, dt=kda.KDA_BF16, scale=1.0, o=BASE + 4 * M)
    a.update(over)
    return L.kda_lin_decode_step(a["q"], a["k"], a["v"], a["g"], a["state"], a["slots"],
                                 a["pool"], a["B"], a["H"], a["dk"], a["dv"], a["dt"],
                                 a["scale"], a["o"], None)


@pytest.mark.parametrize("over,expect", [
    (dict(dk=16), UNS), (dict(dt=3), UNS), (dict(H=0), INV), (dict(B=-1), INV),
    (dict(pool=3), INV), (dict(pool=-1), INV), (dict(state=None), INV), (dict(g=None), INV),
    (dict(o=None), INV), (dict(scale=float("nan")), INV),
    (dict(k=BASE + M + 4), ALI), (dict(state=BASE + 16 * M + 8), ALI),
    (dict(slots=BASE + 5 * M + 2), ALI), (dict(g=BASE + 3 * M + 1), ALI),
    (dict(o=BASE + 16), INV), (dict(o=BASE + 16 * M), INV), (dict(state=BASE + M), INV),
    (dict(B=0), kda.KDA_OK),
])
def test_decode_refusals(L, over, expect):
    assert _decode(L, **over) == expect


def _backward(L, **over):
    a = dict(q=BASE, k=BASE + M, v=BASE + 2 * M, g=BASE + 3 * M, S0=None, cu=None, cu_host=None,
             N=1, T=64, H=2, dk=32, dv=32, dt=kda.KDA_F32, scale=1.0, flags=0, dO=BASE + 4 * M,
             dS=None, dq=BASE + 5 * M, dk_=BASE + 6 * M, dv_=BASE + 7 * M, dS0=BASE + 8 * M,
             ws=BASE + 16 * M, ws_bytes=16 * M)
    a.update(over)
    return L.kda_lin_backward(a["q"], a["k"], a["v"], a["g"], a["S0"], a["cu"], a["cu_host"],
                              a["N"], a["T"], a["H"], a["dk"], a["dv"], a["dt"], a["scale"],
                              a["flags"], a["dO"], a["dS"], a["dq"], a["dk_"], a["dv_"],
                              a["dS0"], a["ws"], a["ws_bytes"], None)


@pytest.mark.parametrize("over,expect", [
    (dict(dk=96), UNS), (dict(dt=9), UNS), (dict(N=0), INV), (dict(T=-5), INV),
    (dict(dO=None), INV), (dict(dq=None), INV), (dict(dv_=None), INV), (dict(g=None), INV),
    (dict(flags=16), INV), (dict(N=5), INV), (dict(scale=float("-inf")), INV),
    (dict(ws=None), WS), (dict(ws_bytes=0), WS),
    (dict(dO=BASE + 4 * M + 8), ALI), (dict(dS0=BASE + 8 * M + 4), ALI),
    (dict(dS=BASE + 9 * M + 4), ALI), (dict(ws=BASE + 16 * M + 64), ALI),
    (dict(dq=BASE + 4 * M), INV), (dict(dk_=BASE + 5 * M), INV),    # on dO, on dq
    (dict(dS=BASE + 8 * M), INV), (dict(ws=BASE + 6 * M), INV),     # dS0 on dS, workspace on dk
])
def test_backward_refusals(L, over, expect):
    assert _backward(L, **over) == expect


def test_lin_workspace_bytes(L):
    for f in (L.kda_lin_prefill_workspace_bytes, L.kda_lin_backward_workspace_bytes):
        assert f(0, 64, 2, 32, 32, kda.KDA_F32) == 0
        assert f(1, 64, 2, 48, 32, kda.KDA_F32) == 0
        assert f(1, 64, 2, 32, 32, 7) == 0
        assert f(1, -1, 2, 32, 32, kda.KDA_F32) == 0
        assert f(1, 0, 1, 128, 128, kda.KDA_BF16) >= 256
        # many pairs fill the machine uncut: no state per segment
        assert f(64, 1 << 20, 64, 128, 128, kda.KDA_BF16) == 256
        # one long sequence is cut; the room stays below a state for each 128 tokens
        b = f(1, 1 << 17, 1, 128, 128, kda.KDA_BF16)
        assert 256 < b <= 256 + (1024 + 1) * 128 * 128 * 4


def _norm(L, **over):
    a = dict(y=BASE, wp=BASE + M, gate=BASE + 2 * M, x=BASE + 3 * M, rs=BASE + 4 * M,
             wn=BASE + 5 * M, rows=4, D=256, group=256, dt=kda.KDA_BF16, act=0, eps=1e-6,
             out=BASE + 6 * M, h=BASE + 7 * M)
    a.update(over)
    return L.kda_block_norm(a["y"], a["wp"], a["gate"], a["x"], a["rs"], a["wn"], a["rows"],
                            a["D"], a["group"], a["dt"], a["act"], a["eps"], a["out"], a["h"],
                            None)


@pytest.mark.parametrize("over,expect", [
    (dict(dt=5), UNS), (dict(D=260, group=260), UNS), (dict(D=16392, group=16392), UNS),
    (dict(group=16), UNS), (dict(D=160, group=64), UNS), (dict(group=512), UNS),
    (dict(rows=-1), INV), (dict(D=0), INV), (dict(group=0), INV), (dict(act=2), INV),
    (dict(eps=0.0), INV), (dict(eps=float("nan")), INV), (dict(eps=-1e-6), INV),
    (dict(y=None), INV), (dict(wp=None), INV), (dict(out=None), INV), (dict(h=None), INV),
    (dict(wn=None), INV),                                  # h without its weights
    (dict(y=BASE + 8), ALI), (dict(wp=BASE + M + 4), ALI), (dict(rs=BASE + 4 * M + 8), ALI),
    (dict(h=BASE + 7 * M + 2), ALI),
    (dict(out=BASE + 16), INV), (dict(h=BASE + 6 * M), INV), (dict(out=BASE + M - 512), INV),
    (dict(rows=0), kda.KDA_OK),
])
def test_norm_refusals(L, over, expect):
    assert _norm(L, **over) == expect


def _norm_backward(L, **over):
    a = dict(y=BASE, wp=BASE + M, gate=BASE + 2 * M, xo=BASE + 3 * M, rs=BASE + 4 * M,
             wn=BASE + 5 * M, dxo=BASE + 6 * M, dh=BASE + 7 * M, rows=4, D=256, group=256,
             dt=kda.KDA_BF16, act=1, eps=1e-6, dy=BASE + 8 * M, dg=BASE + 9 * M,
             dx=BASE + 10 * M, dwp=BASE + 11 * M, drs=BASE + 12 * M, dwn=BASE + 13 * M,
             ws=BASE + 14 * M, ws_bytes=M)
    a.update(over)
    return L.kda_block_norm_backward(
        a["y"], a["wp"], a["gate"], a["xo"], a["rs"], a["wn"], a["dxo"], a["dh"], a["rows"],
        a["D"], a["group"], a["dt"], a["act"], a["eps"], a["dy"], a["dg"], a["dx"], a["dwp"],
        a["drs"], a["dwn"], a["ws"], a["ws_bytes"], None)


@pytest.mark.parametrize("over,expect", [
    (dict(dt=-1), UNS), (dict(group=48), UNS), (dict(rows=-2), INV), (dict(act=-1), INV),
    (dict(eps=0.0), INV), (dict(dy=None), INV), (dict(dg=None), INV), (dict(dwp=None), INV),
    (dict(drs=None), INV), (dict(dwn=None), INV), (dict(dh=None), INV), (dict(xo=None), INV),
    (dict(gate=None), INV), (dict(rs=None), INV), (dict(wn=None), INV),
    (dict(dxo=None, wn=None, dwn=None, dh=None), INV),      # no gradient comes in
    (dict(ws=None), WS), (dict(ws_bytes=16), WS),
    (dict(dy=BASE + 8 * M + 4), ALI), (dict(dwn=BASE + 13 * M + 4), ALI),
    (dict(ws=BASE + 14 * M + 8), ALI),
    (dict(dx=BASE + 6 * M), INV), (dict(dy=BASE), INV), (dict(dg=BASE + 8 * M), INV),
    (dict(ws=BASE + 11 * M), INV),
])
def test_norm_backward_refusals(L, over, expect):
    assert _norm_backward(L, **over) == expect


def test_norm_workspace_bytes(L):
    f = L.kda_block_norm_backward_workspace_bytes
    assert f(0, 256, 256) == 3 * 256 * 4 and f(-1, 256, 256) == 0 and f(4, 260, 260) == 0
    assert f(10 ** 6, 4096, 4096) <= 304 * 3 * 4096 * 4


def test_binding_refuses_cpu_tensors_and_shapes():
    q, g = torch.zeros(4, 1, 32), torch.zeros(1)
    with pytest.raises(ValueError):
        kda.kda_lin_prefill(q, q, q, g)
    with pytest.raises(ValueError):
        kda.kda_lin_decode_step(q, q, q, g, torch.zeros(4, 1, 32, 32))
    with pytest.raises(ValueError):
        kda.kda_lin_backward(q, q, q, g, q)
    with pytest.raises(ValueError):
        kda.kda_block_norm(torch.zeros(2, 32), torch.zeros(32))
    with pytest.raises(ValueError):
        kda.kda_block_norm_backward(torch.zeros(2, 32), torch.zeros(32), torch.zeros(2, 32))


# ----------------------------------------------------------- the references
def test_reference_backward_against_differences():
    x = R.make([5, 0, 3], 2, 4, 3, torch.float64, seed=3, state=True)
    a = {n: R.f64(t) for n, t in x.items() if isinstance(t, torch.Tensor)}
    lens, scale = x["lens"], 0.7
    rng = np.random.RandomState(0)

    def loss(q, k, v, S0):
        o, S = R.lin_forward(q, k, v, a["log_decay"], lens, S0, scale)
        return (o * a["dO"]).sum() + (S * a["dS"]).sum()

    g = R.lin_backward(a["q"], a["k"], a["v"], a["log_decay"], lens, a["dO"], a["S0"], a["dS"],
                       scale)
    args = [a["q"], a["k"], a["v"], a["S0"]]
    for i, name in enumerate(("dq", "dk", "dv", "dS0")):
        step = rng.standard_normal(args[i].shape)
        e = 1e-6
        hi, lo = ([y + s * e * step if j == i else y for j, y in enumerate(args)]
                  for s in (1, -1))
        # the loss is quadratic at most in each argument: a central difference is exact but
        # for rounding, 2^-53 of the loss over the step
        assert abs((loss(*hi) - loss(*lo)) / (2 * e) - (g[name] * step).sum()) < 1e-7


def test_reference_forward_closed_forms():
    # no decay: causal attention without softmax; infinite decay: the token alone
    x = R.make([6], 1, 4, 4, torch.float64, seed=1, state=True)
    a = {n: R.f64(t) for n, t in x.items() if isinstance(t, torch.Tensor)}
    o, S = R.lin_forward(a["q"], a["k"], a["v"], np.zeros(1), [6], None, 2.0)
    att = np.tril(a["q"][:, 0] @ a["k"][:, 0].T)
    assert np.allclose(o[:, 0], 2.0 * att @ a["v"][:, 0], rtol=0, atol=1e-12)
    o, S = R.lin_forward(a["q"], a["k"], a["v"], np.array([-np.inf]), [6], a["S0"], 1.0)
    want = (a["q"][:, 0] * a["k"][:, 0]).sum(1, keepdims=True) * a["v"][:, 0]
    assert np.allclose(o[:, 0], want, rtol=0, atol=1e-12)
    assert np.allclose(S[0, 0], np.outer(a["k"][5, 0], a["v"][5, 0]), rtol=0, atol=1e-12)


def test_reference_norm_against_differences():
    gen = torch.Generator().manual_seed(5)
    n = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64)  # noqa: E731
    y, gate, x, dxo, dh = (n(3, 8) for _ in range(5))
    w_post, rs, w_pre = n(4), n(8), n(8)
    out, h = R.norm_forward(y, w_post, gate, x, rs, w_pre, "silu", 1e-3)
    g = R.norm_backward(y, w_post, dxo, gate, out, rs, w_pre, dh, "silu", 1e-3)
    args = dict(y=y, w_post=w_post, gate=gate, x=x, res_scale=rs, w_pre=w_pre)
    for name, t in args.items():
        step, e = n(*t.shape), 1e-6
        diff = []
        for s in (1, -1):
            o2, h2 = R.norm_forward(**{**args, name: t + s * e * step}, act="silu", eps=1e-3)
            diff.append((o2 * dxo).sum() + (h2 * dh).sum())
        want = (g["d" + name] * step).sum()
        assert abs((diff[0] - diff[1]) / (2 * e) - want) < 1e-6 * max(1.0, abs(want))
