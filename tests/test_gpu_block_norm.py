"""GPU parity of the block norms against 64-bit autograd of the formulas.

An fp32 value carries a few roundings of its own products and those of a
mean over the row, whose relative error is at most (terms) 2^-24; a stored
bf16 value half a step, 2^-8, more.  A weight's gradient is a sum over rows,
bounded against the sum of its absolute terms."""
import pytest
import torch

import kimi_delta_attention_12_gb300 as kda
import lin_reference as R

pytestmark = pytest.mark.gpu

BF, F = torch.bfloat16, torch.float32

CASES = [
    # rows, D, group, gate, residual, scale, pre, dtype
    (1, 8, 0, "sigmoid", True, True, True, F),
    (3, 32, 32, "silu", False, False, False, BF),
    (7, 40, 0, "none", True, False, True, BF),
    (5, 96, 32, "sigmoid", True, True, True, F),
    (130, 256, 64, "sigmoid", False, False, False, BF),
    (33, 384, 128, "silu", True, True, True, BF),
    (9, 768, 0, "none", False, False, True, F),
    (6, 1000, 0, "silu", True, True, True, F),
    (700, 1024, 128, "sigmoid", False, True, False, BF),
    (401, 2304, 0, "sigmoid", True, True, True, BF),
    (4, 4096, 0, "sigmoid", True, False, True, BF),
    (333, 4096, 0, "sigmoid", True, True, True, BF),
    (607, 4096, 128, "silu", False, True, True, BF),
    (5, 4096, 0, "none", False, True, False, BF),
    (3, 4104, 0, "silu", True, True, True, F),
    (5, 7168, 64, "silu", False, False, True, BF),
    (2, 8200, 0, "sigmoid", True, True, True, BF),
    (3, 12288, 128, "sigmoid", False, False, False, BF),
    (2, 16384, 0, "silu", True, True, True, F),
]
IDS = ["-".join(map(str, c[:4])) + f"-{int(c[4])}{int(c[5])}{int(c[6])}-{str(c[7])[6:]}"
       for c in CASES]


def make(rows, D, group, gate, residual, scale, pre, dtype, seed=0):
    gen = torch.Generator().manual_seed(seed)

    def n(*s):
        return torch.randn(*s, generator=gen)

    return dict(y=(2 * n(rows, D)).to(dtype), w_post=1 + 0.2 * n(group or D),
                gate=n(rows, D).to(dtype) if gate != "none" else None,
                x=n(rows, D).to(dtype) if residual else None,
                res_scale=1 + 0.2 * n(D) if scale else None,
                w_pre=1 + 0.2 * n(D) if pre else None)


def cuda(t):
    return None if t is None else t.cuda()


def near(name, got, want, mag, terms, dtype):
    want = want.double()
    bound = terms * R.U32 * mag + 1e-30
    if dtype == BF:
        bound = bound + R.U16 * (want.abs() + bound)
    bad = ~((got.double().cpu() - want).abs() <= bound)
    assert not bad.any(), (name, int(bad.sum()), bad.numel(),
                           float(((got.double().cpu() - want).abs() / bound).max()))


def forward_mag(x, act, eps):
    """Sizes that the relative roundings apply to: |u|, |x| and what they make."""
    u, _ = R.norm_forward(x["y"], x["w_post"], x["gate"], None, x["res_scale"], None, act, eps)
    out, h = R.norm_forward(x["y"], x["w_post"], x["gate"], x["x"], x["res_scale"], x["w_pre"],
                            act, eps)
    m = u.abs() + (0 if x["x"] is None else x["x"].double().abs())
    if h is None:
        return out, h, m, None
    # h = x' r w: the error of x' and of r, whose mean's terms are squares
    r = 1 / (out.pow(2).mean(-1, keepdim=True) + eps).sqrt()
    mh = m * r * x["w_pre"].double().abs() + h.abs() * (m * m).mean(-1, keepdim=True) * r * r
    return out, h, m, mh


@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_forward(case):
    rows, D, group, gate, residual, scale, pre, dtype = case
    x = make(*case, seed=D)
    o, h = kda.kda_block_norm(cuda(x["y"]), cuda(x["w_post"]), cuda(x["gate"]), cuda(x["x"]),
                              cuda(x["res_scale"]), cuda(x["w_pre"]), gate_act=gate)
    wo, wh, mo, mh = forward_mag(x, gate, 1e-6)
    # products, the sigmoid's few units and half the mean's terms (a square root halves them)
    near("x_out", o, wo, mo, D / 2 + 24, dtype)
    assert (h is None) == (wh is None)
    if h is not None:
        near("h", h, wh, mh, D + 32, dtype)


@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_backward(case):
    rows, D, group, gate, residual, scale, pre, dtype = case
    x = make(*case, seed=D + 1)
    gen = torch.Generator().manual_seed(D)
    dxo = torch.randn(rows, D, generator=gen).to(dtype)
    dh = torch.randn(rows, D, generator=gen).to(dtype) if pre else None
    xo = R.norm_forward(x["y"], x["w_post"], x["gate"], x["x"], x["res_scale"], None, gate)[0]
    xo = xo.to(dtype) if pre else None
    g = kda.kda_block_norm_backward(cuda(x["y"]), cuda(x["w_post"]), cuda(dxo), cuda(x["gate"]),
                                    cuda(xo), cuda(x["res_scale"]), cuda(x["w_pre"]), cuda(dh),
                                    gate_act=gate, residual=residual)
    want = R.norm_backward(x["y"], x["w_post"], dxo, x["gate"], xo, x["res_scale"], x["w_pre"],
                           dh, gate)
    if not residual:
        want.pop("dx")
    assert set(want) == {n for n, t in g.items() if t is not None}
    # magnitudes: the terms of each gradient, their signs dropped
    ye, G = x["y"].double(), group or D
    total = dxo.double().abs()
    if pre:
        r = 1 / (xo.double().pow(2).mean(-1, keepdim=True) + 1e-6).sqrt()
        t = dh.double().abs() * x["w_pre"].double().abs()
        xa = xo.double().abs()
        total = total + r * t + xa * r ** 3 * (t * xa).mean(-1, keepdim=True)
        near("dw_pre", g["dw_pre"], want["dw_pre"], (dh.double().abs() * xa * r).sum(0),
             D + rows + 32, F)
    if residual:
        near("dx", g["dx"], want["dx"], total, D + 32, dtype)
    blocks = ye.unflatten(-1, (-1, G))
    ry = 1 / (blocks.pow(2).mean(-1, keepdim=True) + 1e-6).sqrt()
    ya = blocks.abs()
    n = (ya * ry * x["w_post"].double().abs()).flatten(-2)
    act = torch.ones_like(ye)
    if gate != "none":
        t = x["gate"].double()
        s = torch.sigmoid(t)
        act = s if gate == "sigmoid" else (t * s).abs()
        # 1 - s and 1 + t (1 - s) cancel: their terms, not their values, carry the roundings
        da = s if gate == "sigmoid" else s * (1 + t.abs())
        du = total * (1 if not scale else x["res_scale"].double().abs())
        near("dgate", g["dgate"], want["dgate"], du * n * da, 2 * D + 64, dtype)
    if scale:
        near("dres_scale", g["dres_scale"], want["dres_scale"], (total * n * act).sum(0),
             2 * D + rows + 64, F)
    du = total * act * (1 if not scale else x["res_scale"].double().abs())
    dub = du.unflatten(-1, (-1, G))
    near("dw_post", g["dw_post"], want["dw_post"], (dub * ya * ry).sum((0, 1)),
         2 * D + rows * (D // G) + 64, F)
    dn = dub * x["w_post"].double().abs()
    dy = ry * dn + ya * ry ** 3 * (dn * ya).mean(-1, keepdim=True)
    near("dy", g["dy"], want["dy"], dy.flatten(-2), 3 * D + 64, dtype)


def test_backward_without_stream_gradient_and_empty():
    x = make(12, 256, 0, "silu", True, True, True, F)
    xo = R.norm_forward(x["y"], x["w_post"], x["gate"], x["x"], x["res_scale"], None, "silu")[0]
    xo = xo.float()
    dh = torch.randn(12, 256, generator=torch.Generator().manual_seed(1))
    args = [cuda(x["y"]), cuda(x["w_post"]), None, cuda(x["gate"]), cuda(xo),
            cuda(x["res_scale"]), cuda(x["w_pre"]), cuda(dh)]
    g = kda.kda_block_norm_backward(*args, gate_act="silu")
    want = R.norm_backward(x["y"], x["w_post"], None, x["gate"], xo, x["res_scale"], x["w_pre"],
                           dh, "silu")
    for n in want:
        assert R.rel_fro(g[n], want[n].numpy()) <= 2e-6, n
    none = [t[:0] if t is not None and t.dim() == 2 else t for t in args]
    none[2] = none[0]
    g = kda.kda_block_norm_backward(*none, gate_act="silu")
    for n in ("dw_post", "dres_scale", "dw_pre"):
        assert bool((g[n] == 0).all())
    o, h = kda.kda_block_norm(none[0], args[1], none[3], none[0], args[5], args[6])
    assert o.shape == (0, 256) and h.shape == (0, 256)


def test_rows_of_zeros_and_of_non_numbers():
    x = make(6, 512, 128, "sigmoid", True, True, True, BF)
    x["y"][1] = 0
    x["x"][1] = 0
    for t, v in ((2, float("nan")), (3, float("inf"))):
        x["y"][t, 5] = v
    o, h = kda.kda_block_norm(*(cuda(x[n]) for n in ("y", "w_post", "gate", "x", "res_scale",
                                                     "w_pre")))
    assert bool((o[1] == 0).all()) and bool((h[1] == 0).all())
    assert bool(torch.isfinite(o[[0, 1, 4, 5]]).all() and torch.isfinite(h[[0, 1, 4, 5]]).all())
    # only the head with the bad value, and the whole row after the pre norm
    for t in (2, 3):
        assert torch.isnan(o[t, 5]) and bool(torch.isfinite(o[t, 128:]).all())
        assert torch.isnan(h[t]).all()


def test_in_place_streams_and_graphs():
    x = make(65, 2304, 0, "sigmoid", True, True, True, BF)
    names = ("y", "w_post", "gate", "x", "res_scale", "w_pre")
    a = [cuda(x[n]) for n in names]
    o, h = kda.kda_block_norm(*a)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    o2, h2 = kda.kda_block_norm(*a, stream=side)
    side.synchronize()
    assert torch.equal(o, o2) and torch.equal(h, h2)
    b = [t.clone() for t in a]
    o3, h3 = kda.kda_block_norm(*b, x_out=b[3], h=b[0])
    assert o3 is b[3] and h3 is b[0] and torch.equal(o, o3) and torch.equal(h, h3)
    dxo = torch.randn_like(o)
    bargs = (a[0], a[1], dxo, a[2], o, a[4], a[5], dxo)
    g = kda.kda_block_norm_backward(*bargs)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g2 = kda.kda_block_norm_backward(*bargs)
    for t in g2.values():
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(g[n], g2[n]) for n in g)


def test_more_than_32_bits_of_elements():
    rows, D = 262200, 8192                       # 2.15e9 elements
    if torch.cuda.mem_get_info()[0] < 30e9:
        pytest.skip("needs 30 GB")
    y = torch.ones(rows, D, dtype=BF, device="cuda")
    y[-1] = 3.0
    w = torch.full((128,), 2.0, device="cuda")
    o, _ = kda.kda_block_norm(y, w, x_out=y)
    assert bool((o[-2:] == 2.0).all()) and bool((o[:2] == 2.0).all())


def test_binding_refusals():
    y, w = torch.zeros(4, 64, device="cuda"), torch.ones(64, device="cuda")
    with pytest.raises(ValueError):
        kda.kda_block_norm(y, w, gate=y[:2])
    with pytest.raises(ValueError):
        kda.kda_block_norm(y, w, gate=y, gate_act="tanh")
    with pytest.raises(ValueError):
        kda.kda_block_norm(y.t(), w)
    with pytest.raises(TypeError):
        kda.kda_block_norm(y, w.double())
    with pytest.raises(TypeError):
        kda.kda_block_norm(y.half(), w)
    with pytest.raises(kda.KDAError):
        kda.kda_block_norm(y, torch.ones(16, device="cuda"))
    with pytest.raises(kda.KDAError):
        kda.kda_block_norm(y, w, x=y, x_out=torch.empty(4, 64, device="cuda"), eps=0.0)
    with pytest.raises(kda.KDAError):
        kda.kda_block_norm_backward(y, w, None)
