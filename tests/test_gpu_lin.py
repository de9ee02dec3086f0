"""GPU parity of the decayed linear attention against the 64-bit recurrence.

Bounds count roundings (lin_reference): the fp32 form has only its sums'; the
tensor-core form (bf16, d = 128) rounds the products x.y and the carried state
to bf16 where they multiply, one operand each, and its fp32 states keep fp32
sums."""
import numpy as np
import pytest
import torch

import kimi_delta_attention_12_gb300 as kda
import lin_reference as R

pytestmark = pytest.mark.gpu

BF, F = torch.bfloat16, torch.float32

SHAPES = [
    # lens, H, dk, dv, dtype, states
    ([64], 2, 32, 32, F, False),
    ([1], 1, 32, 64, F, True),
    ([3, 0, 33, 1], 3, 64, 32, F, True),
    ([31, 32, 0, 65], 2, 128, 64, F, True),
    ([700], 1, 64, 128, F, True),               # cut into segments
    ([129, 0, 300], 1, 128, 128, F, False),
    ([50, 70], 2, 64, 64, BF, True),
    ([257], 1, 32, 128, BF, True),
    ([1], 1, 128, 128, BF, True),
    ([0, 2, 0], 2, 128, 128, BF, True),
    ([127], 3, 128, 128, BF, False),
    ([128], 2, 128, 128, BF, True),
    ([129, 255, 256, 257], 2, 128, 128, BF, True),
    ([640], 1, 128, 128, BF, True),             # cut into segments
    ([900, 5, 0, 131], 1, 128, 128, BF, False),
]
IDS = [f"{'_'.join(map(str, s[0]))}-H{s[1]}-{s[2]}x{s[3]}-{str(s[4])[6:]}-{int(s[5])}"
       for s in SHAPES]


def tensor_core(dk, dv, dtype, recurrent=False):
    return dtype == BF and dk == 128 and dv == 128 and not recurrent


def forward_bounds(x, scale, dk, dtype, tc):
    a = {n: R.f64(t) for n, t in x.items() if isinstance(t, torch.Tensor)}
    want = R.lin_forward(a["q"], a["k"], a["v"], a["log_decay"], x["lens"], a.get("S0"), scale)
    mags = R.lin_forward(*R.absolute(a["q"], a["k"], a["v"]), a["log_decay"], x["lens"],
                         None if x["S0"] is None else np.abs(a["S0"]), abs(scale))
    return want, mags


def check_forward(x, o, S, scale, dk, dtype, tc):
    (wo, wS), (mo, mS) = forward_bounds(x, scale, dk, dtype, tc)
    terms = R.fp32_terms(x["lens"], dk)
    R.check("o", o, wo, mo, terms, dtype == BF, 1 if tc else 0)
    R.check("final state", S, wS, mS, terms)
    if dtype == BF and wo.size > 1000:
        # independent roundings of random sign: below half a step of bf16 in the norm
        assert R.rel_fro(o, wo) <= R.U16
    if wS.size > 1000:
        assert R.rel_fro(S, wS) <= 2e-6


@pytest.mark.parametrize("lens,H,dk,dv,dtype,state", SHAPES, ids=IDS)
@pytest.mark.parametrize("recurrent", [True, False])
def test_prefill(lens, H, dk, dv, dtype, state, recurrent):
    x = R.make(lens, H, dk, dv, dtype, seed=len(lens) + dk, state=state)
    d = R.dev(x)
    o, S = kda.kda_lin_prefill(d["q"], d["k"], d["v"], d["log_decay"], d["S0"], d["cu"], x["cu"],
                               scale=0.75, recurrent=recurrent)
    assert o.dtype == dtype and S.dtype == F
    check_forward(x, o, S, 0.75, dk, dtype, tensor_core(dk, dv, dtype, recurrent))


@pytest.mark.parametrize("lens,H,dk,dv,dtype,state", SHAPES, ids=IDS)
@pytest.mark.parametrize("recurrent", [True, False])
def test_backward(lens, H, dk, dv, dtype, state, recurrent):
    x = R.make(lens, H, dk, dv, dtype, seed=7 + dv, state=state)
    d = R.dev(x)
    g = kda.kda_lin_backward(d["q"], d["k"], d["v"], d["log_decay"], d["dO"], d["S0"], d["cu"],
                             x["cu"], d["dS"], scale=0.75, recurrent=recurrent)
    a = {n: R.f64(t) for n, t in x.items() if isinstance(t, torch.Tensor)}
    want = R.lin_backward(a["q"], a["k"], a["v"], a["log_decay"], lens, a["dO"], a.get("S0"),
                          a.get("dS"), 0.75)
    mag = R.lin_backward(*R.absolute(a["q"], a["k"], a["v"]), a["log_decay"], lens,
                         np.abs(a["dO"]), *R.absolute(a.get("S0"), a.get("dS")), 0.75)
    tc = tensor_core(dk, dv, dtype, recurrent)
    terms = R.fp32_terms(lens, max(dk, dv))
    for n in ("dq", "dk", "dv"):
        assert g[n].dtype == dtype
        R.check(n, g[n], want[n], mag[n], terms, dtype == BF, 1 if tc else 0)
        if dtype == BF and want[n].size > 1000:
            assert R.rel_fro(g[n], want[n]) <= R.U16
    R.check("dS0", g["dS0"], want["dS0"], mag["dS0"], terms)


def test_backward_without_upstream_state_or_initial_state():
    x = R.make([40, 90], 2, 64, 32, F, seed=4, state=True)
    d = R.dev(x)
    a = {n: R.f64(t) for n, t in x.items() if isinstance(t, torch.Tensor)}
    for S0, dS in ((None, "dS"), ("S0", None), (None, None)):
        g = kda.kda_lin_backward(d["q"], d["k"], d["v"], d["log_decay"], d["dO"],
                                 d["S0"] if S0 else None, d["cu"], x["cu"],
                                 d["dS"] if dS else None)
        want = R.lin_backward(a["q"], a["k"], a["v"], a["log_decay"], x["lens"], a["dO"],
                              a["S0"] if S0 else None, a["dS"] if dS else None)
        for n in want:
            assert R.rel_fro(g[n], want[n]) <= 2e-6, n


@pytest.mark.parametrize("dtype,d", [(F, 64), (BF, 128)])
@pytest.mark.parametrize("decay", [0.0, -1e-9, -3.0, -40.0, -1e30, float("-inf")])
def test_decay_extremes(dtype, d, decay):
    x = R.make([300, 17], 2, d, d, dtype, seed=2, state=True, g=[decay, -0.1])
    dv = R.dev(x)
    o, S = kda.kda_lin_prefill(dv["q"], dv["k"], dv["v"], dv["log_decay"], dv["S0"], dv["cu"],
                               x["cu"])
    check_forward(x, o, S, 1.0, d, dtype, dtype == BF)
    st = dv["S0"].clone()
    od = kda.kda_lin_decode_step(dv["q"][:2], dv["k"][:2], dv["v"][:2], dv["log_decay"], st)
    one = {**x, "lens": [1, 1], **{n: x[n][:2] for n in ("q", "k", "v")}}
    check_forward(one, od, st, 1.0, d, dtype, False)
    g = kda.kda_lin_backward(dv["q"], dv["k"], dv["v"], dv["log_decay"], dv["dO"], dv["S0"],
                             dv["cu"], x["cu"], dv["dS"])
    assert all(bool(torch.isfinite(t).all()) for t in g.values())


@pytest.mark.parametrize("dtype,d", [(F, 32), (BF, 128)])
def test_state_in_place_equal_lengths_and_4d(dtype, d):
    x = R.make([500, 500], 1, d, d, dtype, seed=9, state=True)
    v = R.dev(x)
    o, S = kda.kda_lin_prefill(v["q"], v["k"], v["v"], v["log_decay"], v["S0"], v["cu"], x["cu"])
    st = v["S0"].clone()
    o2, S2 = kda.kda_lin_prefill(v["q"], v["k"], v["v"], v["log_decay"], st, v["cu"],
                                 final_state=st)           # no host mirror either
    assert S2 is st and torch.equal(o, o2) and torch.equal(S, st)
    four = [v[n].view(2, 500, 1, d) for n in ("q", "k", "v")]
    o3, S3 = kda.kda_lin_prefill(*four, v["log_decay"], v["S0"])
    assert o3.shape == (2, 500, 1, d) and torch.equal(o3.view_as(o), o) and torch.equal(S3, S)
    o4, none = kda.kda_lin_prefill(*four, v["log_decay"], v["S0"], output_final_state=False)
    assert none is None and torch.equal(o4, o3)


@pytest.mark.parametrize("dtype,d", [(F, 64), (BF, 64), (BF, 128)])
def test_prefill_then_decode(dtype, d):
    """Prompt, then tokens one at a time in a shared pool, against the whole recurrence."""
    lens, more = [45, 130], 3
    total = [n + more for n in lens]
    x = R.make(total, 2, d, d, dtype, seed=11, state=True)
    cu = R.bounds_of(total)
    head = torch.cat([torch.arange(cu[n], cu[n] + lens[n]) for n in range(2)])
    hcu = torch.tensor(R.bounds_of(lens), dtype=torch.int32)
    v = R.dev(x)
    part = [v[n][head.cuda()] for n in ("q", "k", "v")]
    _, S = kda.kda_lin_prefill(*part, v["log_decay"], v["S0"], hcu.cuda(), hcu)
    pool = torch.full((5, 2, d, d), 7.0, device="cuda")
    slots = torch.tensor([3, 1], dtype=torch.int32, device="cuda")
    kda.kda_state_io(kda.KDA_STATE_SCATTER, pool, S, slots)
    outs = []
    for i in range(more):
        at = torch.tensor([cu[n] + lens[n] + i for n in range(2)], device="cuda")
        outs.append(kda.kda_lin_decode_step(*(v[n][at] for n in ("q", "k", "v")), v["log_decay"],
                                            pool, slots))
    (wo, wS), (mo, mS) = forward_bounds(x, 1.0, d, dtype, False)
    terms = R.fp32_terms(total, d)
    for i in range(more):
        rows = [cu[n] + lens[n] + i for n in range(2)]
        R.check("o", outs[i], wo[rows], mo[rows], terms, dtype == BF)
    R.check("pool", pool[slots.long()], wS, mS, terms)
    assert bool((pool[[0, 2, 4]] == 7.0).all())


@pytest.mark.parametrize("dk,dv", [(32, 32), (64, 128), (128, 32), (128, 128)])
@pytest.mark.parametrize("dtype", [F, BF])
def test_decode(dk, dv, dtype):
    B, H = 5, 3
    x = R.make([1] * B, H, dk, dv, dtype, seed=dk + dv, state=True)
    v = R.dev(x)
    st = v["S0"].clone()
    o = kda.kda_lin_decode_step(v["q"], v["k"], v["v"], v["log_decay"], st, scale=-0.5)
    (wo, wS), (mo, mS) = forward_bounds(x, -0.5, dk, dtype, False)
    R.check("o", o, wo, mo, R.fp32_terms([1], dk), dtype == BF)
    R.check("state", st, wS, mS, R.fp32_terms([1], dk))


def test_decode_bad_slots_leave_the_pool_alone():
    x = R.make([1] * 4, 2, 128, 128, BF, seed=1, state=True)
    v = R.dev(x)
    pool = v["S0"].clone()
    slots = torch.tensor([2, -1, 4, 0], dtype=torch.int32, device="cuda")
    o = kda.kda_lin_decode_step(v["q"], v["k"], v["v"], v["log_decay"], pool, slots)
    assert torch.isnan(o[1:3]).all() and torch.isfinite(o[[0, 3]]).all()
    assert torch.equal(pool[[1, 3]], v["S0"][[1, 3]])
    assert not torch.equal(pool[2], v["S0"][2])


@pytest.mark.parametrize("dtype,d", [(F, 64), (BF, 128)])
def test_same_bits_on_other_streams_and_in_graphs(dtype, d):
    x = R.make([300, 20, 513], 2, d, d, dtype, seed=5, state=True)
    v = R.dev(x)
    args = (v["q"], v["k"], v["v"], v["log_decay"])

    def both(stream=None):
        o, S = kda.kda_lin_prefill(*args, v["S0"], v["cu"], x["cu"], stream=stream)
        g = kda.kda_lin_backward(*args, v["dO"], v["S0"], v["cu"], x["cu"], v["dS"],
                                 stream=stream)
        return [o, S, *g.values()]

    first = both()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    other = both(side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, other))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = both()
    for t in captured:
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, captured))


@pytest.mark.parametrize("dtype,d", [(F, 64), (BF, 128)])
def test_neighbours_do_not_mix(dtype, d):
    """NaN and infinity in one sequence stay in it, also where a chunk ends inside a tile."""
    x = R.make([70, 100, 40], 2, d, d, dtype, seed=6, state=True)
    v = R.dev(x)

    def run():
        o, S = kda.kda_lin_prefill(v["q"], v["k"], v["v"], v["log_decay"], v["S0"], v["cu"],
                                   x["cu"])
        g = kda.kda_lin_backward(v["q"], v["k"], v["v"], v["log_decay"], v["dO"], v["S0"],
                                 v["cu"], x["cu"], v["dS"])
        return [o, g["dq"], g["dk"], g["dv"]], [S, g["dS0"]]

    rows, states = run()
    for n in ("q", "k", "v", "dO"):
        v[n][70:170] = float("nan")
        v[n][75:90] = float("inf")
    for n in ("S0", "dS"):
        v[n][1] = float("nan")
    rows2, states2 = run()
    keep = torch.cat([torch.arange(70), torch.arange(170, 210)]).cuda()
    assert all(torch.equal(a[keep], b[keep]) for a, b in zip(rows, rows2))
    assert all(torch.equal(a[[0, 2]], b[[0, 2]]) for a, b in zip(states, states2))
    assert torch.isnan(rows2[0][70:170]).any()


@pytest.mark.parametrize("dtype,d", [(F, 32), (BF, 128)])
def test_malformed_device_seqlens_stay_inside(dtype, d):
    """Without the host mirror the kernels bound what they touch themselves."""
    T, H, pad = 256, 1, 64
    x = R.make([T], H, d, d, dtype, seed=3)
    v = R.dev(x)
    for cu in ([0, 256, 0, 256, 0], [-5, 300, 10 ** 9, -10 ** 9, 7], [256, 0, 256, 0, 256],
               [0, 1, 2, 3, 10 ** 6]):
        N = len(cu) - 1
        buf = torch.full((T + 2 * pad, H, d), 3.0, dtype=dtype, device="cuda")
        sbuf = torch.full((N + 2, H, d, d), 3.0, device="cuda")
        need = kda.lin_prefill_workspace_bytes(N, T, H, d, d, dtype)
        wbuf = torch.full((need + 512,), 9, dtype=torch.uint8, device="cuda")
        kda.kda_lin_prefill(v["q"], v["k"], v["v"], v["log_decay"], None,
                            torch.tensor(cu, dtype=torch.int32, device="cuda"),
                            o=buf[pad:pad + T], final_state=sbuf[1:N + 1],
                            workspace=wbuf[256:256 + need])
        torch.cuda.synchronize()
        assert bool((buf[:pad] == 3.0).all()) and bool((buf[pad + T:] == 3.0).all())
        assert bool((sbuf[[0, N + 1]] == 3.0).all())
        assert bool((wbuf[:256] == 9).all()) and bool((wbuf[256 + need:] == 9).all())


def test_malformed_device_seqlens_of_sequences_cut_in_two():
    T, H, pad = 33000, 40, 64
    x = R.make([T], H, 128, 128, BF, seed=3)
    v = R.dev(x)
    for cu in ([0, T, 0], [-5, T + 3, 7], [T, 1, 10 ** 9]):
        N = len(cu) - 1
        buf = torch.full((T + 2 * pad, H, 128), 3.0, dtype=BF, device="cuda")
        sbuf = torch.full((N + 2, H, 128, 128), 3.0, device="cuda")
        need = kda.lin_prefill_workspace_bytes(N, T, H, 128, 128, BF)
        wbuf = torch.full((need + 512,), 9, dtype=torch.uint8, device="cuda")
        kda.kda_lin_prefill(v["q"], v["k"], v["v"], v["log_decay"], None,
                            torch.tensor(cu, dtype=torch.int32, device="cuda"),
                            o=buf[pad:pad + T], final_state=sbuf[1:N + 1],
                            workspace=wbuf[256:256 + need])
        torch.cuda.synchronize()
        assert int(wbuf[256:260].view(torch.int32)) == 0
        assert bool((buf[:pad] == 3.0).all()) and bool((buf[pad + T:] == 3.0).all())
        assert bool((sbuf[[0, N + 1]] == 3.0).all())
        assert bool((wbuf[:256] == 9).all()) and bool((wbuf[256 + need:] == 9).all())


def test_offsets_past_32_bits():
    """2.2e9 elements per tensor: the last tokens, whose decay forgets what came before."""
    T, H, d = 136000, 128, 128
    free, _ = torch.cuda.mem_get_info()
    if free < 60e9:
        pytest.skip("needs 60 GB")
    gen = torch.Generator(device="cuda").manual_seed(0)
    q, k, v = (torch.empty(T, H, d, dtype=BF, device="cuda").normal_(generator=gen)
               for _ in range(3))
    g = torch.full((H,), -1.0, device="cuda")
    o, S = kda.kda_lin_prefill(q, k, v, g, scale=0.01)
    tail = 160     # e^-160 of anything earlier is below fp32
    heads = [0, 77, 127]
    qs, ks, vs = (t[-tail:][:, heads].contiguous() for t in (q, k, v))
    wo, wS = R.lin_forward(*(R.f64(t) for t in (qs, ks, vs)), -np.ones(3), [tail], None, 0.01)
    assert R.rel_fro(o[-16:][:, heads], wo[-16:]) <= R.U16
    assert R.rel_fro(S[0, heads], wS[0]) <= 2e-6


def test_decode_offsets_past_32_bits():
    B, H, d = 4, 128, 128
    pool = torch.empty(1200, H, d, d, device="cuda")       # 2.5e9 floats
    x = R.make([1] * B, H, d, d, BF, seed=1, state=True)
    v = R.dev(x)
    slots = torch.tensor([0, 1199, 1023, 1024], dtype=torch.int32, device="cuda")
    pool[slots.long()] = v["S0"]
    o = kda.kda_lin_decode_step(v["q"], v["k"], v["v"], v["log_decay"], pool, slots)
    (wo, wS), (mo, mS) = forward_bounds(x, 1.0, d, BF, False)
    R.check("o", o, wo, mo, R.fp32_terms([1], d), True)
    R.check("state", pool[slots.long()], wS, mS, R.fp32_terms([1], d))


def test_binding_refusals():
    x = R.dev(R.make([8, 8], 2, 32, 32, F, state=True))
    a = (x["q"], x["k"], x["v"], x["log_decay"])
    with pytest.raises(ValueError):
        kda.kda_lin_prefill(x["q"], x["k"][:8], x["v"], x["log_decay"])
    with pytest.raises(TypeError):
        kda.kda_lin_prefill(x["q"], x["k"].bfloat16(), x["v"], x["log_decay"])
    with pytest.raises(TypeError):
        kda.kda_lin_prefill(x["q"].half(), x["k"].half(), x["v"].half(), x["log_decay"])
    with pytest.raises(ValueError):
        kda.kda_lin_prefill(*a, x["S0"])                    # one sequence, two states
    with pytest.raises(TypeError):
        kda.kda_lin_prefill(*a[:3], x["log_decay"].double())
    with pytest.raises(ValueError):
        kda.kda_lin_prefill(x["q"].transpose(0, 1).contiguous().transpose(0, 1), *a[1:])
    with pytest.raises(ValueError):
        kda.kda_lin_prefill(*a, None, x["cu"].long())
    with pytest.raises(ValueError):
        kda.kda_lin_decode_step(*a, x["S0"][0])
    with pytest.raises(ValueError):
        kda.kda_lin_backward(*a, x["dO"][:4])
    with pytest.raises(kda.KDAError):
        kda.kda_lin_prefill(*a, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(kda.KDAError):
        kda.kda_lin_prefill(*a, o=x["v"])                   # onto an input


def test_many_ragged_sequences_in_any_order():
    """More (sequence, head) pairs than SMs: whole sequences, taken longest first."""
    lens = [5, 300, 0, 129, 128, 1, 257, 40] * 5          # 40 sequences, ties among them
    x = R.make(lens, 4, 128, 128, BF, seed=12, state=True)
    v = R.dev(x)
    for n in (40, 70):                                     # ranked, and past the ranked range
        cu = torch.cat([x["cu"], x["cu"][-1:].repeat(n - 40)])
        S0 = torch.cat([v["S0"], v["S0"][:n - 40]])
        o, S = kda.kda_lin_prefill(v["q"], v["k"], v["v"], v["log_decay"], S0, cu.cuda(), cu)
        assert torch.equal(S[40:], S0[40:])                # empty ones hand theirs on
        check_forward(x, o, S[:40], 1.0, 128, BF, True)


def heads(x, keep):
    """The same sequences with some of the heads: what heads do is independent."""
    axis = {"q": 1, "k": 1, "v": 1, "dO": 1, "log_decay": 0, "S0": 1, "dS": 1}
    return {n: t.index_select(axis[n], torch.tensor(keep)) if n in axis and t is not None else t
            for n, t in x.items()}


# Pairs of sequences and heads that fill more than half of the SMs but not all:
# the sequences are cut into a head of a few segments and a tail.
CUT_IN_TWO = [([16509], 96, True), ([31000, 1850], 39, True), ([12000, 24000, 0, 30500], 20, False),
              ([16400] * 2, 40, False)]


@pytest.mark.parametrize("lens,H,state", CUT_IN_TWO, ids=["1x96", "2x39", "4x20", "2x40"])
def test_prefill_of_sequences_cut_in_two(lens, H, state):
    x = R.make(lens, H, 128, 128, BF, seed=H, state=state, g=[-0.3 * h / H for h in range(H)])
    d = R.dev(x)
    cu = (None, None) if len(set(lens)) == 1 and len(lens) > 1 else (d["cu"], x["cu"])
    S0 = None if x["S0"] is None else d["S0"].clone()
    shape = (len(lens), -1, H, 128) if cu[0] is None else (-1, H, 128)
    o, S = kda.kda_lin_prefill(d["q"].reshape(shape), d["k"].reshape(shape),
                               d["v"].reshape(shape), d["log_decay"], S0, *cu, scale=0.75,
                               final_state=S0)      # in place, where there is one
    keep = [0, H // 2, H - 1]
    o = o.reshape(-1, H, 128)
    check_forward(heads(x, keep), o[:, keep], S[:, keep], 0.75, 128, BF, True)


@pytest.mark.parametrize("lens,H", [([16509], 26), ([31000, 1850], 13)], ids=["1x26", "2x13"])
def test_backward_of_sequences_cut_in_two(lens, H):
    x = R.make(lens, H, 128, 128, BF, seed=H, state=True, g=[-0.3 * h / H for h in range(H)])
    d = R.dev(x)
    g = kda.kda_lin_backward(d["q"], d["k"], d["v"], d["log_decay"], d["dO"], d["S0"], d["cu"],
                             x["cu"], d["dS"], scale=0.75)
    keep = [0, H - 1]
    x = heads(x, keep)
    a = {n: R.f64(t) for n, t in x.items() if isinstance(t, torch.Tensor)}
    want = R.lin_backward(a["q"], a["k"], a["v"], a["log_decay"], lens, a["dO"], a["S0"], a["dS"],
                          0.75)
    mag = R.lin_backward(*R.absolute(a["q"], a["k"], a["v"]), a["log_decay"], lens,
                         np.abs(a["dO"]), *R.absolute(a["S0"], a["dS"]), 0.75)
    terms = R.fp32_terms(lens, 128)
    for n in ("dq", "dk", "dv"):
        R.check(n, g[n][:, keep], want[n], mag[n], terms, True, 1)
        assert R.rel_fro(g[n][:, keep], want[n]) <= R.U16
    R.check("dS0", g["dS0"][:, keep], want["dS0"], mag["dS0"], terms)


@pytest.mark.parametrize("scale", [0.0, -0.75, 2.5])
def test_scales(scale):
    for dtype, d in ((F, 32), (BF, 128)):
        x = R.make([150, 20], 2, d, d, dtype, seed=13, state=True)
        v = R.dev(x)
        o, S = kda.kda_lin_prefill(v["q"], v["k"], v["v"], v["log_decay"], v["S0"], v["cu"],
                                   x["cu"], scale=scale)
        check_forward(x, o, S, scale, d, dtype, dtype == BF)
        g = kda.kda_lin_backward(v["q"], v["k"], v["v"], v["log_decay"], v["dO"], v["S0"],
                                 v["cu"], x["cu"], v["dS"], scale=scale)
        a = {n: R.f64(t) for n, t in x.items() if isinstance(t, torch.Tensor)}
        want = R.lin_backward(a["q"], a["k"], a["v"], a["log_decay"], x["lens"], a["dO"],
                              a["S0"], a["dS"], scale)
        for n in want:
            assert R.rel_fro(g[n], want[n]) <= (R.U16 if g[n].dtype == BF else 2e-6), n


def test_growing_decay():
    """log_decay above zero: the formula as it stands."""
    for dtype, d in ((F, 64), (BF, 128)):
        x = R.make([200], 2, d, d, dtype, seed=14, state=True, g=[0.02, 0.005])
        v = R.dev(x)
        o, S = kda.kda_lin_prefill(v["q"], v["k"], v["v"], v["log_decay"], v["S0"])
        check_forward(x, o, S, 1.0, d, dtype, dtype == BF)


@pytest.mark.parametrize("dtype,d", [(F, 32), (BF, 128)])
def test_status_word(dtype, d):
    x = R.make([200], 1, d, d, dtype)
    v = R.dev(x)
    args = (v["q"], v["k"], v["v"], v["log_decay"])
    for size, call in ((kda.lin_prefill_workspace_bytes, lambda w: kda.kda_lin_prefill(
            *args, workspace=w)), (kda.lin_backward_workspace_bytes,
                                   lambda w: kda.kda_lin_backward(*args, v["dO"], workspace=w))):
        w = torch.full((size(1, 200, 1, d, d, dtype),), 255, dtype=torch.uint8, device="cuda")
        call(w)
        assert kda.workspace_status(w) == kda.KDA_OK
