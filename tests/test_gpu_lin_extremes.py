"""GPU parity of the decayed linear attention where decays are extreme, against the 64-bit
recurrence with test_gpu_lin's bounds."""
import pytest
import torch

import lin_reference as R
import test_gpu_lin as L
import kimi_delta_attention_12_gb300 as kda

pytestmark = pytest.mark.gpu

BF, F = torch.bfloat16, torch.float32


@pytest.mark.parametrize("dtype,d", [(F, 32), (F, 64), (BF, 64), (BF, 128)])
def test_decays_that_grow_past_fp32_within_a_chunk(dtype, d):
    """e^{20} a token: the powers up to the sequences' own lengths are finite, those up to a
    whole chunk's are not, and count for nothing."""
    x = R.make([1, 2, 4, 1], 2, d, d, dtype, seed=2, state=True, g=[3.0, 20.0])
    v = R.dev(x)
    args = (v["q"], v["k"], v["v"], v["log_decay"])
    o, S = kda.kda_lin_prefill(*args, v["S0"], v["cu"], x["cu"])
    L.check_forward(x, o, S, 1.0, d, dtype, L.tensor_core(d, d, dtype))
    g = kda.kda_lin_backward(*args, v["dO"], v["S0"], v["cu"], x["cu"], v["dS"])
    check_backward(x, g, 1.0, L.tensor_core(d, d, dtype))


def check_backward(x, g, scale, tc):
    """Every gradient within the roundings counted, as test_gpu_lin.test_backward has them."""
    a = {n: R.f64(t) for n, t in x.items() if isinstance(t, torch.Tensor)}
    inputs = [a[n] for n in ("q", "k", "v")]
    want = R.lin_backward(*inputs, a["log_decay"], x["lens"], a["dO"], a.get("S0"), a.get("dS"),
                          scale)
    mag = R.lin_backward(*R.absolute(*inputs), a["log_decay"], x["lens"],
                         *R.absolute(a["dO"], a.get("S0"), a.get("dS")), abs(scale))
    terms = R.fp32_terms(x["lens"], max(inputs[0].shape[2], inputs[2].shape[2]))
    for n in want:
        assert bool(torch.isfinite(g[n]).all()), n
        rows = n != "dS0"
        R.check(n, g[n], want[n], mag[n], terms, rows and g[n].dtype == BF,
                1 if rows and tc else 0)


@pytest.mark.parametrize("dtype,d", [(F, 64), (BF, 64), (BF, 128)])
@pytest.mark.parametrize("decay", [0.0, -1e-9, -3.0, -40.0, -87.0, -1e30, float("-inf")])
@pytest.mark.parametrize("lens", [[300, 17], [641, 0, 1]], ids=["two", "cut"])
def test_gradients_at_extreme_decays(dtype, d, decay, lens):
    x = R.make(lens, 2, d, d, dtype, seed=3, state=True, g=[decay, -0.1])
    v = R.dev(x)
    g = kda.kda_lin_backward(v["q"], v["k"], v["v"], v["log_decay"], v["dO"], v["S0"], v["cu"],
                             x["cu"], v["dS"], scale=0.75)
    check_backward(x, g, 0.75, L.tensor_core(d, d, dtype))


@pytest.mark.parametrize("dtype,d", [(F, 64), (BF, 128)])
def test_a_factor_of_zero_on_states_that_are_not_finite(dtype, d):
    """log_decay of -infinity is the factor 0: finite states are dropped, and 0 times infinity is
    NaN, as in the formula."""
    x = R.make([1, 1], 1, d, d, dtype, seed=4, state=True, g=[float("-inf")])
    x["S0"][1, 0, 3, 5] = float("inf")
    v = R.dev(x)
    args = (v["q"], v["k"], v["v"], v["log_decay"])
    o, S = kda.kda_lin_prefill(*args, v["S0"], v["cu"], x["cu"])
    pool = v["S0"].clone()
    od = kda.kda_lin_decode_step(*args, pool)
    for out, state in ((o, S), (od, pool)):
        assert bool(torch.isfinite(state[0]).all()) and bool(torch.isnan(state[1, 0, 3, 5]))
        assert bool(torch.isfinite(out[0]).all()) and bool(torch.isnan(out[1, 0, 5]))


def one_sign(T, H, d=128):
    gen = torch.Generator(device="cuda").manual_seed(T + H)
    q, k, v = (torch.rand(T, H, d, generator=gen, device="cuda").add(0.5).to(BF)
               for _ in range(3))
    g = torch.zeros(H, device="cuda")
    g[1::3], g[2::3] = -1e-6, -2e-5
    return q, k, v, g


@pytest.mark.parametrize("T,H", [(65536, 64), (65536, 96), (20000, 4)],
                         ids=["segments", "cut_in_two", "short_segments"])
def test_long_sums_of_one_sign(T, H):
    """States of slow decays whose terms all have one sign: what the tensor core cuts off the
    sums is cut off the same side each time.  It adds up four chunks at most, 96 additions that
    each lose less than 2^-23; everything after them is rounded, an addition a chunk."""
    q, k, v, g = one_sign(T, H)
    o, S = kda.kda_lin_prefill(q, k, v, g, scale=1.0 / T)
    bound = (2 * 96 + T / 128 + 64) * R.U32
    t = torch.arange(T, device="cuda", dtype=torch.float64)
    for h in range(3):
        w = torch.exp(g[h].double() * (T - 1 - t))[:, None]
        want = (k[:, h].double() * w).T @ v[:, h].double()
        assert float(((S[0, h].double() - want) / want).abs().max()) <= bound, h
    H = max(1, H // 3)
    g = g[:H].contiguous()
    q, k, v = (a[:, :H].contiguous() for a in (q, k, v))
    dS0 = kda.kda_lin_backward(q, k, v, g, v, scale=1.0 / T)["dS0"]
    for h in range(min(H, 3)):
        w = torch.exp(g[h].double() * (t + 1))[:, None] / T
        want = (q[:, h].double() * w).T @ v[:, h].double()
        assert float(((dS0[0, h].double() - want) / want).abs().max()) <= bound, h
