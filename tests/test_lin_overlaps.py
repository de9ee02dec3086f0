"""Host-side refusals of buffers on top of one another: addresses that nothing dereferences,
and calls that are refused before anything is launched."""
import pytest

import kimi_delta_attention_12_gb300 as kda
import test_lin_abi as A
from test_lin_abi import BASE, INV, L, M  # noqa: F401 (L is the fixture)


@pytest.mark.parametrize("at", [BASE, BASE + M + 16384 - 16, BASE + 2 * M],
                         ids=["q", "k's end", "v"])
def test_a_state_in_place_may_not_lie_on_an_input(L, at):  # noqa: F811
    """final_state may be initial_state itself, and nothing else."""
    assert A._prefill(L, S0=at, Sf=at) == INV


# An output or the workspace on the decays, on the sequences' starts or on the slots: sizes as
# the argument tables of test_lin_abi have them (rows of 16 KB, states of 8 KB).
@pytest.mark.parametrize("call,over", [
    (A._prefill, dict(o=BASE + 3 * M)), (A._prefill, dict(o=BASE + 3 * M - 16384 + 16)),
    (A._prefill, dict(Sf=BASE + 3 * M - 8192 + 16)), (A._prefill, dict(ws=BASE + 3 * M)),
    (A._prefill, dict(cu=BASE + 4 * M + 4)), (A._prefill, dict(cu=BASE + 5 * M + 8188)),
    (A._prefill, dict(cu=BASE + 6 * M + 252)),
    (A._decode, dict(o=BASE + 3 * M)), (A._decode, dict(g=BASE + 16 * M + 64)),
    (A._decode, dict(slots=BASE + 4 * M)), (A._decode, dict(slots=BASE + 16 * M + 64)),
    (A._backward, dict(g=BASE + 5 * M)), (A._backward, dict(g=BASE + 8 * M + 8188)),
    (A._backward, dict(ws=BASE + 3 * M)), (A._backward, dict(cu=BASE + 6 * M + 16)),
    (A._backward, dict(cu=BASE + 7 * M)), (A._backward, dict(cu=BASE + 16 * M)),
])
def test_outputs_may_not_lie_on_decays_starts_or_slots(L, call, over):  # noqa: F811
    assert call(L, **over) == INV


def test_decays_may_lie_beside_an_output(L):  # noqa: F811
    """Sizes are the call's: 2 heads of decays end where o begins.  (Without a device, a call that
    passes the checks ends at its launch.)"""
    if kda.torch.cuda.is_available():
        pytest.skip("the addresses are not a device's")
    assert A._prefill(L, g=BASE + 4 * M - 8) == kda.KDA_ERR_CUDA
    assert A._decode(L, g=BASE + 4 * M - 8) == kda.KDA_ERR_CUDA
    assert A._backward(L, g=BASE + 5 * M - 8) == kda.KDA_ERR_CUDA
