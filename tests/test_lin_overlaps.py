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
