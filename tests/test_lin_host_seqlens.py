"""The host's copy of the sequences' starts beside, and without, the device's."""
import ctypes

import pytest

import kimi_delta_attention_12_gb300 as kda
import test_lin_abi as A
from test_lin_abi import BASE, INV, L, M  # noqa: F401 (L is the fixture)


def starts(*at):
    return (ctypes.c_int32 * len(at))(*at)


@pytest.mark.parametrize("call", [A._prefill, A._backward])
def test_ragged_lengths_on_the_host_alone_are_refused(L, call):  # noqa: F811
    """Without the device's array the call is one of equal lengths."""
    assert call(L, N=2, cu_host=starts(0, 10, 64)) == INV
    assert call(L, N=4, cu_host=starts(0, 16, 32, 64, 64)) == INV
    if not kda.torch.cuda.is_available():     # (accepted: the call ends at its launch)
        assert call(L, N=2, cu_host=starts(0, 32, 64)) == kda.KDA_ERR_CUDA
        assert call(L, N=2, cu=BASE + 9 * M, cu_host=starts(0, 10, 64)) == kda.KDA_ERR_CUDA
