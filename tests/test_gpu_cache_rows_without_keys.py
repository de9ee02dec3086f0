"""A row that sees no key is zero whatever the values of the other rows' keys are."""
import pytest
import torch

import kimi_delta_attention_12_gb300 as kda
from test_gpu_cache_attention import Batch, _tensor_cores

pytestmark = pytest.mark.gpu


def _nan_at(b, request, token):
    b.v[b.table[request][token // b.block], :, token % b.block] = 0x7f


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("d", [32, 64, 128])
def test_values_that_are_nan_beside_rows_without_keys(d, dtype):
    """3, 30 and 200 cached tokens, 5, 33 and 203 new ones: the first rows of each see nothing."""
    b = Batch([0, 0, 0], [5, 33, 203], 16, 8, 2, d, dtype, seed=d)
    b.context = [3, 30, 200]
    for i, at in enumerate((1, 0, 7)):
        _nan_at(b, i, at)
    args = b.args()
    for got in (kda.kda_cache_attention(*args, max_new=1),                          # clusters
                kda.kda_cache_attention(*args[:5], b.wide(), *args[6:], max_new=1),  # stretches
                kda.kda_cache_attention(*args[:5], b.wide(), *args[6:], max_new=33)):
        assert not got[:2].any() and not got[5:8].any() and not got[38:41].any()
        assert torch.isnan(got[3:5]).all() and torch.isnan(got[8:38]).all()
        assert torch.isnan(got[48:]).all()


@pytest.mark.parametrize("new,context,heads,at", [
    ([140, 100], [100, 30], (16, 4), 20),      # items that a block has whole
    ([1870], [1760], (20, 20), 20),            # and some of which it has a part
])
@pytest.mark.parametrize("d", [64, 128])
def test_the_same_on_the_tensor_cores(new, context, heads, at, d):
    b = Batch([0] * len(new), new, 16, *heads, d, torch.bfloat16, seed=d)
    b.context = context
    for i in range(len(new)):
        _nan_at(b, i, at)
    args, most = _tensor_cores(b)
    got = kda.kda_cache_attention(*args, max_new=most)
    for i, (n, c) in enumerate(zip(new, context)):
        rows = got[b.cu[i]:b.cu[i + 1]]
        assert not rows[:n - c].any()
        assert torch.isnan(rows[n - c + at:]).all()
