"""GPU parity of the block norm's backward over the widths at which its launch changes: rows
past what a ring in shared memory holds, whose only dynamic shared memory is the room of the
sums.  Bounds and references are test_gpu_block_norm's."""
import pytest
import torch

import test_gpu_block_norm as B

pytestmark = pytest.mark.gpu

BF, F = torch.bfloat16, torch.float32
GATES = ("none", "sigmoid", "silu")


def case_id(c):
    return "-".join(map(str, c[:4])) + f"-{int(c[4])}{int(c[5])}{int(c[6])}-{str(c[7])[6:]}"


# The sums' room, 4 D bytes, is below 48 KB here, and with the kernel's own buffer above.
AROUND_48K = [(3, D, 0, gate, True, True, True, dtype)
              for D in (11528, 12288) for gate in GATES for dtype in (F, BF)]
AROUND_48K += [(2, 12288, 128, "sigmoid", True, True, True, dtype) for dtype in (F, BF)]


@pytest.mark.parametrize("case", AROUND_48K, ids=case_id)
def test_backward_of_rows_whose_sums_fill_48_kb(case):
    B.test_backward(case)
