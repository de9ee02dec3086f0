"""GPU parity of the block norms over the widths at which a launch changes: what a block keeps
in shared memory, rows too wide for it, and the room of the sums.  Bounds and references are
test_gpu_block_norm's."""
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


# Every part there: the weights stay in shared memory beside the ring while that has room, one
# row a block or two (an SM would hold one block: 3,584 and 4,096 columns of bf16), with and
# without columns to spare in the last vectors; past that they do not.  Some with more rows
# than blocks, so that the ring goes round.
KEPT = [(rows, D, 0, gate, True, True, True, BF)
        for rows, D in ((9, 264), (1300, 1000), (700, 1024), (650, 2048), (5, 2304), (633, 2560),
                        (5, 3584), (333, 4096), (4, 4096), (5, 4104), (161, 5000), (7, 5120),
                        (313, 7168), (3, 7176), (3, 8192)) for gate in GATES]
KEPT += [(rows, D, 0, gate, True, True, True, F)
         for rows, D in ((9, 264), (650, 1024), (633, 1000), (311, 2304), (5, 2560), (155, 4096),
                         (5, 4408), (5, 4416)) for gate in GATES]
KEPT += [(160, 4096, 0, "silu", True, False, True, BF), (5, 7168, 0, "sigmoid", True, False, True, BF),
         (333, 2304, 0, "none", True, False, True, F)]


@pytest.mark.parametrize("case", KEPT, ids=case_id)
def test_backward_with_every_part(case):
    B.test_backward(case)


# Rows too wide for a ring, which are read into registers, and those whose two vectors a thread
# take the form for four (fp32, 5,640 to 8,192 columns).
WIDE = [(3, D, 0, gate, True, True, True, BF) for D in (11264, 11272, 16384) for gate in GATES]
WIDE += [(3, D, 0, gate, True, True, True, F) for D in (5632, 5640, 7168, 8192, 8200, 16384)
         for gate in GATES]
WIDE += [(155, 7168, 0, "sigmoid", False, True, True, F), (155, 12288, 64, "silu", True, True, True, BF)]


@pytest.mark.parametrize("case", WIDE, ids=case_id)
def test_backward_of_wide_rows(case):
    B.test_backward(case)


# Parts left out: the same widths without the weights kept.
PARTS = [(313, D, group, gate, residual, scale, pre, dtype)
         for D, group in ((4096, 0), (7168, 0), (2048, 128))
         for gate, residual, scale, pre in (("silu", False, True, True), ("none", True, True, False),
                                            ("sigmoid", True, False, False))
         for dtype in (F, BF)]


@pytest.mark.parametrize("case", PARTS, ids=case_id)
def test_backward_with_parts_left_out(case):
    B.test_backward(case)


FORWARD = [(3, D, 0, gate, True, True, True, dtype) for D in (7168, 8200, 16384)
           for gate in GATES for dtype in (F, BF)]


@pytest.mark.parametrize("case", FORWARD, ids=case_id)
def test_forward_of_wide_rows(case):
    B.test_forward(case)
