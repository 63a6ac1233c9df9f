"""The residual RMS norm's backward where its ring of rows goes round several times: all of dX and dweight against 64
bits, at widths whose teams, rows of a slot and slots fit together differently.  A turn of the ring is about 5 million
elements of each tensor on 152 SMs; tolerances as in test_gpu_block_fp8."""
import pytest

import test_gpu_block_fp8 as block

pytestmark = pytest.mark.gpu

# (rows, width, chunks): ragged last groups, groups that cross chunks, widths of each kind of team
SHAPES = [(300001, 64, 1), (140002, 136, 2), (70007, 264, 7), (45003, 504, 3), (40003, 520, 1), (30000, 688, 8), (24013, 832, 1),
          (21001, 896, 1), (20014, 1024, 2), (20000, 1032, 5), (16003, 1152, 1), (11001, 1792, 3), (8192, 2880, 8), (8001, 2816, 1),
          (8192, 3584, 8), (6001, 3456, 1), (8192, 4096, 8), (5000, 4104, 1), (3000, 8192, 1), (2601, 12296, 3), (2000, 16384, 1)]


@pytest.mark.parametrize("T,d,N", SHAPES)
@pytest.mark.parametrize("residual", [True, False])
def test_norm_backward_over_several_turns_of_the_ring(T, d, N, residual):
    block.test_rmsnorm_add_backward(T, d, N, residual)
