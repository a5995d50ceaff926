"""tv_rope_rows at the row counts where a block of the grid takes two rows instead of one, with
test_gpu_rope.py's tolerance."""
import pytest
import torch

from speculative_tree_verify_gb300 import abi
from test_gpu_rope import Rows

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("more", [-1, 0, 1, 16])
@pytest.mark.parametrize("interleaved,in_place", [(False, True), (False, False), (True, True), (True, False)])
@pytest.mark.parametrize("heads,dim,rot", [(3, 64, 32), (2, 128, 112), (5, 128, 128)])
def test_one_row_a_block_or_two(gpu, heads, dim, rot, interleaved, in_place, more):
    """Sixteen rows an SM, or one less, or an odd one more."""
    rows = 16 * torch.cuda.get_device_properties(0).multi_processor_count + more
    Rows(rows, heads, dim, seed=rot + more, pad=8).run(abi.tv_rope_init(rot, interleaved, gain=1.1), in_place)
