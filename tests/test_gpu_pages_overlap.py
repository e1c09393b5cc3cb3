"""Pages given back with an output that lies in the stack or the table are refused."""
import numpy as np
import pytest
import torch

from memory_bound_gemv_row_amd import binding

from gpu_util import say
from test_gpu_pages import _ints

pytestmark = pytest.mark.gpu


def test_release_over_its_stack_or_table(gpu):
    say("[release] outputs in the stack and the table")
    free, count, keep = _ints(range(8)), _ints([3, 0]), _ints([0, 0])
    wide = _ints([[3, 4, -1, -1, 9, 9], [5, -1, -1, -1, 9, 9]])
    table = wide[:, :4]
    before = free.clone(), wide.clone()
    for out in (free[:2], free[6:], wide[0, :2], wide[0, 2:4], wide[0, 4:], wide[1, 2:4], keep, count):
        with pytest.raises(ValueError):
            binding.release_pages(free, count, table, keep, 16, out=out)
    assert torch.equal(free, before[0]) and torch.equal(wide, before[1])
    out = binding.release_pages(free, count, table, keep, 16, out=_ints([0, 0]))
    assert out.tolist() == [6, 0] and free.tolist()[:6] == [0, 1, 2, 3, 4, 5] and np.all(table.cpu().numpy() == -1)
    assert torch.all(wide[:, 4:] == 9)
    # an empty pool and no sequences
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    assert binding.release_pages(none, _ints([0, 0]), none.view(0, 4), none, 16, out=_ints([7, 7])).tolist() == [0, 0]
