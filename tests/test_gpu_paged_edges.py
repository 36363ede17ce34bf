"""GPU tests of the paged-attention operators beyond those beside their forms:
places that a first version got wrong or that its tests could not tell apart."""
import pytest
import torch

import paged_ref as ref
from test_gpu_paged import Dev, _check_attn

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("group", [5, 11, 13, 25])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
def test_joining_tiles_whose_rows_are_no_multiple_of_four(group, dim, e4m3):
    """Items of 250, 242 and 234 rows cut among many ranges.  The joining kernel takes
    rows in pairs, two pairs a warp at head_dim 64: the last warp's second pair is
    behind the tile, and behind the partial result (its maxima and totals would be
    the next one's first sums).  Full items, and one with a last row alone in its pair."""
    tokens = 2 * (128 // group)
    _check_attn(ref.Batch([tokens, tokens + 1, 1 + 16 // group], [3000, 700, 1500], heads=group, kv_heads=1, dim=dim, e4m3=e4m3,
                          seed=20))


@pytest.mark.parametrize("group", [5, 11, 13, 25])
def test_joining_reads_nothing_of_an_unwritten_neighbour(group):
    """The same with a workspace of NaN around a single item: the parts behind the
    last range's are never written."""
    b = ref.Batch([2 * (128 // group)], [18 * 128], heads=group, kv_heads=1, dim=64, seed=21)
    d = Dev(b)
    d.ws.view(torch.float32).fill_(float("nan"))
    out = d.run().cpu().double()
    want, tol = b.reference()
    assert int(d.status[0]) == 0 and ((out - want).abs() <= tol).all()
