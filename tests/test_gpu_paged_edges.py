"""GPU tests of the paged-attention operators beyond those beside their forms:
places that a first version got wrong or that its tests could not tell apart."""
import time

import pytest
import torch

import mixture_experts_layer_22_b200 as moe
import paged_cases as cases
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


# ------------------------------------------- weights in two parts beside a bf16 cache
def _check_two_parts(b, max_q=None):
    d = Dev(b, max_q)
    out = d.run().cpu().double()
    n = sum(b.q_lens)
    want, tol = b.reference(cases.U_TWO_BF16)
    err = (out[:n] - want).abs()
    assert int(d.status[0]) == 0 and (err <= tol).all(), f"{float((err / tol).max()):.2f} of the bound"


@pytest.mark.parametrize("x", [1 - 2.0 ** -9, 0.7519, 0.3])
@pytest.mark.parametrize("heads,kv_heads,dim", [(4, 2, 64), (8, 8, 64), (8, 1, 128), (16, 1, 128), (4, 2, 256), (16, 1, 256)])
def test_few_rows_keep_both_parts_of_a_weight(heads, kv_heads, dim, x):
    """Up to 16 query rows a key/value head: sums of 2^-8 of their terms."""
    few = 16 * kv_heads // heads
    _check_two_parts(cases.cancelling([1, min(few, 3), 1, 1, few], [2, 48, 1001, 130, 300], x, heads=heads, kv_heads=kv_heads, dim=dim,
                                      seed=22))


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_a_hint_of_few_rows_keeps_both_parts_in_all(dim):
    _check_two_parts(cases.cancelling([40, 1, 17], [90, 300, 701], 0.7519, heads=4, kv_heads=2, dim=dim, seed=23), max_q=1)


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("q,kv", [([1], [1]), ([1, 1, 1, 1], [1, 17, 64, 300]), ([1] * 6, [2000, 1, 65, 700, 3, 129]),
                                  ([6, 3], [4, 3]), ([2, 3, 4, 1], [128, 64, 256, 192])])
def test_few_rows_of_ordinary_batches_within_the_bound_of_two_parts(q, kv, dim):
    _check_two_parts(ref.Batch(q, kv, heads=4, kv_heads=2, dim=dim, seed=24))


# -------------------------------------------------------------- the failure path
def test_the_attentions_bounded_wait_runs_out_and_the_context_stays_usable():
    """Both kinds of wait on barriers that nothing arrives on, one after the other: each
    lasts its limit of 2 s, either's abort flag ends the other warp's wait, and the
    status is MOE_ERR_TIMEOUT."""
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    gave_up = torch.full((1,), -1, dtype=torch.int32, device="cuda")
    b = ref.Batch([70, 1], [200, 90], heads=4, kv_heads=2, dim=64, seed=25)
    before = Dev(b).run().clone()
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    moe.selftest_wait_timeout(ws, gave_up)
    torch.cuda.synchronize()
    dt = time.perf_counter() - t0
    assert int(gave_up[0]) == 2 and int(ws[:4].view(torch.int32)[0]) == -6
    assert 3.9 < dt < 30.0                               # two clocks
    assert torch.equal(Dev(b).run(), before)
