"""That the cancelling batches tell a weight in two bf16 parts from a weight in one, on
the host: mistakes are planted in the 64-bit form."""
import pytest
import torch

import paged_cases as cases
import paged_ref as ref


def _bf16(p):
    return p.to(torch.bfloat16).double()


ROUNDED = {"exact": lambda p: p, "two parts": lambda p: _bf16(p) + _bf16(p - _bf16(p))}
MISTAKEN = {"high part alone": _bf16, "low part twice": lambda p: _bf16(p) + 2 * _bf16(p - _bf16(p)),
            "low part's sign": lambda p: _bf16(p) - _bf16(p - _bf16(p)),
            "low part of the next key": lambda p: _bf16(p) + torch.roll(_bf16(p - _bf16(p)), 1, -1)}


@pytest.mark.parametrize("x", [1 - 2.0 ** -9, 0.7519, 0.3])
@pytest.mark.parametrize("q,kv", [([1, 1], [2, 48]), ([1, 3], [1001, 130])])
def test_cancelling_batches_show_one_rounding(x, q, kv):
    b = cases.cancelling(q, kv, x, heads=4, kv_heads=2, dim=64)
    want, tight = b.reference(cases.U_TWO_BF16)
    _, wide = b.reference(ref.U_BF16)
    for name, f in ROUNDED.items():
        assert ((cases.weighted(b, f) - want).abs() <= tight).all(), name
    for name, f in MISTAKEN.items():
        assert ((cases.weighted(b, f) - want).abs() > tight).any(), name
    # the allowance for a weight that is rounded once does not
    assert ((cases.weighted(b, _bf16) - want).abs() <= wide).all()
