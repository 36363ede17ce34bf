"""What the paged-attention entry points refuse, one argument changed at a time: every
buffer of the unchanged call has addresses of its own, and that call is refused by
nothing but the missing GPU."""
import ctypes as C

import pytest
import torch

import mixture_experts_layer_22_b200 as moe
from mixture_experts_layer_22_b200 import build as mbuild

# The addresses are made up: a call that is not refused may only run where nothing can
# be launched.
pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="made-up addresses: for hosts without a GPU")

INVALID, NO_GPU = -1, -4          # MOE_ERR_INVALID_ARG, MOE_ERR_CUDA


@pytest.fixture(scope="module")
def lib():
    mbuild.build()
    return moe.lib()


def _apart(names):
    """An address for each name, 256 MB apart."""
    return {n: (i + 1) << 28 for i, n in enumerate(names)}


# ------------------------------------------------------------- the attention
ATTN = dict(B=4, num_tokens=8, n_heads=8, n_kv_heads=2, head_dim=128, page_size=16, num_pages=64, max_pages=8, causal=1, max_q=0,
            cache_dtype=0, scale=0.1, k_scale=1.0, v_scale=1.0)
ATTN_AT = _apart(["q", "k_cache", "v_cache", "block_table", "q_start", "kv_len", "out", "status", "ws"])


def _attention(lib, shape=None, ws_bytes=None, **at):
    s = moe.AttnShape(**{**ATTN, **(shape or {})})
    p = {**ATTN_AT, **at}
    return lib.moe_paged_attention(C.byref(s), *(p[n] for n in ATTN_AT), moe.attn_workspace_size(s) if ws_bytes is None else ws_bytes,
                                   None)


def _attn_bytes(shape=None):
    a = {**ATTN, **(shape or {})}
    esz = 1 if a["cache_dtype"] else 2
    row, page = a["n_heads"] * a["head_dim"], a["page_size"] * a["n_kv_heads"] * a["head_dim"]
    q = (a["num_tokens"] - 1) * (a.get("q_stride") or row) + row
    cache = (a["num_pages"] - 1) * (a.get("page_stride") or page) + page
    return dict(q=2 * q, k_cache=esz * cache, v_cache=esz * cache, block_table=4 * a["B"] * a["max_pages"], q_start=4 * (a["B"] + 1),
                kv_len=4 * a["B"], out=2 * a["num_tokens"] * row, status=4, ws=moe.attn_workspace_size(moe.AttnShape(**a)))


def _up(x, a):
    return -(-x // a) * a


@pytest.mark.parametrize("shape", [{}, dict(cache_dtype=1), dict(q_stride=12 * 128), dict(page_stride=2 * 16 * 2 * 128)], ids=str)
@pytest.mark.parametrize("written,align", [("out", 16), ("ws", 256), ("status", 4)])
@pytest.mark.parametrize("over", ["q", "k_cache", "v_cache", "block_table", "q_start", "kv_len", "out", "ws", "status"])
def test_attention_writes_over_nothing_else(lib, shape, written, align, over):
    if written == over:
        return
    n = _attn_bytes(shape)
    assert _attention(lib, shape) == NO_GPU
    at = ATTN_AT[over]
    # the same address, the first byte on the other's last, the last byte on its first
    first_on_last, last_on_first = (at + n[over] - 1) // align * align, _up(at - n[written] + 1, align)
    for x in (at, first_on_last, last_on_first):
        assert _attention(lib, shape, **{written: x}) == INVALID
    # side by side
    for x in (_up(at + n[over], align), (at - n[written]) // align * align):
        assert _attention(lib, shape, **{written: x}) == NO_GPU


def test_attention_output_shifted_within_the_queries(lib):
    row = 8 * 128 * 2
    for shift in (-7 * row, -row, -16, 16, row, 7 * row):
        assert _attention(lib, out=ATTN_AT["q"] + shift) == INVALID
    assert _attention(lib, out=ATTN_AT["q"] + 8 * row) == NO_GPU


def test_attention_takes_buffers_between_the_rows_of_others(lib):
    """One token's output beside its queries in a fused projection's row; K and V pages
    that alternate, with the output in a gap of theirs; one cache for both."""
    head = 128 * 2
    fused = dict(num_tokens=1, q_stride=40 * 128)
    assert _attention(lib, fused, out=ATTN_AT["q"] + 8 * head) == NO_GPU
    assert _attention(lib, fused, out=ATTN_AT["q"] + 7 * head) == INVALID
    page = 16 * 2 * 128
    gaps = dict(page_stride=4 * page)
    k = ATTN_AT["k_cache"]
    assert _attention(lib, gaps, v_cache=k + 2 * page) == NO_GPU
    assert _attention(lib, gaps, v_cache=k + 2 * page, out=k + 2 * 2 * page) == NO_GPU
    assert _attention(lib, gaps, v_cache=k + 2 * page, out=k + 2 * 2 * page - 16) == INVALID
    assert _attention(lib, gaps, v_cache=k + 2 * page, out=k + 2 * 9 * 4 * page + 16) == INVALID
    assert _attention(lib, v_cache=k) == NO_GPU
