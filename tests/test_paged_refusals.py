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


# ---------------------------------------------------------------- the append
APPEND = dict(num_tokens=8, n_heads=8, n_kv_heads=2, head_dim=128, rot_dim=128, max_pos=64, interleaved=0, page_size=16,
              num_pages=64, cache_dtype=0, k_scale=1.0, v_scale=1.0)
APPEND_AT = _apart(["q", "k", "v", "positions", "slots", "cos_sin", "q_out", "k_cache", "v_cache", "status"])


def _append(lib, shape=None, **at):
    s = moe.AppendShape(**{**APPEND, **(shape or {})})
    p = {**APPEND_AT, **at}
    return lib.moe_rope_append(C.byref(s), *(p[n] for n in APPEND_AT), None)


def _append_bytes(shape=None):
    a = {**APPEND, **(shape or {})}
    esz, n = 1 if a["cache_dtype"] else 2, a["num_tokens"]
    q, kv = a["n_heads"] * a["head_dim"], a["n_kv_heads"] * a["head_dim"]
    page = a["page_size"] * kv
    cache = esz * ((a["num_pages"] - 1) * (a.get("page_stride") or page) + page)
    rows = {x: 2 * ((n - 1) * (a.get(x + "_stride") or w) + w) for x, w in (("q", q), ("k", kv), ("v", kv))}
    return dict(**rows, positions=4 * n, slots=4 * n, cos_sin=4 * a["max_pos"] * a["rot_dim"], q_out=2 * n * q, k_cache=cache,
                v_cache=cache, status=4)


@pytest.mark.parametrize("shape", [{}, dict(cache_dtype=1), dict(q_stride=12 * 128, k_stride=12 * 128, v_stride=12 * 128),
                                   dict(page_stride=2 * 16 * 2 * 128)], ids=str)
@pytest.mark.parametrize("written,align", [("q_out", 16), ("k_cache", 16), ("v_cache", 16), ("status", 4)])
@pytest.mark.parametrize("over", list(APPEND_AT))
def test_append_writes_over_nothing_else(lib, shape, written, align, over):
    if written == over:
        return
    n = _append_bytes(shape)
    assert _append(lib, shape) == NO_GPU
    at = APPEND_AT[over]
    step = align if over != "q" or written != "q_out" else 2 * align
    for x in (at, (at + n[over] - 1) // align * align, _up(at - n[written] + 1, align), at + step):
        if x >= at + n[over] or (x == at and {written, over} in ({"q_out", "q"}, {"k_cache", "v_cache"})):
            continue                                     # behind it, or one of the two forms that are allowed
        assert _append(lib, shape, **{written: x}) == INVALID
    for x in (_up(at + n[over], align), (at - n[written]) // align * align):
        assert _append(lib, shape, **{written: x}) == NO_GPU


def test_append_in_place_and_one_cache(lib):
    """q_out on q where q's rows are adjacent, one cache for both; neither shifted."""
    row, page = 8 * 128 * 2, 16 * 2 * 128 * 2
    assert _append(lib, q_out=APPEND_AT["q"]) == NO_GPU
    assert _append(lib, dict(q_stride=12 * 128), q_out=APPEND_AT["q"]) == INVALID
    for shift in (-row, -256, 256, row):
        assert _append(lib, q_out=APPEND_AT["q"] + shift) == INVALID
    assert _append(lib, v_cache=APPEND_AT["k_cache"]) == NO_GPU
    for shift in (-page, -256, 256, page):
        assert _append(lib, v_cache=APPEND_AT["k_cache"] + shift) == INVALID


def test_append_takes_alternating_pages_and_unread_tables(lib):
    page = 16 * 2 * 128
    k = APPEND_AT["k_cache"]
    assert _append(lib, dict(page_stride=2 * page), v_cache=k + 2 * page) == NO_GPU
    assert _append(lib, dict(page_stride=2 * page), v_cache=k + 2 * page - 16) == INVALID
    assert _append(lib, dict(page_stride=2 * page, cache_dtype=1), v_cache=k + page) == NO_GPU
    # without a rotation the positions and the table are not read
    assert _append(lib, dict(rot_dim=0), positions=APPEND_AT["q_out"], cos_sin=APPEND_AT["k_cache"]) == NO_GPU
    # a fused projection's rows, one buffer for q, k and v
    st = dict(q_stride=12 * 128, k_stride=12 * 128, v_stride=12 * 128)
    q = APPEND_AT["q"]
    assert _append(lib, st, k=q + 8 * 256, v=q + 10 * 256) == NO_GPU
    assert _append(lib, {**st, "num_tokens": 1}, k=q + 8 * 256, v=q + 10 * 256, q_out=q + 12 * 256) == NO_GPU


# ------------------------------------------------------------------ the plan
PLAN = dict(B=4, max_tokens=16, max_pages=8, page_size=16, num_pages=64, n_free=10)
PLAN_AT = _apart(["cached", "fresh", "free_pages", "free_pos", "block_table", "q_start", "kv_len", "positions", "slots", "free_next",
                  "status"])
PLAN_WORDS = dict(cached=4, fresh=4, free_pages=10, free_pos=1, block_table=32, q_start=5, kv_len=4, positions=16, slots=16,
                  free_next=1, status=1)


def _plan(lib, shape=None, **at):
    p = {**PLAN_AT, **at}
    return lib.moe_page_plan(C.byref(moe.PageShape(**{**PLAN, **(shape or {})})), *(p[n] for n in PLAN_AT), None)


@pytest.mark.parametrize("written", list(PLAN_AT)[4:])
@pytest.mark.parametrize("over", list(PLAN_AT))
def test_plan_writes_over_nothing_else(lib, written, over):
    if written == over:
        return
    assert _plan(lib) == NO_GPU
    at, n, m = PLAN_AT[over], 4 * PLAN_WORDS[over], 4 * PLAN_WORDS[written]
    for x in (at, at + n - 4, at - m + 4):
        assert _plan(lib, **{written: x}) == INVALID
    for x in (at + n, at - m):
        assert _plan(lib, **{written: x}) == NO_GPU
