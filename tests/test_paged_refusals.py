"""What the paged-attention entry points refuse, one argument changed at a time: every
buffer of the unchanged call has addresses of its own, and that call is refused by
nothing but the missing GPU."""
import ctypes as C
import math
import time

import pytest
import torch

import mixture_experts_layer_22_b200 as moe
from mixture_experts_layer_22_b200 import build as mbuild

# The addresses are made up: a call that is not refused may only run where nothing can
# be launched.
pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="made-up addresses: for hosts without a GPU")

INVALID, UNSUPPORTED, TOO_SMALL, NO_GPU = -1, -2, -3, -4          # MOE_ERR_*; the last is what a launch gives here


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


@pytest.mark.parametrize("kw", [dict(B=0), dict(B=-1), dict(B=4097), dict(max_tokens=-1), dict(max_tokens=(1 << 30) + 1), dict(max_pages=0),
                                dict(page_size=0), dict(num_pages=0), dict(n_free=-1), dict(num_pages=1 << 20, page_size=1 << 11),
                                dict(max_pages=1 << 20, page_size=1 << 11)], ids=str)
def test_plan_refuses_each_bad_size(lib, kw):
    assert _plan(lib) == NO_GPU
    # far apart: some of these sizes would reach the next buffer
    far = {n: a << 16 for n, a in PLAN_AT.items()}
    assert _plan(lib, **far) == NO_GPU and _plan(lib, kw, **far) == INVALID


@pytest.mark.parametrize("name", ["cached", "fresh", "free_pages", "block_table", "q_start", "kv_len", "positions", "slots"])
def test_plan_refuses_each_null(lib, name):
    assert _plan(lib, **{name: None}) == INVALID


def test_plan_takes_what_may_be_missing(lib):
    for name in ("free_pos", "free_next", "status"):
        assert _plan(lib, **{name: None}) == NO_GPU
    assert _plan(lib, dict(n_free=0), free_pages=None) == NO_GPU
    assert _plan(lib, dict(max_tokens=0), positions=None, slots=None) == NO_GPU
    # the cursor is not its own successor, and that alone is refused
    assert _plan(lib, free_next=PLAN_AT["free_pos"]) == INVALID
    assert lib.moe_page_plan(None, *PLAN_AT.values(), None) == INVALID


@pytest.mark.parametrize("kw,code", [
    (dict(num_tokens=-1), -1), (dict(n_heads=0), -1), (dict(n_heads=65537), -1), (dict(n_kv_heads=0), -1), (dict(n_kv_heads=65537), -1),
    (dict(rot_dim=-2), -1), (dict(rot_dim=130), -1), (dict(rot_dim=7), -1), (dict(rot_dim=24), -2), (dict(max_pos=0), -1),
    (dict(interleaved=2), -1), (dict(page_size=0), -1), (dict(num_pages=0), -1), (dict(cache_dtype=2), -1),
    (dict(head_dim=96, rot_dim=96), -2), (dict(q_stride=1016), -1), (dict(q_stride=1028), -1), (dict(k_stride=128), -1),
    (dict(k_stride=260), -1), (dict(v_stride=128), -1), (dict(v_stride=260), -1), (dict(page_stride=4088), -1),
    (dict(page_stride=4080), -1), (dict(page_stride=4104), -1), (dict(cache_dtype=1, k_scale=0.0), -1),
    (dict(cache_dtype=1, v_scale=-1.0), -1), (dict(cache_dtype=1, k_scale=math.nan), -1), (dict(cache_dtype=1, v_scale=math.nan), -1),
    (dict(cache_dtype=1, k_scale=math.inf), -1), (dict(cache_dtype=1, v_scale=math.inf), -1), (dict(num_pages=1 << 27), -1),
    (dict(q_stride=1 << 62), -1), (dict(k_stride=1 << 62), -1), (dict(v_stride=1 << 62), -1), (dict(page_stride=1 << 62), -1)], ids=str)
def test_append_refuses_each_bad_size(lib, kw, code):
    far = {n: a << 16 for n, a in APPEND_AT.items()}
    assert _append(lib, **far) == NO_GPU and _append(lib, kw, **far) == code


def test_append_refuses_each_null_and_misaligned(lib):
    for name in list(APPEND_AT)[:-1]:
        assert _append(lib, **{name: None}) == INVALID
    for name in ("q", "k", "v", "q_out", "k_cache", "v_cache"):
        assert _append(lib, **{name: APPEND_AT[name] + 8}) == INVALID
    assert _append(lib, cos_sin=APPEND_AT["cos_sin"] + 2) == INVALID
    assert lib.moe_rope_append(None, *APPEND_AT.values(), None) == INVALID
    assert _append(lib, status=None) == NO_GPU
    assert _append(lib, dict(rot_dim=0), positions=None, cos_sin=None) == NO_GPU
    assert _append(lib, dict(num_tokens=0), **{n: None for n in APPEND_AT}) == 0


BAD_ATTN = [
    (dict(B=0), -1), (dict(B=4097), -1), (dict(num_tokens=-1), -1), (dict(n_heads=0), -1), (dict(n_heads=9), -1),
    (dict(n_heads=65538), -1), (dict(n_kv_heads=0), -1), (dict(n_kv_heads=3), -1), (dict(head_dim=96), -2), (dict(page_size=0), -1),
    (dict(num_pages=0), -1), (dict(max_pages=0), -1), (dict(causal=2), -1), (dict(max_q=-1), -1), (dict(cache_dtype=2), -1),
    (dict(q_stride=1000), -1), (dict(q_stride=1016), -1), (dict(q_stride=1028), -1), (dict(page_stride=4080), -1),
    (dict(page_stride=4104), -1), (dict(scale=math.nan), -1), (dict(scale=math.inf), -1), (dict(scale=-math.inf), -1),
    (dict(cache_dtype=1, k_scale=0.0), -1), (dict(cache_dtype=1, k_scale=math.inf), -1), (dict(cache_dtype=1, v_scale=math.nan), -1),
    (dict(cache_dtype=1, v_scale=-1.0), -1), (dict(num_pages=1 << 27), -1), (dict(max_pages=1 << 27), -1), (dict(q_stride=1 << 62), -1),
    (dict(page_stride=1 << 62), -1), (dict(num_tokens=1 << 29), -1),
    # times log2(e), and with codes times k_scale, beyond fp32: 0 x infinity is no score
    (dict(scale=3e38), -1), (dict(scale=-3e38), -1), (dict(cache_dtype=1, scale=1e20, k_scale=1e20), -1)]


@pytest.mark.parametrize("kw,code", BAD_ATTN, ids=str)
def test_attention_refuses_each_bad_size(lib, kw, code):
    s = moe.AttnShape(**{**ATTN, **kw})
    far = {n: a << 16 for n, a in ATTN_AT.items()}
    assert _attention(lib, ws_bytes=1 << 40, **far) == NO_GPU
    assert lib.moe_attn_workspace_size(C.byref(s), C.byref(C.c_size_t())) == code
    assert _attention(lib, kw, ws_bytes=1 << 40, **far) == code


def test_attention_refuses_each_null_misaligned_and_small(lib):
    for name in ("q", "k_cache", "v_cache", "block_table", "q_start", "kv_len", "out", "ws"):
        assert _attention(lib, **{name: None}) == INVALID
    for name in ("q", "k_cache", "v_cache", "out"):
        assert _attention(lib, **{name: ATTN_AT[name] + 8}) == INVALID
    for off in (8, 16, 128):
        assert _attention(lib, ws=ATTN_AT["ws"] + off) == INVALID
    need = moe.attn_workspace_size(moe.AttnShape(**ATTN))
    assert _attention(lib, ws_bytes=need - 1) == TOO_SMALL and _attention(lib, ws_bytes=need) == NO_GPU
    assert _attention(lib, status=None) == NO_GPU
    assert lib.moe_paged_attention(None, *ATTN_AT.values(), need, None) == INVALID
    assert lib.moe_attn_workspace_size(C.byref(moe.AttnShape(**ATTN)), None) == INVALID
    assert _attention(lib, dict(num_tokens=0), ws_bytes=0, **{n: None for n in ATTN_AT}) == 0


@pytest.mark.parametrize("gap", [0, 3])
def test_append_checks_alternating_pages_at_once(lib, gap):
    """K and V pages that alternate in one buffer, 16 million of each, perhaps of several
    layers: the check does not go from page to page."""
    page = 16 * 2 * 128
    shape = dict(page_stride=(2 + gap) * page, num_pages=1 << 24)
    far = {n: a << 20 for n, a in APPEND_AT.items()}
    far["v_cache"] = far["k_cache"] + 2 * page
    t0 = time.perf_counter()
    for _ in range(20):
        assert _append(lib, shape, **far) == NO_GPU
    assert time.perf_counter() - t0 < 0.3
    for off in (16, -16):
        moved = {**far, "v_cache": far["v_cache"] + off}
        assert _append(lib, shape, **moved) == (INVALID if off < 0 or gap == 0 else NO_GPU)
    # within the first gap of K and behind its last page: only whole pages count
    last = far["k_cache"] + 2 * (2 + gap) * page * ((1 << 24) - 1)
    assert _append(lib, shape, **{**far, "v_cache": last + 2 * page}) == NO_GPU
    assert _append(lib, shape, **{**far, "v_cache": last + 2 * page - 16}) == INVALID
