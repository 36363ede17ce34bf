"""The paged-attention entry points on the host, without a GPU: sizes, refusals
before anything is launched, and the plain forms the GPU tests compare with."""
import ctypes as C
import math

import numpy as np
import pytest
import torch

import mixture_experts_layer_22_b200 as moe
import paged_ref as ref
from mixture_experts_layer_22_b200 import build as mbuild

A = 256          # an address that is aligned for everything; nothing here reaches a launch


@pytest.fixture(scope="module")
def lib():
    mbuild.build()
    return moe.lib()


def _page(**kw):
    base = dict(B=4, max_tokens=16, max_pages=8, page_size=16, num_pages=64, n_free=10)
    base.update(kw)
    return moe.PageShape(**base)


@pytest.mark.parametrize("kw", [dict(B=0), dict(B=4097), dict(max_tokens=-1), dict(max_pages=0), dict(page_size=0),
                                dict(num_pages=0), dict(n_free=-1), dict(num_pages=1 << 20, page_size=1 << 11),
                                dict(max_pages=1 << 20, page_size=1 << 11)])
def test_page_plan_rejects_bad_shapes(lib, kw):
    assert lib.moe_page_plan(C.byref(_page(**kw)), A, A, A, None, A, A, A, A, A, 2 * A, None, None) == -1


@pytest.mark.parametrize("null", [0, 1, 2, 4, 5, 6, 7, 8])
def test_page_plan_rejects_null_pointers(lib, null):
    args = [A, A, A, None, A, A, A, A, A, 2 * A, None]
    args[null] = None
    assert lib.moe_page_plan(C.byref(_page()), *args, None) == -1
    assert lib.moe_page_plan(None, A, A, A, None, A, A, A, A, A, 2 * A, None, None) == -1


def test_page_plan_cursor_must_not_be_its_own_successor(lib):
    assert lib.moe_page_plan(C.byref(_page()), A, A, A, A, A, A, A, A, A, A, None, None) == -1


# cached, fresh, free_pages, free_pos, block_table, q_start, kv_len, positions, slots, free_next, each at
# its own address (nothing here reaches a launch)
APART = [A * (1 << i) for i in range(10)]


@pytest.mark.parametrize("out", [4, 5, 6, 7, 8, 9])
@pytest.mark.parametrize("into", [0, 1, 2, 3])
def test_page_plan_outputs_must_not_overlap_inputs(lib, out, into):
    words = dict(zip(range(10), (4, 4, 10, 1, 32, 5, 4, 16, 16, 1)))
    for at in (APART[into], APART[into] + 4 * (words[into] - 1), APART[into] - 4 * (words[out] - 1)):
        args = list(APART)
        args[out] = at
        assert lib.moe_page_plan(C.byref(_page()), *args, None, None) == -1


def _append(**kw):
    base = dict(num_tokens=8, n_heads=8, n_kv_heads=2, head_dim=128, rot_dim=128, max_pos=64, interleaved=0, page_size=16,
                num_pages=64, cache_dtype=0, k_scale=1.0, v_scale=1.0)
    base.update(kw)
    return moe.AppendShape(**base)


@pytest.mark.parametrize("kw,code", [
    (dict(num_tokens=-1), -1), (dict(n_heads=0), -1), (dict(n_kv_heads=0), -1), (dict(rot_dim=-2), -1),
    (dict(rot_dim=130), -1), (dict(rot_dim=7), -1), (dict(rot_dim=24), -2), (dict(max_pos=0), -1),
    (dict(interleaved=2), -1), (dict(page_size=0), -1), (dict(num_pages=0), -1), (dict(cache_dtype=2), -1),
    (dict(head_dim=96, rot_dim=96), -2), (dict(q_stride=1016), -1), (dict(q_stride=1028), -1), (dict(k_stride=128), -1),
    (dict(v_stride=260), -1), (dict(page_stride=4088), -1), (dict(page_stride=4104), -1),
    (dict(cache_dtype=1, k_scale=0.0), -1), (dict(cache_dtype=1, v_scale=-1.0), -1),
    (dict(cache_dtype=1, v_scale=math.nan), -1), (dict(cache_dtype=1, k_scale=math.inf), -1), (dict(num_pages=1 << 27), -1),
    (dict(q_stride=1 << 62), -1), (dict(page_stride=1 << 62), -1), (dict(num_tokens=0), 0)])
def test_rope_append_checks_shapes(lib, kw, code):
    ptr = None if code == 0 else A
    assert lib.moe_rope_append(C.byref(_append(**kw)), ptr, A, A, A, A, A, 2 * A, A, A, None, None) == code


def test_rope_append_rejects_null_and_misaligned_pointers(lib):
    good = [A, A, A, A, A, A, 2 * A, A, A]
    for i in range(9):
        args = list(good)
        args[i] = None
        assert lib.moe_rope_append(C.byref(_append()), *args, None, None) == -1
    for i in (0, 1, 2, 6, 7, 8):
        args = list(good)
        args[i] = A + 8
        assert lib.moe_rope_append(C.byref(_append()), *args, None, None) == -1
    # in place only where the rows are adjacent
    assert lib.moe_rope_append(C.byref(_append(q_stride=2048)), A, A, A, A, A, A, A, A, A, None, None) == -1


def _attn(**kw):
    base = dict(B=4, num_tokens=8, n_heads=8, n_kv_heads=2, head_dim=128, page_size=16, num_pages=64, max_pages=8, causal=1,
                max_q=0, cache_dtype=0, scale=0.1, k_scale=1.0, v_scale=1.0)
    base.update(kw)
    return moe.AttnShape(**base)


BAD_ATTN = [
    (dict(B=0), -1), (dict(B=4097), -1), (dict(num_tokens=-1), -1), (dict(n_heads=0), -1), (dict(n_heads=9), -1),
    (dict(n_kv_heads=0), -1), (dict(head_dim=96), -2), (dict(page_size=0), -1), (dict(num_pages=0), -1),
    (dict(max_pages=0), -1), (dict(causal=2), -1), (dict(max_q=-1), -1), (dict(cache_dtype=2), -1),
    (dict(q_stride=1000), -1), (dict(q_stride=1028), -1), (dict(page_stride=4088), -1), (dict(page_stride=4104), -1),
    (dict(scale=math.nan), -1), (dict(scale=math.inf), -1), (dict(cache_dtype=1, k_scale=0.0), -1),
    (dict(cache_dtype=1, v_scale=math.nan), -1), (dict(num_pages=1 << 27), -1), (dict(max_pages=1 << 27), -1),
    (dict(cache_dtype=1, k_scale=math.inf), -1), (dict(q_stride=1 << 62), -1), (dict(page_stride=1 << 62), -1),
    (dict(num_tokens=1 << 29), -1)]


@pytest.mark.parametrize("kw,code", BAD_ATTN)
def test_paged_attention_rejects_bad_shapes(lib, kw, code):
    s = _attn(**kw)
    assert lib.moe_attn_workspace_size(C.byref(s), C.byref(C.c_size_t())) == code
    assert lib.moe_paged_attention(C.byref(s), A, A, A, A, A, A, A, None, A, 1 << 40, None) == code


def test_paged_attention_rejects_null_misaligned_and_small(lib):
    s = _attn()
    need = moe.attn_workspace_size(s)
    assert need % 4 == 0
    good = [A, A, A, A, A, A, A, None, A]
    for i in (0, 1, 2, 3, 4, 5, 6, 8):
        args = list(good)
        args[i] = None
        assert lib.moe_paged_attention(C.byref(s), *args, need, None) == -1
    for i in (0, 1, 2, 6, 8):
        args = list(good)
        args[i] = A + 8
        assert lib.moe_paged_attention(C.byref(s), *args, need, None) == -1
    assert lib.moe_paged_attention(C.byref(s), *good, need - 1, None) == -3
    assert lib.moe_attn_workspace_size(C.byref(s), None) == -1
    assert lib.moe_paged_attention(C.byref(_attn(num_tokens=0)), *([None] * 9), 0, None) == 0


def test_paged_attention_output_is_not_q(lib):
    s = _attn()
    assert lib.moe_paged_attention(C.byref(s), A, A, A, A, A, A, A, None, A, moe.attn_workspace_size(s), None) == -1


def test_reference_attention_against_torch():
    """The 64-bit form the kernels are held to, against torch's own attention."""
    b = ref.Batch([3, 1, 5], [3, 40, 21], heads=4, kv_heads=2, dim=64)
    out, tol = b.reference()
    at = 0
    for i, (n, kv) in enumerate(zip(b.q_lens, b.kv_lens)):
        q = b.q[at:at + n].double().transpose(0, 1)
        k, v = (x[i].transpose(0, 1).repeat_interleave(2, 0) for x in (b.k, b.v))
        mask = torch.ones(n, kv, dtype=torch.bool).tril(kv - n)
        want = torch.nn.functional.scaled_dot_product_attention(q, k, v, attn_mask=mask).transpose(0, 1)
        assert torch.allclose(out[at:at + n], want, atol=1e-12)
        at += n
    assert (tol > 0).all() and (tol < 0.1).all()


def test_reference_attention_empty_rows():
    b = ref.Batch([4, 2], [2, 0], heads=2, kv_heads=1, dim=64)
    out, _ = b.reference()
    assert (out[:2] == 0).all() and (out[2:4] != 0).any() and (out[4:] == 0).all()


def test_reference_plan():
    table = np.full((2, 3), -1, np.int32)
    table[0, 0] = 5
    t, qs, kv, pos, slot, nxt, bad = ref.plan([3, 0], [2, 1], [7, 2, 9], 1, table, 4, 10, 4)
    assert t.tolist() == [[5, 2, -1], [9, -1, -1]] and qs.tolist() == [0, 2, 3] and kv.tolist() == [5, 1]
    assert pos.tolist() == [3, 4, 0, 0] and slot.tolist() == [23, 8, 36, -1] and nxt == 3 and not bad
