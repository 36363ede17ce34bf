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


# --------------------------------------------- where the inverse rotary step belongs
@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("il,rot", [(0, 128), (0, 64), (1, 64)])
@pytest.mark.parametrize("shift", [0, 1000])
def test_inverse_rotary_step_behind_keys_that_are_the_values(il, rot, e4m3, shift):
    """Plan, append, attention with the key cache as both caches, inverse rotary step:
    sum_j p_ij R(x_j - x_i) k_j, p = softmax_j(scale q_i . R(x_j - x_i) k_j), a
    function of distances alone, wherever the positions x start."""
    H, D, ps, max_pos = 4, 128, 16, 2048
    lens = [40, 90]
    T = sum(lens)
    g = torch.Generator().manual_seed(26)
    w = 1e4 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    ang = torch.arange(max_pos, dtype=torch.float64)[:, None] * w
    table = torch.cat([ang.cos(), ang.sin()], 1)
    q = (torch.randn(T, H, D, generator=g) * 0.1).to(torch.bfloat16)
    k = torch.randn(T, 1, D, generator=g).to(torch.bfloat16)
    sc = 1 / 64 if e4m3 else 1.0

    def i32(x):
        return torch.tensor(x, dtype=torch.int32, device="cuda")
    pages = 12
    blocks, q_start, kv_len, pos, slots = i32([[-1] * 8] * 2), i32([0] * 3), i32([0] * 2), i32([0] * T), i32([0] * T)
    moe.page_plan(moe.PageShape(B=2, max_tokens=T, max_pages=8, page_size=ps, num_pages=pages, n_free=pages), i32([0, 0]), i32(lens),
                  i32(list(range(pages))[::-1]), blocks, q_start, kv_len, pos, slots)
    pos += shift
    dt = torch.uint8 if e4m3 else torch.bfloat16
    kc, vc = (torch.zeros(pages, ps, 1, D, dtype=dt, device="cuda") for _ in range(2))
    q_rot = torch.empty(T, H, D, dtype=torch.bfloat16, device="cuda")
    cs, status = table.float().cuda(), i32([0])
    dk = k.cuda()
    moe.rope_append(moe.AppendShape(num_tokens=T, n_heads=H, n_kv_heads=1, head_dim=D, rot_dim=rot, max_pos=max_pos, interleaved=il,
                                    page_size=ps, num_pages=pages, cache_dtype=int(e4m3), k_scale=sc, v_scale=sc),
                    q.cuda(), dk, dk, pos, slots, cs, q_rot, kc, vc, status)
    s = moe.AttnShape(B=2, num_tokens=T, n_heads=H, n_kv_heads=1, head_dim=D, page_size=ps, num_pages=pages, max_pages=8, causal=1,
                      max_q=max(lens), cache_dtype=int(e4m3), scale=D ** -0.5, k_scale=sc, v_scale=sc)
    out, codes = torch.empty_like(q_rot), torch.empty(T, H, D, dtype=torch.uint8, device="cuda")
    scales = torch.empty(T, H, device="cuda")
    moe.paged_attention(s, q_rot, kc, kc, blocks, q_start, kv_len, out, moe.attn_workspace(s), status)
    moe.inv_rope_quant(moe.RopeShape(num_tokens=T, n_heads=H, head_dim=D, rot_dim=rot, max_pos=max_pos, interleaved=il), out, pos, cs,
                       codes, scales, status)
    got = codes.view(torch.float8_e4m3fn).cpu().double() * scales.cpu().double()[..., None]
    assert int(status[0]) == 0

    # The key at position x_j rounded in its cache and the query in its buffer: u_k and 2^-8 of each rotated element (a
    # pair's elements mix, so both count by the larger of the pair's, sqrt(2) at most), and the table's fp32.
    u_k, step = (ref.U_E4M3, 2.0 ** -10 * sc) if e4m3 else (ref.U_BF16, 0.0)
    u_q, tab = ref.U_BF16, 4 * ref.U_F32
    at, planted = 0, False
    for n in lens:
        qq, kk = q[at:at + n].double(), k[at:at + n, 0].double()
        far = max_pos // 2                               # distance d in row far + d of a table of its own
        a = (torch.arange(max_pos, dtype=torch.float64) - far)[:, None] * w
        rel = torch.cat([a.cos(), a.sin()], 1)
        for i in range(n):
            # the keys as position i sees them
            seen = ref.rotate(kk[:i + 1, None], rel, torch.arange(i + 1) - i + far, rot, bool(il))[:, 0]
            norm = _pair_norm(seen, rot, il)
            p = torch.softmax(qq[i] @ seen.T * D ** -0.5, -1)
            want = p @ seen
            mag = (_pair_norm(qq[i], rot, il) @ norm.T) * 2 * D ** -0.5
            e_s = mag.amax(-1, keepdim=True) * (u_k + u_q + u_k * u_q + 2 * tab + (D + 8) * ref.U_F32)
            e_s = e_s + _pair_norm(qq[i], rot, il).sum(-1, keepdim=True) * step * D ** -0.5
            A = p @ norm
            u_p = ref.U_F16 if e4m3 else ref.U_BF16
            # in the rotated basis; an element of the result takes its pair's two, at most sqrt(2) of the larger
            err = 2 ** 0.5 * (A * (torch.expm1(2 * e_s) * (1 + u_k) + u_k + 2 * tab + u_p + 2 ** -20) + A * ref.U_BF16 + 2 * step)
            size = (A + err).amax(-1, keepdim=True)
            tol = err * (1 + ref.U_E4M3) + ref.U_E4M3 * want.abs() + size * (2.0 ** -10 / 448 * 1.1 + 2.0 ** -20)
            assert ((got[at + i] - want).abs() <= tol).all()
            # values without a rotation, turned back all the same: what the chain must not be used for
            turned = ref.rotate((p @ kk[:i + 1])[None], torch.cat([table[:, :rot // 2], -table[:, rot // 2:]], 1),
                                torch.tensor([i + shift]), rot, bool(il))[0]
            planted |= bool(((turned - want).abs() > tol).any())
        at += n
    assert planted


def _pair_norm(x, rot, il):
    """Each element's size as a rotation can make it: its pair's length."""
    y = x.abs().clone()
    if il:
        n = (x[..., 0:rot:2] ** 2 + x[..., 1:rot:2] ** 2).sqrt()
        y[..., 0:rot:2], y[..., 1:rot:2] = n, n
    else:
        n = (x[..., :rot // 2] ** 2 + x[..., rot // 2:rot] ** 2).sqrt()
        y[..., :rot // 2], y[..., rot // 2:rot] = n, n
    return y


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("power", [-100, 100, 107])
def test_values_near_either_end_of_the_range(dim, power):
    """Values of up to 2^(power + 2.3), 700 keys: below 2^119 / kv_len.  Times a power of two
    everything keeps its roundings."""
    b = ref.Batch([1, 45, 2, 1], [130, 300, 2, 700], heads=8, kv_heads=2, dim=dim, seed=27)
    assert max(float(v.abs().max()) for v in b.v) < 2 ** 2.3
    d = Dev(b)
    d.v_cache = (d.v_cache.float() * 2.0 ** power).to(torch.bfloat16)
    out = d.run().cpu().double() * 2.0 ** -power
    want, tol = b.reference()
    assert int(d.status[0]) == 0 and ((out - want).abs() <= tol).all()
