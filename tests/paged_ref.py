"""Plain 64-bit forms of the paged-attention operators, on the CPU, and the
batches the tests run them on."""
from __future__ import annotations

import numpy as np
import torch

U_BF16, U_F16, U_F32, U_E4M3 = 2.0 ** -8, 2.0 ** -11, 2.0 ** -24, 2.0 ** -4   # half a step, relative


def plan(cached, fresh, free, free_pos, table, ps, num_pages, max_tokens):
    """(table, q_start, kv_len, positions, slots, free_next, bad) by loops."""
    table = table.copy()
    B, max_pages = table.shape
    q_start, kv_len = [0], []
    pos, slot = np.zeros(max_tokens, np.int32), np.full(max_tokens, -1, np.int32)
    bad = False
    at = free_pos
    if not 0 <= at <= len(free):
        bad, at = True, len(free)
    for b in range(B):
        c, f = int(cached[b]), int(fresh[b])
        if c < 0 or f < 0 or c + f > max_pages * ps:
            bad, c, f = True, 0, 0
        for j in range(-(-c // ps), -(-(c + f) // ps)):
            page = int(free[at]) if at < len(free) else -1
            if not 0 <= page < num_pages:
                bad, page = True, -1
            table[b, j] = page
            at += 1
        for i in range(f):
            t = q_start[-1] + i
            if t >= max_tokens:
                bad = True
                break
            page = int(table[b, (c + i) // ps])
            if not 0 <= page < num_pages:
                bad, page = True, -1
            pos[t] = c + i
            slot[t] = page * ps + (c + i) % ps if page >= 0 else -1
        q_start.append(q_start[-1] + f)
        kv_len.append(c + f)
    return table, np.array(q_start, np.int32), np.array(kv_len, np.int32), pos, slot, min(at, len(free)), bad


def rotate(x, cos_sin, positions, rot, interleaved):
    """x [T, H, D] float64 turned by its positions' angles."""
    y = x.clone()
    if rot == 0:
        return y
    cs = cos_sin.double()[positions.long()][:, None]
    c, s = cs[..., :rot // 2], cs[..., rot // 2:]
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2], y[..., 1:rot:2] = a * c - b * s, b * c + a * s
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y[..., :rot // 2], y[..., rot // 2:rot] = a * c - b * s, b * c + a * s
    return y


def cache_values(cache):
    """A CPU cache in float64 (E4M3 codes decoded)."""
    return (cache.view(torch.float8_e4m3fn) if cache.dtype == torch.uint8 else cache).double()


def attention(q, k, v, q_lens, kv_lens, causal, scale, u_p):
    """Outputs and how far a kernel may be from them.

    q [T, H, D]; k, v: per request [kv, G, D]; all float64.  The bound per
    element, with A = sum_j p_j |v_j| (so |out| <= A):
      out's own rounding            U_BF16 |out|
      p's rounding before p v       u_p A (p in 16 bits; for fp16 p, formed times
                                    2^7 at least, also half its smallest step,
                                    2^-32, per key)
      scores: D products and sums in fp32, the scale and the exponent's argument
      (|s| log2 e large) rounded: an error e_s in s changes p by e_s p, in
      numerator and denominator    2 e_s A
      ex2's 2^-22 and the running sums of n terms, rescaled: 2 (2^-22 + (n + 64) U_F32) A
    """
    T, H, D = q.shape
    out, tol = torch.zeros_like(q), torch.zeros_like(q)
    at = 0
    for b, (n, kv) in enumerate(zip(q_lens, kv_lens)):
        g = k[b].shape[1]
        r = H // g
        for h in range(H):
            kk, vv = k[b][:, h // r], v[b][:, h // r]
            x = q[at:at + n, h] @ kk.T * scale
            mag = q[at:at + n, h].abs() @ kk.abs().T * abs(scale)
            seen = torch.ones(n, kv, dtype=torch.bool)
            if causal:
                seen = torch.arange(kv)[None] <= (kv - n + torch.arange(n))[:, None]
            x = torch.where(seen, x, -torch.inf)
            some = seen.any(1, keepdim=True)
            p = torch.where(some, torch.softmax(x, -1), 0.0) if kv else x
            out[at:at + n, h] = p @ vv
            A = p @ vv.abs()
            e_s = (mag.amax(-1, keepdim=True) if kv else torch.zeros(n, 1)) * (D + 8) * U_F32
            vmax = vv.abs().max() if kv else 0.0
            tol[at:at + n, h] = (U_BF16 * (p @ vv).abs() + A * (u_p + 2 * e_s + 2 * (2.0 ** -22 + (kv + 64) * U_F32)) +
                                 (kv * 2.0 ** -32 * vmax if u_p == U_F16 else 0.0) + 2.0 ** -130)
        at += n
    return out, tol


class Batch:
    """A batch of requests with its cache, as tensors on the CPU; every cache
    position that no request holds is NaN."""

    def __init__(self, q_lens, kv_lens, *, heads=8, kv_heads=2, dim=128, ps=16, causal=True, e4m3=False, seed=0,
                 spread=2.0, pad_rows=0, interleaved_kv=False, qkv=False, scale=None):
        g = torch.Generator().manual_seed(seed)
        self.q_lens, self.kv_lens = list(q_lens), list(kv_lens)
        self.heads, self.kv_heads, self.dim, self.ps, self.causal, self.e4m3 = heads, kv_heads, dim, ps, causal, e4m3
        self.B, self.T = len(q_lens), sum(q_lens) + pad_rows
        pages = [-(-kv // ps) for kv in kv_lens]
        self.num_pages, self.max_pages = sum(pages) + 3, max(max(pages), 1) + 1
        self.table = torch.full((self.B, self.max_pages), -1, dtype=torch.int32)
        order = torch.randperm(self.num_pages, generator=g).to(torch.int32)
        for b, n in enumerate(pages):
            self.table[b, :n] = order[sum(pages[:b]):sum(pages[:b]) + n]
        shape = (self.num_pages, ps, kv_heads, dim)
        dt = torch.uint8 if e4m3 else torch.bfloat16
        if interleaved_kv:                              # K and V pages alternate in one buffer
            both = torch.empty((self.num_pages, 2) + shape[1:], dtype=dt)
            self.k_cache, self.v_cache = both[:, 0], both[:, 1]
        else:
            self.k_cache, self.v_cache = torch.empty(shape, dtype=dt), torch.empty(shape, dtype=dt)
        nan = 0x7F if e4m3 else float("nan")
        self.k_cache.fill_(nan)
        self.v_cache.fill_(nan)
        self.page_stride = self.k_cache.stride(0) if interleaved_kv else 0
        self.kv_scale = 1 / 64 if e4m3 else 1.0
        self.k, self.v = [], []
        for b, kv in enumerate(kv_lens):
            for cache, rows in ((self.k_cache, self.k), (self.v_cache, self.v)):
                x = torch.randn(kv, kv_heads, dim, generator=g)
                stored = (x / self.kv_scale).to(torch.float8_e4m3fn) if e4m3 else x.to(torch.bfloat16)
                rows.append(stored.double() * self.kv_scale)
                for j in range(kv):
                    cache[self.table[b, j // ps], j % ps] = stored[j].view(torch.uint8) if e4m3 else stored[j]
        if qkv:                                         # queries beside keys and values of a fused projection
            whole = (torch.randn(self.T, heads + 2 * kv_heads, dim, generator=g) * spread).to(torch.bfloat16)
            self.q, self.q_stride = whole[:, :heads], whole.stride(0)
        else:
            self.q, self.q_stride = (torch.randn(self.T, heads, dim, generator=g) * spread).to(torch.bfloat16), 0
        self.q_start = torch.tensor([0] + list(np.cumsum(self.q_lens)), dtype=torch.int32)
        self.kv_len = torch.tensor(self.kv_lens, dtype=torch.int32)
        self.scale = dim ** -0.5 if scale is None else scale

    def reference(self, u_p=None):
        if u_p is None:
            u_p = U_F16 if self.e4m3 else U_BF16
        n = sum(self.q_lens)
        return attention(self.q[:n].double(), self.k, self.v, self.q_lens, self.kv_lens, self.causal, self.scale, u_p)
