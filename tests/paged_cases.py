"""Batches on which the places where a weight is rounded show in the output."""
import math

import numpy as np
import torch

import paged_ref as ref

# The weight p enters its product as two bf16, p_h = RN(p) and p_l = RN(p - p_h).  p - p_h is exact in fp32 and at most
# 2^-8 p, and p_l misses it by at most 2^-8 of it.
U_TWO_BF16 = ref.U_BF16 ** 2


def cancelling(q_lens, kv_lens, x, **kw):
    """Keys of weight 1 and value v beside keys of weight x and value -RN(1 / x) v, in turn:
    the sum is at most 2^-8 of its terms, so that neither the output's own rounding
    nor chance hides what happens to the weights."""
    b = ref.Batch(q_lens, kv_lens, scale=float(np.float32(-math.log(x))), **kw)
    b.q.zero_()
    b.q[..., 0] = 1
    w = torch.tensor([1.0, -0.5, 2.0, 0.25]).repeat(b.dim // 4)
    other = torch.tensor(-1 / x).to(torch.bfloat16)
    for i, kv in enumerate(b.kv_lens):
        odd = (torch.arange(kv) % 2 == 1)[:, None, None]
        k = torch.zeros(kv, b.kv_heads, b.dim)
        k[..., :1] = torch.where(odd, 0.0, 1.0)
        v = torch.where(odd, other.float() * w, w).expand(kv, b.kv_heads, b.dim)
        b.k[i], b.v[i] = k.double(), v.double()
        pages = b.table[i, torch.arange(kv) // b.ps].long()
        b.k_cache[pages, torch.arange(kv) % b.ps] = k.to(torch.bfloat16)
        b.v_cache[pages, torch.arange(kv) % b.ps] = v.to(torch.bfloat16)
    return b


def weighted(b, rounded):
    """The batch's output with `rounded` applied to the weights relative to the largest,
    on their way into the product with v only."""
    out = torch.zeros(sum(b.q_lens), b.heads, b.dim, dtype=torch.float64)
    at, r = 0, b.heads // b.kv_heads
    for i, (n, kv) in enumerate(zip(b.q_lens, b.kv_lens)):
        for h in range(b.heads):
            s = b.q[at:at + n, h].double() @ b.k[i][:, h // r].T * b.scale
            if b.causal:
                s = torch.where(torch.arange(kv)[None] <= (kv - n + torch.arange(n))[:, None], s, -torch.inf)
            p = torch.exp(s - s.amax(-1, keepdim=True))
            out[at:at + n, h] = rounded(p) @ b.v[i][:, h // r] / p.sum(-1, keepdim=True)
        at += n
    return out
