"""What the paged-attention operators are measured on: the page plan, the
rotary append into the cache, and attention over the cache.

`listed()` are fixed cases, `draw()` gives more of the same ranges.  Head
layouts follow the library's rotary workloads (32 heads x 128 and 128 heads x
64 interleaved) with grouped key/value heads; batch and token counts follow
its decode (1 to 128 tokens) and prefill (4096, 8192 tokens) configurations.
"""
import random

import torch

own = False

E4M3_MAX = 448.0


# ---------------------------------------------------------------- the cases
def listed():
    plan = dict(op="plan")
    app = dict(op="append", e4m3=False, interleaved=False)
    att = dict(op="attention", e4m3=False, causal=True)
    return [
        # one decode step of a small batch: a launch and little else
        dict(plan, name="plan decode B=64", B=64, q_min=1, q_max=1, kv_max=8192, page=16, pad=0),
        # a full server's step: most requests decode, some bring a chunk, rows padded to a graph's capacity
        dict(plan, name="plan mixed B=1024", B=1024, q_min=1, q_max=64, kv_max=32768, page=16, pad=1000),
        # the cache write of an 8-token decode step
        dict(app, name="append decode T=8", T=8, heads=32, kv_heads=8, dim=128, rot=128, page=16, pad=0),
        # a whole prefill batch in bf16
        dict(app, name="append prefill T=8192", T=8192, heads=32, kv_heads=8, dim=128, rot=128, page=64, pad=0),
        # many narrow heads, interleaved pairs, an E4M3 cache, an odd token count
        dict(app, name="append e4m3 T=4099", T=4099, heads=128, kv_heads=8, dim=64, rot=64, page=32, pad=61,
             e4m3=True, interleaved=True),
        # one user's next token: latency
        dict(att, name="decode B=1 kv=1000", B=1, q_min=1, q_max=1, kv_min=1000, kv_max=1000, heads=32, kv_heads=8,
             dim=128, page=16),
        # a decode batch of ragged lengths: the cache is read once
        dict(att, name="decode B=64 kv<=8192", B=64, q_min=1, q_max=1, kv_min=1, kv_max=8192, heads=32, kv_heads=8,
             dim=128, page=16),
        # the same with codes in the cache, at the headline batch
        dict(att, name="decode e4m3 B=128 kv<=8192", B=128, q_min=1, q_max=1, kv_min=64, kv_max=8192, heads=32,
             kv_heads=8, dim=128, page=64, e4m3=True),
        # decoding requests beside chunks of prompts, odd lengths
        dict(att, name="mixed B=16 q<=250", B=16, q_min=1, q_max=250, kv_min=250, kv_max=4001, heads=32, kv_heads=8,
             dim=128, page=16),
        # whole prompts of a prefill batch
        dict(att, name="prompts B=4 q=2048", B=4, q_min=2048, q_max=2048, kv_min=2048, kv_max=2048, heads=32,
             kv_heads=8, dim=128, page=64),
        # narrow heads, an E4M3 cache, chunks behind a cached prefix
        dict(att, name="chunk e4m3 d64 B=8 q<=512", B=8, q_min=100, q_max=512, kv_min=1000, kv_max=4096, heads=24,
             kv_heads=8, dim=64, page=32, e4m3=True),
        # the last chunk of a long document
        dict(att, name="chunk q=1024 kv=32768", B=1, q_min=1024, q_max=1024, kv_min=32768, kv_max=32768, heads=32,
             kv_heads=8, dim=128, page=64),
    ]


def _log(rng, lo, hi):
    """A whole number whose logarithm is even over [lo, hi]."""
    return min(hi, max(lo, round(lo * (hi / lo) ** rng.random())))


def draw(rng):
    op = rng.choice(["plan", "append", "attention", "attention"])
    page = rng.choice([16, 32, 64, 128])
    if op == "plan":
        B = _log(rng, 1, 1024)
        q_max = _log(rng, 1, min(2048, 65536 // B))
        return dict(op=op, B=B, q_min=rng.choice([0, 1]), q_max=q_max, kv_max=max(q_max, _log(rng, 64, 32768)),
                    page=page, pad=rng.choice([0, rng.randint(1, 1000)]))
    heads, kv_heads = rng.choice([(32, 8), (32, 4), (16, 16), (24, 8), (8, 1), (28, 4), (64, 8)])
    dim = rng.choice([64, 128, 128])
    if op == "append":
        return dict(op=op, T=_log(rng, 1, 8192), heads=heads, kv_heads=kv_heads, dim=dim,
                    rot=rng.choice([dim, dim // 2]), page=page, pad=rng.choice([0, rng.randint(1, 64)]),
                    e4m3=rng.random() < 0.5, interleaved=rng.random() < 0.5)
    while True:
        B = _log(rng, 1, 128)
        q_max = 1 if rng.random() < 0.5 else _log(rng, 2, 2048)
        kv_max = max(_log(rng, 16, 32768), q_max)
        case = dict(op=op, B=B, q_min=rng.choice([1, q_max]), q_max=q_max, kv_min=max(1, kv_max // rng.choice([1, 2, 16])),
                    kv_max=kv_max, heads=heads, kv_heads=kv_heads, dim=dim, page=page, e4m3=rng.random() < 0.4,
                    causal=rng.random() < 0.85)
        # within the largest listed case: scores of the plain form, cache rows, work
        if B * q_max * kv_max * heads <= 1.07e9 and B * kv_max * kv_heads * dim <= 1.07e9:
            return case


def _lengths(case):
    """(new tokens, tokens in all) of each request, the same for every seed."""
    r = random.Random(case["B"] * 1000003 + case["kv_max"] * 101 + case["q_max"])
    q = [r.randint(case["q_min"], case["q_max"]) for _ in range(case["B"])]
    q[r.randrange(case["B"])] = case["q_max"]
    if case["op"] == "plan":
        return q, [n + r.randint(0, case["kv_max"] - n) for n in q]
    kv = [max(n, r.randint(case["kv_min"], case["kv_max"])) for n in q]
    kv[r.randrange(case["B"])] = case["kv_max"]
    return q, kv


def _ceil(a, b):
    return -(-a // b)


def work(case):
    if case["op"] == "plan":
        q, kv = _lengths(case)
        page = case["page"]
        new = sum(_ceil(k, page) - _ceil(k - n, page) for n, k in zip(q, kv))
        partial = sum((k - n) % page != 0 and n > 0 for n, k in zip(q, kv))
        words = 2 * case["B"] + partial + 2 * new + 2 * case["B"] + 1 + 2 * (sum(q) + case["pad"]) + 2
        return {"bytes": 4 * words, "flops": 0}
    esz = 1 if case["e4m3"] else 2
    h, g, d = case["heads"], case["kv_heads"], case["dim"]
    if case["op"] == "append":
        T = case["T"]
        per = 2 * (2 * h * d + 2 * g * d) + esz * 2 * g * d + 4 * case["rot"] + 8
        return {"bytes": T * per + 4 * case["pad"], "flops": T * 3 * case["rot"] * (h + g)}
    q, kv = _lengths(case)
    pages = sum(_ceil(k, case["page"]) for k in kv)
    pairs = sum(n * k - (n * (n - 1) // 2 if case["causal"] else 0) for n, k in zip(q, kv))
    return {"bytes": sum(q) * h * d * 4 + sum(kv) * g * d * 2 * esz + 4 * (pages + 2 * case["B"] + 1),
            "flops": 4 * d * h * pairs}


# --------------------------------------------------------------- the inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _normal(gen, shape, std=1.0, dtype=torch.bfloat16):
    return (torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32) * std).to(dtype)


def _codes(gen, shape):
    """E4M3 codes of normal values of spread 64 (a scale of 1/64 brings them to 1)."""
    return _normal(gen, shape, 64.0, torch.float32).clamp_(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8)


def _plan_inputs(case, seed):
    q, kv = _lengths(case)
    gen, page, B = _gen(seed), case["page"], case["B"]
    cached = [k - n for n, k in zip(q, kv)]
    held, need = sum(_ceil(c, page) for c in cached), sum(_ceil(k, page) for k in kv)
    num_pages = need + 5
    order = torch.randperm(num_pages, generator=gen, device="cuda").to(torch.int32)
    max_pages = _ceil(max(kv) + 1, page)
    table = torch.full((B, max_pages), -1, dtype=torch.int32, device="cuda")
    n_held = _ints([_ceil(c, page) for c in cached]).long()
    at = torch.arange(max_pages, device="cuda")[None] < n_held[:, None]
    table[at] = order[:held]
    rows = sum(q) + case["pad"]
    return dict(case=case, cached=_ints(cached), fresh=_ints(q), free=order[held:].contiguous(), table=table,
                cursor=_ints([0]), num_pages=num_pages, rows=rows,
                q_start=_ints([0] * (B + 1)), kv_len=_ints([0] * B), positions=_ints([0] * rows),
                slots=_ints([0] * rows), cursor_out=_ints([0]))


def _rotary(positions, rot, base):
    w = float(base) ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
    a = torch.arange(positions, dtype=torch.float64, device="cuda")[:, None] * w
    return torch.cat([a.cos(), a.sin()], 1).to(torch.float32)


def _append_inputs(case, seed):
    gen, n, page = _gen(seed), case["T"], case["page"]
    h, g, d = case["heads"], case["kv_heads"], case["dim"]
    rows, num_pages, max_pos = n + case["pad"], _ceil(n, page) + 3, 8192
    # the queries, keys and values of a token lie side by side, as their projection writes them
    qkv = _normal(gen, (rows, h + 2 * g, d))
    slots = torch.full((rows,), -1, dtype=torch.int32, device="cuda")
    slots[:n] = torch.randperm(num_pages * page, generator=gen, device="cuda")[:n].to(torch.int32)
    dt = torch.uint8 if case["e4m3"] else torch.bfloat16
    scale = 1.0 / 64 if case["e4m3"] else 1.0
    return dict(case=case, n=n, q=qkv[:, :h], k=qkv[:, h:h + g], v=qkv[:, h + g:], slots=slots,
                positions=torch.randint(0, max_pos, (rows,), generator=gen, device="cuda", dtype=torch.int32),
                cos_sin=_rotary(max_pos, case["rot"], 1e4 if case["interleaved"] else 1e6),
                q_out=torch.zeros((rows, h, d), dtype=torch.bfloat16, device="cuda"),
                k_cache=torch.zeros((num_pages, page, g, d), dtype=dt, device="cuda"),
                v_cache=torch.zeros((num_pages, page, g, d), dtype=dt, device="cuda"), scale=scale)


def _attention_inputs(case, seed):
    q, kv = _lengths(case)
    gen, page, B = _gen(seed), case["page"], case["B"]
    h, g, d = case["heads"], case["kv_heads"], case["dim"]
    pages = [_ceil(k, page) for k in kv]
    num_pages, max_pages = sum(pages) + 2, max(pages)
    table = torch.full((B, max_pages), -1, dtype=torch.int32, device="cuda")
    at = torch.arange(max_pages, device="cuda")[None] < _ints(pages)[:, None]
    table[at] = torch.randperm(num_pages, generator=gen, device="cuda")[:sum(pages)].to(torch.int32)
    make = _codes if case["e4m3"] else _normal
    start = [0]
    for n in q:
        start.append(start[-1] + n)
    # queries of spread 2: attention that is neither flat nor on one key
    return dict(case=case, q=_normal(gen, (start[-1], h, d), 2.0), k_cache=make(gen, (num_pages, page, g, d)),
                v_cache=make(gen, (num_pages, page, g, d)), table=table, q_start=_ints(start), kv_len=_ints(kv),
                out=torch.zeros((start[-1], h, d), dtype=torch.bfloat16, device="cuda"), scale=d ** -0.5,
                kv_scale=1.0 / 64 if case["e4m3"] else 1.0, q_most=max(q))


def prepare(case, seed):
    return {"plan": _plan_inputs, "append": _append_inputs, "attention": _attention_inputs}[case["op"]](case, seed)


# ---------------------------------------------------------- the plain forms
def _plain_plan(s):
    page = s["case"]["page"]
    cached, fresh, table = s["cached"].long(), s["fresh"].long(), s["table"]
    held, need = (cached + page - 1) // page, (cached + fresh + page - 1) // page
    q_start = torch.nn.functional.pad(fresh.cumsum(0), (1, 0))
    taken = (need - held).cumsum(0)
    col = torch.arange(table.shape[1], device="cuda")[None]
    new = (col >= held[:, None]) & (col < need[:, None])
    at = (s["cursor"] + (taken - need)[:, None] + col).clamp(0, s["free"].numel() - 1)
    table.copy_(torch.where(new, s["free"][at], table))
    t = torch.arange(s["rows"], device="cuda")
    b = torch.searchsorted(q_start[1:], t, right=True).clamp(max=cached.numel() - 1)
    pos = cached[b] + t - q_start[b]
    inside = t < q_start[-1]
    slot = table[b, (pos // page).clamp(max=table.shape[1] - 1)] * page + pos % page
    i32 = torch.int32
    return dict(table=table, q_start=q_start.to(i32), kv_len=(cached + fresh).to(i32),
                positions=torch.where(inside, pos, 0).to(i32), slots=torch.where(inside, slot, -1).to(i32),
                cursor=(s["cursor"] + taken[-1]).to(i32))


def _rotate(x, cos, sin, rot, interleaved):
    y = x.clone()
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if interleaved else (x[..., :rot // 2], x[..., rot // 2:rot])
    ra, rb = a * cos - b * sin, b * cos + a * sin
    if interleaved:
        y[..., 0:rot:2], y[..., 1:rot:2] = ra, rb
    else:
        y[..., :rot // 2], y[..., rot // 2:rot] = ra, rb
    return y


def _values(cache):
    """A cache as the values it holds: E4M3 codes are seen as their type."""
    return cache.view(torch.float8_e4m3fn) if cache.dtype == torch.uint8 else cache


def _plain_append(s):
    c, n = s["case"], s["n"]
    rot = c["rot"]
    at = s["cos_sin"][s["positions"][:n].long()]
    cos, sin = at[:, None, :rot // 2], at[:, None, rot // 2:]
    q = _rotate(s["q"][:n].float(), cos, sin, rot, c["interleaved"])
    k = _rotate(s["k"][:n].float(), cos, sin, rot, c["interleaved"])
    v = s["v"][:n].float()
    s["q_out"][:n] = q.to(torch.bfloat16)
    slots = s["slots"][:n].long()
    if c["e4m3"]:
        k, v = ((x / s["scale"]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8) for x in (k, v))
    else:
        k, v = k.to(torch.bfloat16), v.to(torch.bfloat16)
    s["k_cache"].flatten(0, 1).index_copy_(0, slots, k)
    s["v_cache"].flatten(0, 1).index_copy_(0, slots, v)
    return dict(q=s["q_out"], k_cache=_values(s["k_cache"]), v_cache=_values(s["v_cache"]))


def _plain_attention(s):
    c, table = s["case"], s["table"].long().clamp(min=0)
    g, d = c["kv_heads"], c["dim"]
    r = c["heads"] // g
    B, m = table.shape[0], s["q_most"]
    start, kv_len = s["q_start"].long(), s["kv_len"].long()
    q_len = start[1:] - start[:-1]
    keys = torch.arange(table.shape[1] * c["page"], device="cuda")
    k = _values(s["k_cache"][table]).float().reshape(B, -1, g, d).permute(0, 2, 3, 1) * s["kv_scale"]
    v = _values(s["v_cache"][table]).float().reshape(B, -1, g, d).permute(0, 2, 1, 3) * s["kv_scale"]
    v = torch.where((keys[None] < kv_len[:, None])[:, None, :, None], v, 0.0)
    rows = torch.arange(m, device="cuda")
    t = (start[:-1, None] + rows).clamp(max=s["q"].shape[0] - 1)
    q = s["q"][t].float().reshape(B, m, g, r, d).permute(0, 2, 3, 1, 4)
    x = (q.reshape(B, g, r * m, d) @ k).reshape(B, g, r, m, -1) * s["scale"]
    last = (kv_len - q_len)[:, None] + rows if c["causal"] else (kv_len - 1)[:, None].expand(B, m)
    sees = (keys[None, None] <= last[:, :, None]) & (keys[None, None] < kv_len[:, None, None])
    x = torch.where(sees[:, None, None], x, float("-inf"))
    top = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(top == float("-inf"), 0.0, top))
    total = p.sum(-1, keepdim=True)
    o = (p.reshape(B, g, r * m, -1) @ v).reshape(B, g, r, m, d) / torch.where(total == 0, 1.0, total)
    o = o.permute(0, 3, 1, 2, 4).reshape(B, m, g * r, d)
    at = torch.arange(s["q"].shape[0], device="cuda")
    b = torch.searchsorted(start[1:], at, right=True)
    return o[b, at - start[b]].to(torch.bfloat16)


# ------------------------------------------------------ the library's calls
def _own_plan(s):
    import mixture_experts_layer_22_b200 as moe
    if "shape" not in s:
        B, cols = s["table"].shape
        s["shape"] = moe.PageShape(B=B, max_tokens=s["rows"], max_pages=cols, page_size=s["case"]["page"],
                                   num_pages=s["num_pages"], n_free=s["free"].numel())
    moe.page_plan(s["shape"], s["cached"], s["fresh"], s["free"], s["table"], s["q_start"], s["kv_len"],
                  s["positions"], s["slots"], s["cursor_out"], free_pos=s["cursor"])
    return dict(table=s["table"], q_start=s["q_start"], kv_len=s["kv_len"], positions=s["positions"],
                slots=s["slots"], cursor=s["cursor_out"])


def _own_append(s):
    import mixture_experts_layer_22_b200 as moe
    if "shape" not in s:
        c = s["case"]
        stride = s["q"].stride(0)
        s["shape"] = moe.AppendShape(num_tokens=s["q"].shape[0], n_heads=c["heads"], n_kv_heads=c["kv_heads"],
                                     head_dim=c["dim"], rot_dim=c["rot"], max_pos=s["cos_sin"].shape[0],
                                     interleaved=int(c["interleaved"]), page_size=c["page"],
                                     num_pages=s["k_cache"].shape[0], cache_dtype=moe.E4M3 if c["e4m3"] else moe.BF16,
                                     q_stride=stride, k_stride=stride, v_stride=stride, k_scale=s["scale"],
                                     v_scale=s["scale"])
    moe.rope_append(s["shape"], s["q"], s["k"], s["v"], s["positions"], s["slots"], s["cos_sin"], s["q_out"],
                    s["k_cache"], s["v_cache"])
    return dict(q=s["q_out"], k_cache=_values(s["k_cache"]), v_cache=_values(s["v_cache"]))


def _own_attention(s):
    import mixture_experts_layer_22_b200 as moe
    if "shape" not in s:
        c = s["case"]
        s["shape"] = moe.AttnShape(B=c["B"], num_tokens=s["q"].shape[0], n_heads=c["heads"], n_kv_heads=c["kv_heads"],
                                   head_dim=c["dim"], page_size=c["page"], num_pages=s["k_cache"].shape[0],
                                   max_pages=s["table"].shape[1], causal=int(c["causal"]), max_q=s["q_most"],
                                   cache_dtype=moe.E4M3 if c["e4m3"] else moe.BF16, scale=s["scale"],
                                   k_scale=s["kv_scale"], v_scale=s["kv_scale"])
        s["ws"] = moe.attn_workspace(s["shape"])
    moe.paged_attention(s["shape"], s["q"], s["k_cache"], s["v_cache"], s["table"], s["q_start"], s["kv_len"],
                        s["out"], s["ws"])
    return s["out"]


def run(state):
    op = state["case"]["op"]
    if own:
        return {"plan": _own_plan, "append": _own_append, "attention": _own_attention}[op](state)
    return {"plan": _plain_plan, "append": _plain_append, "attention": _plain_attention}[op](state)


# ------------------------------------------------------------ in 64 bits
def _exact_append(case, s):
    n, rot = case["T"], case["rot"]
    pos = s["positions"][:n].long()
    half = rot // 2
    c, sn = s["cos_sin"][pos, :half].double(), s["cos_sin"][pos, half:].double()
    # each pair is a complex number turned by its angle
    turn = torch.complex(c, sn)[:, None]

    def turned(x):
        x = x[:n].double()
        pairs = x[..., :rot].unflatten(-1, (half, 2)) if case["interleaved"] else x[..., :rot].unflatten(-1, (2, half)).transpose(-1, -2)
        z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
        z = z.flatten(-2) if case["interleaved"] else z.transpose(-1, -2).flatten(-2)
        return torch.cat([z, x[..., rot:]], -1)

    def stored(x, like):
        cache = torch.zeros(like.shape, dtype=torch.float64, device="cuda").flatten(0, 1)
        x = (x / s["scale"]).clamp(-E4M3_MAX, E4M3_MAX) if case["e4m3"] else x
        cache[s["slots"][:n].long()] = x
        return cache.reshape(like.shape)

    q = torch.zeros(s["q_out"].shape, dtype=torch.float64, device="cuda")
    q[:n] = turned(s["q"])
    return dict(q=q, k_cache=stored(turned(s["k"]), s["k_cache"]), v_cache=stored(s["v"][:n].double(), s["v_cache"]))


def _exact_attention(case, s):
    q_lens, kv_lens = _lengths(case)
    page, g, d = case["page"], case["kv_heads"], case["dim"]
    r = case["heads"] // g
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    at = 0
    for b, (n, kv) in enumerate(zip(q_lens, kv_lens)):
        ids = s["table"][b, :_ceil(kv, page)].long()
        hidden = torch.ones(n, kv, dtype=torch.bool, device="cuda").triu(kv - n + 1) if case["causal"] else None
        for j in range(g):
            k = _values(s["k_cache"][ids, :, j].reshape(-1, d)[:kv]).double() * s["kv_scale"]
            v = _values(s["v_cache"][ids, :, j].reshape(-1, d)[:kv]).double() * s["kv_scale"]
            x = torch.einsum("nrd,kd->rnk", s["q"][at:at + n, j * r:(j + 1) * r].double(), k) * s["scale"]
            if hidden is not None:
                x.masked_fill_(hidden, float("-inf"))
            out[at:at + n, j * r:(j + 1) * r] = torch.einsum("rnk,kd->nrd", torch.softmax(x, -1), v)
        at += n
    return out


def exact(case, seed):
    """The results in 64 bits; the plan's are whole numbers and have none."""
    if case["op"] == "plan":
        return None
    return (_exact_append if case["op"] == "append" else _exact_attention)(case, prepare(case, seed))
