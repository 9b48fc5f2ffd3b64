"""Cases, plain forms and 64-bit values of the rotary positions, the MXFP8 key/value cache and its attention.

``run`` computes one pass of an operator, in elementary torch operations or, with ``own`` set, by
the library's calls.  ``exact`` computes the same outputs in binary64.

The cache is paged: codes [pages][kv heads][page][head_dim] (E4M3) and scales [..][head_dim/32]
(E8M0, the smallest power of two that brings the block's largest magnitude to 448 or below) for
keys and values each.  Sequence s has the tokens q_starts[s] .. q_starts[s+1]-1 of a call, the last
ones of its kv_lens[s] positions; position p is in row p % page of page page_table[s][p // page].
8-bit codes and scales are returned as torch's float8_e4m3fn and float8_e8m0fnu views of the bytes.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"


# --- cases ---------------------------------------------------------------------------------

def listed():
    return [
        # queries and keys of a training step, rotated inside the rows of a fused projection (8192 tokens, the
        # benchmark's; 32 query, 8 key and 8 value heads)
        dict(name="rotary 8192 tokens", op="rotary", tokens=8192, heads=40, row_heads=48, head_dim=128, rot=128, layout="half",
             dtype="bf16", backward=False, positions=32768),
        # the gradient of a rotation of part of the head, on a short fp32 batch
        dict(name="rotary grad fp32 short", op="rotary", tokens=1021, heads=12, row_heads=12, head_dim=96, rot=72,
             layout="interleaved", dtype="f32", backward=True, positions=8192),
        # the table that a long-context program makes at its start, low frequencies stretched
        dict(name="table 131072 positions", op="table", positions=131072, rot=128, base=500000.0, factor=16.0, original=8192,
             low=1.0, high=4.0, amplitude=1.1),
        # the table of a small model
        dict(name="table 4097 positions", op="table", positions=4097, rot=64, base=10000.0, factor=1.0, original=0, low=0.0,
             high=0.0, amplitude=1.0),
        # one decoded token's keys and values: latency only
        dict(name="append 1 token", op="append", seqs=1, q_lo=1, q_hi=1, kv_lo=4000, kv_hi=4000, kv_heads=8, head_dim=128, rot=128,
             layout="half", dtype="bf16", page=64),
        # ragged prompts on their way into an empty cache
        dict(name="append prompts", op="append", seqs=5, q_lo=701, q_hi=6001, kv_lo=701, kv_hi=6001, kv_heads=8, head_dim=128,
             rot=128, layout="half", dtype="bf16", page=64),
        # one decoded token of one sequence: the card has to be filled from one cache
        dict(name="attend 1 token", op="attend", seqs=1, q_lo=1, q_hi=1, kv_lo=4000, kv_hi=4000, q_heads=32, kv_heads=8, head_dim=128,
             page=64, window=0, groups=0, shared=0),
        # a decode batch of ragged lengths: the cache's bytes are all that counts
        dict(name="attend 64 sequences", op="attend", seqs=64, q_lo=1, q_hi=1, kv_lo=301, kv_hi=16384, q_heads=32, kv_heads=8,
             head_dim=128, page=64, window=0, groups=0, shared=0),
        # ragged prompts that attend to themselves: matrix products
        dict(name="attend prompts", op="attend", seqs=3, q_lo=1021, q_hi=4096, kv_lo=1021, kv_hi=4096, q_heads=32, kv_heads=8,
             head_dim=128, page=64, window=0, groups=0, shared=0),
        # a few drafted tokens per sequence over a sliding window, every head with keys of its own
        dict(name="attend 5 tokens window", op="attend", seqs=7, q_lo=3, q_hi=5, kv_lo=77, kv_hi=3001, q_heads=12, kv_heads=12,
             head_dim=64, page=16, window=1000, groups=0, shared=0),
        # many answers to one long prompt
        dict(name="shared 64 sequences", op="attend", seqs=64, q_lo=1, q_hi=1, kv_lo=17, kv_hi=700, q_heads=32, kv_heads=8,
             head_dim=128, page=64, window=0, groups=1, shared=16384),
        # several prompts with a few answers each
        dict(name="shared 3 prompts", op="attend", seqs=11, q_lo=1, q_hi=2, kv_lo=5, kv_hi=333, q_heads=16, kv_heads=2, head_dim=64,
             page=32, window=0, groups=3, shared=2048),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rotary", "rotary", "table", "append", "append", "attend", "attend", "attend", "shared", "shared"])
    if op == "table":
        scaled = rng.random() < 0.5
        return dict(op=op, positions=_log(rng, 256, 131072), rot=2 * _log(rng, 8, 64), base=rng.choice([10000.0, 500000.0, 1e6]),
                    factor=rng.choice([2.0, 8.0, 32.0]) if scaled else 1.0, original=rng.choice([2048, 4096, 8192]) if scaled else 0,
                    low=1.0 if scaled else 0.0, high=rng.choice([4.0, 32.0]) if scaled else 0.0, amplitude=rng.choice([1.0, 1.2]))
    dim = rng.choice([64, 128, 256])
    if op in ("rotary", "append"):
        dim = rng.choice([64, 96, 128, 160, 256])
        rot = rng.choice([dim, dim, dim // 2, 2 * rng.randint(1, dim // 2)])
        layout, dtype = rng.choice(["half", "interleaved"]), rng.choice(["bf16", "bf16", "f32"])
        if op == "rotary":
            heads = _log(rng, 1, 64)
            tokens = min(_log(rng, 1, 16384), max(1, 8192 * 20 * 128 // (heads * dim)))
            return dict(op=op, tokens=tokens, heads=heads, row_heads=heads + rng.choice([0, 0, rng.randint(1, 8)]), head_dim=dim, rot=rot,
                        layout=layout, dtype=dtype, backward=rng.random() < 0.5, positions=rng.choice([4096, 32768, 131072]))
        seqs, heads = _log(rng, 1, 64), rng.choice([1, 2, 4, 8, 12])
        q = _log(rng, 1, max(1, 6000 * 8 * 128 // (seqs * heads * dim)))
        kv = q + rng.choice([0, _log(rng, 1, 4096)])
        return dict(op=op, seqs=seqs, q_lo=max(1, q // 3), q_hi=q, kv_lo=max(1, kv // 3), kv_hi=kv, kv_heads=heads, head_dim=dim, rot=rot,
                    layout=layout, dtype=dtype, page=rng.choice([16, 32, 64, 128, 256]))
    kv_heads, group = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 4, 5, 8])
    page, seqs = rng.choice([16, 32, 64, 128, 256]), _log(rng, 2 if op == "shared" else 1, 64)
    c = dict(op="attend", seqs=seqs, q_heads=kv_heads * group, kv_heads=kv_heads, head_dim=dim, page=page)
    if op == "shared":
        q, tail, shared = rng.choice([1, 1, 2, 5]), _log(rng, 8, 800), page * _log(rng, 4, max(5, 16384 // page))
        shared = min(shared, max(page, (64 * 17000 * 1024 // (seqs * kv_heads * dim) - tail) // page * page))
        return dict(c, q_lo=1, q_hi=q, kv_lo=max(q, tail // 5), kv_hi=max(q, tail), window=0, groups=rng.randint(1, min(4, seqs)), shared=shared)
    if rng.random() < 0.4:      # prompts, or chunks of them behind what the cache holds
        seqs = min(seqs, 4)
        q = _log(rng, 16, 2048 // seqs)
        kv = q + rng.choice([0, _log(rng, 1, 2000)])
    else:
        q = rng.choice([1, 1, 1, 2, 5])
        kv = max(q, min(_log(rng, 16, 16384), 64 * 16384 * 1024 // (seqs * kv_heads * dim)))
    return dict(c, seqs=seqs, q_lo=max(1, q // 3), q_hi=q, kv_lo=max(1, kv // 9), kv_hi=kv, window=rng.choice([0, 0, 0, _log(rng, 8, 4096)]),
                groups=0, shared=0)


def _spread(lo, hi, n):
    """n whole numbers from hi down to lo, evenly over their logarithm."""
    return [int(round(hi * (lo / hi) ** (i / max(1, n - 1)))) for i in range(n)]


def _lengths(c):
    """(query tokens, positions, shared positions, group) of each sequence, longest and shortest side by side."""
    n = c["seqs"]
    order = sorted(range(n), key=lambda i: (i * 5 + 3) % n * n + i)
    q, kv = _spread(c["q_lo"], c["q_hi"], n), _spread(c["kv_lo"], c["kv_hi"], n)
    groups = c.get("groups", 0)
    out = []
    for place, i in enumerate(order):
        g = place * groups // n if groups else 0
        shared = c["shared"] // (g + 1) // c["page"] * c["page"] if groups else 0
        out.append((q[i], max(q[i], kv[i]) + shared, shared, g))
    return out


def work(case):
    c, op = case, case["op"]
    esz = 4 if c.get("dtype") == "f32" else 2
    if op == "rotary":
        n = c["tokens"] * c["heads"]
        return {"bytes": n * c["head_dim"] * esz * 2 + 4 * c["tokens"] + 4 * c["rot"] * min(c["tokens"], c["positions"]),
                "flops": 3 * n * c["rot"]}
    if op == "table":
        return {"bytes": 4 * c["positions"] * c["rot"], "flops": 3 * c["positions"] * c["rot"]}
    lens, dim = _lengths(c), c["head_dim"]
    tokens = sum(q for q, _, _, _ in lens)
    if op == "append":
        n = tokens * c["kv_heads"]
        return {"bytes": 2 * n * dim * (esz + 1 + 1 / 32) + 4 * c["rot"] * tokens, "flops": n * (3 * c["rot"] + 4 * dim)}
    keys = seen = 0
    groups = {}
    for q, kv, shared, g in lens:
        w = c["window"] or kv
        first = max(0, kv - q + 1 - w)
        keys += kv - max(first, shared)
        groups[g] = max(groups.get(g, 0), shared - first)
        seen += sum(min(w, p + 1) for p in range(kv - q, kv))
    keys += sum(groups.values())
    return {"bytes": keys * c["kv_heads"] * 2 * dim * (1 + 1 / 32) + tokens * c["q_heads"] * (4 * dim + 4) + 4 * keys / c["page"],
            "flops": 4 * seen * c["q_heads"] * dim}


# --- inputs --------------------------------------------------------------------------------

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def _dtype(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _two(e):
    """2^e, exact: the exponent field of a binary64, for whole e in -1022 .. 1023."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _mxfp8(y):
    """Plain MXFP8 of the last axis: (values as float8_e4m3fn, scale bytes); y in fp32, or in fp64 where its
    rounding to fp32 would count."""
    v = y.unflatten(-1, (-1, 32))
    m, e = torch.frexp(v.abs().amax(-1))
    p = torch.where(m == 0, -127, torch.clamp(torch.where(m > 0.875, e - 8, e - 9), min=-127))
    t = v * _two(-p).to(y.dtype)[..., None]
    step = _two(torch.frexp(t)[1].clamp(min=-5) - 4).to(y.dtype)      # E4M3's grid at t
    q = (torch.round(t / step) * step).float().to(torch.float8_e4m3fn)
    return q.flatten(-2), (p + 127).to(torch.uint8)


def _keys(g, rows, heads, dim):
    """Gaussian, with a few channels of each head several times larger, as keys have."""
    big = torch.rand(heads, 1, dim, generator=g, device=DEV) < 0.02
    return torch.randn(heads, rows, dim, generator=g, device=DEV) * torch.where(big, 4.0, 1.0)


def _cache(g, pages, heads, page, dim):
    """A cache that holds earlier tokens everywhere."""
    s = {}
    for name in ("k", "v"):
        codes = torch.empty(pages, heads, page, dim, dtype=torch.uint8, device=DEV)
        scales = torch.empty(pages, heads, page, dim // 32, dtype=torch.uint8, device=DEV)
        step = max(1, (1 << 26) // (heads * page * dim))
        for p in range(0, pages, step):
            n = min(step, pages - p)
            x = _keys(g, n * page, heads, dim) if name == "k" else torch.randn(heads, n * page, dim, generator=g, device=DEV)
            q, e = _mxfp8(x)
            codes[p:p + n] = q.view(torch.uint8).view(heads, n, page, dim).transpose(0, 1)
            scales[p:p + n] = e.view(heads, n, page, dim // 32).transpose(0, 1)
        s[name + "_codes"], s[name + "_scales"] = codes, scales
    return s


def _batch(c, g):
    """The batch's lengths and a page table of pages in no order; sequences of a group share its first pages."""
    lens, page = _lengths(c), c["page"]
    own_pages = [-(-(kv - sh) // page) for _, kv, sh, _ in lens]
    shared = {gr: sh // page for _, _, sh, gr in lens}
    total = sum(own_pages) + sum(shared.values())
    ids = torch.randperm(total + 3, generator=g, device=DEV).to(torch.int32)
    width = max(-(-kv // page) for _, kv, _, _ in lens)
    table = torch.zeros(len(lens), width, dtype=torch.int32, device=DEV)
    at, first = 0, {}
    for gr, n in shared.items():
        first[gr] = ids[at:at + n]
        at += n
    for i, (_, _, _, gr) in enumerate(lens):
        n = shared[gr]
        table[i, :n] = first[gr]
        table[i, n:n + own_pages[i]] = ids[at:at + own_pages[i]]
        at += own_pages[i]

    def i32(v):
        return torch.tensor(v, dtype=torch.int32, device=DEV)
    b = {"q_starts": i32([0] + list(np.cumsum([q for q, _, _, _ in lens]))), "kv_lens": i32([kv for _, kv, _, _ in lens]),
         "page_table": table, "max_q_len": max(q for q, _, _, _ in lens), "max_kv_len": max(kv for _, kv, _, _ in lens)}
    if c.get("groups"):
        of = [gr for _, _, _, gr in lens]
        b["group_starts"] = i32([of.index(k) for k in range(c["groups"])] + [len(lens)])
        b["shared_lens"] = i32([shared[k] * page for k in range(c["groups"])])
        b["max_shared_len"] = max(shared.values()) * page
    return b, total + 3


def _table(positions, rot, base=10000.0):
    """(cos, sin) of a program's unscaled rotary table, from binary64 angles."""
    f = base ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=DEV) / rot)
    a = torch.arange(positions, dtype=torch.float64, device=DEV)[:, None] * f
    return torch.stack([a.cos(), a.sin()], -1).float()


def prepare(case, seed):
    c, g = case, _gen(seed)
    s = {"case": c}
    if c["op"] == "rotary":
        rows = torch.randn(c["tokens"], c["row_heads"], c["head_dim"], generator=g, device=DEV).to(_dtype(c["dtype"]))
        s["x"] = rows[:, :c["heads"]]
        s["positions"] = torch.randint(0, c["positions"], (c["tokens"],), generator=g, device=DEV, dtype=torch.int32)
        s["table"] = _table(c["positions"], c["rot"])
    elif c["op"] == "table":    # nothing is read: another seed is another base
        s["base"] = c["base"] * (1 + (int(seed) % 1000) / 4096)
    else:
        s["batch"], pages = _batch(c, g)
        tokens = sum(q for q, _, _, _ in _lengths(c))
        s["cache"] = _cache(g, pages, c["kv_heads"], c["page"], c["head_dim"])
        if c["op"] == "append":
            rows = torch.randn(tokens, 2 * c["kv_heads"], c["head_dim"], generator=g, device=DEV)
            rows[:, :c["kv_heads"]] = _keys(g, tokens, c["kv_heads"], c["head_dim"]).transpose(0, 1)
            rows = rows.to(_dtype(c["dtype"]))
            s["k"], s["v"] = rows[:, :c["kv_heads"]], rows[:, c["kv_heads"]:]     # parts of one projection's rows
            s["table"] = _table(s["batch"]["max_kv_len"], c["rot"])
        else:
            s["q"] = torch.randn(tokens, c["q_heads"], c["head_dim"], generator=g, device=DEV).to(torch.bfloat16)
    return s


# --- the plain forms -----------------------------------------------------------------------

def _rotate(x, table, layout, backward=False):
    """x [tokens][heads][head_dim] turned by table [tokens][rot/2][2], both of one type."""
    half = table.shape[1]
    cos, sin = table[:, None, :, 0], table[:, None, :, 1]
    if backward:
        sin = -sin
    if layout == "half":
        a, b = x[..., :half], x[..., half:2 * half]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    else:
        a, b = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    return torch.cat([y, x[..., 2 * half:]], -1)


def _plain_table(s):
    c = s["case"]
    i = torch.arange(0, c["rot"], 2, dtype=torch.float64, device=DEV)
    f = torch.exp(-math.log(s["base"]) * i / c["rot"])
    if c["factor"] != 1.0:
        turns = c["original"] * f / (2 * math.pi)
        keep = torch.clamp((turns - c["low"]) / (c["high"] - c["low"]), 0, 1)
        f = f * (keep + (1 - keep) / c["factor"])
    a = torch.arange(c["positions"], dtype=torch.float64, device=DEV)[:, None] * f
    return (c["amplitude"] * torch.stack([a.cos(), a.sin()], -1)).float()


def _places(b, tokens):
    """(sequence, position) of each token of the call."""
    t = torch.arange(tokens, device=DEV)
    seq = (t[:, None] >= b["q_starts"][None, 1:]).sum(1)
    return seq, b["kv_lens"][seq] - (b["q_starts"][seq + 1] - t)


def _views(cache):
    return {k: v.view(torch.float8_e4m3fn if k.endswith("codes") else torch.float8_e8m0fnu) for k, v in cache.items()}


def _plain_append(s):
    c, b, cache = s["case"], s["batch"], s["cache"]
    seq, pos = _places(b, s["k"].shape[0])
    page, row = b["page_table"][seq, pos // c["page"]].long(), pos % c["page"]
    k = _rotate(s["k"].double(), s["table"][pos].double(), c["layout"])    # in 64 bits: keys next to a border between two codes
    for name, x in (("k", k), ("v", s["v"].float())):
        q, e = _mxfp8(x)
        cache[name + "_codes"][page, :, row] = q.view(torch.uint8)
        cache[name + "_scales"][page, :, row] = e
    return _views(cache)


def _plain_cache(s, name):
    """The batch's keys or values as fp32 [seqs][kv heads][positions][head_dim]."""
    at = s["batch"]["page_table"].long()
    v = s["cache"][name + "_codes"][at].view(torch.float8_e4m3fn).to(torch.float32).unflatten(-1, (-1, 32))
    v = v * _two(s["cache"][name + "_scales"][at].to(torch.int64) - 127).float()[..., None]
    return v.flatten(-2).transpose(1, 2).flatten(2, 3)


def _plain_attend(s):
    c, b, q = s["case"], s["batch"], s["q"]
    heads, group = c["kv_heads"], c["q_heads"] // c["kv_heads"]
    seqs, most = c["seqs"], b["max_q_len"]
    i = torch.arange(most, device=DEV)
    n = b["q_starts"][1:] - b["q_starts"][:-1]
    rows = torch.clamp(b["q_starts"][:-1, None] + i, max=q.shape[0] - 1)                          # [seqs][most]
    x = q.float()[rows].view(seqs, most, heads, group, -1).permute(0, 2, 1, 3, 4).flatten(2, 3)   # [seqs][heads][most group][dim]
    scores = x @ _plain_cache(s, "k").transpose(2, 3) * c["head_dim"] ** -0.5
    last = (b["kv_lens"] - n)[:, None] + i                                                        # each query's position
    key = torch.arange(scores.shape[-1], device=DEV)
    seen = (key <= last[..., None]) & (key < b["kv_lens"][:, None, None])
    if c["window"]:
        seen &= key > last[..., None] - c["window"]
    scores = scores.view(seqs, heads, most, group, -1).masked_fill(~seen[:, None, :, None], -math.inf)
    top = scores.amax(-1, keepdim=True)
    p = torch.exp(scores - top)
    total = p.sum(-1, keepdim=True)
    o = (p / total).flatten(2, 3) @ _plain_cache(s, "v")
    o = o.view(seqs, heads, most, group, -1).permute(0, 2, 1, 3, 4).flatten(2, 3)                 # [seqs][most][q heads][dim]
    lse = (top + torch.log(total)).squeeze(-1).permute(0, 2, 1, 3).flatten(2, 3)
    seq, _ = _places(b, q.shape[0])
    at = torch.arange(q.shape[0], device=DEV) - b["q_starts"][seq]
    return {"out": o[seq, at].to(torch.bfloat16), "lse": lse[seq, at]}


def run(state):
    s, op = state, state["case"]["op"]
    if own:
        return _own(s, op)
    if op == "rotary":
        c = s["case"]
        return {"y": _rotate(s["x"].float(), s["table"][s["positions"]], c["layout"], c["backward"]).to(s["x"].dtype)}
    if op == "table":
        return {"table": _plain_table(s)}
    if op == "append":
        return _plain_append(s)
    return _plain_attend(s)


def _own(s, op):
    from block_scaled_fp4_05_amd import binding as fp4q
    c = s["case"]
    if op == "table":
        return {"table": fp4q.rotary_table(c["positions"], c["rot"], base=s["base"], factor=c["factor"], original=c["original"],
                                           low=c["low"], high=c["high"], amplitude=c["amplitude"])}
    if op == "attend":
        out, lse = fp4q.attention_paged(s["q"], s["cache"], s["batch"], scale=c["head_dim"] ** -0.5, window=c["window"], with_lse=True)
        return {"out": out, "lse": lse}
    layout = fp4q.ROTARY_HALF if c["layout"] == "half" else fp4q.ROTARY_INTERLEAVED
    if op == "rotary":
        return {"y": fp4q.rotary(s["x"], s["table"], s["positions"], layout=layout, backward=c["backward"])}
    fp4q.kv_append(s["cache"], s["batch"], s["k"], s["v"], table=s["table"], layout=layout)
    return _views(s["cache"])


# --- the definitions in binary64 -------------------------------------------------------------

def _exact_mxfp8(y):
    """(element values, scales) of float64 blocks: exponents from frexp, elements rounded on E4M3's grid."""
    v = y.reshape(*y.shape[:-1], -1, 32)
    top = v.abs().amax(-1)
    m, e = torch.frexp(top)                       # top = m 2^e, m in [1/2, 1); 448 = 0.875 * 2^9
    p = torch.where(top > 0, e - 9 + (m > 0.875).int(), torch.full_like(e, -127)).clamp(min=-127)
    q = v * _two(-p)[..., None]
    step = _two(torch.frexp(q)[1].clamp(min=-5) - 4)
    return (torch.round(q / step) * step).reshape(y.shape), _two(p)


def _exact_e4m3(codes):
    c = codes.to(torch.int64)
    e, m, sign = (c >> 3) & 15, c & 7, 1 - 2 * (c >> 7)
    return sign * torch.where(e > 0, (8 + m) * _two(e - 10), m * 2.0 ** -9)


def _exact_rotation(x, table, layout, backward):
    """x [tokens][heads][head_dim] as complex numbers times table [tokens][rot/2][2]."""
    rot = 2 * table.shape[1]
    turn = torch.view_as_complex(table.double().contiguous())[:, None]
    if backward:
        turn = turn.conj()
    a = x[..., :rot].double()
    if layout == "half":
        a = a.unflatten(-1, (2, rot // 2)).transpose(-1, -2)
    else:
        a = a.unflatten(-1, (rot // 2, 2))
    z = torch.view_as_real(torch.view_as_complex(a.contiguous()) * turn)
    z = z.transpose(-1, -2) if layout == "half" else z
    y = x.double().clone()
    y[..., :rot] = z.reshape(*x.shape[:-1], rot)
    return y


def _exact_attend(s):
    c, b, q = s["case"], s["batch"], s["q"].double()
    group, dim = c["q_heads"] // c["kv_heads"], c["head_dim"]
    out = torch.zeros(q.shape, dtype=torch.float64, device=DEV)
    lse = torch.zeros(q.shape[:2], dtype=torch.float64, device=DEV)
    starts = b["q_starts"].tolist()
    for i, kv in enumerate(b["kv_lens"].tolist()):
        at = b["page_table"][i, :-(-kv // c["page"])].long()
        first, end = starts[i], starts[i + 1]
        pos = torch.arange(kv - (end - first), kv, device=DEV)[:, None]
        key = torch.arange(kv, device=DEV)[None]
        hide = (key > pos) | (key <= pos - (c["window"] or kv + 1))
        for h in range(c["kv_heads"]):
            k, v = ((_exact_e4m3(s["cache"][n + "_codes"][at, h]).reshape(-1, dim // 32, 32)
                     * _two(s["cache"][n + "_scales"][at, h].to(torch.int64) - 127).reshape(-1, dim // 32, 1)).reshape(-1, dim)[:kv]
                    for n in ("k", "v"))
            for j in range(h * group, (h + 1) * group):
                w = (q[first:end, j] @ k.t() / math.sqrt(dim)).masked_fill(hide, -math.inf)
                lse[first:end, j] = torch.logsumexp(w, -1)
                out[first:end, j] = torch.softmax(w, -1) @ v
    return {"out": out, "lse": lse}


def exact(case, seed):
    s, c, op = prepare(case, seed), case, case["op"]
    if op == "rotary":
        return {"y": _exact_rotation(s["x"], s["table"][s["positions"].long()], c["layout"], c["backward"])}
    if op == "table":
        f = np.float64(s["base"]) ** (-2.0 * np.arange(c["rot"] // 2) / c["rot"])
        if c["factor"] != 1.0:
            keep = np.clip((c["original"] / (2 * np.pi / f) - c["low"]) / (c["high"] - c["low"]), 0.0, 1.0)
            f = keep * f + (1.0 - keep) * f / c["factor"]
        z = c["amplitude"] * np.exp(1j * np.outer(np.arange(c["positions"]), f))
        return {"table": torch.from_numpy(np.stack([z.real, z.imag], -1)).to(DEV)}
    if op == "attend":
        return _exact_attend(s)
    b, page = s["batch"], c["page"]
    out = {k: _exact_e4m3(v) if k.endswith("codes") else _two(v.to(torch.int64) - 127) for k, v in s["cache"].items()}
    starts = b["q_starts"].tolist()
    for i, kv in enumerate(b["kv_lens"].tolist()):
        first, end = starts[i], starts[i + 1]
        pos = torch.arange(kv - (end - first), kv, device=DEV)
        at, row = b["page_table"][i][pos // page].long(), pos % page
        for name, x in (("k", _exact_rotation(s["k"][first:end], s["table"][pos], c["layout"], False)), ("v", s["v"][first:end].double())):
            v, e = _exact_mxfp8(x)
            out[name + "_codes"][at, :, row] = v
            out[name + "_scales"][at, :, row] = e
    return out
