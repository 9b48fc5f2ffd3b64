"""Cases, plain forms and 64-bit values of the MXFP8 norm, quantizer and product and of the MXFP4 expert layer.

``run`` computes one pass of an operator, in elementary fp32 torch operations or, with ``own``
set, by the library's calls.  ``exact`` computes the same outputs in binary64.

Formats: MXFP4 is E2M1 codes, two per byte, with an E8M0 scale per 32 elements; MXFP8 is E4M3
codes with an E8M0 scale per 32 elements, the smallest power of two that brings the block's
largest magnitude to 448 or below.  8-bit codes and scales are returned as torch's
float8_e4m3fn and float8_e8m0fnu views of the bytes, so each stands for its value.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
EPS = 1e-6
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# --- cases ---------------------------------------------------------------------------------

def listed():
    return [
        # one decoded token's norm: a single row, latency only
        dict(name="norm 1 token", op="norm", rows=1, cols=4096, dtype="bf16", residual=True),
        # the norm of a training step's activation, the benchmark's 8192 x 4096
        dict(name="norm 8192 tokens", op="norm", rows=8192, cols=4096, dtype="bf16", residual=True),
        # a ragged fp32 batch without a residual: odd rows, a width that is no power of two
        dict(name="norm fp32 ragged", op="norm", rows=1021, cols=2080, dtype="f32", residual=False),
        # the norm's gradient in the same training step, with the residual stream's gradient
        dict(name="norm grad 8192 tokens", op="norm_grad", rows=8192, cols=4096, dtype="bf16", residual=True),
        # the gradient for a short fp32 sequence at a narrow odd width
        dict(name="norm grad fp32 short", op="norm_grad", rows=77, cols=1056, dtype="f32", residual=False),
        # an output gradient on its way into the data-gradient product (the benchmark's 16384 x 4096)
        dict(name="quantize 16384 tokens", op="quantize", rows=16384, cols=4096, dtype="bf16"),
        # a few decoded tokens' attention output before the output projection
        dict(name="quantize 33 tokens", op="quantize", rows=33, cols=2080, dtype="f32"),
        # one decoded token through a projection: the weights' bytes are all that counts
        dict(name="product 1 token", op="product", m=1, n=4096, k=4096, out="bf16"),
        # a short ragged prompt: odd rows and columns
        dict(name="product 193 tokens", op="product", m=193, n=4099, k=4224, out="bf16"),
        # a training-size projection, the benchmark's 8192 x 8192 x 8192
        dict(name="product 8192 tokens", op="product", m=8192, n=8192, k=8192, out="bf16"),
        # one decoded token through an expert layer
        dict(name="experts 1 token", op="experts", tokens=1, d=2048, hidden=1024, experts=64, topk=4),
        # a full decode batch: nearly every expert is read
        dict(name="experts 64 tokens", op="experts", tokens=64, d=4096, hidden=2048, experts=32, topk=4),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _mult(rng, step, lo, hi):
    return step * max(1, _log(rng, lo / step, hi / step))


def draw(rng):
    op = rng.choice(["norm", "norm_grad", "quantize", "product", "experts"])
    if op == "norm" or op == "norm_grad":
        rows, cols = _log(rng, 1, 16384), _mult(rng, 32, 64, 16384)
        return dict(op=op, rows=max(1, min(rows, 8192 * 4096 // cols)), cols=cols, dtype=rng.choice(["bf16", "f32"]), residual=rng.random() < 0.5)
    if op == "quantize":
        return dict(op=op, rows=_log(rng, 1, 16384), cols=_mult(rng, 32, 64, 8192), dtype=rng.choice(["bf16", "f32"]))
    if op == "product":
        return dict(op=op, m=_log(rng, 1, 8192), n=_log(rng, 64, 8192), k=_mult(rng, 128, 256, 8192), out="bf16")
    experts = rng.choice([8, 16, 32, 64])
    return dict(op=op, tokens=_log(rng, 1, 64), d=_mult(rng, 128, 512, 4096), hidden=_mult(rng, 128, 256, 2048),
                experts=experts, topk=rng.choice([1, 2, 4, 8][: 4 if experts > 8 else 3]))


def work(case):
    c, op = case, case["op"]
    esz = 2 if c.get("dtype", "bf16") == "bf16" else 4
    if op == "norm":
        n = c["rows"] * c["cols"]
        return {"bytes": n * (esz * (3 if c["residual"] else 1) + 1 + 1 / 32) + 4 * c["cols"] + 4 * c["rows"], "flops": 6 * n}
    if op == "norm_grad":
        n = c["rows"] * c["cols"]
        return {"bytes": n * esz * (4 if c["residual"] else 3) + 8 * c["cols"] + 4 * c["rows"], "flops": 10 * n}
    if op == "quantize":
        n = c["rows"] * c["cols"]
        return {"bytes": n * (esz + 1 + 1 / 32), "flops": 2 * n}
    if op == "product":
        m, n, k = c["m"], c["n"], c["k"]
        return {"bytes": m * k * (1 + 1 / 32) + n * k * (1 / 2 + 1 / 32) + m * n * 2, "flops": 2 * m * n * k}
    t, d, h, e, k = c["tokens"], c["d"], c["hidden"], c["experts"], c["topk"]
    read = e * (1 - (1 - k / e) ** t)   # experts that t tokens of k random choices reach
    return {"bytes": read * 3 * d * h * (1 / 2 + 1 / 32) + 2 * e * d + t * d * (1 + 1 / 32 + 2 + 2) + 8 * t * k,
            "flops": 2 * t * k * 3 * d * h + 2 * t * e * d}


# --- inputs --------------------------------------------------------------------------------

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def _dtype(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _two(e):
    """2^e, exact: the exponent field of a binary64, for whole e in -1022 .. 1023."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _hidden(g, rows, cols, dtype):
    """Activations: Gaussian, with a few channels an order of magnitude larger."""
    x = torch.randn(rows, cols, generator=g, device=DEV)
    big = torch.rand(cols, generator=g, device=DEV) < 0.004
    return (x * torch.where(big, 12.0, 1.0)).to(dtype)


def _weights_mxfp4(g, rows, cols):
    """Gaussian weights of a layer as MXFP4: the scale the power of two nearest max / 6."""
    codes = torch.empty(rows, cols // 2, dtype=torch.uint8, device=DEV)
    scales = torch.empty(rows, cols // 32, dtype=torch.uint8, device=DEV)
    edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=DEV)
    step = max(1, (1 << 27) // cols)
    for r in range(0, rows, step):
        w = torch.randn(min(step, rows - r), cols // 32, 32, generator=g, device=DEV) * cols ** -0.5
        e = torch.round(torch.log2(w.abs().amax(-1) / 6))
        v = w * _two(-e).float()[..., None]
        c = torch.bucketize(v.abs(), edges, out_int32=True).to(torch.uint8) | ((v < 0).to(torch.uint8) << 3)
        c = c.reshape(-1, cols // 2, 2)
        codes[r:r + step] = c[..., 0] | (c[..., 1] << 4)
        scales[r:r + step] = (e + 127).to(torch.uint8)
    return {"codes": codes, "scales": scales}


def _mxfp8(y):
    """Plain MXFP8: y [rows][cols] fp32 -> (values as float8_e4m3fn, exponents of the scales)."""
    v = y.reshape(y.shape[0], -1, 32)
    m, e = torch.frexp(v.abs().amax(-1))
    p = torch.where(m == 0, -127, torch.clamp(torch.where(m > 0.875, e - 8, e - 9), min=-127))
    q = (v * _two(-p).float()[..., None]).to(torch.float8_e4m3fn)
    return q.reshape(y.shape), p


def _bytes8(y):
    q, p = _mxfp8(y)
    return {"codes": q.view(torch.uint8), "scales": (p + 127).to(torch.uint8)}


def prepare(case, seed):
    c, g = case, _gen(seed)
    s = {"case": c}
    if c["op"] in ("norm", "norm_grad"):
        dt = _dtype(c["dtype"])
        s["gain"] = torch.randn(c["cols"], generator=g, device=DEV) * 0.1 + 1.0
        x = _hidden(g, c["rows"], c["cols"], dt)
        if c["op"] == "norm":
            s["x"] = x
            s["residual"] = _hidden(g, c["rows"], c["cols"], dt) if c["residual"] else None
        else:
            s["sum"] = x
            s["rstd"] = 1.0 / torch.sqrt(x.float().square().mean(-1) + EPS)
            s["dy"] = (torch.randn(c["rows"], c["cols"], generator=g, device=DEV) * 1e-2).to(dt)
            s["dsum"] = (torch.randn(c["rows"], c["cols"], generator=g, device=DEV) * 1e-2).to(dt) if c["residual"] else None
    elif c["op"] == "quantize":
        s["x"] = _hidden(g, c["rows"], c["cols"], _dtype(c["dtype"]))
    elif c["op"] == "product":
        s["a"] = _bytes8(_hidden(g, c["m"], c["k"], torch.float32))
        s["b"] = _weights_mxfp4(g, c["n"], c["k"])
    else:
        t, d, h, e = c["tokens"], c["d"], c["hidden"], c["experts"]
        s["router_x"] = _hidden(g, t, d, torch.bfloat16)
        s["x"] = _bytes8(s["router_x"].float())
        s["router_w"] = (torch.randn(e, d, generator=g, device=DEV) * d ** -0.5).to(torch.bfloat16)
        for name, r, k in (("w13", 2 * h, d), ("w2", d, h)):
            w = _weights_mxfp4(g, e * r, k)
            s[name] = {"codes": w["codes"].view(e, r, k // 2), "scales": w["scales"].view(e, r, k // 32)}
    return s


# --- the plain forms -----------------------------------------------------------------------

def _pow2(scales):
    return _two(scales.to(torch.int64) - 127).float()


def _plain_fp4(w):
    """MXFP4 bytes -> fp32 values."""
    t = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=w["codes"].device)
    pairs = torch.stack([t.repeat(16), t.repeat_interleave(16)], -1)   # byte -> its two elements
    v = pairs[w["codes"].int()].flatten(-2)
    return (v.unflatten(-1, (-1, 32)) * _pow2(w["scales"])[..., None]).flatten(-2)


def _plain_fp8(x):
    v = x["codes"].view(torch.float8_e4m3fn).to(torch.float32)
    return (v.unflatten(-1, (-1, 32)) * _pow2(x["scales"])[..., None]).flatten(-2)


def _out8(q, p):
    return q, (p + 127).to(torch.uint8).view(torch.float8_e8m0fnu)


def _plain_norm(s):
    x = s["x"].float()
    if s["residual"] is not None:
        x = x + s["residual"].float()
    r = 1.0 / torch.sqrt(x.square().mean(-1) + EPS)
    codes, scales = _out8(*_mxfp8(x * r[:, None] * s["gain"]))
    return {"codes": codes, "scales": scales, "rstd": r, "sum": x.to(s["x"].dtype) if s["residual"] is not None else None}


def _plain_norm_grad(s):
    x, dy, r = s["sum"].float(), s["dy"].float(), s["rstd"][:, None]
    a = dy * s["gain"]
    dx = a * r - x * (r * r * r * (a * x).mean(-1, keepdim=True))
    if s["dsum"] is not None:
        dx = dx + s["dsum"].float()
    return {"dx": dx.to(s["dy"].dtype), "dgain": (dy * x * r).sum(0)}


def _plain_experts(s):
    c = s["case"]
    logits = s["router_x"].float() @ s["router_w"].float().t()
    top, ids = torch.sort(logits, dim=-1, descending=True, stable=True)
    top, ids = top[:, :c["topk"]], ids[:, :c["topk"]]
    w = torch.exp(top - top[:, :1])
    w = w / w.sum(-1, keepdim=True)
    x, h = _plain_fp8(s["x"]), c["hidden"]
    gather = c["tokens"] * c["topk"] < c["experts"]
    if gather:      # fewer choices than experts: each choice's own weights
        flat = ids.reshape(-1)
        w13 = {k: v[flat] for k, v in s["w13"].items()}
        w2 = {k: v[flat] for k, v in s["w2"].items()}
        x = x.repeat_interleave(c["topk"], 0)[:, None]                    # [choices][1][d]
    else:           # every expert on every token, the choices picked at the end
        w13, w2, x = s["w13"], s["w2"], x[None]                           # [1][tokens][d]
    gu = torch.matmul(x, _plain_fp4(w13).transpose(1, 2))
    g, u = gu[..., :h], gu[..., h:]
    act = g / (1.0 + torch.exp(-g)) * u
    q, p = _mxfp8(act.reshape(-1, h))
    act = (q.to(torch.float32).unflatten(-1, (-1, 32)) * _two(p).float()[..., None]).reshape(act.shape)
    y = torch.matmul(act, _plain_fp4(w2).transpose(1, 2))
    if gather:
        y = (y.reshape(c["tokens"], c["topk"], -1) * w[..., None]).sum(1)
    else:
        share = torch.zeros(c["tokens"], c["experts"], device=w.device).scatter_(1, ids, w)
        y = (y * share.t()[..., None]).sum(0)
    return {"y": y.to(torch.bfloat16), "ids": ids.to(torch.int32), "weights": w}


def run(state):
    s, op = state, state["case"]["op"]
    if own:
        return _own(s, op)
    if op == "norm":
        return _plain_norm(s)
    if op == "norm_grad":
        return _plain_norm_grad(s)
    if op == "quantize":
        codes, scales = _out8(*_mxfp8(s["x"].float()))
        return {"codes": codes, "scales": scales}
    if op == "product":
        return {"c": (_plain_fp8(s["a"]) @ _plain_fp4(s["b"]).t()).to(_dtype(s["case"]["out"]))}
    return _plain_experts(s)


def _own(s, op):
    from block_scaled_fp4_05_amd import binding as fp4q
    if op == "norm":
        o = fp4q.rmsnorm_mxfp8(s["x"], s["gain"], residual=s["residual"], eps=EPS)
        return {"codes": o["codes"].view(torch.float8_e4m3fn), "scales": o["scales"].view(torch.float8_e8m0fnu),
                "rstd": o["rstd"], "sum": o["sum"] if s["residual"] is not None else None}
    if op == "norm_grad":
        dx, dgain = fp4q.rmsnorm_backward(s["dy"], s["sum"], s["gain"], s["rstd"], dsum=s["dsum"])
        return {"dx": dx, "dgain": dgain}
    if op == "quantize":
        o = fp4q.quantize_mxfp8(s["x"])
        return {"codes": o["codes"].view(torch.float8_e4m3fn), "scales": o["scales"].view(torch.float8_e8m0fnu)}
    if op == "product":
        return {"c": fp4q.gemm_mxfp8_mxfp4(s["a"], s["b"], _dtype(s["case"]["out"]))}
    o = fp4q.moe_mxfp4(s["x"], s["w13"], s["w2"], s["case"]["topk"], router_x=s["router_x"], router_w=s["router_w"])
    return {"y": o["y"], "ids": o["ids"], "weights": o["weights"]}


# --- the definitions in binary64 -------------------------------------------------------------

def _exact_mxfp8(y):
    """(element values, scales) of float64 rows: exponents from frexp, elements rounded on E4M3's grid."""
    v = y.reshape(y.shape[0], -1, 32)
    top = v.abs().amax(-1)
    m, e = torch.frexp(top)                       # top = m 2^e, m in [1/2, 1); 448 = 0.875 * 2^9
    p = torch.where(top > 0, e - 9 + (m > 0.875).int(), torch.full_like(e, -127)).clamp(min=-127)
    q = v * _two(-p)[..., None]
    step = _two(torch.frexp(q)[1].clamp(min=-5) - 4)
    return (torch.round(q / step) * step).reshape(y.shape), _two(p)


def _exact_fp4(codes, scales):
    c = codes.to(torch.int64)
    n = torch.stack([c & 15, c >> 4], -1).flatten(-2)
    e, m, sign = (n >> 1) & 3, n & 1, 1 - 2 * (n >> 3)
    mag = torch.where(e > 0, (2 + m) * _two(e - 2), m * 0.5)
    return sign * mag * _two(scales.to(torch.int64) - 127).repeat_interleave(32, -1)


def _exact_fp8(codes, scales):
    c = codes.to(torch.int64)
    e, m, sign = (c >> 3) & 15, c & 7, 1 - 2 * (c >> 7)
    mag = torch.where(e > 0, (8 + m) * _two(e - 10), m * 2.0 ** -9)
    return sign * mag * _two(scales.to(torch.int64) - 127).repeat_interleave(32, -1)


def exact(case, seed):
    s, c, op = prepare(case, seed), case, case["op"]
    if op == "norm":
        x = s["x"].double()
        if s["residual"] is not None:
            x = x + s["residual"].double()
        r = torch.rsqrt((x * x).sum(1) / c["cols"] + EPS)
        q, p = _exact_mxfp8(s["gain"].double() * (r[:, None] * x))
        return {"codes": q, "scales": p, "rstd": r, "sum": x if s["residual"] is not None else None}
    if op == "norm_grad":
        x, dy, r, g = s["sum"].double(), s["dy"].double(), s["rstd"].double(), s["gain"].double()
        dot = (dy * g * x).sum(1)
        dx = r[:, None] * dy * g - (r ** 3 * dot / c["cols"])[:, None] * x
        if s["dsum"] is not None:
            dx = dx + s["dsum"].double()
        return {"dx": dx, "dgain": ((r[:, None] * x) * dy).sum(0)}
    if op == "quantize":
        q, p = _exact_mxfp8(s["x"].double())
        return {"codes": q, "scales": p}
    if op == "product":
        return {"c": _exact_fp8(s["a"]["codes"], s["a"]["scales"]) @ _exact_fp4(s["b"]["codes"], s["b"]["scales"]).t()}
    logits = s["router_x"].double() @ s["router_w"].double().t()
    t, k, h = c["tokens"], c["topk"], c["hidden"]
    host = logits.cpu().numpy()
    ids = np.lexsort((np.broadcast_to(np.arange(host.shape[1]), host.shape), -host), axis=-1)[:, :k].copy()
    w = torch.softmax(torch.gather(logits, 1, torch.from_numpy(ids).to(DEV)), -1)
    x = _exact_fp8(s["x"]["codes"], s["x"]["scales"])
    y = torch.zeros(t, c["d"], dtype=torch.float64, device=DEV)
    for e in sorted(set(ids.reshape(-1).tolist())):
        tok, slot = (torch.from_numpy(v).to(DEV) for v in np.nonzero(ids == e))
        gu = x[tok] @ _exact_fp4(s["w13"]["codes"][e], s["w13"]["scales"][e]).t()
        q, p = _exact_mxfp8(gu[:, :h] * torch.sigmoid(gu[:, :h]) * gu[:, h:])
        act = q * p.repeat_interleave(32, -1)
        y[tok] += w[tok, slot][:, None] * (act @ _exact_fp4(s["w2"]["codes"][e], s["w2"]["scales"][e]).t())
    return {"y": y, "ids": torch.from_numpy(ids.astype(np.int32)), "weights": w}
