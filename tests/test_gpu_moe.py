"""The MXFP4 expert layer (GPU) against binary64.

The hidden activations are rounded to MXFP8 inside the layer, so a value next to a rounding
boundary may take either neighbour.  The reference therefore follows the layer's own hidden
rounding to within the error of the sums: |y - exact| is bounded by
 - the down product's own arithmetic: of 16 neighbouring products each is cut at most 2^-13 of the
   largest, and fp32 sums of depth at most 64;
 - for each hidden value whose distance to a boundary is within the first products' bound, the step
   across it times the largest weight it meets;
 - the softmax weights: 16 roundings, 2^-20.
With small whole values that the arithmetic holds exactly (a gate of 0 or large, weights given) the
layer must be equal to the reference.
"""
import numpy as np
import pytest
import torch

import mxfp8_ref as ref
from block_scaled_fp4_05_amd import binding as B

pytestmark = pytest.mark.gpu
DEV = "cuda"
VAL8 = ref.e4m3_values()


def _experts(e, rows, k, seed, spread=1):
    rng = np.random.default_rng(seed)
    codes = rng.integers(0, 256, (e, rows, k // 2), dtype=np.uint8)
    scales = rng.integers(120 - spread, 121 + spread, (e, rows, k // 32)).astype(np.uint8)
    return codes, scales


def _tokens(t, d, seed):
    g = torch.Generator().manual_seed(seed)
    return B.quantize_mxfp8(torch.randn(t, d, generator=g).to(DEV))


def _dev(w):
    return {"codes": torch.from_numpy(w[0]).to(DEV), "scales": torch.from_numpy(w[1]).to(DEV)}


def _np(t):
    return t.float().cpu().numpy().astype(np.float64) if t.is_floating_point() else t.cpu().numpy()


def _cut(a, b):
    """Bound of the matrix instruction's cuts in a @ b.T, 16 neighbours at a time."""
    a, b = np.abs(a), np.abs(b)
    out = np.zeros((a.shape[0], b.shape[0]))
    for t in range(0, a.shape[1], 16):
        out += (a[:, None, t:t + 16] * b[None, :, t:t + 16]).max(-1)
    return out * 16 * 2.0 ** -13 + 2.0 ** -24 * 2 * (32 + a.shape[1] / 64) * (a @ b.T)


def _layer(x, w13, w2, ids, weights):
    """(y, bound) in binary64 with the given choices."""
    t, d = x.shape
    y, bound = np.zeros((t, d)), np.zeros((t, d))
    for e in sorted({int(v) for v in ids.reshape(-1)}):
        if not 0 <= e < w13[0].shape[0]:
            continue
        tok = [i for i in range(t) if e in ids[i]]
        share = np.array([weights[i][ids[i] == e].sum() for i in tok])[:, None]
        a, b = ref.fp4(w13[0][e], w13[1][e]), ref.fp4(w2[0][e], w2[1][e])
        gu, ge = x[tok] @ a.T, _cut(x[tok], a)
        n = gu.shape[1] // 2
        g, u, dg, du = gu[:, :n], gu[:, n:], ge[:, :n], ge[:, n:]
        with np.errstate(over="ignore"):
            silu = g / (1 + np.exp(-g))
        h = silu * u
        # |silu'| <= 1.1; the exponential, the division and the product round at most 8 times
        dh = 1.1 * dg * (np.abs(u) + du) + np.abs(silu) * du + 2.0 ** -21 * np.abs(h)
        v, c = ref.quantize(h)
        step = np.repeat(np.ldexp(1.0, (c - 127).astype(np.int32)), 32, axis=-1)
        q = v * step
        lo, hi = ref.quantize(h - dh), ref.quantize(h + dh)
        vals = [w * np.repeat(np.ldexp(1.0, (k - 127).astype(np.int32)), 32, axis=-1) for w, k in (lo, hi)]
        # the block's scale may move with its largest value: then every element may round on the other grid
        bm, dm = np.abs(h).reshape(*h.shape[:1], -1, 32).max(-1), dh.reshape(*h.shape[:1], -1, 32).max(-1)
        moved = np.repeat(ref.scale_code(np.maximum(bm - dm, 0)) != ref.scale_code(bm + dm), 32, axis=-1)
        flip = np.maximum(np.abs(vals[0] - q), np.abs(vals[1] - q)) + np.where(moved, np.abs(q) * 2.0 ** -3 + step * 2.0 ** -8, 0)
        y[tok] += share * (q @ b.T)
        bound[tok] += np.abs(share) * (flip @ np.abs(b).T + _cut(q, b)) + 2.0 ** -19 * np.abs(share) * (np.abs(q) @ np.abs(b).T)
    return y, bound


def _route(rx, rw, topk):
    logits = rx @ rw.T
    order = np.lexsort((np.broadcast_to(np.arange(logits.shape[1]), logits.shape), -logits), axis=-1)[:, :topk]
    top = np.take_along_axis(logits, order, 1)
    w = np.exp(top - top[:, :1])
    return order, w / w.sum(1, keepdims=True)


CASES = [  # tokens, d, hidden, experts, topk
    (1, 128, 128, 1, 1), (1, 256, 128, 8, 2), (1, 512, 384, 64, 4), (1, 128, 256, 512, 16), (2, 384, 128, 16, 3),
    (3, 256, 256, 5, 5), (5, 128, 640, 40, 8), (15, 256, 128, 7, 2), (16, 128, 128, 3, 1), (17, 256, 128, 4, 2),
    (31, 128, 256, 130, 4), (33, 640, 128, 2, 2), (40, 128, 128, 1, 1), (48, 256, 128, 6, 1), (64, 128, 256, 16, 4),
    (64, 256, 128, 8, 8), (64, 128, 128, 512, 16), (50, 1152, 128, 3, 2)]


@pytest.mark.parametrize("router", ["bf16", "f32"])
@pytest.mark.parametrize("case", CASES)
def test_layer_with_its_router(case, router):
    t, d, h, e, k = case
    x, w13, w2 = _tokens(t, d, t + d), _experts(e, 2 * h, d, 1), _experts(e, d, h, 2)
    g = torch.Generator().manual_seed(7)
    dt = torch.bfloat16 if router == "bf16" else torch.float32
    rx, rw = (torch.randn(n, d, generator=g).to(dt).to(DEV) for n in (t, e))
    print("moe", case, router, flush=True)
    o = B.moe_mxfp4(x, _dev(w13), _dev(w2), k, router_x=rx, router_w=rw, out_dtype=torch.float32)
    ids, w = _route(_np(rx), _np(rw), k)
    assert np.array_equal(_np(o["ids"]), ids)
    # a logit is off by at most (d / 16 + 24) roundings of its magnitudes; so is the exponential's argument
    err = (d / 16 + 24) * 2.0 ** -24 * (np.abs(_np(rx)) @ np.abs(_np(rw)).T).max()
    assert np.all(np.abs(_np(o["weights"]) - w) <= (4 * err + 2.0 ** -19) * w + 1e-30)
    xv = ref.dequantize(_np(x["codes"]), _np(x["scales"]))
    y, bound = _layer(xv, w13, w2, ids, _np(o["weights"]))
    assert np.all(np.abs(_np(o["y"]) - y) <= bound)
    half = B.moe_mxfp4(x, _dev(w13), _dev(w2), k, router_x=rx, router_w=rw)
    assert torch.equal(half["y"], o["y"].to(torch.bfloat16)) and torch.equal(half["ids"], o["ids"])
    again = B.moe_mxfp4(x, _dev(w13), _dev(w2), k, ids=o["ids"], weights=o["weights"], out_dtype=torch.float32)
    assert torch.equal(again["y"], o["y"])               # the same choices given: the same bits


def _whole_layer(t, d, h, e, seed):
    """Operands whose products, activations and sums the layer holds exactly: tokens of 0, 1 and 2,
    gates of 0 or at least 64 (silu(g) = g there), hidden values of few bits."""
    rng = np.random.default_rng(seed)
    xc = np.zeros((t, d), np.uint8)
    xc[:, 0] = 0x38                                              # x[:, 0] = 1
    xc[np.arange(t), 1 + np.arange(t) % (d - 1)] = rng.choice(np.array([0x38, 0xB8, 0x40], np.uint8), t)
    n = np.zeros((e, 2 * h, d), np.uint8)
    n[:, :h, 0] = rng.choice(np.array([0, 2, 4], np.uint8), (e, h))   # gate: 0, 1 or 2 (times 2^6)
    n[:, h:, 1:] = rng.choice(np.array([0, 2, 10], np.uint8), (e, h, d - 1))   # up: 0, 1, -1
    s13 = np.full((e, 2 * h, d // 32), 127, np.uint8)
    s13[:, :h, :] = 127 + 6
    n2 = rng.integers(0, 16, (e, d, h)).astype(np.uint8)
    pack = lambda v: (v[..., 0::2] | (v[..., 1::2] << 4)).astype(np.uint8)
    return ((xc, np.full((t, d // 32), 127, np.uint8)), (pack(n), s13),
            (pack(n2), rng.integers(126, 129, (e, d, h // 32)).astype(np.uint8)))


@pytest.mark.parametrize("t,d,h,e,k", [(1, 128, 128, 4, 2), (7, 256, 128, 9, 3), (16, 128, 256, 2, 2), (33, 128, 128, 5, 4),
                                       (64, 256, 256, 3, 1), (64, 128, 128, 40, 4), (4, 1024, 128, 6, 2), (2, 128, 1024, 33, 5)])
def test_whole_values_are_exact(t, d, h, e, k):
    x, w13, w2 = _whole_layer(t, d, h, e, t + h)
    rng = np.random.default_rng(1)
    ids = np.stack([rng.permutation(e)[:k] for _ in range(t)]).astype(np.int32)
    weights = rng.choice([0.5, 1.0, 2.0, -1.0], (t, k)).astype(np.float32)
    xv = ref.dequantize(*x)
    gu = np.stack([xv @ ref.fp4(w13[0][i], w13[1][i]).T for i in range(e)])      # [e][t][2h]
    hid = gu[..., :h] * gu[..., h:]
    v, c = ref.quantize(hid.reshape(e * t, h))
    q = (v * np.repeat(np.ldexp(1.0, (c - 127).astype(np.int32)), 32, axis=-1)).reshape(e, t, h)
    assert np.array_equal(q, hid)
    out = np.stack([q[i] @ ref.fp4(w2[0][i], w2[1][i]).T for i in range(e)])
    y = sum(weights[:, j, None] * out[ids[:, j], np.arange(t)] for j in range(k))
    print("moe whole", t, d, h, e, k, flush=True)
    o = B.moe_mxfp4(_dev(x), _dev(w13), _dev(w2), k, ids=torch.from_numpy(ids).to(DEV),
                    weights=torch.from_numpy(weights).to(DEV), out_dtype=torch.float32)
    assert np.array_equal(_np(o["y"]), y)


@pytest.mark.parametrize("t,e", [(3, 64), (6, 4), (40, 3)])
def test_choices_that_take_no_part_and_repeats(t, e):
    d, h, k = 128, 128, 3
    x, w13, w2 = _whole_layer(t, d, h, e, 5)
    dx, d13, d2 = _dev(x), _dev(w13), _dev(w2)
    run = lambda i, w: B.moe_mxfp4(dx, d13, d2, i.shape[1], ids=i, weights=w, out_dtype=torch.float32)["y"]
    ids = torch.randint(0, e, (t, 1), dtype=torch.int32, device=DEV)
    one = torch.ones(t, 1, device=DEV)
    base = run(ids, one)
    none = torch.full((t, 1), -1, dtype=torch.int32, device=DEV)
    big = torch.full((t, 1), e, dtype=torch.int32, device=DEV)
    junk = torch.full((t, 1), float("nan"), device=DEV)
    assert torch.equal(run(torch.cat([none, ids, big], 1), torch.cat([junk, one, junk], 1)), base)
    assert torch.all(run(torch.cat([none, big, none], 1), torch.cat([junk, junk, junk], 1)) == 0)
    assert torch.equal(run(torch.cat([ids, ids, none], 1), torch.cat([one, one, one], 1)), 2 * base)
    mixed = torch.cat([ids, none, none], 1)
    mixed[0] = -1                                         # one empty row among full ones
    y = run(mixed, torch.cat([one, one, one], 1))
    assert torch.all(y[0] == 0) and torch.equal(y[1:], base[1:])


def test_router_ties_and_not_finite_logits():
    t, d, h, e, k = 6, 128, 128, 70, 4
    x, w13, w2 = _whole_layer(t, d, h, e, 9)
    rx, rw = torch.zeros(t, d, device=DEV), torch.zeros(e, d, device=DEV)
    rx[:, 0] = 1.0
    rw[:, 0] = -1.0
    rw[[5, 66, 3], 0] = 2.0                                # ties: 3, 5, 66 by index, then the rest by index
    rx[1, 1], rw[60, 1] = 1.0, float("nan")                # token 1: expert 60's logit is NaN (0 * NaN: all tokens')
    o = B.moe_mxfp4(_dev(x), _dev(w13), _dev(w2), k, router_x=rx, router_w=rw)
    assert o["ids"].tolist() == [[60, 3, 5, 66]] * t and torch.isnan(o["weights"]).all() and torch.isnan(o["y"]).all()
    rw[60, 1] = 0.0
    o = B.moe_mxfp4(_dev(x), _dev(w13), _dev(w2), k, router_x=rx, router_w=rw)
    assert o["ids"].tolist() == [[3, 5, 66, 0]] * t
    third = 1.0 / (3.0 + np.exp(-3.0))
    assert np.allclose(_np(o["weights"]), [third, third, third, third * np.exp(-3.0)], rtol=1e-6, atol=0)
    rw[:, 0] = 0.0
    rw[::2, 0] = -0.0                                      # -0 and +0 tie
    o = B.moe_mxfp4(_dev(x), _dev(w13), _dev(w2), k, router_x=rx, router_w=rw)
    assert o["ids"].tolist() == [[0, 1, 2, 3]] * t and torch.all(o["weights"] == 0.25)
    rw[9, 0] = float("-inf")
    rw[10:, 0] = float("-inf")
    rw[1:9, 0] = float("-inf")                             # one finite logit: the others weigh nothing
    o = B.moe_mxfp4(_dev(x), _dev(w13), _dev(w2), k, router_x=rx, router_w=rw)
    assert o["ids"].tolist() == [[0, 1, 2, 3]] * t and o["weights"][0].tolist() == [1, 0, 0, 0]


def test_graph_stream_and_a_not_finite_hidden_value():
    t, d, h, e, k = 20, 256, 128, 8, 2
    w13, w2 = _dev(_experts(e, 2 * h, d, 1)), _dev(_experts(e, d, h, 2))
    rw = torch.randn(e, d, device=DEV)
    xs = torch.randn(t, d, device=DEV)
    gain = torch.ones(d, device=DEV)

    def step():
        n = B.rmsnorm_mxfp8(xs, gain, with_y=True)
        return B.moe_mxfp4(n, w13, w2, k, router_x=n["y"], router_w=rw)["y"]

    step()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = step()
    for _ in range(4):
        xs.copy_(torch.randn(t, d, device=DEV))
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, step())
        torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    n = B.rmsnorm_mxfp8(xs, gain, with_y=True, stream=side)
    z = B.moe_mxfp4(n, w13, w2, k, router_x=n["y"], router_w=rw, stream=side)["y"]
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(y, z)
    # a NaN token: its row is NaN, the others' are untouched
    xs2 = xs.clone()
    xs2[3, 9] = float("nan")
    n = B.rmsnorm_mxfp8(xs2, gain, with_y=True)
    o = B.moe_mxfp4(n, w13, w2, k, router_x=n["y"], router_w=rw)["y"]
    keep = torch.arange(t, device=DEV) != 3
    assert torch.isnan(o[3]).all() and torch.equal(o[keep], y[keep])


def test_refusals_on_the_device():
    t, d, h, e, k = 2, 128, 128, 4, 2
    x, w13, w2 = _tokens(t, d, 0), _dev(_experts(e, 2 * h, d, 1)), _dev(_experts(e, d, h, 2))
    rx, rw = torch.zeros(t, d, device=DEV), torch.zeros(e, d, device=DEV)
    ids, wt = torch.zeros(t, k, dtype=torch.int32, device=DEV), torch.ones(t, k, device=DEV)
    for kw in (dict(), dict(router_x=rx), dict(ids=ids), dict(router_x=rx, router_w=rw, ids=ids, weights=wt)):
        with pytest.raises(ValueError):
            B.moe_mxfp4(x, w13, w2, k, **kw)
    for kw in (dict(router_x=rx, router_w=rw.bfloat16()), dict(ids=ids.long(), weights=wt)):
        with pytest.raises(TypeError):
            B.moe_mxfp4(x, w13, w2, k, **kw)
    for kw in (dict(router_x=rx, router_w=rw[:3]), dict(ids=ids[:, :1], weights=wt)):
        with pytest.raises(ValueError):
            B.moe_mxfp4(x, w13, w2, k, **kw)
    with pytest.raises(ValueError):
        B.moe_mxfp4(x, w2, w13, k, router_x=rx, router_w=rw)
    with pytest.raises(B.Fp4qError):                       # topk > experts
        B.moe_mxfp4(x, w13, w2, 5, router_x=rx, router_w=rw)
    with pytest.raises(B.Fp4qError):                       # over 64 tokens
        B.moe_mxfp4(_tokens(65, d, 0), w13, w2, k, router_x=torch.zeros(65, d, device=DEV), router_w=rw)
