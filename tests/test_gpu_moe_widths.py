"""The MXFP4 expert layer (GPU) at the widths of real layers, against binary64.

Whole values that the layer holds exactly, with their nonzero channels spread over every K step, so that the
result must be equal in any order of summation and a wrong step, row, block or scale shows.  The cases reach
each kernel of the up product (its groups of 16 tokens, four and eight waves) with two and more groups of four
K steps per wave, even and uneven shares, and the down product with one and several workgroups per row tile.
"""
import numpy as np
import pytest
import torch

from block_scaled_fp4_05_amd import binding as B

pytestmark = pytest.mark.gpu
DEV = "cuda"
E2M1 = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64)


def _pack(n):
    return n[..., 0::2] | (n[..., 1::2] << 4)


def _layer(t, d, h, e, seed):
    """Tokens with one gate channel (5 of a K step of 128, any step) of 1 and seven other channels of 1 or -1;
    gate weights of 0, 1 or 2 times 2^6 on the gate channels only (silu(g) = g there), up weights of 0, 1 or -1 on
    the others, so that |up| <= 7 and a hidden value has four significant bits; any down weights."""
    g = torch.Generator(device=DEV).manual_seed(seed)

    def pick(values, *shape):
        v = torch.tensor(values, dtype=torch.uint8, device=DEV)
        return v[torch.randint(0, len(values), shape, generator=g, device=DEV)]
    xc = torch.zeros(t, d, dtype=torch.uint8, device=DEV)
    others = torch.arange(d, device=DEV)
    others = others[others % 128 != 5]
    for i in range(t):
        at = others[torch.randperm(len(others), generator=g, device=DEV)[:7]]
        xc[i, at] = pick([0x38, 0xB8], 7)                               # 1, -1
        xc[i, 5 + 128 * ((3 * i + seed) % (d // 128))] = 0x38
    w13 = torch.zeros(e, 2 * h, d, dtype=torch.uint8, device=DEV)
    w13[:, :h, 5::128] = pick([0, 2, 4], e, h, d // 128)                # 0, 1, 2
    w13[:, h:] = pick([0, 2, 10], e, h, d)                              # 0, 1, -1
    w13[:, h:, 5::128] = 0
    s13 = torch.full((e, 2 * h, d // 32), 127, dtype=torch.uint8, device=DEV)
    s13[:, :h] = 127 + 6
    w2 = pick(list(range(16)), e, d, h)
    s2 = torch.randint(126, 129, (e, d, h // 32), generator=g, device=DEV).to(torch.uint8)
    return ({"codes": xc, "scales": torch.full((t, d // 32), 127, dtype=torch.uint8, device=DEV)},
            {"codes": _pack(w13), "scales": s13}, {"codes": _pack(w2), "scales": s2})


def _values4(codes, scales):
    v = E2M1.to(DEV)[torch.stack([codes & 15, codes >> 4], -1).flatten(-2).long()]
    return v * torch.exp2(scales.double() - 127).repeat_interleave(32, -1)


def _exact(x, w13, w2, ids, weights):
    value = torch.zeros(256, dtype=torch.float64, device=DEV)
    value[0x38], value[0xB8] = 1.0, -1.0
    xv, h = value[x["codes"].long()], w2["codes"].shape[2] * 2
    y = torch.zeros(xv.shape, dtype=torch.float64, device=DEV)
    for e in range(w2["codes"].shape[0]):
        share = (weights.double() * (ids == e)).sum(1)
        tok = (ids == e).any(1).nonzero().flatten()
        if len(tok):
            gu = xv[tok] @ _values4(w13["codes"][e], w13["scales"][e]).t()
            hid = gu[:, :h] * gu[:, h:]
            assert hid.abs().max() <= 128 * 7
            y[tok] += share[tok, None] * (hid @ _values4(w2["codes"][e], w2["scales"][e]).t())
    return y


#  tokens, d, hidden, experts, topk, hot (every token's first choice is one expert)
CASES = [
    (64, 1024, 2048, 16, 4, False), (64, 4096, 2048, 16, 4, False), (64, 1152, 2048, 16, 4, True),
    (64, 4096, 512, 16, 4, False), (64, 2304, 2176, 8, 4, False),
    (64, 1024, 2048, 12, 4, False),   # two groups of tokens, four waves, two K steps each; down in three parts
    (64, 4096, 2048, 12, 4, False),   # eight steps each; down in two parts
    (64, 1152, 2048, 12, 4, True),    # nine steps over four waves; a hot expert
    (64, 4096, 512, 12, 4, False),    # two groups, eight waves, four steps each
    (32, 1280, 4352, 4, 4, False),    # two groups, 32 tokens, four waves
    (64, 2304, 2816, 6, 4, False),    # four groups, four waves, 18 steps; down in two parts
    (64, 4096, 1024, 8, 8, False),    # four groups, eight waves
    (64, 2816, 1024, 32, 4, False),   # one group, four waves, 22 steps
    (64, 2816, 1024, 32, 4, True),    # one group, four passes over a hot expert
    (64, 4096, 1024, 32, 4, False),   # one group, four waves, eight steps each
    (64, 8192, 512, 30, 4, False),    # one group, eight waves, eight steps each
    (24, 8192, 256, 32, 4, True),     # eight steps each; two passes
    (33, 4224, 640, 24, 3, False),    # 33 steps over eight waves
    (17, 2048, 1024, 64, 8, False), (8, 4096, 2048, 32, 4, False), (3, 2944, 1024, 16, 2, False),
    (12, 1024, 2048, 32, 4, True),    # down in four parts, 16 tokens' kernel
    (1, 2048, 1024, 64, 4, False), (1, 4096, 2048, 8, 2, False), (1, 2816, 4096, 16, 8, False),
    (1, 2048, 8192, 8, 4, False),     # one token, four waves
    (1, 1024, 4096, 8, 8, False),     # as many choices as experts
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
def test_whole_values_are_exact(case):
    t, d, h, e, k, hot = case
    x, w13, w2 = _layer(t, d, h, e, t + e)
    g = torch.Generator().manual_seed(1)
    ids = torch.stack([torch.randperm(e, generator=g)[:k] for _ in range(t)]).to(torch.int32)
    if hot:
        ids[ids == 1] = ids[:, :1].expand(-1, k)[ids == 1]            # nobody's other choice ...
        ids[:, 0] = 1                                                   # ... everybody's first
    weights = torch.tensor([0.5, 1.0, 2.0, -1.0])[torch.randint(0, 4, (t, k), generator=g)]
    ids, weights = ids.to(DEV), weights.to(DEV)
    print("moe widths", case, flush=True)
    run = lambda: B.moe_mxfp4(x, w13, w2, k, ids=ids, weights=weights, out_dtype=torch.float32)["y"]
    y = run()
    assert torch.equal(y.double(), _exact(x, w13, w2, ids, weights))
    assert torch.equal(run(), y)


@pytest.mark.parametrize("router", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("case", [c for c in CASES if not c[5]], ids=lambda c: "-".join(map(str, c[:5])))
def test_the_router_at_these_widths(case, router):
    """Whole router operands: logits exact in fp32, so the choices are those of binary64, ties and all; the
    result is the bits of the layer with these choices given."""
    t, d, h, e, k, _ = case
    x, w13, w2 = _layer(t, d, h, e, t + e)
    g = torch.Generator(device=DEV).manual_seed(2)
    rx = torch.randint(-2, 3, (t, d), generator=g, device=DEV).to(router)
    rw = (torch.randint(-2, 3, (e, d), generator=g, device=DEV) / 64).to(router)
    logits = (rx.double() @ rw.double().t()).cpu().numpy()
    order = np.lexsort((np.broadcast_to(np.arange(e), logits.shape), -logits), axis=-1)[:, :k]
    top = np.take_along_axis(logits, order, 1)
    w = np.exp(top - top[:, :1])
    w /= w.sum(1, keepdims=True)
    print("moe router", case, router, flush=True)
    o = B.moe_mxfp4(x, w13, w2, k, router_x=rx, router_w=rw, out_dtype=torch.float32)
    assert np.array_equal(o["ids"].cpu().numpy(), order)
    # exact logits and differences; the exponential, a sum of at most 16 and the division round: 2^-19 at most
    assert np.all(np.abs(o["weights"].cpu().numpy() - w) <= 2.0 ** -19 * w + 1e-37)
    again = B.moe_mxfp4(x, w13, w2, k, ids=o["ids"], weights=o["weights"], out_dtype=torch.float32)
    assert torch.equal(again["y"], o["y"])
    half = B.moe_mxfp4(x, w13, w2, k, router_x=rx, router_w=rw)
    assert torch.equal(half["y"], o["y"].to(torch.bfloat16))
