"""The MXFP8 activation path of a decoder layer: norm -> projection -> norm -> experts, and the
norm's gradient.

    python examples/moe_decoder.py [--tokens 8] [--d 2048] [--hidden 1024] [--experts 32] [--topk 4]

``decode`` is what a serving loop runs per layer and step: every activation stays in MXFP8 between
operators, every weight in MXFP4.  ``fit_gain`` is a training loop's part: the norm's gain is
learned through the quantized projection (the gradient passes straight through the rounding).
Both print how far they are from the same layer computed in float32 on unquantized activations.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))

from block_scaled_fp4_05_amd import binding as fp4q  # noqa: E402

EPS = 1e-6


def mxfp4(w: torch.Tensor) -> dict:
    """Row-wise MXFP4 of the last axis of a weight of two or three axes."""
    q = fp4q.quantize_mxfp4(w.reshape(-1, w.shape[-1]))
    return {k: q[k].reshape(*w.shape[:-1], -1) for k in ("codes", "scales")}


def mxfp4_values(q: dict) -> torch.Tensor:
    codes = q["codes"].reshape(-1, q["codes"].shape[-1])
    scales = q["scales"].reshape(-1, q["scales"].shape[-1])
    rows, cols = codes.shape[0], codes.shape[1] * 2
    return fp4q.dequantize(fp4q.FMT_MXFP4, codes, scales, None, rows, cols).reshape(*q["codes"].shape[:-1], cols)


class Layer:
    def __init__(self, d: int, hidden: int, experts: int, topk: int, seed: int = 0):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def weight(*shape):
            return (torch.randn(*shape, generator=g, device="cuda") * shape[-1] ** -0.5).to(torch.bfloat16)

        self.topk = topk
        self.gain_in = torch.ones(d, device="cuda")
        self.gain_mid = torch.ones(d, device="cuda")
        self.proj = mxfp4(weight(d, d))
        self.router = weight(experts, d)
        self.w13 = mxfp4(weight(experts, 2 * hidden, d))
        self.w2 = mxfp4(weight(experts, d, hidden))


def decode(layer: Layer, stream: torch.Tensor, branch: torch.Tensor) -> tuple[torch.Tensor, dict]:
    """One step of at most 64 tokens: the residual stream and the last branch's output (bf16
    [tokens][d]) to the stream before the experts and the experts' output."""
    n = fp4q.rmsnorm_mxfp8(branch, layer.gain_in, residual=stream, eps=EPS)
    p = fp4q.gemm_mxfp8_mxfp4(n, layer.proj, torch.bfloat16)
    n = fp4q.rmsnorm_mxfp8(p, layer.gain_mid, residual=n["sum"], eps=EPS, with_y=True)
    return n["sum"], fp4q.moe_mxfp4(n, layer.w13, layer.w2, layer.topk, router_x=n["y"], router_w=layer.router)


def plain_norm(x: torch.Tensor, gain: torch.Tensor) -> torch.Tensor:
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * gain


def plain_decode(layer: Layer, stream: torch.Tensor, branch: torch.Tensor, ids: torch.Tensor, weights: torch.Tensor):
    """decode in float32 on the weights' quantized values, with given experts."""
    s = stream.float() + branch.float()
    s = s + plain_norm(s, layer.gain_in) @ mxfp4_values(layer.proj).t()
    n = plain_norm(s, layer.gain_mid)
    w13, w2 = mxfp4_values(layer.w13), mxfp4_values(layer.w2)
    y = torch.zeros_like(s)
    for t in range(s.shape[0]):
        for e, w in zip(ids[t].tolist(), weights[t].tolist()):
            gate, up = (w13[e] @ n[t]).chunk(2)
            y[t] += w * (w2[e] @ (torch.nn.functional.silu(gate) * up))
    return s, y


def fit_gain(layer: Layer, x: torch.Tensor, steps: int = 8) -> list[float]:
    """Gradient steps on the first norm's gain towards a projection with a gain of 1.25; the losses."""
    w = mxfp4_values(layer.proj)
    target = plain_norm(x.float(), torch.full_like(layer.gain_in, 1.25)) @ w.t()
    losses = []
    for _ in range(steps):
        n = fp4q.rmsnorm_mxfp8(x, layer.gain_in, eps=EPS)
        miss = fp4q.gemm_mxfp8_mxfp4(n, layer.proj, torch.float32) - target
        losses.append(miss.square().mean().item())
        dy = (miss @ w).to(x.dtype)
        _, dgain = fp4q.rmsnorm_backward(dy, n["sum"], layer.gain_in, n["rstd"])
        # the loss is close to |gain - 1.25|^2 times the tokens' squares: a Newton step of one half
        layer.gain_in -= 0.5 * dgain / (x.shape[0] * w.square().sum(0))
    return losses


def run(tokens: int, d: int, hidden: int, experts: int, topk: int) -> tuple[float, float, list[float]]:
    layer = Layer(d, hidden, experts, topk)
    g = torch.Generator(device="cuda").manual_seed(1)
    stream, branch, batch = (torch.randn(n, d, generator=g, device="cuda").to(torch.bfloat16)
                             for n in (tokens, tokens, 512))
    s, out = decode(layer, stream, branch)
    s_plain, y_plain = plain_decode(layer, stream, branch, out["ids"], out["weights"])

    def off(a, b):
        return ((a.float() - b).norm() / b.norm()).item()

    return off(s, s_plain), off(out["y"], y_plain), fit_gain(layer, batch)


def main() -> None:
    ap = argparse.ArgumentParser()
    for name, default in (("tokens", 8), ("d", 2048), ("hidden", 1024), ("experts", 32), ("topk", 4)):
        ap.add_argument(f"--{name}", type=int, default=default)
    s, y, losses = run(**vars(ap.parse_args()))
    print(f"residual stream: {s:.2e} of its norm from float32; experts' output: {y:.2e}")
    print("losses of the gain's fit:", " ".join(f"{v:.3g}" for v in losses))


if __name__ == "__main__":
    main()
