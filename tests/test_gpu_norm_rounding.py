"""The RMS norm's MXFP8 codes (GPU) next to rounding boundaries, against binary64.

Rows of ones: the sum of squares is exact, r = 1 / sqrt(1 + eps) is known to binary64 and the library holds it to
at least 2^-46.  The gain is the fp32 value next to (boundary / r), so n = r gain lies within 2^-23 of a boundary
of E4M3, or of the scale, and about 2^-25 from it on either side: half of these n round to the boundary itself in
fp32.  n is to be rounded from its value, not from its fp32 rounding: the codes and scales are equal."""
import numpy as np
import pytest
import torch

import mxfp8_ref as ref
from block_scaled_fp4_05_amd import binding as B

pytestmark = pytest.mark.gpu
DEV = "cuda"
VAL = ref.e4m3_values()


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("cols", [64, 1024, 4096, 8192, 20000])
def test_codes_next_to_a_boundary(cols, dtype, residual):
    eps = float(np.float32(3e-3))
    r = 1.0 / np.sqrt(1.0 + eps)
    rng = np.random.default_rng(cols)
    # halfway between two codes: odd sixteenths from 1/2 up to 448, odd multiples of 2^-10 below 2^-6; some negative
    half = np.where(rng.random(cols) < 0.8, (17 + 2 * rng.integers(0, 8, cols)) * 2.0 ** (rng.integers(-6, 8, cols) - 4),
                    (2 * rng.integers(0, 8, cols) + 1) * 2.0 ** -10)
    half *= np.where(rng.random(cols) < 0.5, -1, 1)
    half[::32] = 448.0 * 2.0 ** rng.integers(0, 2, cols // 32)      # the block's largest: a boundary of the scale
    gain = (half / r).astype(np.float32)
    y = r * gain.astype(np.float64)
    near = np.abs(y / half - 1)
    assert near.max() < 2.0 ** -23 and (y.astype(np.float32) == half).mean() > 0.3
    x = torch.ones(3, cols, dtype=dtype, device=DEV)
    res = torch.zeros_like(x) if residual else None
    print("norm rounding", cols, dtype, residual, flush=True)
    o = B.rmsnorm_mxfp8(x, torch.from_numpy(gain).to(DEV), residual=res, eps=eps, with_y=True)
    v, c = ref.quantize(np.broadcast_to(y, (3, cols)))
    assert np.array_equal(o["scales"].cpu().numpy(), c)
    assert np.array_equal(VAL[o["codes"].cpu().numpy()], v)
    assert torch.equal(o["y"].cpu(), torch.from_numpy(np.broadcast_to(y.astype(np.float32), (3, cols)).copy()).to(dtype))


def test_zeros_and_exact_products():
    x = torch.zeros(4, 256, device=DEV)
    x[1:, ::2] = 2.0
    x[2, 1::2] = -2.0
    x[3, :] = -0.0
    gain = torch.tensor([1.0625, -0.53125, 448.0, 0.0], device=DEV).repeat(64)
    o = B.rmsnorm_mxfp8(x, gain, eps=0.25, with_y=True)
    _, _, y = ref.rmsnorm(x.cpu().numpy(), gain.cpu().numpy(), None, 0.25)
    v, c = ref.quantize(y)
    assert np.array_equal(o["scales"].cpu().numpy(), c) and np.array_equal(VAL[o["codes"].cpu().numpy()], v)
    sign = torch.signbit(x) ^ torch.signbit(gain)           # also of a zero: s is x itself, -0 too
    assert torch.equal(o["codes"] >> 7, sign.to(torch.uint8))


def test_products_that_leave_fp32():
    """n past the largest fp32 number is infinite (a NaN code), below the smallest zero; between, ties of fp32 itself."""
    x = torch.full((2, 96), 1.5, device=DEV)
    gain = torch.ones(96, device=DEV)
    gain[3], gain[40], gain[41], gain[70], gain[71] = 3e38, 1e-45, -1e-45, 2.0 ** -127, 3.4e38
    eps = 0.5
    o = B.rmsnorm_mxfp8(x, gain, eps=eps, with_y=True)
    _, _, y = ref.rmsnorm(x.cpu().numpy(), gain.cpu().numpy(), None, eps)
    assert np.array_equal(o["y"].cpu().numpy(), y.astype(np.float32))
    v, c = ref.quantize(y)
    assert np.array_equal(o["scales"].cpu().numpy(), c) and np.array_equal(VAL[o["codes"].cpu().numpy()], v)
    wide = torch.zeros(1, 64, device=DEV)
    wide[0, 0], wide[0, 33] = 8.0, -8.0                                     # r = sqrt(1/2): n = 5.66 gain
    g = torch.ones(64, device=DEV)
    g[0], g[33] = 1e38, 2e38
    o = B.rmsnorm_mxfp8(wide, g, eps=0.0, with_y=True)
    assert o["y"][0, 0] == float("inf") and o["y"][0, 33] == float("-inf")
    codes = VAL[o["codes"].cpu().numpy()][0]
    assert np.isnan(codes[[0, 33]]).all() and np.all(np.delete(codes, [0, 33]) == 0)


def test_few_codes_differ_from_binary64():
    """8192 x 4096 bf16 with a residual.  The fp32 sum of squares is off by at most 32 roundings of 2^-24 of it
    and r by half of that, 2^-20; a boundary is crossed where n is as close as that to one, and at least
    2^-4 lies between two: at most one code in 2^16 / 2."""
    g = torch.Generator(device=DEV).manual_seed(3)
    x, res = (torch.randn(8192, 4096, generator=g, device=DEV).bfloat16() for _ in range(2))
    gain = torch.randn(4096, generator=g, device=DEV) * 0.1 + 1
    o = B.rmsnorm_mxfp8(x, gain, residual=res, eps=1e-6)
    s = x.double() + res.double()
    y = (s * torch.rsqrt(s.square().mean(1, keepdim=True) + 1e-6) * gain.double()).view(8192, -1, 32)
    m, e = torch.frexp(y.abs().amax(-1))
    p = e - 9 + (m > 0.875).int()
    q = y * torch.exp2(-p.double())[..., None]
    step = torch.exp2(torch.frexp(q)[1].clamp(min=-5).double() - 4)
    v = (torch.round(q / step) * step).view(8192, 4096)
    off = torch.tensor(VAL, device=DEV)[o["codes"].long()] != v
    assert off.sum().item() <= y.numel() / 2 ** 17
    assert (o["scales"].long() != p + 127).sum().item() <= p.numel() / 2 ** 17
