"""The RMS norm's gradient (GPU) on rows far from ordinary size, against binary64.

dx = r a - s r^3 mean(a s): the two terms are of one size whatever the row's, so the bound is the one of
ordinary rows, 64 roundings of the terms' magnitudes (54 for the mean, at most 10 around it), and dgain's is
44 roundings of its terms' magnitudes (one row per partial sum, 37 additions, two products)."""
import numpy as np
import pytest
import torch

import mxfp8_ref as ref
from block_scaled_fp4_05_amd import binding as B

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -24


def _np(t):
    return t.float().cpu().numpy().astype(np.float64)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("cols", [256, 2080, 4096, 20000])
@pytest.mark.parametrize("size,eps", [(1e-17, 0.0), (1e-13, 0.0), (1e-9, 1e-30), (1e-3, 1e-6), (1e13, 1e-6), (1e15, 1e-6),
                                      (3e16, 0.0), (1e18, 1e-6)])
def test_gradient_of_rows_of_any_size(size, eps, cols, dtype):
    g = torch.Generator().manual_seed(cols)
    x = (torch.randn(5, cols, generator=g) * size).to(dtype).to(DEV)
    dy = torch.randn(5, cols, generator=g).to(dtype).to(DEV)
    dy += (x / size).to(dtype)                              # so that the projection is as large as the rest
    gain = (torch.randn(cols, generator=g) * 0.2 + 1).to(DEV)
    print("norm gradient", size, eps, cols, dtype, flush=True)
    o = B.rmsnorm_mxfp8(x, gain, eps=eps)
    _, r, _ = ref.rmsnorm(_np(x), _np(gain), None, eps)
    assert np.all(np.abs(_np(o["rstd"]) - r) <= 32 * U * r)
    dx, dg = B.rmsnorm_backward(dy, x, gain, o["rstd"])
    wx, wg, mx, mg = ref.rmsnorm_backward(_np(dy), _np(x), _np(gain), _np(o["rstd"]))
    half = 2.0 ** -8 if dtype == torch.bfloat16 else U
    assert np.all(np.abs(_np(dx) - wx) <= 1.01 * half * np.abs(wx) + 64 * U * mx + 1e-45)
    assert np.all(np.abs(_np(dg) - wg) <= 44 * U * mg + 1e-45)
