"""The MXFP8 x MXFP4 product (GPU) against binary64.

Small whole values make every partial sum exact in fp32 (magnitudes below 2^21 in steps of 2^-3),
so the result must be equal in any order of summation and any wrong row, block or scale shows.
On real operands the bound is derived from the instruction: of 16 neighbouring products each is
cut at most 2^-13 of their largest, and the joins are fp32 sums (depth at most 8 per instruction
plus one per instruction, plus 16 for the waves' join), doubled.
"""
import numpy as np
import pytest
import torch

import mxfp8_ref as ref
from block_scaled_fp4_05_amd import binding as B

pytestmark = pytest.mark.gpu
DEV = "cuda"
VAL8 = ref.e4m3_values()


def _whole(rows, k, bits, seed):
    """Codes of small whole values (a few halves for the 4-bit side) with scales 2^-1, 1, 2."""
    rng = np.random.default_rng(seed)
    if bits == 8:
        small = np.array([0x00, 0x80, 0x38, 0xB8, 0x40, 0xC0, 0x44, 0xC4, 0x48, 0xC8], np.uint8)   # 0, 1, 2, 3, 4 and signs
        codes = small[rng.integers(0, len(small), (rows, k))]
    else:
        codes = rng.integers(0, 256, (rows, k // 2), dtype=np.uint8)
    return codes, rng.integers(126, 129, (rows, k // 32), dtype=np.uint8)


def _dev(codes, scales):
    return {"codes": torch.from_numpy(codes).to(DEV), "scales": torch.from_numpy(scales).to(DEV)}


def _check_whole(m, n, k, seed=0):
    a, b = _whole(m, k, 8, seed), _whole(n, k, 4, seed + 1)
    exact = (torch.from_numpy(ref.dequantize(*a)).to(DEV) @ torch.from_numpy(ref.fp4(*b)).to(DEV).t()).float()
    print("gemm8", m, n, k, flush=True)
    da, db = _dev(*a), _dev(*b)
    got = B.gemm_mxfp8_mxfp4(da, db, torch.float32)
    assert torch.equal(got, exact)
    assert torch.equal(B.gemm_mxfp8_mxfp4(da, db, torch.bfloat16), exact.to(torch.bfloat16))


@pytest.mark.parametrize("k", [128, 256, 384, 640, 1152, 4224])
@pytest.mark.parametrize("m,n", [(1, 1), (1, 16), (2, 100), (15, 33), (16, 260), (17, 64), (33, 255), (64, 48), (65, 130),
                                 (130, 67), (193, 257)])
def test_whole_values_are_exact(m, n, k):
    _check_whole(m, n, k, m + n + k)


@pytest.mark.parametrize("m,n,k", [(1, 4096, 8192), (64, 2050, 2048), (70, 13000, 512), (1000, 3000, 640),
                                   (1500, 2301, 256), (3600, 3601, 384), (4096, 8192, 256), (65, 70000, 128),
                                   (20000, 65, 128), (3600, 3601, 512), (3600, 3601, 640), (3500, 3700, 1536),
                                   (1000, 3000, 1024), (900, 3001, 2688), (193, 4099, 640), (193, 4099, 1536),
                                   (1, 33000, 256), (16, 8200, 640), (5, 40001, 1152), (32, 8193, 384),
                                   (20, 8193, 1280), (3, 70000, 512), (4, 10300, 1152), (5, 10241, 640), (1, 300, 16384),
                                   (17, 4100, 2176), (24, 6145, 896), (33, 4096, 640), (64, 4001, 4480), (70, 1900, 1152),
                                   (200, 1000, 1536), (449, 500, 384), (1600, 130, 640)])
def test_whole_values_large(m, n, k):
    _check_whole(m, n, k)


@pytest.mark.parametrize("m,n,k", [(2, (1 << 25) + 33, 256), (3, (1 << 26) + 17, 128), (70000, 65540, 128)])
def test_offsets_past_32_bits(m, n, k):
    """Codes of B past 4 GiB (few rows, and the tiles that take over), or 2^32 outputs: the last
    rows against the same rows multiplied alone."""
    g = torch.Generator(device=DEV).manual_seed(1)
    a, b = _dev(*_whole(min(m, 1000), k, 8, 0)), _dev(*_whole(1000, k, 4, 1))
    a = {key: v.repeat(-(-m // v.shape[0]), 1)[:m].contiguous() for key, v in a.items()}
    codes = torch.randint(0, 256, (n, k // 2), dtype=torch.uint8, device=DEV, generator=g)
    scales = torch.randint(126, 129, (n, k // 32), dtype=torch.uint8, device=DEV, generator=g)
    print("gemm8", m, n, k, flush=True)
    c = B.gemm_mxfp8_mxfp4(a, {"codes": codes, "scales": scales}, torch.bfloat16)
    rows = slice(max(0, m - 70), m)
    last = {key: v[rows].clone() for key, v in a.items()}
    for at in (0, n // 2, n - 300):
        part = {"codes": codes[at:at + 300].clone(), "scales": scales[at:at + 300].clone()}
        assert torch.equal(c[rows, at:at + 300], B.gemm_mxfp8_mxfp4(last, part, torch.bfloat16))


@pytest.mark.parametrize("m,n,k", [(1, 64, 4096), (5, 33, 1152), (48, 40, 640), (130, 70, 512), (260, 96, 256)])
def test_real_operands(m, n, k):
    g = torch.Generator().manual_seed(m + k)
    x = torch.randn(m, k, generator=g)
    x[:, ::61] *= 30.0
    w = torch.randn(n, k, generator=g) * k ** -0.5
    a, b = B.quantize_mxfp8(x.to(DEV)), B.quantize_mxfp4(w.to(DEV))
    av = ref.dequantize(a["codes"].cpu().numpy(), a["scales"].cpu().numpy())
    bv = ref.fp4(b["codes"].cpu().numpy(), b["scales"].cpu().numpy())
    exact, mag = av @ bv.T, np.abs(av) @ np.abs(bv).T
    cut = np.zeros_like(exact)
    for t in range(0, k, 16):
        cut += (np.abs(av)[:, None, t:t + 16] * np.abs(bv)[None, :, t:t + 16]).max(-1) * 16 * 2.0 ** -13
    bound = cut + 2 * (8 + k / 64 + 16) * 2.0 ** -24 * mag
    got = B.gemm_mxfp8_mxfp4(a, b, torch.float32).cpu().numpy()
    assert np.all(np.abs(got - exact) <= bound)
    half = B.gemm_mxfp8_mxfp4(a, b, torch.bfloat16).float().cpu().numpy()
    assert np.all(np.abs(half - exact) <= bound + 2.0 ** -8 * np.abs(exact))


@pytest.mark.parametrize("m,n", [(3, 40), (70, 130), (300, 90)])
def test_extreme_scales_and_nan(m, n):
    k = 256
    a, b = _whole(m, k, 8, 1), _whole(n, k, 4, 2)
    # scales far apart whose products stay in range: 2^100 and 2^-100, and zeros of scale 0
    a[1][0, :], b[1][:, :] = 227, 27
    a[1][m - 1, :] = 0
    a[0][m - 1, :] = 0
    exact = (torch.from_numpy(ref.dequantize(*a)).to(DEV) @ torch.from_numpy(ref.fp4(*b)).to(DEV).t()).float()
    got = B.gemm_mxfp8_mxfp4(_dev(*a), _dev(*b))
    assert torch.equal(got[0], exact[0]) and torch.all(got[m - 1] == 0)
    a, b = _whole(m, k, 8, 3), _whole(n, k, 4, 4)
    clean = B.gemm_mxfp8_mxfp4(_dev(*a), _dev(*b))
    a[0][1, 77] = 0x7F                       # a NaN code in row 1
    b[1][7, 2] = 255                         # a NaN scale in column 7
    got = B.gemm_mxfp8_mxfp4(_dev(*a), _dev(*b))
    nan = torch.isnan(got)
    assert nan[1].all() and nan[:, 7].all()
    keep = torch.ones_like(nan)
    keep[1], keep[:, 7] = False, False
    assert torch.equal(got[keep], clean[keep])


def test_the_norm_feeds_the_product_and_graphs_replay():
    x = torch.randn(40, 1024, device=DEV).bfloat16()
    gain = torch.ones(1024, device=DEV)
    w = B.quantize_mxfp4(torch.randn(515, 1024, device=DEV) * 0.03)
    B.gemm_mxfp8_mxfp4(B.rmsnorm_mxfp8(x, gain), w, torch.bfloat16)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = B.gemm_mxfp8_mxfp4(B.rmsnorm_mxfp8(x, gain), w, torch.bfloat16)
    for k in range(4):
        x.copy_(torch.randn(40, 1024, device=DEV))
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, B.gemm_mxfp8_mxfp4(B.rmsnorm_mxfp8(x, gain), w, torch.bfloat16))
        torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    a = B.rmsnorm_mxfp8(x, gain, stream=s)
    z = B.gemm_mxfp8_mxfp4(a, w, torch.bfloat16, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(y, z)


def test_refusals_on_the_device():
    a, b = _dev(*_whole(4, 256, 8, 0)), _dev(*_whole(8, 256, 4, 1))
    short = {"codes": b["codes"][:, :64].contiguous(), "scales": b["scales"]}
    for bad in (short, {"codes": b["codes"], "scales": b["scales"][:, :4].contiguous()},
                {"codes": b["codes"].repeat(1, 2)[:, ::2], "scales": b["scales"]}):
        with pytest.raises(ValueError):
            B.gemm_mxfp8_mxfp4(a, bad)
    with pytest.raises(TypeError):
        B.gemm_mxfp8_mxfp4({"codes": a["codes"].view(torch.int8), "scales": a["scales"]}, b)
    with pytest.raises(B.Fp4qError):                       # k % 128
        B.gemm_mxfp8_mxfp4(_dev(*_whole(4, 96, 8, 0)), _dev(*_whole(8, 96, 4, 0)))
