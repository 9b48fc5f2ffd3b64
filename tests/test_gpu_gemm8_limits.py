"""The MXFP8 x MXFP4 product (GPU) at the largest number of columns: column indexes next to 2^31."""
import numpy as np
import pytest
import torch

from block_scaled_fp4_05_amd import binding as B

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _past_the_end(n):
    """Tiles of the last 256 columns store 8 columns at a time where n % 8 == 0.  The columns that the
    condition `col + 8 <= n` passes in 32-bit arithmetic without being columns of C."""
    col = np.arange(n - n % 256, n - n % 256 + 256, 8).astype(np.int64)
    wrapped = ((col + 8 + 2 ** 31) % 2 ** 32 - 2 ** 31) <= n
    return col[wrapped & (col + 8 > n)]


def test_nothing_is_written_past_the_last_row():
    n, m, k, guard = 2 ** 31 - 8, 1, 128, 256
    assert list(_past_the_end(n)) == [n]                   # this many columns is where the sum wraps
    torch.cuda.empty_cache()
    g = torch.Generator(device=DEV).manual_seed(0)
    codes = torch.empty(n, k // 2, dtype=torch.uint8, device=DEV)      # 137 GB, any values but the last rows'
    scales = torch.empty(n, k // 32, dtype=torch.uint8, device=DEV)
    codes[-300:] = torch.randint(0, 256, (300, k // 2), dtype=torch.uint8, device=DEV, generator=g)
    scales[-300:] = 127
    a = B.quantize_mxfp8(torch.randn(m, k, device=DEV, generator=g))
    c = torch.full((m * n + guard,), 7.0, dtype=torch.bfloat16, device=DEV)
    print("gemm8", m, n, k, flush=True)
    B.fp4q_gemm_mxfp8_mxfp4(a["codes"], a["scales"], codes, scales, m, n, k, B.BF16, c)
    torch.cuda.synchronize()
    assert torch.all(c[m * n:] == 7.0)
    last = {"codes": codes[-300:].clone(), "scales": scales[-300:].clone()}
    assert torch.equal(c[m * n - 300:m * n], B.gemm_mxfp8_mxfp4(a, last, torch.bfloat16)[0])
    del codes, scales, c
    torch.cuda.empty_cache()


@pytest.mark.parametrize("m,n,k", [(1, 4096, 4096), (16, 4096, 1152), (32, 8200, 4096), (64, 4096, 2048), (193, 4099, 4224),
                                   (1000, 1000, 1024), (2048, 4096, 4096)])
def test_the_same_bits_on_every_call(m, n, k):
    g = torch.Generator(device=DEV).manual_seed(m)
    a = B.quantize_mxfp8(torch.randn(m, k, device=DEV, generator=g))
    b = B.quantize_mxfp4(torch.randn(n, k, device=DEV, generator=g))
    print("gemm8", m, n, k, flush=True)
    c = B.gemm_mxfp8_mxfp4(a, b)
    for _ in range(8):
        assert torch.equal(B.gemm_mxfp8_mxfp4(a, b), c)
